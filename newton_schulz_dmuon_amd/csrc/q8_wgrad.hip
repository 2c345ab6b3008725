// The weight gradient from an 8-bit checkpoint on gfx950 matrix cores.
//
//   out[n][k] = base[n][k] + sum_t dy[t][n] 2^e[k / 128][t] x[t][k]
//
// The sum runs over t, along which the checkpoint's scales change, so they
// cannot ride on an 8-bit matrix instruction.  Code times scale is exact in
// bf16 (four significant bits, an exponent within bf16's normal range), so x
// is expanded to bf16 on its way into LDS and multiplied with the bf16
// gradient; sums are fp32.

#include "device_common.h"
#include "q8_internal.h"

namespace dmuon {

namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(1))) uint32_t g_u32;
typedef __attribute__((address_space(1))) uint8_t g_u8;

// 64 x 64 outputs per work-group of four waves (32 x 32 each), 32 rows of t
// per step, both operands transposed into LDS as [column][t].
constexpr int kTile = 64, kStep = 32, kPitch = kStep + 8;  // elements; 80-byte rows

__global__ __launch_bounds__(256) void q8_wgrad64_kernel(Q8WeightGrad p) {
  __shared__ __align__(16) uint16_t l[kTile * kPitch], r[kTile * kPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, g4 = lane >> 4;
  const uint32_t kt = static_cast<uint32_t>((p.cols + kTile - 1) / kTile);
  const int64_t k0 = static_cast<int64_t>(blockIdx.x % kt) * kTile, n0 = static_cast<int64_t>(blockIdx.x / kt) * kTile;
  const int64_t t4 = (p.rows + 3) & ~static_cast<int64_t>(3);
  const uint8_t *const sx = p.sx + (k0 / kQ8Block) * t4;
  const int wn = (wave >> 1) * 32, wk = (wave & 1) * 32;
  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t tb = 0; tb < p.rows; tb += kStep) {
    // thread: row tid / 8 of the step, columns (tid % 8) * 8 .. + 7
    const int row = tid >> 3, c = (tid & 7) * 8;
    const int64_t t = tb + row;
    const bool in = t < p.rows;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t n = n0 + c + k;
      l[(c + k) * kPitch + row] = in && n < p.outs ? ((const g_u16 *)p.dy)[t * p.outs + n] : 0;
    }
    uint32_t q[2] = {0, 0};
    float s = 1.f;
    if (in) {
      q[0] = *(const g_u32 *)(p.x + t * p.kp + k0 + c);
      q[1] = *(const g_u32 *)(p.x + t * p.kp + k0 + c + 4);
      s = __uint_as_float(static_cast<uint32_t>(((const g_u8 *)sx)[t]) << 23);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[h], s, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[h], s, true);
      const uint32_t u[2] = {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        r[(c + 4 * h + k) * kPitch + row] = static_cast<uint16_t>(u[k >> 1] >> (16 * (k & 1)));
    }
    __syncthreads();
    bf16x8 fl[2], fr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fl[i] = *reinterpret_cast<const bf16x8 *>(&l[(wn + i * 16 + r16) * kPitch + g4 * 8]);
      fr[i] = *reinterpret_cast<const bf16x8 *>(&r[(wk + i * 16 + r16) * kPitch + g4 * 8]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fl[i], fr[j], acc[i][j], 0, 0, 0);
    __syncthreads();
  }
  // lane: rows n = 4 g4 + v, column k = r16 of each 16 x 16 block
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t n = n0 + wn + i * 16 + 4 * g4 + v, k = k0 + wk + j * 16 + r16;
        if (n < p.outs && k < p.cols) {
          const int64_t at = n * p.cols + k;
          const float b = p.base ? load_elem(p.base, p.out_dt, at) : 0.f;
          store_elem(p.out, p.out_dt, at, b + acc[i][j][v]);
        }
      }
}

}  // namespace

size_t q8_wgrad_workspace(int64_t rows, int64_t outs, int64_t cols) { return 0; }

hipError_t launch_q8_wgrad(const Q8WeightGrad &p, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>((p.cols + kTile - 1) / kTile * ((p.outs + kTile - 1) / kTile)));
  hipLaunchKernelGGL(q8_wgrad64_kernel, grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace dmuon
