// Products of bf16 rows with 4-bit block weights on gfx950 matrix cores.
//
//   out[t][n] = sum_b 2^eb[b][n] sum_{k in b} a[t][k] b[n][k]
//
// The codes are expanded to bf16, code times half the scale, which is exact (two
// significant bits; 4 * 2^125 is in range, 4 * 2^126, the code of the largest
// bf16 and fp32 values, would not be, and 0.5 * 2^-126 is a subnormal that
// expansion and product keep), and multiplied by v_mfma_f32_16x16x32_bf16: every
// product is exact and every sum fp32's.  The sums are half the result's and are
// doubled.
//
// Weights b are the instruction's first operand and rows a the second: a lane
// then holds four consecutive outputs of one row.

#include "q4_device.h"

namespace dmuon {

namespace {

constexpr int64_t kSide = 64;  // of a work-group's tile

// A work-group of four waves (2 x 2) computes 64 outputs by 64 rows; rows and
// outputs behind the last are clamped for the loads and not stored.
__global__ __launch_bounds__(256) void q4_rows_tile_kernel(Q4Product p, uint32_t na) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g4 = lane >> 4;
  const uint32_t tb = blockIdx.x / na;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x - tb * na) * kSide + (wave & 1) * 32;
  const int64_t t0 = static_cast<int64_t>(tb) * kSide + (wave >> 1) * 32;
  const int64_t rb = (p.outs + 15) / 16 * 16;
  const int64_t n1[2] = {min(n0 + r16, p.outs - 1), min(n0 + 16 + r16, p.outs - 1)};
  const int64_t t1[2] = {min(t0 + r16, p.rows - 1), min(t0 + 16 + r16, p.rows - 1)};
  f32x4 acc[2][2] = {};
  for (int64_t k = 0; k < p.kp; k += 32) {
    const int64_t kl = k + g4 * 8;
    bf16x8 fb[2], fa[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = *(const g_u32 *)(p.b + n1[i] * (p.kp / 2) + kl / 2);
      fb[i] = q4_expand8(w, q4_half_scale(((const g_u8 *)p.sb)[k / kQ4Block * rb + n1[i]]));
#pragma unroll
      for (int e = 0; e < 8; ++e)
        fa[i][e] = kl + e < p.inner ? static_cast<__bf16>(load_elem(p.a, kBF16, t1[i] * p.inner + kl + e))
                                    : static_cast<__bf16>(0.f);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[i], fa[j], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t t = t0 + j * 16 + r16, n = n0 + i * 16 + 4 * g4;
      if (t >= p.rows) continue;
      float v[4] = {2 * acc[i][j][0], 2 * acc[i][j][1], 2 * acc[i][j][2], 2 * acc[i][j][3]};
      finish_run<4>(nullptr, p.out, p.out_dt, t * p.outs + n, p.outs - n, v);
    }
}

}  // namespace

size_t q4_rows_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_q4_rows(const Q4Product &p, hipStream_t st) {
  const int64_t na = (p.outs + kSide - 1) / kSide, nb = (p.rows + kSide - 1) / kSide;
  hipLaunchKernelGGL(q4_rows_tile_kernel, dim3(static_cast<uint32_t>(na * nb)), dim3(256), 0, st, p,
                     static_cast<uint32_t>(na));
  return hipGetLastError();
}

}  // namespace dmuon
