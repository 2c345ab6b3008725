// Products of 4-bit block operands on gfx950 matrix cores.
//
//   out[t][n] = base[t][n] + sum_b 2^(ea[b][t] + eb[b][n]) sum_{k in b} a[t][k] b[n][k]
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 by 128 x 16 codes and
// applies each operand's scale, one per 32 codes, inside the instruction: a lane
// holds 32 codes of one row, one block of the format, and its scale byte.  The
// sums are fp32's: a product of two codes is a multiple of 1/4 up to 36, so a
// block's 32 products add up exactly, and the blocks add in fp32 (checked against
// 64 bits with scales over the format's whole range: within 2^-22 of the sum of
// magnitudes an instruction, without a bias, and exact where the scales agree).
//
// Weights b are the instruction's first operand and rows a the second: a lane
// then holds four consecutive outputs of one row.

#include "q4_device.h"

namespace dmuon {

namespace {

constexpr int64_t kSide = 64;  // of a work-group's tile

// A work-group of four waves (2 x 2) computes 64 outputs by 64 rows; rows and
// outputs behind the last are clamped for the loads and not stored.
__global__ __launch_bounds__(256) void q4_tile_kernel(Q4Product p, uint32_t na) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g4 = lane >> 4;
  const uint32_t tb = blockIdx.x / na;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x - tb * na) * kSide + (wave & 1) * 32;
  const int64_t t0 = static_cast<int64_t>(tb) * kSide + (wave >> 1) * 32;
  const int64_t ra = (p.rows + 15) / 16 * 16, rb = (p.outs + 15) / 16 * 16;
  const int64_t n1[2] = {min(n0 + r16, p.outs - 1), min(n0 + 16 + r16, p.outs - 1)};
  const int64_t t1[2] = {min(t0 + r16, p.rows - 1), min(t0 + 16 + r16, p.rows - 1)};
  f32x4 acc[2][2] = {};
  for (int64_t k = 0; k < p.kp; k += 128) {
    const int64_t block = k / kQ4Block + g4;
    u32x4 fb[2], fa[2];
    uint32_t sb[2], sa[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fb[i] = *(const g_u32x4 *)(p.b + n1[i] * (p.kp / 2) + k / 2 + g4 * 16);
      fa[i] = *(const g_u32x4 *)(static_cast<const uint8_t *>(p.a) + t1[i] * (p.kp / 2) + k / 2 + g4 * 16);
      sb[i] = ((const g_u8 *)p.sb)[block * rb + n1[i]];
      sa[i] = ((const g_u8 *)p.sa)[block * ra + t1[i]];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = q4_product<0, 0>(fb[i], sb[i], fa[j], sa[j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t t = t0 + j * 16 + r16, n = n0 + i * 16 + 4 * g4;
      if (t >= p.rows) continue;
      float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      finish_run<4>(p.base, p.out, p.out_dt, t * p.outs + n, p.outs - n, v);
    }
}

}  // namespace

size_t q4_matmul_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_q4_matmul(const Q4Product &p, hipStream_t st) {
  const int64_t na = (p.outs + kSide - 1) / kSide, nb = (p.rows + kSide - 1) / kSide;
  hipLaunchKernelGGL(q4_tile_kernel, dim3(static_cast<uint32_t>(na * nb)), dim3(256), 0, st, p,
                     static_cast<uint32_t>(na));
  return hipGetLastError();
}

}  // namespace dmuon
