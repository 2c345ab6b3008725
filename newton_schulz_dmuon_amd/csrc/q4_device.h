// Device helpers shared by the 4-bit products' kernels.
#pragma once

#include "q4_internal.h"
#include "q8_device.h"

namespace dmuon {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// A lane's 32 codes as a matrix operand: 4-bit operands take the first four words.
__device__ __forceinline__ i32x8 codes_operand(const u32x4 &w) {
  return i32x8{static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z), static_cast<int>(w.w), 0, 0, 0, 0};
}

// acc += 16 outputs by 16 rows over 128 codes: a lane's 32 codes of each operand
// (one block of the format) and the words whose bytes IB and IA are their scales.
template <int IB, int IA>
__device__ __forceinline__ f32x4 q4_product(const u32x4 &b, uint32_t sb, const u32x4 &a, uint32_t sa, f32x4 acc) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes_operand(b), codes_operand(a), acc, 4, 4, IB,
                                                          static_cast<int>(sb), IA, static_cast<int>(sa));
}

// 2^(byte - 128) as fp32, half of a scale byte's scale; infinity for kQ4Nan, with
// which every conversion from a code gives NaN.
__device__ __forceinline__ float q4_half_scale(uint32_t byte) { return __uint_as_float(byte << 23) * 0.5f; }

// Eight codes (a word) times a power of two as bf16, exactly.
__device__ __forceinline__ bf16x8 q4_expand8(uint32_t w, float s) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// The streaming kernels' outputs tile of a work-group: a line of a scale table holds
// 128 outputs' bytes of a block, so the 8 / NN work-groups that share it are eight
// apart, on one XCD and its L2 (work-groups go to the XCDs in turn): one row by 4096 x
// 14336 8.1 us, in the grid's order 9.3, of which every XCD read most of the table.
template <int NN>
__device__ __forceinline__ uint32_t line_tile(uint32_t n, uint32_t count) {
  constexpr uint32_t kShare = 8 / NN, kChunk = 8 * kShare;
  const uint32_t first = n / kChunk * kChunk, q = n - first;
  return first + kChunk <= count ? first + q % 8 * kShare + q / 8 : n;
}

// Adds the sums of two waves that share a tile and split k: wave `half` 0 keeps the
// rows' blocks j < FN / 2, half 1 the others, and each gets the other's part of its
// own through LDS (slot: 1 KB times FM FN / 2 of each of the pair's waves).  The
// first half's sum is the first operand.  `mine` and `other` are the two waves'
// slots; every wave of the work-group takes part.
template <int FM, int FN>
__device__ __forceinline__ void exchange_halves(f32x4 (&acc)[FM][FN], int half, lds_char *mine, lds_char *other) {
  const int at = (threadIdx.x & 63) * 16;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN / 2; ++j) {
      const f32x4 give = half == 0 ? acc[i][j + FN / 2] : acc[i][j];
      *(lds_f32x4 *)(mine + (i * (FN / 2) + j) * 1024 + at) = give;
    }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN / 2; ++j) {
      const f32x4 got = *(const lds_f32x4 *)(other + (i * (FN / 2) + j) * 1024 + at);
      acc[i][j] = half == 0 ? acc[i][j] + got : got + acc[i][j + FN / 2];
    }
}

// R runs of N elements of base, `step` apart, `left` > 0 of which exist from the
// first on (zeros behind them), a run's or all loads before the first use.  The kernels add
// base before their first store: a load may not pass a store, since base may be out,
// and each run would wait for its own.
template <int N, int R>
__device__ __forceinline__ void load_base(const void *base, int32_t dt, int64_t at, int step, int64_t left, float (&v)[R][N]) {
  if (left >= (R - 1) * step + N) {
    load_runs<N, R>(base, dt, at, step, v);
    return;
  }
  // run by run, element by element
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint32_t w[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t i = at + min(static_cast<int64_t>(r * step + k), left - 1);
      w[k] = dt == kF32 ? ((const g_u32 *)base)[i] : static_cast<uint32_t>(((const g_u16 *)base)[i]) << 16;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[r][k] = r * step + k < left ? __uint_as_float(w[k]) : 0.f;
    __builtin_amdgcn_sched_barrier(0);
  }
}

}  // namespace dmuon
