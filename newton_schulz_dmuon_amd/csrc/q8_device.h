// Device helpers shared by the 8-bit block products' kernels.
#pragma once

#include "device_common.h"
#include "q8_internal.h"

namespace dmuon {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(1))) u32x4 g_u32x4;
// ... at the address of any 2-byte or 4-byte element
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
typedef __attribute__((address_space(1))) u32x4_at2 g_u32x4_at2;
typedef __attribute__((address_space(1))) u32x4_at4 g_u32x4_at4;
typedef __attribute__((address_space(1))) u32x2_at2 g_u32x2_at2;
typedef __attribute__((address_space(1))) f32x4_at4 g_f32x4_at4;
typedef __attribute__((address_space(1))) u32x2 g_u32x2;
typedef __attribute__((address_space(1))) f32x4 g_f32x4;
typedef __attribute__((address_space(1))) uint32_t g_u32;
typedef __attribute__((address_space(1))) uint8_t g_u8;
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;
typedef __attribute__((address_space(3))) uint16_t lds_u16;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

// A value that is the same in every lane, as a scalar (integer divisions run
// on the vector unit).
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
}

// This lane's index, made anew: where registers are short, nothing need be kept
// for it.
__device__ __forceinline__ int lane_index() {
  return static_cast<int>(__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)));
}

// Work-group barriers.  The memory clobbers keep the compiler from moving LDS
// accesses across them.
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }
// ... once this wave's LDS accesses are complete
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// ... once this wave's loads have landed
__device__ __forceinline__ void load_barrier() { asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory"); }

// The place in a list of `total` entries that work-group `w` takes: neighbours
// in the list run together on one XCD (work-group w runs on XCD w % 8).
__device__ __forceinline__ uint32_t xcd_order(uint32_t w, uint32_t total) {
  const uint32_t x = w % kXcds, q = total / kXcds, rem = total % kXcds;
  return x * q + min(x, rem) + w / kXcds;
}

// Tile (a, b) at place `idx` of the list of na * nb tiles: bands of four b,
// whose neighbours share operand panels in an XCD's L2.
__device__ __forceinline__ void tile_at(uint32_t idx, uint32_t na, uint32_t nb, uint32_t &a, uint32_t &b) {
  const uint32_t band = idx / (4 * na), r = idx - band * 4 * na;
  const uint32_t h = min(4u, nb - band * 4);
  a = uniform(r / h);
  b = uniform(band * 4 + r % h);
}

// What a work-group of a tiled launch computes: tile (a, b), steps [begin,
// end), and where to: the result, or slot `slot` of the workspace.
struct TileWork {
  uint32_t a, b;
  int begin, end;
  int64_t slot;  // -1: the result
};
__device__ __forceinline__ TileWork tile_work(const TileSplit &sp, uint32_t w, uint32_t steps) {
  TileWork t;
  t.begin = 0;
  t.end = static_cast<int>(steps);
  t.slot = -1;
  uint32_t idx;
  if (w < sp.whole) {
    idx = xcd_order(w, sp.whole);
  } else {
    const uint32_t r = w - sp.whole, piece = uniform(r / sp.tail), place = uniform(r - piece * sp.tail);
    idx = sp.whole + xcd_order(place, sp.tail);
    if (sp.pieces > 1) {
      // steps * pieces fits 32 bits: 2^23 steps, 2^4 pieces
      t.begin = static_cast<int>(uniform(steps * piece / sp.pieces));
      t.end = static_cast<int>(uniform(steps * (piece + 1) / sp.pieces));
      t.slot = static_cast<int64_t>(idx - sp.whole) * sp.pieces + piece;
    }
  }
  tile_at(idx, sp.na, sp.nb, t.a, t.b);
  return t;
}

// Where a tile's results go: the result matrix (rows x cols), or the tile's
// slot of the workspace, which takes all of them as fp32.
struct TileOut {
  const void *base;
  void *out;
  int32_t dt;
  int64_t at, ld;   // the tile's first element, and a row's length
  int64_t rows, cols;  // of the tile that exist
};
__device__ __forceinline__ TileOut tile_out(const TileWork &w, int ta, int tb, const void *base, void *out, int32_t dt,
                                            int64_t rows, int64_t cols, void *ws) {
  if (w.slot >= 0) return TileOut{nullptr, ws, kF32, w.slot * ta * tb, ta, tb, ta};
  const int64_t r = static_cast<int64_t>(w.b) * tb, c = static_cast<int64_t>(w.a) * ta;
  return TileOut{base, out, dt, r * cols + c, cols, rows - r, cols - c};
}

// R runs of N (4 or 8) consecutive elements of base, `step` apart, all loads
// before the first use.
template <int N, int R>
__device__ __forceinline__ void load_runs(const void *base, int32_t dt, int64_t at, int step, float (&v)[R][N]) {
  if (dt == kF32) {
    f32x4 w[R][N / 4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < N / 4; ++h) w[r][h] = *(const g_f32x4_at4 *)(static_cast<const float *>(base) + at + r * step + 4 * h);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < N; ++k) v[r][k] = w[r][k / 4][k % 4];
  } else {
    u32x2 w[R][N / 4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < N / 4; ++h)
        w[r][h] = *(const g_u32x2_at2 *)(static_cast<const uint16_t *>(base) + at + r * step + 4 * h);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        v[r][2 * k] = __uint_as_float(w[r][k / 2][k % 2] << 16);
        v[r][2 * k + 1] = __uint_as_float(w[r][k / 2][k % 2] & 0xffff0000u);
      }
  }
}

// N (4 or 8) consecutive outputs, plus base where there is one; `left` of them
// exist.  Vector accesses at any element's address (8192 rows x 4095 bf16 outputs
// of 512 codes each: 34 us, element by element 83); base may be out.
template <int N>
__device__ __forceinline__ void finish_run(const void *base, void *out, int32_t dt, int64_t at, int64_t left,
                                           float (&v)[N]) {
  if (left >= N) {
    if (dt == kF32) {
      if (base) {
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
          const f32x4 b = *(const g_f32x4_at4 *)(static_cast<const float *>(base) + at + 4 * h);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[4 * h + k] += b[k];
        }
      }
#pragma unroll
      for (int h = 0; h < N / 4; ++h)
        *(g_f32x4_at4 *)(static_cast<float *>(out) + at + 4 * h) = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    } else {
      if (base) {
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
          const u32x2 b = *(const g_u32x2_at2 *)(static_cast<const uint16_t *>(base) + at + 4 * h);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            v[4 * h + 2 * k] += __uint_as_float(b[k] << 16);
            v[4 * h + 2 * k + 1] += __uint_as_float(b[k] & 0xffff0000u);
          }
        }
      }
      uint32_t u[N / 2];
#pragma unroll
      for (int k = 0; k < N / 2; ++k)
        u[k] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * k])) |
               (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * k + 1])) << 16);
      if constexpr (N == 8)
        *(g_u32x4_at2 *)(static_cast<uint16_t *>(out) + at) = u32x4{u[0], u[1], u[2], u[3]};
      else
        *(g_u32x2_at2 *)(static_cast<uint16_t *>(out) + at) = u32x2{u[0], u[1]};
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < left) store_elem(out, dt, at + k, base ? load_elem(base, dt, at + k) + v[k] : v[k]);
  }
}

}  // namespace dmuon
