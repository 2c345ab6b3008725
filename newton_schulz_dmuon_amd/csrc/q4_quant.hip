// Quantisation to the 4-bit block format on gfx950, and back: E2M1 codes, two to
// a byte, and one power-of-two scale 2^e per block of 32 along the direction
// that a product will sum over.
//
// e is the smallest integer with max|block| <= 6 * 2^e, clamped to [kQ4MinExp,
// kQ4MaxExp].  6 = 1.5 * 2^2, so with max = m * 2^p (1 <= m < 2) e = p - 2, or
// p - 1 when m > 1.5: read off the fp32 bits of the maximum, with no logarithm.
// No value saturates, so rounding by random bytes has no bias at the top.  A code
// is the value times 2^-e (exact: a power of two) rounded once, to nearest even
// or by the element's random byte.  A block with a NaN or an infinity, which no
// code stands for, gets the scale byte 255, which the matrix instruction reads as
// NaN, and zero codes.
//
// Bound by memory: 8192 x 4096 bf16 in both forms reads 67 and writes 36 MB in 24.8
// us (4.1 TB/s; a large copy 5.0), fp32 40 us, a list of matrices of 218 M elements
// 164 us (4.1 TB/s).  Rounding by random bytes is bound by the vector ALUs (busy 87%
// of the time): 36 to 39 us in both forms (41 with the scale always in two factors), 28
// in one.  One row 3.9 us, a launch's latency.

#include <algorithm>
#include <type_traits>

#include "q4_internal.h"
#include "q8_device.h"

namespace dmuon {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;
// Rows read back per launch: its threads along the grid stay below 2^32.
constexpr int64_t kLaunchRows = int64_t(1) << 28;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
// eight bytes at any address
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));
typedef __attribute__((address_space(1))) u32x2_at1 g_u32x2_at1;
typedef u32x2 u32x2_at4 __attribute__((aligned(4)));
typedef __attribute__((address_space(1))) u32x2_at4 g_u32x2_at4;

// The scale byte of a block whose largest magnitude has these fp32 bits.
__device__ __forceinline__ int scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return kQ4Nan;
  const int e = static_cast<int>(amax >> 23) - 127 - 2 + ((amax & 0x7fffffu) > 0x400000u ? 1 : 0);
  return min(max(e, kQ4MinExp), kQ4MaxExp) + 127;
}

// 2^e as fp32, for a scale byte e + 127 of the format (a normal number); infinity
// for kQ4Nan, with which every conversion from a code gives NaN.
__device__ __forceinline__ float scale_of(int byte) { return __uint_as_float(static_cast<uint32_t>(byte) << 23); }

// Eight elements as loaded: four words of bf16 pairs, or eight of fp32.
template <bool F32> struct Eight {
  uint32_t w[F32 ? 8 : 4];
  // at any element's address, all loads before the first use
  __device__ __forceinline__ void load(const void *x, int64_t i) {
    if constexpr (F32) {
      const u32x4 a = *(const g_u32x4_at4 *)(static_cast<const float *>(x) + i);
      const u32x4 b = *(const g_u32x4_at4 *)(static_cast<const float *>(x) + i + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = a[k];
        w[4 + k] = b[k];
      }
    } else {
      const u32x4 a = *(const g_u32x4_at2 *)(static_cast<const uint16_t *>(x) + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = a[k];
    }
  }
  // element by element, each at its own place; elements `left` on are zero
  template <typename P>
  __device__ __forceinline__ void load_each(const void *x, P place, int64_t left) {
    uint32_t e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if constexpr (F32)
        e[k] = ((const g_u32 *)x)[place(k)];
      else
        e[k] = ((const g_u16 *)x)[place(k)];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = k < left ? e[k] : 0;
#pragma unroll
    for (int k = 0; k < (F32 ? 8 : 4); ++k) w[k] = F32 ? e[k] : e[2 * k % 8] | e[(2 * k + 1) % 8] << 16;
  }
  __device__ __forceinline__ void zero_unless(bool is) {
#pragma unroll
    for (int k = 0; k < (F32 ? 8 : 4); ++k) w[k] = is ? w[k] : 0;
  }
};

// Magnitudes as ordered bits: fp32's, or two bf16's in the halves of a word.
template <bool F32> __device__ __forceinline__ uint32_t magnitude(uint32_t w) { return w & (F32 ? 0x7fffffffu : 0x7fff7fffu); }
template <bool F32> __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  if constexpr (F32) return max(a, b);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// The larger of this lane's value and that of the lane DPP control CTRL names.
template <bool F32, int CTRL>
__device__ __forceinline__ uint32_t larger_dpp(uint32_t v) {
  return larger<F32>(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true)));
}
// ... over the four lanes of a quad
template <bool F32> __device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  return larger_dpp<F32, 0x4e>(larger_dpp<F32, 0xb1>(v));
}
// ... over the lanes l, l + 4, l + 8 and l + 12 of a row of 16 (rotations by 4 and 8)
template <bool F32> __device__ __forceinline__ uint32_t stride4_max(uint32_t v) {
  return larger_dpp<F32, 0x128>(larger_dpp<F32, 0x124>(v));
}

// Two values times 2^-e rounded by their random bytes n: in units of 2^-10, of which
// a step between codes has 512, 1024 or 2048 (values below 2, 4 and 6), up iff what
// lies above the code below is at least 255.5 - n of 256 parts.  Cutting a value to
// whole units changes no comparison, since every threshold is a whole number of
// them.  more * unit: 2^(10 - e), in two factors where fp32 does not hold it.
template <bool TINY>
__device__ __forceinline__ u16x2 random_codes(float a, float b, float more, float unit, u16x2 n) {
  const float x = TINY ? __builtin_fabsf(a) * more : __builtin_fabsf(a);
  const float y = TINY ? __builtin_fabsf(b) * more : __builtin_fabsf(b);
  const u16x2 u = {static_cast<unsigned short>(static_cast<uint32_t>(x * unit)),
                   static_cast<unsigned short>(static_cast<uint32_t>(y * unit))};
  const u16x2 wide = __builtin_elementwise_min(u >> 11, u16x2{2, 2});
  return ((u + ((n + n + 1) << wide)) >> (wide + 9)) + (wide + wide);
}

// Four pairs of elements, as the halves of a word in bf16 or as two words in fp32.
template <bool F32> struct Pairs {
  uint32_t w[F32 ? 8 : 4];
  __device__ __forceinline__ float get(int k) const {
    if constexpr (F32) return __uint_as_float(w[k % 8]);
    return __uint_as_float(k % 2 ? w[k / 2 % 4] & 0xffff0000u : w[k / 2 % 4] << 16);
  }
};

// The codes of eight elements, the first in the lowest four bits.  n(k): the random
// bytes of pair k, in the halves of a word.  Without TINY byte is at least kTinyByte.
constexpr int kTinyByte = 10;
template <bool F32, bool RANDOM, bool TINY, typename N>
__device__ __forceinline__ uint32_t codes8(const Pairs<F32> &x, int byte, N n) {
  uint32_t w = 0;
  if constexpr (RANDOM) {
    const float unit = __uint_as_float(static_cast<uint32_t>(min(264 - byte, 254)) << 23);
    const float more = __uint_as_float(static_cast<uint32_t>(127 + max(kTinyByte - byte, 0)) << 23);
    uint32_t two[4];  // a pair's two codes in the lowest byte
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t c = __builtin_bit_cast(
          uint32_t, random_codes<TINY>(x.get(2 * k), x.get(2 * k + 1), more, unit, __builtin_bit_cast(u16x2, n(k))));
      const uint32_t sign = F32 ? __builtin_amdgcn_perm(x.w[(2 * k + 1) % (F32 ? 8 : 4)], x.w[2 * k % (F32 ? 8 : 4)], 0x07060302u)
                                : x.w[k];  // in bits 15 and 31
      const uint32_t s = (sign >> 12 & 0x00080008u) | c;
      two[k] = s | s >> 12;
    }
    w = __builtin_amdgcn_perm(__builtin_amdgcn_perm(two[3], two[2], 0x0c0c0400u),
                              __builtin_amdgcn_perm(two[1], two[0], 0x0c0c0400u), 0x05040100u);
  } else if constexpr (F32) {
    const float s = scale_of(byte);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x.get(0), x.get(1), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x.get(2), x.get(3), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x.get(4), x.get(5), s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x.get(6), x.get(7), s, 3);
  } else {
    const float s = scale_of(byte);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.w[0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.w[1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.w[2]), s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.w[3]), s, 3);
  }
  return byte == kQ4Nan ? 0u : w;
}

// Eight bytes from `at` on, of eight rows `step` apart.  Loads at any byte's address
// are slow (8192 x 4095 elements 61 us): whole words are loaded and shifted, where
// none of a wave's lies behind the `size` bytes.  The branch is the wave's: where each
// lane took its own, the built code lost the elements that lanes of the first side
// had loaded before.
__device__ __forceinline__ void load_bytes(const uint8_t *p, int64_t at, int64_t step, int64_t size, u32x2 (&n)[8]) {
  const bool behind = at + 7 * step + 12 > size;
  if (((step & 7) == 0) | (__builtin_amdgcn_ballot_w64(behind) != 0)) {
#pragma unroll
    for (int r = 0; r < 8; ++r) n[r] = *(const g_u32x2_at1 *)(p + at + r * step);
    return;
  }
  u32x2 lo[8];
  uint32_t hi[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int64_t word = (at + r * step) & ~int64_t(3);
    lo[r] = *(const g_u32x2_at4 *)(p + word);
    hi[r] = *(const g_u32 *)(p + word + 8);
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const uint32_t shift = static_cast<uint32_t>(at + r * step) & 3;
    n[r] = u32x2{__builtin_amdgcn_alignbyte(lo[r].y, lo[r].x, shift), __builtin_amdgcn_alignbyte(hi[r], lo[r].y, shift)};
  }
}

// Whether rounding by random bytes takes its scale in two factors somewhere in the
// wave.
template <bool RANDOM> __device__ __forceinline__ bool any_tiny(const int (&b)[8]) {
  if (!RANDOM) return false;
  int least = b[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) least = min(least, b[k]);
  return __builtin_amdgcn_ballot_w64(least < kTinyByte) != 0;
}

// Eight scale bytes as two words.
__device__ __forceinline__ u32x2 pack8(const int (&b)[8]) {
  u32x2 w = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k / 4] |= static_cast<uint32_t>(b[k]) << (8 * (k % 4));
  return w;
}

// One tile of 128 x 128, which both forms read once.  A lane holds an 8 x 8 patch; a quad's lanes lie side by
// side along a row (a row's block of 32), the lanes 4 apart of a row of 16 below
// each other (a column's block), the four rows of 16 cover 128 columns and the
// four waves 128 rows.  Both directions' maxima are then taken by DPP alone.  The
// transposed codes leave through LDS, 64 bytes of a column at a time.  Patches at an
// edge take clamped places, all loads in flight at once (8192 x 4095 to nearest 33 us,
// with a load and a wait an element 42; by random bytes 51 and 89).
constexpr int kPitch = kTile / 2 + 4;  // bytes of a column in LDS

template <bool F32, bool RANDOM>
__device__ __forceinline__ void quantise_tile(const Q4Batch &b, int32_t mi, int64_t tile, char *smem) {
  const int64_t rows = b.rows[mi], cols = b.cols[mi];
  const int64_t kp = (cols + kQ4Pad - 1) / kQ4Pad * kQ4Pad, rp = (rows + kQ4Pad - 1) / kQ4Pad * kQ4Pad;
  const int64_t r16 = (rows + kQ4ScaleRow - 1) / kQ4ScaleRow * kQ4ScaleRow;
  const int64_t c16 = (cols + kQ4ScaleRow - 1) / kQ4ScaleRow * kQ4ScaleRow;
  uint8_t *const codes = b.codes[mi], *const codes_t = b.codes_t[mi];
  const uint32_t tc = static_cast<uint32_t>(((codes ? kp : c16) + kTile - 1) / kTile);
  const uint32_t ti = uniform(static_cast<uint32_t>(tile) / tc), tj = uniform(static_cast<uint32_t>(tile) - ti * tc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rl = wave * 32 + (lane >> 2 & 3) * 8, cl = (lane >> 4) * 32 + (lane & 3) * 8;
  const int64_t r0 = static_cast<int64_t>(ti) * kTile + rl, c0 = static_cast<int64_t>(tj) * kTile + cl;
  Eight<F32> x[8];
  u32x2 n[8];
  if (r0 + 8 <= rows && c0 + 8 <= cols) {
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r].load(b.x[mi], (r0 + r) * cols + c0);
    if constexpr (RANDOM) load_bytes(b.random[mi], r0 * cols + c0, cols, rows * cols, n);
  } else if (c0 + 8 <= cols) {
    // rows behind the last: the last one's elements, then zeros
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r].load(b.x[mi], min(r0 + r, rows - 1) * cols + c0);
    if constexpr (RANDOM)
#pragma unroll
      for (int r = 0; r < 8; ++r) n[r] = *(const g_u32x2_at1 *)(b.random[mi] + min(r0 + r, rows - 1) * cols + c0);
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r].zero_unless(r0 + r < rows);
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int64_t row = min(r0 + r, rows - 1) * cols;
      auto place = [&](int k) { return row + min(c0 + k, cols - 1); };
      x[r].load_each(b.x[mi], place, r0 + r < rows ? cols - c0 : 0);
      if constexpr (RANDOM) {
        n[r] = u32x2{0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k) n[r][k / 4] |= static_cast<uint32_t>(((const g_u8 *)b.random[mi])[place(k)]) << (8 * (k % 4));
      }
    }
  }
  constexpr int W = F32 ? 8 : 4;
  uint32_t col_max[W];
#pragma unroll
  for (int k = 0; k < W; ++k) col_max[k] = 0;
  int bytes[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    uint32_t a = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const uint32_t m = magnitude<F32>(x[r].w[k]);
      a = larger<F32>(a, m);
      col_max[k] = larger<F32>(col_max[k], m);
    }
    a = quad_max<F32>(a);
    bytes[r] = scale_byte(F32 ? a : max(a << 16, a & 0xffff0000u));
  }
  if (codes) {
    auto write_rows = [&](auto tiny) {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        Pairs<F32> v;
#pragma unroll
        for (int k = 0; k < W; ++k) v.w[k] = x[r].w[k];
        // bytes 2 k and 2 k + 1 of the row's
        const uint32_t w = codes8<F32, RANDOM, tiny>(v, bytes[r], [&](int k) {
          return __builtin_amdgcn_perm(0, n[r][k / 2], k % 2 ? 0x0c030c02u : 0x0c010c00u);
        });
        if (r0 + r < rows && c0 < kp) *(g_u32 *)(codes + (r0 + r) * (kp / 2) + c0 / 2) = w;
      }
    };
    if (any_tiny<RANDOM>(bytes))
      write_rows(std::true_type{});
    else
      write_rows(std::false_type{});
    if ((lane & 3) == 0 && r0 < r16 && c0 < kp) *(g_u32x2 *)(b.scales[mi] + c0 / kQ4Block * r16 + r0) = pack8(bytes);
  }
  if (!codes_t) return;
  lds_char *const lds = (lds_char *)smem;
#pragma unroll
  for (int k = 0; k < W; ++k) col_max[k] = stride4_max<F32>(col_max[k]);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    bytes[k] = scale_byte(F32 ? col_max[k % W] : k % 2 ? col_max[k / 2 % W] & 0xffff0000u : col_max[k / 2 % W] << 16);
  auto put_columns = [&](auto tiny) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      Pairs<F32> v;
#pragma unroll
      for (int r = 0; r < W; ++r) {
        if constexpr (F32)
          v.w[r] = x[r].w[k];
        else
          v.w[r] = __builtin_amdgcn_perm(x[2 * r + 1].w[k / 2], x[2 * r].w[k / 2], k % 2 ? 0x07060302u : 0x05040100u);
      }
      // byte k of two rows'
      *(lds_u32 *)(lds + (cl + k) * kPitch + rl / 2) = codes8<F32, RANDOM, tiny>(v, bytes[k], [&](int q) {
        return __builtin_amdgcn_perm(n[2 * q + 1][k / 4], n[2 * q][k / 4], 0x0c040c00u + (k % 4) * 0x00010001u);
      });
    }
  };
  if (any_tiny<RANDOM>(bytes))
    put_columns(std::true_type{});
  else
    put_columns(std::false_type{});
  if ((lane & 12) == 0 && c0 < c16 && r0 < rp) *(g_u32x2 *)(b.scales_t[mi] + r0 / kQ4Block * c16 + c0) = pack8(bytes);
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = h * 64 + static_cast<int>(threadIdx.x >> 2), at = (threadIdx.x & 3) * 16;
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = *(const lds_u32 *)(lds + c * kPitch + at + 4 * k);
    const int64_t col = static_cast<int64_t>(tj) * kTile + c, row = static_cast<int64_t>(ti) * kTile + 2 * at;
    if (col < cols && row < rp) *(g_u32x4 *)(codes_t + col * (rp / 2) + row / 2) = w;
  }
}

template <bool F32, bool RANDOM>
__global__ __launch_bounds__(kThreads) void q4_quantise_kernel(Q4Batch b) {
  __shared__ __align__(16) char smem[kTile * kPitch];
  const int64_t w = blockIdx.x;
  const int32_t mi = find_range(b.n, w, [&](int32_t i) { return b.first_tile[i]; });
  quantise_tile<F32, RANDOM>(b, mi, w - b.first_tile[mi], smem);
}

template <bool F32, bool RANDOM>
hipError_t launch_quantise(const Q4Batch &b, hipStream_t st) {
  hipLaunchKernelGGL((q4_quantise_kernel<F32, RANDOM>), dim3(static_cast<uint32_t>(b.first_tile[b.n])), dim3(kThreads),
                     0, st, b);
  return hipGetLastError();
}

// Values of codes.  A work-group takes 256 columns (32 lanes of 8 codes) of 32
// rows, so that the lines of the scale table it touches serve them all (8192 x 4096 to
// bf16 21.5 us, 4.0 TB/s; 13.6 out of the memory-side cache).  Every
// code times its scale is a bf16 number, but for 4 * 2^126, which the largest
// values round to and which becomes infinite.
template <bool F32>
__global__ __launch_bounds__(kThreads) void q4_dequantise_kernel(const uint8_t *__restrict__ codes,
                                                                 const uint8_t *__restrict__ scales, int64_t first,
                                                                 int64_t rows, int64_t cols, void *__restrict__ out) {
  const int64_t kp = (cols + kQ4Pad - 1) / kQ4Pad * kQ4Pad;
  const int64_t r16 = (rows + kQ4ScaleRow - 1) / kQ4ScaleRow * kQ4ScaleRow;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + (threadIdx.x & 31) * 8;
  const int64_t r0 = first + static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x >> 5);
  if (c >= cols) return;
  uint32_t w[4];
  int byte[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = min(r0 + 8 * i, rows - 1);
    w[i] = *(const g_u32 *)(codes + r * (kp / 2) + c / 2);
    byte[i] = ((const g_u8 *)scales)[c / kQ4Block * r16 + r];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 8 * i;
    if (r >= rows) return;
    const float s = scale_of(byte[i]);
    u32x4 p;
    p.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 0));
    p.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 1));
    p.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 2));
    p.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 3));
    const int64_t at = r * cols + c;
    if (!F32 && c + 8 <= cols) {
      *(g_u32x4_at2 *)(static_cast<uint16_t *>(out) + at) = p;
      continue;
    }
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(k % 2 ? p[k / 2] & 0xffff0000u : p[k / 2] << 16);
    finish_run<8>(nullptr, out, F32 ? kF32 : kBF16, at, cols - c, v);
  }
}

// Codes and scales whose bytes lie apart, copied to where a product's loads find them:
// out[r][c] = src[r * row_step + c * col_step].  128 x 128 bytes a work-group, in 4 x 4
// patches turned in registers and, through LDS, written 16 bytes a lane.  With WORDS
// the rows of a column are consecutive (a transposed view) and whole words are loaded,
// otherwise bytes.  Bound by memory: 14336 x 4096 transposed bytes, 59 MB read and
// written, 24 us (4.9 TB/s, a large copy's rate).
constexpr int kCopyTile = 128, kCopyPitch = kCopyTile / 4 + 1;  // words of a row in LDS

template <bool WORDS>
__global__ __launch_bounds__(kThreads) void q4_copy_kernel(const uint8_t *__restrict__ src, int64_t rows, int64_t cols,
                                                           int64_t row_step, int64_t col_step,
                                                           uint8_t *__restrict__ out) {
  __shared__ __align__(16) char smem[kCopyTile * kCopyPitch * 4];
  lds_char *const lds = (lds_char *)smem;
  const uint32_t across = static_cast<uint32_t>((cols + kCopyTile - 1) / kCopyTile);
  const uint32_t ti = uniform(blockIdx.x / across), tj = uniform(blockIdx.x - ti * across);
  const int64_t r0 = static_cast<int64_t>(ti) * kCopyTile, c0 = static_cast<int64_t>(tj) * kCopyTile;
  const bool along_rows = row_step <= col_step;  // the direction of a wave's lanes
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = i * kThreads + static_cast<int>(threadIdx.x), fast = q & 31, slow = q >> 5;
    const int pr = along_rows ? fast : slow, pc = along_rows ? slow : fast;
    const int64_t r = r0 + 4 * pr;
    uint32_t w[4];  // four rows' bytes of a column; behind the last row and column those of the last
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint8_t *const p = src + min(c0 + 4 * pc + k, cols - 1) * col_step;
      if (WORDS && r + 4 <= rows) {
        w[k] = *(const g_u32 *)(p + r);
        continue;
      }
      w[k] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        w[k] |= static_cast<uint32_t>(((const g_u8 *)p)[min(r + b, rows - 1) * row_step]) << (8 * b);
    }
    const uint32_t lo01 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), lo23 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
    const uint32_t hi01 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), hi23 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    const uint32_t row[4] = {__builtin_amdgcn_perm(lo23, lo01, 0x05040100u), __builtin_amdgcn_perm(lo23, lo01, 0x07060302u),
                             __builtin_amdgcn_perm(hi23, hi01, 0x05040100u), __builtin_amdgcn_perm(hi23, hi01, 0x07060302u)};
#pragma unroll
    for (int b = 0; b < 4; ++b) *(lds_u32 *)(lds + ((4 * pr + b) * kCopyPitch + pc) * 4) = row[b];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = i * kThreads + static_cast<int>(threadIdx.x), r = q >> 3, c = (q & 7) * 16;
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = *(const lds_u32 *)(lds + r * kCopyPitch * 4 + c + 4 * k);
    if (r0 + r < rows && c0 + c < cols) *(g_u32x4 *)(out + (r0 + r) * cols + c0 + c) = w;
  }
}

int64_t up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }

}  // namespace

int64_t q4_tiles(int64_t rows, int64_t cols, bool plain, bool transposed) {
  const int64_t r = transposed ? up(rows, kQ4Pad) : up(rows, kQ4ScaleRow);
  const int64_t c = plain ? up(cols, kQ4Pad) : up(cols, kQ4ScaleRow);
  return up(r, kTile) / kTile * (up(c, kTile) / kTile);
}

hipError_t launch_q4_quantize(const Q4Batch &b, hipStream_t st) {
  if (b.n == 0) return hipSuccess;
  if (b.random[0]) return b.dt == kF32 ? launch_quantise<true, true>(b, st) : launch_quantise<false, true>(b, st);
  return b.dt == kF32 ? launch_quantise<true, false>(b, st) : launch_quantise<false, false>(b, st);
}

hipError_t launch_q4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *out,
                                int32_t dt, hipStream_t st) {
  for (int64_t first = 0; first < rows; first += kLaunchRows) {
    const int64_t here = std::min(rows - first, kLaunchRows);
    const dim3 grid(static_cast<uint32_t>((here + 31) / 32), static_cast<uint32_t>((cols + 255) / 256));
    if (dt == kF32)
      hipLaunchKernelGGL(q4_dequantise_kernel<true>, grid, dim3(kThreads), 0, st, codes, scales, first, rows, cols, out);
    else
      hipLaunchKernelGGL(q4_dequantise_kernel<false>, grid, dim3(kThreads), 0, st, codes, scales, first, rows, cols, out);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_q4_copy(const uint8_t *src, int64_t rows, int64_t cols, int64_t row_step, int64_t col_step,
                          uint8_t *out, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(up(rows, kCopyTile) / kCopyTile * (up(cols, kCopyTile) / kCopyTile)));
  const bool words = row_step == 1 && col_step % 4 == 0 && reinterpret_cast<uintptr_t>(src) % 4 == 0;
  if (words)
    hipLaunchKernelGGL(q4_copy_kernel<true>, grid, dim3(kThreads), 0, st, src, rows, cols, row_step, col_step, out);
  else
    hipLaunchKernelGGL(q4_copy_kernel<false>, grid, dim3(kThreads), 0, st, src, rows, cols, row_step, col_step, out);
  return hipGetLastError();
}

}  // namespace dmuon
