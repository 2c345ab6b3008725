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

#include <algorithm>

#include "q4_internal.h"
#include "q8_device.h"

namespace dmuon {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;

// The scale byte of a block whose largest magnitude has these fp32 bits.
__device__ __forceinline__ int scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return kQ4Nan;
  const int e = static_cast<int>(amax >> 23) - 127 - 2 + ((amax & 0x7fffffu) > 0x400000u ? 1 : 0);
  return min(max(e, kQ4MinExp), kQ4MaxExp) + 127;
}

// 2^e as fp32, for a scale byte e + 127 of the format (a normal number); infinity
// for kQ4Nan, with which every conversion from a code gives NaN.
__device__ __forceinline__ float scale_of(int byte) { return __uint_as_float(static_cast<uint32_t>(byte) << 23); }

// |v| * 2^-e rounded by a random byte: up iff the part of a step that is left is
// at least (255.5 - n) / 256, so by n + 0.5 of 256 equally likely cases.  All of
// it is exact in fp32.
__device__ __forceinline__ uint32_t random_code(float v, float inv, uint32_t n) {
  const float a = __builtin_fabsf(v) * inv;
  const float per = a < 2.f ? 2.f : a < 4.f ? 1.f : 0.5f;  // codes per unit
  const float at = a * per, whole = __builtin_floorf(at);
  // codes below 2, 4 and 6: 0 .. 3, 4 and 5, 6 and 7
  const uint32_t first = a < 2.f ? 0u : a < 4.f ? 2u : 4u;
  const uint32_t up = at - whole >= (255.5f - static_cast<float>(n)) * 0.00390625f ? 1u : 0u;
  return (static_cast<uint32_t>(whole) + first + up) | (__float_as_uint(v) >> 31 << 3);
}

// The codes of eight elements, the first in the lowest four bits.
template <bool RANDOM>
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], int byte, const uint8_t (&n)[8]) {
  if (byte == kQ4Nan) return 0;
  uint32_t w = 0;
  if constexpr (RANDOM) {
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k) w |= random_code(v[k], inv, n[k]) << (4 * k);
  } else {
    const float s = scale_of(byte);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
  }
  return w;
}

// The larger of this lane's value and that of the lane DPP control CTRL names.
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true)));
}
// ... over the four lanes of a quad
__device__ __forceinline__ uint32_t quad_max(uint32_t v) { return max_dpp<0x4e>(max_dpp<0xb1>(v)); }
// ... over the lanes l, l + 4, l + 8 and l + 12 of a row of 16 (rotations by 4 and 8)
__device__ __forceinline__ uint32_t stride4_max(uint32_t v) { return max_dpp<0x128>(max_dpp<0x124>(v)); }

// Eight scale bytes as two words.
__device__ __forceinline__ u32x2 pack8(const int (&b)[8]) {
  u32x2 w = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k / 4] |= static_cast<uint32_t>(b[k]) << (8 * (k % 4));
  return w;
}

// One tile of 128 x 128.  A lane holds an 8 x 8 patch; a quad's lanes lie side by
// side along a row (a row's block of 32), the lanes 4 apart of a row of 16 below
// each other (a column's block), the four rows of 16 cover 128 columns and the
// four waves 128 rows.
template <bool F32, bool RANDOM>
__device__ __forceinline__ void quantise_tile(const Q4Batch &b, int32_t mi, int64_t tile) {
  const int64_t rows = b.rows[mi], cols = b.cols[mi];
  const int64_t kp = (cols + kQ4Pad - 1) / kQ4Pad * kQ4Pad, rp = (rows + kQ4Pad - 1) / kQ4Pad * kQ4Pad;
  const int64_t r16 = (rows + kQ4ScaleRow - 1) / kQ4ScaleRow * kQ4ScaleRow;
  const int64_t c16 = (cols + kQ4ScaleRow - 1) / kQ4ScaleRow * kQ4ScaleRow;
  uint8_t *const codes = b.codes[mi], *const codes_t = b.codes_t[mi];
  const int64_t tc = ((codes ? kp : c16) + kTile - 1) / kTile;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r0 = tile / tc * kTile + wave * 32 + (lane >> 2 & 3) * 8;
  const int64_t c0 = tile % tc * kTile + (lane >> 4) * 32 + (lane & 3) * 8;
  float v[8][8];
  uint8_t n[8][8] = {};
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool is = r0 + r < rows && c0 + k < cols;
      const int64_t at = (r0 + r) * cols + c0 + k;
      v[r][k] = is ? load_elem(b.x[mi], F32 ? kF32 : kBF16, at) : 0.f;
      if constexpr (RANDOM) n[r][k] = is ? ((const g_u8 *)b.random[mi])[at] : 0;
    }
  if (codes) {
    int bytes[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint32_t a = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) a = max(a, __float_as_uint(v[r][k]) & 0x7fffffffu);
      bytes[r] = scale_byte(quad_max(a));
      if (r0 + r < rows && c0 < kp) *(g_u32 *)(codes + (r0 + r) * (kp / 2) + c0 / 2) = codes8<RANDOM>(v[r], bytes[r], n[r]);
    }
    if ((lane & 3) == 0 && r0 < r16 && c0 < kp) *(g_u32x2 *)(b.scales[mi] + c0 / kQ4Block * r16 + r0) = pack8(bytes);
  }
  if (codes_t) {
    int bytes[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float col[8];
      uint8_t nc[8];
      uint32_t a = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        col[r] = v[r][k];
        nc[r] = n[r][k];
        a = max(a, __float_as_uint(col[r]) & 0x7fffffffu);
      }
      bytes[k] = scale_byte(stride4_max(a));
      if (c0 + k < cols && r0 < rp) *(g_u32 *)(codes_t + (c0 + k) * (rp / 2) + r0 / 2) = codes8<RANDOM>(col, bytes[k], nc);
    }
    if ((lane & 12) == 0 && c0 < c16 && r0 < rp) *(g_u32x2 *)(b.scales_t[mi] + r0 / kQ4Block * c16 + c0) = pack8(bytes);
  }
}

__global__ __launch_bounds__(kThreads) void q4_quantise_kernel(Q4Batch b) {
  const int64_t w = blockIdx.x;
  const int32_t mi = find_range(b.n, w, [&](int32_t i) { return b.first_tile[i]; });
  const int64_t tile = w - b.first_tile[mi];
  if (b.random[mi]) {
    if (b.dt[mi] == kF32)
      quantise_tile<true, true>(b, mi, tile);
    else
      quantise_tile<false, true>(b, mi, tile);
  } else {
    if (b.dt[mi] == kF32)
      quantise_tile<true, false>(b, mi, tile);
    else
      quantise_tile<false, false>(b, mi, tile);
  }
}

// Values of codes.  A work-group takes 256 columns (32 lanes of 8 codes) of 32
// rows, so that the lines of the scale table it touches serve them all.  Every
// code times its scale is a bf16 number, but for 4 * 2^126, which the largest
// values round to and which becomes infinite.
__global__ __launch_bounds__(kThreads) void q4_dequantise_kernel(const uint8_t *__restrict__ codes,
                                                                 const uint8_t *__restrict__ scales, int64_t rows,
                                                                 int64_t cols, void *__restrict__ out, int32_t dt) {
  const int64_t kp = (cols + kQ4Pad - 1) / kQ4Pad * kQ4Pad;
  const int64_t r16 = (rows + kQ4ScaleRow - 1) / kQ4ScaleRow * kQ4ScaleRow;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + (threadIdx.x & 31) * 8;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x >> 5);
  if (c >= cols) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 8 * i;
    if (r >= rows) return;
    const uint32_t w = *(const g_u32 *)(codes + r * (kp / 2) + c / 2);
    const float s = scale_of(((const g_u8 *)scales)[c / kQ4Block * r16 + r]);
    bf16x2 p[4];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = static_cast<float>(p[k].x);
      v[2 * k + 1] = static_cast<float>(p[k].y);
    }
    finish_run<8>(nullptr, out, dt, r * cols + c, cols - c, v);
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
  hipLaunchKernelGGL(q4_quantise_kernel, dim3(static_cast<uint32_t>(b.first_tile[b.n])), dim3(kThreads), 0, st, b);
  return hipGetLastError();
}

hipError_t launch_q4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *out,
                                int32_t dt, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>((rows + 31) / 32), static_cast<uint32_t>((cols + 255) / 256));
  hipLaunchKernelGGL(q4_dequantise_kernel, grid, dim3(kThreads), 0, st, codes, scales, rows, cols, out, dt);
  return hipGetLastError();
}

}  // namespace dmuon
