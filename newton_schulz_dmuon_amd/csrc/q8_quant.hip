// Quantisation to the 8-bit block format on gfx950: E4M3 codes and one
// power-of-two scale 2^e per block of 128.
//
// e is the smallest integer with max|block| <= 448 * 2^e, clamped to
// [kQ8MinExp, kQ8MaxExp].  448 = 1.75 * 2^8, so with max = m * 2^p (1 <= m <
// 2) e = p - 8, or p - 7 when m > 1.75: read off the fp32 bits of the maximum,
// with no logarithm.  A code is the value times 2^-e rounded to nearest even:
// the product is exact in fp32 (a power of two; where it falls below fp32's
// normal range it is far below the smallest code), so each code carries one
// rounding.  NaN and infinities take no part in the maximum and become the
// code NaN.
//
// Both kernels are one pass over the data and bound by HBM: every element is
// read once and every code written once.  16384 x 14336 bf16 rows take 133 us,
// 5.3 TB/s, and the 218 M bf16 elements of a Llama-3.1-8B layer's weights, with
// their transposed codes, 171 us, 5.1 TB/s; a large device copy reaches 4.9.

#include <algorithm>

#include "q8_device.h"

namespace dmuon {

namespace {

constexpr int kThreads = 256;
// Rows per launch: its threads along the grid stay below 2^32.
constexpr int64_t kLaunchRows = int64_t(1) << 24;

// |v| as ordered bits, 0 for NaN and infinities.
__device__ __forceinline__ uint32_t finite_magnitude(float v) {
  const uint32_t a = __float_as_uint(v) & 0x7fffffffu;
  return a < 0x7f800000u ? a : 0u;
}

// The scale byte e + 127 of a block whose largest finite magnitude has these
// bits.
__device__ __forceinline__ int scale_byte(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kQ8MinExp), kQ8MaxExp) + 127;
}

// 2^-e as fp32, for the scale byte e + 127 (e within the format's range, so
// the power is a normal number).
__device__ __forceinline__ float inverse_scale(int byte) {
  return __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
}

// A value's scaled form; infinities become NaN, which the conversion keeps.
__device__ __forceinline__ float scaled(float v, float inv) {
  return (__float_as_uint(v) & 0x7fffffffu) < 0x7f800000u ? v * inv : __uint_as_float(0x7fc00000u);
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(a, inv), scaled(b, inv), 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(scaled(c, inv), scaled(d, inv), r, true));
}

// Eight consecutive elements as loaded, so that several loads can be in flight
// before the first is used.  The address is that of any element: global loads of
// 16 bytes need no more (8192 x 4097 bf16 rows 22 us, element by element 51; a
// 8001 x 7999 bf16 weight 59 us and 119).
template <bool F32> struct Raw8;
template <> struct Raw8<false> {
  u32x4 a;
  __device__ __forceinline__ void load(const void *x, int64_t i) {
    a = *(const g_u32x4_at2 *)(static_cast<const uint16_t *>(x) + i);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(a[k] << 16);
      v[2 * k + 1] = __uint_as_float(a[k] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<true> {
  u32x4 a, b;
  __device__ __forceinline__ void load(const void *x, int64_t i) {
    a = *(const g_u32x4_at4 *)(static_cast<const float *>(x) + i);
    b = *(const g_u32x4_at4 *)(static_cast<const float *>(x) + i + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = __uint_as_float(a[k]);
      v[4 + k] = __uint_as_float(b[k]);
    }
  }
};

// Eight columns from c on of N consecutive rows from t on: all loads first
// where every element exists, else row by row with zeros for those that do
// not.  (8192 x 4096 bf16 rows: 20.4 us so, 24 row by row.)
template <bool F32, int N>
__device__ __forceinline__ void load_patch(const void *x, int64_t t, int64_t c, int64_t rows, int64_t cols,
                                           float (&v)[N][8]) {
  if (c + 8 <= cols && t + N <= rows) {
    Raw8<F32> raw[N];
#pragma unroll
    for (int r = 0; r < N; ++r) raw[r].load(x, (t + r) * cols + c);
#pragma unroll
    for (int r = 0; r < N; ++r) raw[r].get(v[r]);
  } else {
#pragma unroll
    for (int r = 0; r < N; ++r) {
      const int64_t left = t + r < rows ? cols - c : 0;
      if (left >= 8) {
        Raw8<F32> raw;
        raw.load(x, (t + r) * cols + c);
        raw.get(v[r]);
        continue;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v[r][k] = k < left ? load_elem(x, F32 ? kF32 : kBF16, (t + r) * cols + c + k) : 0.f;
    }
  }
}

// Rows.  A wave takes 512 columns (4 blocks, 16 lanes of 8 elements each) of
// four consecutive rows: four loads in flight a lane, and the four scale bytes
// of a block's column, which one lane then holds, leave as one word of the
// [block][row] table.  Rows behind the last are zero rows (scale byte of a zero
// block).
template <bool F32>
__global__ __launch_bounds__(kThreads) void q8_rows_kernel(const void *__restrict__ x, int64_t first, int64_t rows,
                                                           int64_t cols, int64_t kp, uint8_t *__restrict__ codes,
                                                           uint8_t *__restrict__ scales, int64_t t4) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = first + static_cast<int64_t>(blockIdx.x) * 4;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 4 + wave) * 512 + lane * 8;
  if (c >= kp) return;
  float v[4][8];
  load_patch<F32, 4>(x, t, c, rows, cols, v);
  uint32_t bytes = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    uint32_t a = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) a = max(a, finite_magnitude(v[r][k]));
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), m)));
    const int byte = scale_byte(a);
    bytes |= static_cast<uint32_t>(byte) << (8 * r);
    if (t + r < rows) {
      const float inv = inverse_scale(byte);
      *(g_u32x2 *)(codes + (t + r) * kp + c) = u32x2{codes4(v[r][0], v[r][1], v[r][2], v[r][3], inv),
                                                     codes4(v[r][4], v[r][5], v[r][6], v[r][7], inv)};
    }
  }
  if ((lane & 15) == 0) *(g_u32 *)(scales + c / kQ8Block * t4 + t) = bytes;
}

// 4 x 4 byte transpose: r[i] holds bytes (i, 0..3); the result's word j holds
// bytes (0..3, j).
__device__ __forceinline__ void transpose4(const uint32_t (&r)[4], uint32_t (&o)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u);  // r0.0 r1.0 r0.1 r1.1
  const uint32_t b = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);  // r0.2 r1.2 r0.3 r1.3
  const uint32_t c = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
  o[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// Weights: one work-group per 128 x 128 block.  A thread holds an 8 x 8 patch
// (eight 16-byte loads in flight for bf16), so that the transposed codes are a
// byte transpose in registers and leave through LDS in whole rows.
template <bool F32>
__device__ __forceinline__ void q8_weight_block(const Q8WeightBatch &b, int32_t mi, int64_t blk, uint32_t *red,
                                                char *lds) {
  const int64_t rows = b.rows[mi], cols = b.cols[mi];
  const int64_t nb = (rows + kQ8Block - 1) / kQ8Block, kb = (cols + kQ8Block - 1) / kQ8Block;
  const int64_t bi = blk / kb, bj = blk % kb;
  const int64_t kp = kb * kQ8Block, np = nb * kQ8Block;
  const int tid = threadIdx.x;
  const int kc = tid & 15, ng = tid >> 4;  // patch: columns 8 kc, rows 8 ng
  const int64_t n0 = bi * kQ8Block + ng * 8, k0 = bj * kQ8Block + kc * 8;
  float v[8][8];
  load_patch<F32, 8>(b.param[mi], n0, k0, rows, cols, v);
  uint32_t a = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int k = 0; k < 8; ++k) a = max(a, finite_magnitude(v[r][k]));
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), m)));
  if ((tid & 63) == 0) red[tid >> 6] = a;
  __syncthreads();
  a = max(max(red[0], red[1]), max(red[2], red[3]));
  const int byte = scale_byte(a);
  const float inv = inverse_scale(byte);
  if (tid == 0) {
    ((g_u8 *)b.scales[mi])[bi * kb + bj] = static_cast<uint8_t>(byte);
    if (b.scales_t[mi]) ((g_u8 *)b.scales_t[mi])[bj * nb + bi] = static_cast<uint8_t>(byte);
  }
  uint32_t q[8][2];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    q[r][0] = codes4(v[r][0], v[r][1], v[r][2], v[r][3], inv);
    q[r][1] = codes4(v[r][4], v[r][5], v[r][6], v[r][7], inv);
    if (n0 + r < rows) *(g_u32x2 *)(b.codes[mi] + (n0 + r) * kp + k0) = u32x2{q[r][0], q[r][1]};
  }
  if (!b.codes_t[mi]) return;
  // LDS row k (128 bytes) holds the block's column k; its 8-byte chunk ng sits
  // at ng ^ kc, so that the 16 lanes of a row group write distinct chunks.
  lds_char *const l = (lds_char *)lds;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo[4] = {q[0][h], q[1][h], q[2][h], q[3][h]}, hi[4] = {q[4][h], q[5][h], q[6][h], q[7][h]};
    uint32_t tl[4], th[4];
    transpose4(lo, tl);
    transpose4(hi, th);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *(lds_u32x2 *)(l + (kc * 8 + h * 4 + j) * kQ8Block + ((ng ^ kc) * 8)) = u32x2{tl[j], th[j]};
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int k = p * 16 + (tid >> 4), chunk = tid & 15;
    if (bj * kQ8Block + k < cols)
      *(g_u32x2 *)(b.codes_t[mi] + (bj * kQ8Block + k) * np + bi * kQ8Block + chunk * 8) =
          *(const lds_u32x2 *)(l + k * kQ8Block + ((chunk ^ (k >> 3)) * 8));
  }
}

__global__ __launch_bounds__(kThreads) void q8_weights_kernel(Q8WeightBatch b) {
  __shared__ uint32_t red[4];
  __shared__ __align__(16) char lds[kQ8Block * kQ8Block];
  const int64_t w = blockIdx.x;
  const int32_t mi = find_range(b.n, w, [&](int32_t i) { return b.first_block[i]; });
  if (b.param_dt[mi] == kF32)
    q8_weight_block<true>(b, mi, w - b.first_block[mi], red, lds);
  else
    q8_weight_block<false>(b, mi, w - b.first_block[mi], red, lds);
}

}  // namespace

hipError_t launch_q8_rows(const void *x, int32_t dt, int64_t rows, int64_t cols, uint8_t *codes, uint8_t *scales,
                          hipStream_t st) {
  const int64_t kp = (cols + kQ8Block - 1) / kQ8Block * kQ8Block;
  const int64_t t4 = (rows + kQ8ScaleRow - 1) / kQ8ScaleRow * kQ8ScaleRow;
  for (int64_t first = 0; first < t4; first += kLaunchRows) {
    const dim3 grid(static_cast<uint32_t>(std::min(t4 - first, kLaunchRows) / 4), static_cast<uint32_t>((kp + 2047) / 2048));
    if (dt == kF32)
      hipLaunchKernelGGL(q8_rows_kernel<true>, grid, dim3(kThreads), 0, st, x, first, rows, cols, kp, codes, scales, t4);
    else
      hipLaunchKernelGGL(q8_rows_kernel<false>, grid, dim3(kThreads), 0, st, x, first, rows, cols, kp, codes, scales, t4);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_q8_weights(const Q8WeightBatch &b, hipStream_t st) {
  if (b.n == 0) return hipSuccess;
  hipLaunchKernelGGL(q8_weights_kernel, dim3(static_cast<uint32_t>(b.first_block[b.n])), dim3(kThreads), 0, st, b);
  return hipGetLastError();
}

}  // namespace dmuon
