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
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(1))) u32x4 g_u32x4;
typedef __attribute__((address_space(1))) f32x4 g_f32x4;
typedef __attribute__((address_space(1))) uint8_t g_u8;
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

constexpr int kThreads = 512;
constexpr int kStep = 64;               // rows of t per step
constexpr int kHalfBytes = kStep * 256;  // 128 bf16 columns of a step

__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
}

// Work-group barriers.  The memory clobbers keep the compiler from moving LDS
// accesses across them.
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }
// ... once this wave's LDS accesses are complete
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// LDS holds an operand as halves of 128 columns, a row of a half being one t
// (256 bytes).  The 16-byte chunk of a row is XORed with this, so that the
// transposing reads below (16 rows x 32 bytes) touch distinct banks.
__device__ __forceinline__ int swz(int row) { return ((row & 3) | (((row >> 3) & 1) << 2)) << 1; }

// Four consecutive t of one column: within 16 lanes, lane 4 e + q names row
// t0 + e, columns 4 q .. 4 q + 3, and lane j receives rows t0 .. t0 + 3 of
// column j.
__device__ __forceinline__ i16x4 read_transposed(const lds_char *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4 *)p);
}

// TS x TS outputs (TS columns k of x by TS columns n of dy) per work-group of
// 8 waves (2 x 4), each wave TS/2 k by TS/4 n.  Per step of 64 t, dy goes from
// global memory into LDS by LDS-bound loads, and x through registers, where
// its codes become bf16.  A ring of two stages; the two halves of the
// work-group (wm) run in ping-pong, one reading while the other multiplies.
//
// Half wm = 0 loads dy in its read phase and waits for it at the end of its
// product phase, before either half reads that stage.  Each wave writes its
// share of x's next stage in its read phase, from codes loaded a step before;
// the barrier that ends the phase makes it visible before either half reads
// it.  A stage is only written once both halves have read it.
//
// x's columns are placed in LDS so that a lane's results are consecutive: in
// each run of 32 columns, those of 4-column group g (of 8) sit in block g % 2,
// group g / 2; the lane of quarter q then holds columns 8 q .. 8 q + 7 of the
// run in its blocks 2 i and 2 i + 1.
template <int TS>
__device__ __forceinline__ void q8_wgrad_tile(lds_char *const lds, const Q8WeightGrad &p, int64_t k0, int64_t n0,
                                              int tbeg, int tend, f32x4 (&acc)[TS / 32][TS / 64]) {
  constexpr int FM = TS / 32, FN = TS / 64, kHalves = TS / 128;
  constexpr int kOperand = kHalves * kHalfBytes, kStage = 2 * kOperand;
  constexpr int kRowPieces = TS / 16;                          // 16-code pieces of a row of x
  constexpr int kPieces = kStep * kRowPieces / kThreads;       // per thread: 2 or 1
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int g4 = lane >> 4;
  // An opaque copy of the thread's index: what is derived from it is computed
  // again at every step instead of being kept live across the loop, whose
  // accumulators and fragments take most of the registers.
  auto this_thread = [&]() {
    int t = tid;
    asm volatile("" : "+v"(t));
    return t;
  };

  // dy: load j of half h, wave wn: rows 16 j + 4 wn + lane / 16, one 16-byte
  // chunk a lane; chunks behind the last column are clamped to it
  const uint32_t ld = static_cast<uint32_t>(p.dy_ld) * 2;  // bytes
  const int drow = 4 * wn + (lane >> 4);
  uint32_t dcol[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
    dcol[h] = static_cast<uint32_t>(min((n0 + 128 * h) / 8 + ((lane & 15) ^ swz(drow)), p.dy_ld / 8 - 1) * 16);
  // rows of t that exist from a step on, at most kStep
  auto rows_left = [&](int step) {
    return static_cast<int>(min(p.rows - static_cast<int64_t>(step) * kStep, static_cast<int64_t>(kStep)));
  };
  auto issue_dy = [&](int slot, int step) {
    lds_char *const st = lds + slot * kStage + kOperand;
    const char *const src = static_cast<const char *>(p.dy) + static_cast<int64_t>(step) * kStep * ld;
    const int last = rows_left(step) - 1;
    const int r = 4 * wn + ((this_thread() & 63) >> 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t off = static_cast<uint32_t>(min(r + 16 * j, last)) * ld;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        __builtin_amdgcn_global_load_lds((const void *)(src + (off + dcol[h])),
                                         (__attribute__((address_space(3))) void *)(st + h * kHalfBytes + (j * 4 + wn) * 1024),
                                         16, 0, 0);
    }
  };
  // Rows behind the last were loaded as copies of it: once this wave's loads
  // have landed, it zeroes those that it loaded (x's rows there are zero too,
  // but an infinity times zero would not be).
  auto zero_tail = [&](int slot, int step) {
    const int left = rows_left(step);
    if (left == kStep) return;
    const int l = this_thread() & 63, r = 4 * wn + (l >> 4);
    lds_char *const st = lds + slot * kStage + kOperand + wn * 1024 + l * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (r + 16 * j >= left)
#pragma unroll
        for (int h = 0; h < kHalves; ++h) *(lds_u32x4 *)(st + h * kHalfBytes + j * 4096) = u32x4{0, 0, 0, 0};
  };

  // x: piece q of a thread: row q * (512 / kRowPieces) + tid / kRowPieces,
  // codes 16 m .. 16 m + 15; columns behind the last block are clamped to it.
  // Offsets from a step's uniform base fit 32 bits: 64 rows of at most 2^22
  // codes, and two scale rows of at most 2^31 bytes.
  const int64_t t4 = (p.rows + 3) & ~static_cast<int64_t>(3);
  const int last_col = static_cast<int>(min(p.kp - 16 - k0, static_cast<int64_t>(TS)));
  u32x4 codes[kPieces];
  uint32_t sbyte[kPieces];
  auto load_x = [&](int step) {
    const int64_t t0 = static_cast<int64_t>(step) * kStep;
    const uint8_t *const xs = p.x + t0 * p.kp + k0, *const ss = p.sx + k0 / kQ8Block * t4 + t0;
    const int last = rows_left(step) - 1;
    const int th = this_thread(), xrow = th / kRowPieces;
    const uint32_t xcol = static_cast<uint32_t>(min(16 * (th % kRowPieces), last_col));
    const uint32_t scol = xcol / kQ8Block * static_cast<uint32_t>(t4);
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const int row = min(xrow + q * (kThreads / kRowPieces), last);
      codes[q] = *(const g_u32x4 *)(xs + (static_cast<uint32_t>(row) * static_cast<uint32_t>(p.kp) + xcol));
      sbyte[q] = *(const g_u8 *)(ss + (scol + static_cast<uint32_t>(row)));
    }
  };
  // expands the loaded codes into stage `slot`; rows behind the last are zero
  auto write_x = [&](int slot, int step) {
    const int left = rows_left(step);
    const int th = this_thread(), m = th % kRowPieces, xrow = th / kRowPieces;
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const int row = xrow + q * (kThreads / kRowPieces);
      const bool in = row < left;
      const float s = __uint_as_float(sbyte[q] << 23);
      uint32_t u[8];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int c = in ? static_cast<int>(codes[q][w]) : 0;
        u[2 * w] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, false));
        u[2 * w + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, true));
      }
      // groups 0 and 2 of the four are neighbours in the run's first block,
      // 1 and 3 in its second
      lds_char *const at = lds + slot * kStage + (m >> 3) * kHalfBytes + row * 256;
      const int chunk = ((m & 7) >> 1) * 4 + (m & 1);
      *(lds_u32x4 *)(at + ((chunk ^ swz(row)) * 16)) = u32x4{u[0], u[1], u[4], u[5]};
      *(lds_u32x4 *)(at + (((chunk + 2) ^ swz(row)) * 16)) = u32x4{u[2], u[3], u[6], u[7]};
    }
  };

#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // fragments: lane (g4, e, q) names row 32 s + 8 g4 + 4 h + e, columns
  // c + 4 q .. c + 4 q + 3 of its 16-column block
  const int e = (lane >> 2) & 3, tq = lane & 3;
  const int rs = swz(8 * g4 + e);
  // (the column block's bits are XORed into the lane's swizzled chunk)
  const uint32_t rbase = static_cast<uint32_t>((8 * g4 + e) * 256 + (tq & 1) * 8 + (((tq >> 1) ^ rs) * 16));
  auto fragment = [&](const lds_char *op, uint32_t rb, int col, int s) {
    const lds_char *const at = op + (col >> 7) * kHalfBytes + (rb ^ ((col & 127) * 2)) + s * (32 * 256);
    const i16x4 lo = read_transposed(at), hi = read_transposed(at + 4 * 256);
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  load_x(tbeg);
  if (wm == 0) issue_dy(tbeg & 1, tbeg);
  write_x(tbeg & 1, tbeg);
  load_x(min(tbeg + 1, tend - 1));
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if (wm == 0) zero_tail(tbeg & 1, tbeg);
  lds_barrier();
  if (wm == 1) barrier();
  for (int t = tbeg; t < tend; ++t) {
    const lds_char *const st = lds + (t & 1) * kStage;
    // the last step writes its own rows again, into the free stage, which
    // keeps the loop free of branches
    write_x((t + 1) & 1, min(t + 1, tend - 1));
    __builtin_amdgcn_sched_barrier(0);
    bf16x8 fx[2][FM], fd[2][FN];
    uint32_t rb = rbase;
    // opaque: the fragments' addresses are rebuilt at every step
    asm volatile("" : "+v"(rb));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < FM; ++i) fx[s][i] = fragment(st, rb, wm * (TS / 2) + i * 16, s);
#pragma unroll
      for (int j = 0; j < FN; ++j) fd[s][j] = fragment(st + kOperand, rb, wn * (TS / 4) + j * 16, s);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (wm == 0) issue_dy((t + 1) & 1, min(t + 1, tend - 1));
    load_x(min(t + 2, tend - 1));
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[s][i], fd[s][j], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (wm == 0) zero_tail((t + 1) & 1, min(t + 1, tend - 1));
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }
  if (wm == 0) barrier();
}

// Eight consecutive outputs plus base; vec: their addresses are 16-byte aligned.
__device__ __forceinline__ void finish8(const void *base, void *out, int32_t dt, int64_t at, int64_t left, bool vec,
                                        float (&v)[8]) {
  if (vec && left >= 8) {
    if (dt == kF32) {
      if (base) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 b = *(const g_f32x4 *)(static_cast<const float *>(base) + at + 4 * h);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[4 * h + k] += b[k];
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *(g_f32x4 *)(static_cast<float *>(out) + at + 4 * h) = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    } else {
      if (base) {
        const u32x4 b = *(const g_u32x4 *)(static_cast<const uint16_t *>(base) + at);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[2 * k] += __uint_as_float(b[k] << 16);
          v[2 * k + 1] += __uint_as_float(b[k] & 0xffff0000u);
        }
      }
      u32x4 u;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        u[k] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * k])) |
               (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * k + 1])) << 16);
      *(g_u32x4 *)(static_cast<uint16_t *>(out) + at) = u;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) store_elem(out, dt, at + k, base ? load_elem(base, dt, at + k) + v[k] : v[k]);
  }
}

// Tile `w` of `total`, in an order that keeps the tiles running together on
// one XCD (work-group w runs on XCD w % 8) in bands of four n tiles, which
// share operand columns in its L2.
__device__ __forceinline__ void tile_of(uint32_t w, uint32_t total, uint32_t kt, uint32_t nt, uint32_t &ik,
                                        uint32_t &in) {
  const uint32_t x = w % kXcds, q = total / kXcds, rem = total % kXcds;
  const uint32_t idx = x * q + min(x, rem) + w / kXcds;
  const uint32_t band = idx / (4 * kt), r = idx - band * 4 * kt;
  const uint32_t h = min(4u, nt - band * 4);
  ik = r / h;
  in = band * 4 + r % h;
}

template <int TS>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(TS == 256 ? 2 : 4)))
void q8_wgrad_kernel(Q8WeightGrad p, int32_t pieces, int64_t pitch) {
  constexpr int FM = TS / 32, FN = TS / 64;
  __shared__ __attribute__((aligned(1024))) char smem[4 * (TS / 128) * kHalfBytes];
  const uint32_t kt = static_cast<uint32_t>((p.cols + TS - 1) / TS), nt = static_cast<uint32_t>((p.outs + TS - 1) / TS);
  // divisions run on the vector unit: their results are made scalar again
  const uint32_t piece = uniform(blockIdx.x / (kt * nt));
  uint32_t ik, in;
  tile_of(blockIdx.x - piece * kt * nt, kt * nt, kt, nt, ik, in);
  const int64_t k0 = static_cast<int64_t>(uniform(ik)) * TS, n0 = static_cast<int64_t>(uniform(in)) * TS;
  // a piece's steps: rows / 64 < 2^25 steps, at most 2^6 pieces
  const uint32_t steps = static_cast<uint32_t>((p.rows + kStep - 1) / kStep);
  const int tbeg = static_cast<int>(uniform(steps * piece / static_cast<uint32_t>(pieces)));
  const int tend = static_cast<int>(uniform(steps * (piece + 1) / static_cast<uint32_t>(pieces)));
  f32x4 acc[FM][FN];
  q8_wgrad_tile<TS>((lds_char *)smem, p, k0, n0, tbeg, tend, acc);

  void *out = p.out;
  const void *base = p.base;
  int32_t dt = p.out_dt;
  int64_t ldo = p.cols;
  if (pieces > 1) {
    out = static_cast<float *>(p.ws) + static_cast<int64_t>(piece) * p.outs * pitch;
    base = nullptr;
    dt = kF32;
    ldo = pitch;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 2, wn = wave & 3, r16 = lane & 15, g4 = lane >> 4;
  const bool vec = ldo % (dt == kF32 ? 4 : 8) == 0;
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int64_t n = n0 + wn * (TS / 4) + j * 16 + r16;
    if (n >= p.outs) continue;
#pragma unroll
    for (int i = 0; i < FM; i += 2) {
      const int64_t k = k0 + wm * (TS / 2) + i * 16 + g4 * 8;
      float v[8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[4 * h + c] = acc[i + h][j][c];
      finish8(base, out, dt, n * ldo + k, p.cols - k, vec, v);
    }
  }
}

// No rows: out = base, or zero.
__global__ __launch_bounds__(256) void q8_wgrad_empty_kernel(Q8WeightGrad p) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int64_t left = p.outs * p.cols - at;
  if (left > 0) finish8(p.base, p.out, p.out_dt, at, left, true, v);
}

// A copy of dy with rows of a multiple of 8 elements (zeros behind the last
// column), for a dy whose rows are not: the LDS-bound loads take 16 bytes.
__global__ __launch_bounds__(256) void q8_pad_rows_kernel(const uint16_t *__restrict__ dy, int64_t rows, int64_t cols,
                                                          int64_t ld, uint16_t *__restrict__ out) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (at >= rows * ld) return;
  const int64_t t = at / ld, c = at - t * ld;
  uint32_t e[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) e[k] = c + k < cols ? ((const g_u16 *)dy)[t * cols + c + k] : 0;
  *(g_u32x4 *)(out + at) = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
}

// How a weight gradient runs: the tile, the pieces of its rows, and the bytes
// of its workspace's two parts, the padded dy and the pieces' results.
struct Plan {
  int tile, pieces;
  int64_t dy_ld, pitch;
  size_t pad_bytes, piece_bytes;
};

Plan plan_of(int64_t rows, int64_t outs, int64_t cols) {
  Plan pl;
  pl.tile = 256;
  pl.pieces = 1;
  pl.dy_ld = (outs + 7) & ~static_cast<int64_t>(7);
  pl.pitch = (cols + 7) & ~static_cast<int64_t>(7);
  auto up = [](int64_t b) { return (static_cast<size_t>(b) + 255) & ~static_cast<size_t>(255); };
  pl.pad_bytes = pl.dy_ld != outs ? up(rows * pl.dy_ld * 2) : 0;
  pl.piece_bytes = pl.pieces > 1 ? up(pl.pieces * outs * pl.pitch * 4) : 0;
  return pl;
}

template <int TS>
void launch_tiles(const Q8WeightGrad &p, const Plan &pl, hipStream_t st) {
  const int64_t tiles = ((p.outs + TS - 1) / TS) * ((p.cols + TS - 1) / TS);
  hipLaunchKernelGGL((q8_wgrad_kernel<TS>), dim3(static_cast<uint32_t>(tiles * pl.pieces)), dim3(kThreads), 0, st, p,
                     pl.pieces, pl.pitch);
}

}  // namespace

size_t q8_wgrad_workspace(int64_t rows, int64_t outs, int64_t cols) {
  const Plan pl = plan_of(rows, outs, cols);
  return pl.pad_bytes + pl.piece_bytes;
}

hipError_t launch_q8_wgrad(const Q8WeightGrad &args, hipStream_t st) {
  Q8WeightGrad p = args;
  if (p.rows == 0) {
    hipLaunchKernelGGL(q8_wgrad_empty_kernel, dim3(static_cast<uint32_t>((p.outs * p.cols + 2047) / 2048)), dim3(256), 0,
                       st, p);
    return hipGetLastError();
  }
  const Plan pl = plan_of(p.rows, p.outs, p.cols);
  p.dy_ld = pl.dy_ld;
  if (pl.pad_bytes) {
    const int64_t groups = (p.rows * pl.dy_ld / 8 + 255) / 256;
    hipLaunchKernelGGL(q8_pad_rows_kernel, dim3(static_cast<uint32_t>(groups)), dim3(256), 0, st,
                       static_cast<const uint16_t *>(p.dy), p.rows, p.outs, pl.dy_ld, static_cast<uint16_t *>(p.ws));
    p.dy = p.ws;
    p.ws = static_cast<char *>(p.ws) + pl.pad_bytes;
  }
  if (pl.tile == 256)
    launch_tiles<256>(p, pl, st);
  else
    launch_tiles<128>(p, pl, st);
  return hipGetLastError();
}

}  // namespace dmuon
