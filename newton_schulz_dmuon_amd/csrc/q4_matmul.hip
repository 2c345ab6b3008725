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

#include <algorithm>
#include <utility>

#include "q4_device.h"

namespace dmuon {

namespace {

// f(0), ..., f(N - 1) with constant indices (a scale's byte is an immediate of the
// instruction).
template <int... I, typename F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  each(std::make_integer_sequence<int, N>{}, f);
}

// ---- tiles: many rows ----
//
// One work-group of 8 waves (2 x 4) computes TA outputs of the weight by TB
// rows; each wave TA/2 x TB/4 in 16 x 16 blocks.  K advances 256 codes (128 bytes,
// 8 blocks of the format) per step.  Both operand tiles go from global memory into
// LDS by LDS-bound loads (16 bytes a lane, 128-byte rows, the 16-byte chunk, a
// block of the format, XORed with (row / 2) mod 8, which keeps the fragment reads
// off each other's banks), a ring of two stages, with the step's scales behind
// them.  The two halves of the work-group (wm) run in ping-pong: one half's waves
// read fragments and issue the next stage's loads while the other half's multiply,
// switching at every barrier.
//
// The order of rows in LDS is free, since every lane of a load picks its global
// row, and is chosen for the ends of the pipeline: a wave's block i, row q holds
// output ((q % 4) * 4 + q / 4) * FM + i, so that a lane's FM results of one row (FM
// blocks) are consecutive and its quarter-wave neighbours' follow, and block j,
// column r of the rows' operand holds row r * FN + j.  A lane's FM or FN scale bytes
// of a block of k are then consecutive bytes of the scale table's row.
constexpr int kTileThreads = 512;
constexpr int kRowBytes = 128;
constexpr int kStepBlocks = kQ4Pad / kQ4Block;

template <int TA, int TB>
__device__ __forceinline__ void q4_tile(lds_char *const lds, const Q4Product &p, int64_t n0, int64_t t0, int kbeg,
                                        int kend, f32x4 (&acc)[TA / 32][TB / 64]) {
  constexpr int FM = TA / 32, FN = TB / 64;
  // a stage: the weight's tile, the rows', the weight's scales (each half's [block]
  // [output]), the rows' ([block][row])
  constexpr int kWeight = TA * kRowBytes, kScaleA = kWeight + TB * kRowBytes, kScaleB = kScaleA + TA * kStepBlocks;
  constexpr int kStage = kScaleB + TB * kStepBlocks;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int r16 = lane & 15, g4 = lane >> 4;
  const uint32_t kpb = static_cast<uint32_t>(p.kp / 2);
  const int64_t ra = (p.rows + kQ4ScaleRow - 1) & ~static_cast<int64_t>(kQ4ScaleRow - 1);
  const int64_t rb = (p.outs + kQ4ScaleRow - 1) & ~static_cast<int64_t>(kQ4ScaleRow - 1);

  const uint8_t *const gb = p.b + n0 * kpb, *const ga = static_cast<const uint8_t *>(p.a) + t0 * kpb;
  // the last output and row of the tile that exist
  const int lim_n = static_cast<int>(min(p.outs - 1 - n0, static_cast<int64_t>(TA - 1)));
  const int lim_t = static_cast<int>(min(p.rows - 1 - t0, static_cast<int64_t>(TB - 1)));
  // scales: 16 outputs or rows a lane, TA/32 or TB/16 lanes a block
  const uint8_t *const gsb = p.sb + lane / (TA / 32) * rb + min(n0 + wm * (TA / 2) + lane % (TA / 32) * 16, rb - 16);
  const uint8_t *const gsa = p.sa + lane / (TB / 16) * ra + min(t0 + lane % (TB / 16) * 16, ra - 16);
  // loads: lane l of 1 KB load j of a half fills LDS row (j * 4 + wn) * 8 + l / 8,
  // physical chunk l % 8
  const int q = (wn & 1) * 8 + (lane >> 3);
  const uint32_t chunk = static_cast<uint32_t>((lane & 7) ^ (((wn & 1) * 4 + (lane >> 4)) & 7)) * 16;
  const int base_n = ((q & 3) * 4 + (q >> 2)) * FM + (wn >> 1) + wm * (TA / 2);
  const int base_t = q * FN + (wn >> 1);
  auto issue = [&](int slot, int kb) {
    lds_char *const st = lds + slot * kStage;
    const uint8_t *const bb = gb + static_cast<int64_t>(kb) * kRowBytes, *const ba = ga + static_cast<int64_t>(kb) * kRowBytes;
    auto piece = [&](const uint8_t *src, int at) {
      __builtin_amdgcn_global_load_lds((const void *)src, (__attribute__((address_space(3))) void *)(st + at), 16, 0, 0);
    };
    auto load = [&](const uint8_t *src, int row, int at) {
      piece(src + (__umul24(static_cast<uint32_t>(row), kpb) + chunk), at + wn * 1024);
    };
    int bn = base_n, bt = base_t;
    // opaque: the offsets are rebuilt at every issue instead of being kept
    // live across the loop
    asm volatile("" : "+v"(bn), "+v"(bt));
#pragma unroll
    for (int j = 0; j < TA / 64; ++j) load(bb, min(bn + 2 * j, lim_n), wm * (kWeight / 2) + j * 4096);
    if (wn == 3 && lane < TA / 4)
      piece(gsb + static_cast<int64_t>(kb) * kStepBlocks * rb, kScaleA + wm * (TA / 2 * kStepBlocks));
    if (wm == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < TB / 64; ++j) {
          // row s of the tile's LDS rows: quarter s / (TB / 4), then block and column
          const int s = h * (TB / 2) + j * 32, in_quarter = s % (TB / 4);
          const int row = s / (TB / 4) * (TB / 4) + in_quarter / 16;
          load(ba, min(bt + row, lim_t), kWeight + s * kRowBytes);
        }
      // 1024 / TB blocks a load
      if (wn < TB / 128)
        piece(gsa + (static_cast<int64_t>(kb) * kStepBlocks + wn * (1024 / TB)) * ra, kScaleB + wn * 1024);
    }
  };

#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // 16 bytes (chunk sub * 4 + g4, one block) of row r16 of 16-row block i of an
  // operand; the swizzle is the same in every block
  const uint32_t at0 = static_cast<uint32_t>(r16 * kRowBytes + ((g4 ^ (r16 >> 1)) & 7) * 16);
  auto read = [&](const lds_char *op, int i, int sub) {
    return *(const lds_u32x4 *)(op + (sub ? at0 ^ 64 : at0) + i * (16 * kRowBytes));
  };
  const uint32_t at_b = static_cast<uint32_t>(kScaleA + wm * (TA / 2 * kStepBlocks) + g4 * (TA / 2) + ((r16 & 3) * 4 + (r16 >> 2)) * FM);
  const uint32_t at_a = static_cast<uint32_t>(kScaleB + g4 * TB + wn * (TB / 4) + r16 * FN);

  issue(kbeg & 1, kbeg);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if (wm == 1) barrier();
  for (int kb = kbeg; kb < kend; ++kb) {
    const lds_char *const st = lds + (kb & 1) * kStage;
    const lds_char *const opb = st + wm * (kWeight / 2), *const opa = st + kWeight + wn * (TB / 4 * kRowBytes);
    // the last step loads its own block again, into the free stage, which
    // keeps the loop free of a branch
    issue((kb + 1) & 1, min(kb + 1, kend - 1));
    u32x4 fb[FM][2], fa[FN][2];
    uint32_t sb[FM / 4][2], sa[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if constexpr (FM == 8) {
        const u32x2 w = *(const lds_u32x2 *)(st + at_b + s * (4 * TA / 2));
        sb[0][s] = w.x;
        sb[1][s] = w.y;
      } else {
        sb[0][s] = *(const lds_u32 *)(st + at_b + s * (4 * TA / 2));
      }
      if constexpr (FN == 4)
        sa[s] = *(const lds_u32 *)(st + at_a + s * (4 * TB));
      else
        sa[s] = *(const lds_u16 *)(st + at_a + s * (4 * TB));
#pragma unroll
      for (int i = 0; i < FM; ++i) fb[i][s] = read(opb, i, s);
#pragma unroll
      for (int j = 0; j < FN; ++j) fa[j][s] = read(opa, j, s);
    }
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
      each<FM>([&](auto i) {
        each<FN>([&](auto j) {
          acc[i][j] = q4_product<i % 4, j>(fb[i][s], sb[i / 4][s], fa[j][s], sa[s], acc[i][j]);
        });
      });
    __builtin_amdgcn_sched_barrier(0);
    load_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }
  if (wm == 0) barrier();
}

template <int TA, int TB>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(TB == 256 ? 2 : 4)))
void q4_tile_kernel(Q4Product p, TileSplit sp) {
  constexpr int FM = TA / 32, FN = TB / 64;
  __shared__ __attribute__((aligned(1024))) char smem[2 * (TA + TB) * (kRowBytes + kStepBlocks)];
  const TileWork w = tile_work(sp, blockIdx.x, static_cast<uint32_t>(p.kp / kQ4Pad));
  const int64_t n0 = static_cast<int64_t>(w.a) * TA, t0 = static_cast<int64_t>(w.b) * TB;
  f32x4 acc[FM][FN];
  q4_tile<TA, TB>((lds_char *)smem, p, n0, t0, w.begin, w.end, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 2, wn = wave & 3, r16 = lane & 15, g4 = lane >> 4;
  const TileOut o = tile_out(w, TA, TB, p.base, p.out, p.out_dt, p.rows, p.outs, p.ws);
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int r = wn * (TB / 4) + r16 * FN + j;
    if (r >= o.rows) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int c = wm * (TA / 2) + (v * 4 + g4) * FM;
      float run[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i) run[i] = acc[i][j][v];
      finish_run<FM>(o.base, o.out, o.dt, o.at + r * o.ld + c, o.cols - c, run);
    }
  }
}

// A sum of nothing: out = base, or zero.
__global__ __launch_bounds__(256) void q4_empty_kernel(Q4Product p) {
  const int64_t n = p.rows * p.outs;
  for (int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8; at < n; at += gridDim.x * int64_t(2048)) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    finish_run<8>(p.base, p.out, p.out_dt, at, n - at, v);
  }
}

constexpr std::initializer_list<TileCost> kCosts = {
    {256, 256, 1, 1.03f, 1.5f}, {128, 256, 1, 0.8f, 0.97f}, {128, 128, 2, 0.6f, 1.06f}};

TileSplit plan_of(int64_t rows, int64_t outs, int64_t kp) {
  if (rows == 0 || kp == 0) return TileSplit{};
  return choose_split(outs, rows, kp / kQ4Pad, kCosts);
}

template <int TA, int TB>
hipError_t launch_tiles(const Q4Product &p, const TileSplit &sp, hipStream_t st) {
  hipLaunchKernelGGL((q4_tile_kernel<TA, TB>), dim3(sp.whole + sp.tail * sp.pieces), dim3(kTileThreads), 0, st, p, sp);
  return hipGetLastError();
}

}  // namespace

size_t q4_matmul_workspace(int64_t rows, int64_t outs, int64_t kp) { return plan_of(rows, outs, kp).ws_bytes(); }

hipError_t launch_q4_matmul(const Q4Product &p, hipStream_t st) {
  if (p.kp == 0) {
    const int64_t groups = std::min<int64_t>((p.rows * p.outs + 2047) / 2048, 1 << 20);
    hipLaunchKernelGGL(q4_empty_kernel, dim3(static_cast<uint32_t>(groups)), dim3(256), 0, st, p);
    return hipGetLastError();
  }
  const TileSplit sp = plan_of(p.rows, p.outs, p.kp);
  const hipError_t e = sp.ta == 256   ? launch_tiles<256, 256>(p, sp, st)
                       : sp.tb == 256 ? launch_tiles<128, 256>(p, sp, st)
                                      : launch_tiles<128, 128>(p, sp, st);
  if (e != hipSuccess || sp.pieces == 1) return e;
  return launch_q8_reduce(static_cast<const float *>(p.ws), sp, p.rows, p.outs, p.base, p.out, p.out_dt, st);
}

}  // namespace dmuon
