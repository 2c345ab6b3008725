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

// ---- few rows: the weight's bytes ----
//
// A work-group takes 16 NN outputs of up to 16 NT rows, its WAVES waves every
// WAVES-th block of 256 codes; the waves' sums are added through LDS in wave order.
// Each wave has a ring of stages of its own in LDS, and no barrier: it waits for
// its own loads.  A block comes by LDS-bound loads of eight whole rows' 128 bytes,
// the 16-byte chunks XORed with (row / 2) mod 8 against bank conflicts, its scales
// by one more.  The weight's bytes are read once, the rows' from L2 once per 16 NN
// outputs; of up to eight rows, XR = 8, eight are loaded.  Rows and outputs behind
// the last are clamped for the loads and not stored.  Column r of row block j is
// row r * NT + j, so that a lane's NT scale bytes are one LDS word.
//
// Bound by the weight's bytes (one row by 14336 x 4096, 31 MB, 8.2 us out of HBM, 7.2
// out of the memory-side cache: 3.8 TB/s with the launch, 2 us of it, 5.0 without),
// from about 24 rows on by what a CU takes in (64 rows 10.8 us, 64 of 4096 x 14336
// 12.5).  Wider work-groups read the rows' codes less often and have fewer waves a CU:
// of 100 rows by 8192 x 8192 4 x 4 takes 14.0 us, 4 x 2 20.5, the tiles below 18.8; of
// 64 by 4096 x 14336 2 x 2 12.5, 4 x 4 21.6, tiles 17.3.  2 x 1 and 4 x 1 were never
// the best by more than 2%.
constexpr int stream_stage(int nt, int nn, int xr) { return nn * 2048 + nt * xr * 128 + (nn + nt) * 128; }
// Blocks in flight a wave.
constexpr int stream_ahead(int nt, int nn, int waves) { return waves == 8 || nt * nn > 2 ? 2 : 3; }

template <int NT, int NN, int WAVES, int XR>
__global__ __launch_bounds__(WAVES * 64) void q4_stream_kernel(Q4Product p) {
  constexpr int kAhead = stream_ahead(NT, NN, WAVES);
  constexpr int kRows = NN * 2048, kScales = kRows + NT * XR * 128, kStage = stream_stage(NT, NN, XR);
  constexpr int kLoads = 2 * NN + NT * XR / 8 + 1;  // vector loads a block
  static_assert(XR == 16 || (XR == 8 && NT == 1));
  __shared__ __attribute__((aligned(1024))) char smem[WAVES * kAhead * kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const uint32_t nt = static_cast<uint32_t>((p.outs + 16 * NN - 1) / (16 * NN)), tb = uniform(blockIdx.x / nt);
  const int64_t n0 = static_cast<int64_t>(line_tile<NN>(blockIdx.x - tb * nt, nt)) * (16 * NN);
  const int64_t t0 = static_cast<int64_t>(tb) * (16 * NT);
  const int nkb = static_cast<int>(p.kp / kQ4Pad);
  const uint32_t kpb = static_cast<uint32_t>(p.kp / 2);
  const int64_t ra = (p.rows + kQ4ScaleRow - 1) & ~static_cast<int64_t>(kQ4ScaleRow - 1);
  const int64_t rb = (p.outs + kQ4ScaleRow - 1) & ~static_cast<int64_t>(kQ4ScaleRow - 1);
  lds_char *const ring = (lds_char *)smem + wave * (kAhead * kStage);
  // lane l of 1 KB load h of a block fills LDS row 8 h + l / 8, physical chunk l % 8
  const uint8_t *const gb = p.b + n0 * kpb, *const ga = static_cast<const uint8_t *>(p.a) + t0 * kpb;
  const int lim_n = static_cast<int>(min(p.outs - 1 - n0, static_cast<int64_t>(16 * NN - 1)));
  const int lim_t = static_cast<int>(min(p.rows - 1 - t0, static_cast<int64_t>(16 * NT - 1)));
  uint32_t ob[NN][2], oa[NT][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = 8 * h + (lane >> 3);
    const uint32_t chunk = static_cast<uint32_t>((lane & 7) ^ ((row >> 1) & 7)) * 16;
#pragma unroll
    for (int i = 0; i < NN; ++i)
      ob[i][h] = __umul24(static_cast<uint32_t>(min(i * 16 + row, lim_n)), kpb) + chunk;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      oa[j][h] = __umul24(static_cast<uint32_t>(min(row * NT + j, lim_t)), kpb) + chunk;
  }
  // the scales of a stage, 16 bytes a lane: [block][16 NN outputs], then [block]
  // [16 NT rows]
  const int sl = lane < 8 * NN ? lane : lane - 8 * NN;
  // both tables' addresses are read here: chosen by lane as they stand in p, they
  // come by a vector load, which the first stages' loads wait for
  const uint8_t *sb0 = p.sb, *sa0 = p.sa;
  asm volatile("" : "+s"(sb0), "+s"(sa0));
  const uint8_t *const scale0 =
      lane < 8 * NN ? sb0 + sl / NN * rb + min(n0 + sl % NN * 16, rb - 16)
                    : sa0 + sl / NT * ra + min(t0 + sl % NT * 16, ra - 16);
  const int64_t scale_step = (lane < 8 * NN ? rb : ra) * (kQ4Pad / kQ4Block);
  f32x4 acc[NN][NT];
#pragma unroll
  for (int i = 0; i < NN; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto load = [&](int u, int block) {
    const int kb = min(block, nkb - 1);
    lds_char *const st = ring + u * kStage;
    auto piece = [&](const uint8_t *src, int at) {
      __builtin_amdgcn_global_load_lds((const void *)src, (__attribute__((address_space(3))) void *)(st + at), 16, 0, 0);
    };
    const uint8_t *const bb = gb + static_cast<int64_t>(kb) * 128, *const ba = ga + static_cast<int64_t>(kb) * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < NN; ++i) piece(bb + ob[i][h], i * 2048 + h * 1024);
      if (8 * h < XR)
#pragma unroll
        for (int j = 0; j < NT; ++j) piece(ba + oa[j][h], kRows + j * (XR * 128) + h * 1024);
    }
    if (lane < 8 * (NN + NT)) piece(scale0 + kb * scale_step, kScales);
    __builtin_amdgcn_sched_barrier(0);
  };
  // a lane's codes of row r16 of a block: chunks g4 and g4 + 4
  auto at = [&](int row) { return static_cast<uint32_t>(row * 128 + ((g4 ^ (row >> 1)) & 7) * 16); };
  const uint32_t at_b = at(r16), at_a = at(r16 & (XR - 1));
  u32x4 fb[NN][2], fa[NT][2];
  uint32_t sb[NN][2], sa[2];
  auto read = [&](int u) {
    const lds_char *const st = ring + u * kStage;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < NN; ++i) {
        fb[i][s] = *(const lds_u32x4 *)(st + i * 2048 + (s ? at_b ^ 64 : at_b));
        sb[i][s] = *(const lds_u8 *)(st + kScales + (4 * s + g4) * (16 * NN) + i * 16 + r16);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) fa[j][s] = *(const lds_u32x4 *)(st + kRows + j * (XR * 128) + (s ? at_a ^ 64 : at_a));
      const lds_char *const ws = st + kScales + NN * 128 + (4 * s + g4) * (16 * NT) + r16 * NT;
      if constexpr (NT == 4)
        sa[s] = *(const lds_u32 *)ws;
      else if constexpr (NT == 2)
        sa[s] = *(const lds_u16 *)ws;
      else
        sa[s] = *(const lds_u8 *)ws;
    }
    // all are in registers before the stage is loaded again
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&]() {
#pragma unroll
    for (int s = 0; s < 2; ++s)
      each<NN>([&](auto i) {
        each<NT>([&](auto j) { acc[i][j] = q4_product<0, j>(fb[i][s], sb[i][s], fa[j][s], sa[s], acc[i][j]); });
      });
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, wave + u * WAVES);
  // each stage takes the block kAhead further on as soon as its codes have been
  // read; the last kAhead blocks load nothing more
  int k0 = wave;
  for (; k0 + WAVES * kAhead < nkb; k0 += WAVES * kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 1) * kLoads) : "memory");
      read(u);
      load(u, k0 + (kAhead + u) * WAVES);
      multiply();
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (k0 + u * WAVES < nkb) {
      read(u);
      multiply();
    }
  constexpr int kRuns = (NN * NT + WAVES - 1) / WAVES;
  float b[kRuns][1][4];
#pragma unroll
  for (int q = 0; q < kRuns; ++q) {
    const int at = q * WAVES + wave;
    const int64_t t = t0 + r16 * NT + at % NT, n = n0 + at / NT * 16 + 4 * g4;
    if (p.base && at < NN * NT && t < p.rows && n < p.outs)
      load_base<4, 1>(p.base, p.out_dt, t * p.outs + n, 0, p.outs - n, b[q]);
    else
      b[q][0][0] = b[q][0][1] = b[q][0][2] = b[q][0][3] = 0.f;
  }
  // the waves' sums, each in its own part of the ring
  auto part = [&](int w, int b) { return (lds_f32x4 *)((lds_char *)smem + w * (kAhead * kStage) + b * 1024 + lane * 16); };
  static_assert(NN * NT * 1024 <= kAhead * kStage);
#pragma unroll
  for (int i = 0; i < NN; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) *part(wave, i * NT + j) = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kRuns; ++q) {
    const int at = q * WAVES + wave;
    if (at >= NN * NT) return;
    f32x4 sum = *part(0, at);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += *part(w, at);
    const int64_t t = t0 + r16 * NT + at % NT, n = n0 + at / NT * 16 + 4 * g4;
    if (t >= p.rows) continue;
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = p.base ? b[q][0][k] + sum[k] : sum[k];
    finish_run<4>(nullptr, p.out, p.out_dt, t * p.outs + n, p.outs - n, v);
  }
}

// ---- tiles: many rows ----
//
// One work-group of 8 waves (2 x 4) computes TA (128 or 256) outputs of the weight
// by 256 rows, TB below; each wave TA/2 x TB/4 in 16 x 16 blocks.  K advances 256 codes (128 bytes,
// 8 blocks of the format) per step.  Both operand tiles go from global memory into
// LDS by LDS-bound loads (16 bytes a lane, 128-byte rows, the 16-byte chunk, a
// block of the format, XORed with (row / 2) mod 8, which keeps the fragment reads
// off each other's banks), a ring of two stages, with the step's scales behind
// them.  The two halves of the work-group (wm) run in ping-pong: one half's waves
// read fragments and issue the next stage's loads while the other half's multiply,
// switching at every barrier.
//
// 8192 rows by 14336 x 4096: 239 us, 4.0 PFLOP/s (a library product of the same type
// 350).  Not bound by the matrix instructions, which are busy 45% of the cycles: they
// alone, their operands left in registers, take 145 us, everything else without them
// 152, without the loads 164, without the stores 205.  So the loads into LDS beside the
// instructions and fragment reads cost 75 us, and the stores, beside which nothing runs,
// 34.  The power that the instructions draw takes some of the clock: on zero codes the
// whole takes 190 us, the instructions alone 117 (a loop of nothing else reaches 7.1
// PFLOP/s on random codes and 9.6 on zeros).  With four waves of 128 x 128 it took 293
// us for 290, with the next tile's first loads sent before the stores 296 for 295:
// neither was kept.
//
// The order of rows in LDS is free, since every lane of a load picks its global
// row, and is chosen for the ends of the pipeline: a wave's block i, row q holds
// output ((q % 4) * 4 + q / 4) * FM + i, so that a lane's FM results of one row (FM
// blocks) are consecutive and its quarter-wave neighbours' follow, and block j,
// column r of the rows' operand holds row r * FN + j.  A lane's FM or FN scale bytes
// of a block of k are then consecutive bytes of the scale table's row.
constexpr int kTileThreads = 512, kTileRows = 256;
constexpr int kRowBytes = 128;
constexpr int kStepBlocks = kQ4Pad / kQ4Block;

template <int TA>
__device__ __forceinline__ void q4_tile(lds_char *const lds, const Q4Product &p, int64_t n0, int64_t t0, int kbeg,
                                        int kend, f32x4 (&acc)[TA / 32][kTileRows / 64]) {
  constexpr int TB = kTileRows, FM = TA / 32, FN = TB / 64;
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
  const uint32_t at_b = static_cast<uint32_t>(kScaleA + wm * (TA / 2 * kStepBlocks) + g4 * (TA / 2) +
                                              ((r16 & 3) * 4 + (r16 >> 2)) * FM);
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
      sa[s] = *(const lds_u32 *)(st + at_a + s * (4 * TB));
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

template <int TA>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(2)))
void q4_tile_kernel(Q4Product p, TileSplit sp) {
  constexpr int TB = kTileRows, FM = TA / 32, FN = TB / 64;
  __shared__ __attribute__((aligned(1024))) char smem[2 * (TA + TB) * (kRowBytes + kStepBlocks)];
  const TileWork w = tile_work(sp, blockIdx.x, static_cast<uint32_t>(p.kp / kQ4Pad));
  const int64_t n0 = static_cast<int64_t>(w.a) * TA, t0 = static_cast<int64_t>(w.b) * TB;
  f32x4 acc[FM][FN];
  q4_tile<TA>((lds_char *)smem, p, n0, t0, w.begin, w.end, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 2, wn = wave & 3, r16 = lane & 15, g4 = lane >> 4;
  const TileOut o = tile_out(w, TA, TB, p.base, p.out, p.out_dt, p.rows, p.outs, p.ws);
  // a tile of whole columns; at a ragged edge the runs, of which some end, wait each
  // for its own
  const bool base_first = o.base && o.cols >= TA;
  if (base_first) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int r = wn * (TB / 4) + r16 * FN + j;
      if (r >= o.rows) continue;
      float b[4][FM];
      load_runs<FM, 4>(o.base, o.dt, o.at + r * o.ld + wm * (TA / 2) + g4 * FM, 4 * FM, b);
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[i][j][v] += b[v][i];
    }
  }
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
      finish_run<FM>(base_first ? nullptr : o.base, o.out, o.dt, o.at + r * o.ld + c, o.cols - c, run);
    }
  }
}

// ---- small tiles: a deep ring ----
//
// 128 outputs by TB (64 or 128) rows, one work-group a CU, for launches of few tiles,
// which the latency of a step bounds.  Eight waves: 2 x 2 parts of 64 x TB / 2, and
// two halves of a step's 256 codes, whose sums are added at the end (one wave for
// all codes and half the part would read half as much again from LDS).  A ring of
// four stages (six of 64 rows): a step waits for its own stage, loaded three steps ago, meets the
// other waves once, loads the stage that all of them have left and multiplies.  The
// two waves of a SIMD hide each other's reads.  A step of 128 x 128 takes 0.44 us so;
// with two stages and ping-pong 0.75, with whole steps a wave 0.59.  128 rows by 14336
// x 4096: 13.3 us (128 x 128 16.2, streamed 16.7), 256: 16.6 (128 x 64 23.6, 128 x 256
// 24.7).
//
// A lane's four rows of a weight block (q = 4 g4 + v) and FM blocks are consecutive
// outputs: block i, row q holds output q * FM + i of the wave's part, block j,
// column r of the rows' operand row r * FN + j.
constexpr int kMidThreads = 512;

template <int TB>
__global__ __launch_bounds__(kMidThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void q4_mid_kernel(Q4Product p, TileSplit sp) {
  constexpr int TA = 128, FM = TA / 32, FN = TB / 32, kMidStages = TB == 128 ? 4 : 6;
  constexpr int kRows = TA * kRowBytes, kScaleB = kRows + TB * kRowBytes, kScaleA = kScaleB + TA * kStepBlocks;
  constexpr int kStage = kScaleA + TB * kStepBlocks;
  constexpr int kLoads = (TA + TB) / 64 + 1;  // vector loads a wave and stage
  constexpr int kScaleLanes = (TA + TB) * kStepBlocks / 16 / 8;  // 16 bytes each
  __shared__ __attribute__((aligned(1024))) char smem[kMidStages * kStage];
  lds_char *const lds = (lds_char *)smem;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave >> 2, wm = wave >> 1 & 1, wn = wave & 1, r16 = lane & 15, g4 = lane >> 4;
  const TileWork w = tile_work(sp, blockIdx.x, static_cast<uint32_t>(p.kp / kQ4Pad));
  const int64_t n0 = static_cast<int64_t>(w.a) * TA, t0 = static_cast<int64_t>(w.b) * TB;
  const uint32_t kpb = static_cast<uint32_t>(p.kp / 2);
  const int64_t ra = (p.rows + kQ4ScaleRow - 1) & ~static_cast<int64_t>(kQ4ScaleRow - 1);
  const int64_t rb = (p.outs + kQ4ScaleRow - 1) & ~static_cast<int64_t>(kQ4ScaleRow - 1);
  const int lim_n = static_cast<int>(min(p.outs - 1 - n0, static_cast<int64_t>(TA - 1)));
  const int lim_t = static_cast<int>(min(p.rows - 1 - t0, static_cast<int64_t>(TB - 1)));
  // load j of a wave fills LDS rows 8 (wave + 8 j) ..: lane l row l / 8, physical
  // chunk l % 8
  uint32_t ob[TA / 64], oa[TB / 64];
#pragma unroll
  for (int j = 0; j < TA / 64; ++j) {
    const int l = 8 * (wave + 8 * j) + (lane >> 3), part = l / (16 * FM), i = l / 16 % FM, q = l % 16;
    ob[j] = __umul24(static_cast<uint32_t>(min(part * (16 * FM) + q * FM + i, lim_n)), kpb) +
            static_cast<uint32_t>((lane & 7) ^ ((q >> 1) & 7)) * 16;
  }
#pragma unroll
  for (int j = 0; j < TB / 64; ++j) {
    const int l = 8 * (wave + 8 * j) + (lane >> 3), part = l / (16 * FN), i = l / 16 % FN, q = l % 16;
    oa[j] = __umul24(static_cast<uint32_t>(min(part * (16 * FN) + q * FN + i, lim_t)), kpb) +
            static_cast<uint32_t>((lane & 7) ^ ((q >> 1) & 7)) * 16;
  }
  const uint8_t *const gb = p.b + n0 * kpb, *const ga = static_cast<const uint8_t *>(p.a) + t0 * kpb;
  // scales, 16 bytes a lane: the weight's [block][output], then the rows'
  const int s16 = wave * kScaleLanes + lane, s_rows = s16 - TA / 2;
  const uint8_t *const gs =
      s16 < TA / 2 ? p.sb + s16 / (TA / 16) * rb + min(n0 + s16 % (TA / 16) * 16, rb - 16)
                   : p.sa + s_rows / (TB / 16) % kStepBlocks * ra + min(t0 + s_rows % (TB / 16) * 16, ra - 16);
  const int64_t gs_step = (s16 < TA / 2 ? rb : ra) * kStepBlocks;
  auto issue = [&](int kb) {
    lds_char *const st = lds + static_cast<uint32_t>(kb) % kMidStages * kStage;
    const int64_t k = min(kb, w.end - 1);
    auto piece = [&](const uint8_t *src, int at) {
      __builtin_amdgcn_global_load_lds((const void *)src, (__attribute__((address_space(3))) void *)(st + at), 16, 0, 0);
    };
#pragma unroll
    for (int j = 0; j < TA / 64; ++j) piece(gb + k * kRowBytes + ob[j], (wave + 8 * j) * 1024);
#pragma unroll
    for (int j = 0; j < TB / 64; ++j) piece(ga + k * kRowBytes + oa[j], kRows + (wave + 8 * j) * 1024);
    if (lane < kScaleLanes) piece(gs + k * gs_step, kScaleB + wave * (kScaleLanes * 16));
    __builtin_amdgcn_sched_barrier(0);
  };
  // this lane's block of its half, chunk half * 4 + g4
  const int block = 4 * half + g4;
  const uint32_t at = static_cast<uint32_t>(r16 * kRowBytes + ((block ^ (r16 >> 1)) & 7) * 16);
  u32x4 fb[2][FM], fa[2][FN];
  uint32_t sb[2], sa[2];
  auto read = [&](auto set, int kb) {
    const lds_char *const st = lds + static_cast<uint32_t>(kb) % kMidStages * kStage;
    sb[set] = *(const lds_u32 *)(st + kScaleB + block * TA + wm * (16 * FM) + r16 * FM);
    if constexpr (FN == 4)
      sa[set] = *(const lds_u32 *)(st + kScaleA + block * TB + wn * (16 * FN) + r16 * FN);
    else
      sa[set] = *(const lds_u16 *)(st + kScaleA + block * TB + wn * (16 * FN) + r16 * FN);
#pragma unroll
    for (int i = 0; i < FM; ++i) fb[set][i] = *(const lds_u32x4 *)(st + at + (wm * FM + i) * (16 * kRowBytes));
#pragma unroll
    for (int j = 0; j < FN; ++j) fa[set][j] = *(const lds_u32x4 *)(st + kRows + at + (wn * FN + j) * (16 * kRowBytes));
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](auto set, int kb) {
    // this wave's part of the next stage has landed; all waves have used the
    // fragments of the stage before
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((kMidStages - 3) * kLoads) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue(kb + kMidStages - 1);
    // the wait for this step's fragments, before the next step's are read
#pragma unroll
    for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(fb[set][i]));
#pragma unroll
    for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(fa[set][j]));
    asm volatile("" : "+v"(sb[set]), "+v"(sa[set]));
    read(std::integral_constant<int, 1 - set>{}, kb + 1);
    each<FM>([&](auto i) {
      each<FN>([&](auto j) { acc[i][j] = q4_product<i, j>(fb[set][i], sb[set], fa[set][j], sa[set], acc[i][j]); });
    });
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> even{};
  constexpr std::integral_constant<int, 1> odd{};
#pragma unroll
  for (int u = 0; u < kMidStages - 1; ++u) issue(w.begin + u);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((kMidStages - 2) * kLoads) : "memory");
  read(even, w.begin);
  for (int kb = w.begin; kb < w.end; kb += 2) {
    step(even, kb);
    if (kb + 1 == w.end) break;
    step(odd, kb + 1);
  }
  // every wave has read its last stage, and the loads that the last steps repeated
  // have landed
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  const TileOut o = tile_out(w, TA, TB, p.base, p.out, p.out_dt, p.rows, p.outs, p.ws);
  // base comes while the halves are added
  float b[FN / 2][2][8];
  if (o.base) {
#pragma unroll
    for (int j = 0; j < FN / 2; ++j) {
      const int r = wn * (16 * FN) + r16 * FN + half * (FN / 2) + j, c = wm * (16 * FM) + g4 * (4 * FM);
      if (r >= o.rows || c >= o.cols) continue;
      load_base<8, 2>(o.base, o.dt, o.at + r * o.ld + c, 8, o.cols - c, b[j]);
    }
  }
  constexpr int kSlot = FM * FN / 2 * 1024;
  static_assert(8 * kSlot <= kMidStages * kStage);
  exchange_halves<FM, FN>(acc, half, lds + wave * kSlot, lds + (wave ^ 4) * kSlot);
#pragma unroll
  for (int j = 0; j < FN / 2; ++j) {
    const int r = wn * (16 * FN) + r16 * FN + half * (FN / 2) + j;
    if (r >= o.rows) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // eight consecutive outputs of the lane's sixteen
      const int c = wm * (16 * FM) + g4 * (4 * FM) + h * 8;
      float run[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        run[e] = acc[(h * 8 + e) % FM][j][(h * 8 + e) / FM];
        if (o.base) run[e] += b[j][h][e];
      }
      finish_run<8>(nullptr, o.out, o.dt, o.at + r * o.ld + c, o.cols - c, run);
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

// A step's time in microseconds with few work-groups on the chip and with all, from
// the slopes of times over the length of the sum.
constexpr std::initializer_list<TileCost> kCosts = {
    {256, 256, 1, 1.2f, 1.85f}, {128, 256, 1, 0.85f, 1.04f}, {128, 128, 1, 0.44f, 0.58f}, {128, 64, 1, 0.34f, 0.4f}};

// How a product runs: streamed (row blocks, output blocks and waves of a
// work-group) or in tiles.
struct Plan {
  int nt, nn, waves;  // nt = 0: tiles
  TileSplit split;
};

// Waves of a streaming work-group: one block of 16 x 16 is shared by eight where the
// sum is long enough for each to take two blocks of codes.
int stream_waves(int64_t kp, int nt, int nn) { return nt * nn == 1 && kp >= 16 * kQ4Pad ? 8 : 4; }

// The weight's time from memory at 4.9 TB/s, in microseconds.
float memory_us(int64_t outs, int64_t kp) { return static_cast<float>(outs * kp) * 0.53f / 4.9e6f; }

// The streaming kernel's time in microseconds: a work-group takes in its weight's
// and rows' codes at 53 GB/s, 256 of them at a time, while the weight comes from
// memory; a quarter of the shorter of the two does not hide.  Beside them the launch,
// the waves' sums, the start of more work-groups than CUs, and where LDS does not hold
// all of them at once the first loads' latency of the rest, which the others of a CU
// hide (100 rows of 16384 x 256, 4 x 4: 512 work-groups in two rounds, one a CU, 8.9
// us, tiles 5.4; one row of 18944 x 3584, 1 x 1: 1184 in two rounds, four a CU, 8.9,
// tiles 11.1).
float stream_us(int64_t rows, int64_t outs, int64_t kp, int nt, int nn) {
  const int64_t groups = (rows + 16 * nt - 1) / (16 * nt) * ((outs + 16 * nn - 1) / (16 * nn));
  const int xr = rows <= 8 && nt == 1 ? 8 : 16, waves = stream_waves(kp, nt, nn);
  const int64_t resident = 160 * 1024 / (waves * stream_ahead(nt, nn, waves) * stream_stage(nt, nn, xr));  // a CU
  const float sums = 0.2f + 0.09f * static_cast<float>(nt * nn);
  const float bytes = static_cast<float>((16 * nn + nt * xr) * kp) * 0.53f, turns = static_cast<float>((groups + 255) / 256);
  const float taken = turns * bytes / 53e3f, memory = memory_us(outs, kp);
  return 1.5f + sums + std::max(taken, memory) + 0.25f * std::min(taken, memory) +
         0.1f * static_cast<float>(nt * nn) * (turns - 1.f) +
         static_cast<float>((groups - 1) / (256 * resident)) * (1.f + sums) / static_cast<float>(resident);
}
// Rows up to which it is considered: 1000 of 1000 x 1000 5.6 us, tiles 6.3; 2000 of
// 1024 x 1024 are 6.7 in tiles.
constexpr int64_t kStreamRows = 1024;

Plan make_plan(int64_t rows, int64_t outs, int64_t kp) {
  Plan pl{};
  if (rows == 0 || kp == 0) return pl;
  float us;
  pl.split = choose_split(outs, rows, kp / kQ4Pad, kCosts, &us);
  us += 0.35f * memory_us(outs, kp);  // of which the steps hide the rest
  if (rows <= kStreamRows) {
    for (const int nt : {1, 2, 4})
      for (const int nn : {1, 2, 4}) {
        if (nn != 2 && nn != nt) continue;  // 1 x 1, 1 x 2, 2 x 2, 4 x 2 and 4 x 4
        const float s = stream_us(rows, outs, kp, nt, nn);
        if (s >= us) continue;
        us = s;
        pl.nt = nt;
        pl.nn = nn;
      }
    if (pl.nt) {
      pl.waves = stream_waves(kp, pl.nt, pl.nn);
      pl.split = TileSplit{};
    }
  }
  return pl;
}

// ... kept for the next call, which asks for the same sizes again: the workspace's
// bytes, the check of the workspace and the launch of one product.
Plan plan_of(int64_t rows, int64_t outs, int64_t kp) {
  static thread_local struct {
    int64_t rows, outs, kp;
    Plan plan;  // of no rows, as at first, all zero
  } last;
  if (last.rows != rows || last.outs != outs || last.kp != kp) {
    last.plan = make_plan(rows, outs, kp);
    last.rows = rows;
    last.outs = outs;
    last.kp = kp;
  }
  return last.plan;
}

template <int TA>
hipError_t launch_tiles(const Q4Product &p, const TileSplit &sp, hipStream_t st) {
  hipLaunchKernelGGL(q4_tile_kernel<TA>, dim3(sp.whole + sp.tail * sp.pieces), dim3(kTileThreads), 0, st, p, sp);
  return hipGetLastError();
}

template <int TB>
hipError_t launch_mid(const Q4Product &p, const TileSplit &sp, hipStream_t st) {
  hipLaunchKernelGGL(q4_mid_kernel<TB>, dim3(sp.whole + sp.tail * sp.pieces), dim3(kMidThreads), 0, st, p, sp);
  return hipGetLastError();
}

template <int NT, int NN, int WAVES, int XR>
hipError_t launch_stream(const Q4Product &p, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>((p.outs + 16 * NN - 1) / (16 * NN) * ((p.rows + 16 * NT - 1) / (16 * NT))));
  hipLaunchKernelGGL((q4_stream_kernel<NT, NN, WAVES, XR>), grid, dim3(WAVES * 64), 0, st, p);
  return hipGetLastError();
}

// One row block: of up to eight rows, eight are loaded.
template <int NN, int WAVES>
hipError_t launch_stream(const Q4Product &p, hipStream_t st) {
  return p.rows <= 8 ? launch_stream<1, NN, WAVES, 8>(p, st) : launch_stream<1, NN, WAVES, 16>(p, st);
}

}  // namespace

size_t q4_matmul_workspace(int64_t rows, int64_t outs, int64_t kp) { return plan_of(rows, outs, kp).split.ws_bytes(); }

Q4Choice q4_matmul_choice(int64_t rows, int64_t outs, int64_t kp) {
  const Plan pl = plan_of(rows, outs, kp);
  return Q4Choice{pl.nt, pl.nn, pl.waves, pl.nt == 0 ? 0 : pl.nt > 1 || rows > 8 ? 16 : 8, pl.split};
}

hipError_t launch_q4_matmul(const Q4Product &p, hipStream_t st) {
  if (p.kp == 0) {
    const int64_t groups = std::min<int64_t>((p.rows * p.outs + 2047) / 2048, 1 << 20);
    hipLaunchKernelGGL(q4_empty_kernel, dim3(static_cast<uint32_t>(groups)), dim3(256), 0, st, p);
    return hipGetLastError();
  }
  const Plan pl = plan_of(p.rows, p.outs, p.kp);
  if (pl.nt == 1 && pl.nn == 2) return launch_stream<2, 4>(p, st);
  if (pl.nt == 1) return pl.waves == 8 ? launch_stream<1, 8>(p, st) : launch_stream<1, 4>(p, st);
  if (pl.nt == 2) return launch_stream<2, 2, 4, 16>(p, st);
  if (pl.nt == 4) return pl.nn == 2 ? launch_stream<4, 2, 4, 16>(p, st) : launch_stream<4, 4, 4, 16>(p, st);
  const TileSplit &sp = pl.split;
  const hipError_t e = sp.ta == 256   ? launch_tiles<256>(p, sp, st)
                       : sp.tb == 256 ? launch_tiles<128>(p, sp, st)
                       : sp.tb == 128 ? launch_mid<128>(p, sp, st)
                                      : launch_mid<64>(p, sp, st);
  if (e != hipSuccess || sp.pieces == 1) return e;
  return launch_q8_reduce(static_cast<const float *>(p.ws), sp, p.rows, p.outs, p.base, p.out, p.out_dt, st);
}

}  // namespace dmuon
