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

#include <algorithm>
#include <type_traits>

#include "q4_device.h"

namespace dmuon {

namespace {

// Rows as the kernels read them: ld elements, a multiple of 8, zeros behind the
// last.  The LDS-bound loads take 16-byte chunks; those of a row's last block that
// lie behind its end come from kZeros.
struct Rows {
  const uint8_t *x;
  int64_t ld;
};
__device__ const __attribute__((aligned(16))) uint32_t kZeros[4] = {0, 0, 0, 0};

// ---- few rows: the weight's bytes ----
//
// A work-group takes 16 NN outputs of up to 16 rows, its four waves every fourth
// block of 256 codes; the waves' sums are added through LDS in wave order.
// Each wave has a ring of stages of its own in LDS, and no barrier: it waits for
// its own loads.  A block comes by LDS-bound loads: eight outputs' 128 bytes of
// codes each, the 16-byte chunks XORed with (output / 2) mod 8; two rows' 512 bytes
// each, the chunks XORed with the row; and the scales.  The weight's bytes are read
// once, the rows', four times as wide, from L2 once per 16 NN outputs: of up to XR
// rows XR are loaded.  Rows and outputs behind the last are clamped for the loads
// and not stored.
//
// Bound by the weight's bytes (one row by 14336 x 4096 8.7 us out of HBM, 7.8 out of
// the memory-side cache), with more than a few rows by what a CU takes in (16 rows
// 10.0 us, 16 of 4096 x 14336 13.1).  Two row blocks a work-group, and eight waves,
// were no faster.
//
// A lane's 32 codes of a chunk (one block of the format) are multiplied eight an
// instruction.
constexpr int kStreamWaves = 4;
constexpr int stream_stage(int nn, int xr) { return nn * (2048 + 128) + xr * 512; }
// Blocks in flight a wave.
constexpr int stream_ahead(int nn, int xr) { return 3 * kStreamWaves * stream_stage(nn, xr) <= 80 * 1024 ? 3 : 2; }

template <int NN, int XR>
__global__ __launch_bounds__(kStreamWaves * 64) void q4_rows_stream_kernel(Q4Product p, Rows x) {
  constexpr int kAhead = stream_ahead(NN, XR);
  constexpr int kScales = NN * 2048, kRows = kScales + NN * 128, kStage = stream_stage(NN, XR);
  constexpr int kLoads = 2 * NN + XR / 2 + 1;  // vector loads a block
  __shared__ __attribute__((aligned(1024))) char smem[kStreamWaves * kAhead * kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const uint32_t nt = static_cast<uint32_t>((p.outs + 16 * NN - 1) / (16 * NN)), tb = uniform(blockIdx.x / nt);
  const int64_t n0 = static_cast<int64_t>(line_tile<NN>(blockIdx.x - tb * nt, nt)) * (16 * NN);
  const int64_t t0 = static_cast<int64_t>(tb) * 16;
  const int nkb = static_cast<int>(p.kp / kQ4Pad), chunks = static_cast<int>(x.ld / 8);
  const uint32_t kpb = static_cast<uint32_t>(p.kp / 2), ldb = static_cast<uint32_t>(x.ld * 2);
  const int64_t rb = (p.outs + kQ4ScaleRow - 1) & ~static_cast<int64_t>(kQ4ScaleRow - 1);
  lds_char *const ring = (lds_char *)smem + wave * (kAhead * kStage);
  // lane l of 1 KB load h of the codes fills LDS row 8 h + l / 8, physical chunk
  // l % 8; of the rows LDS row 2 h + l / 32, physical chunk l % 32
  const uint8_t *const gb = p.b + n0 * kpb, *const ga = x.x + t0 * ldb;
  const int lim_n = static_cast<int>(min(p.outs - 1 - n0, static_cast<int64_t>(16 * NN - 1)));
  const int lim_t = static_cast<int>(min(p.rows - 1 - t0, static_cast<int64_t>(15)));
  uint32_t ob[NN][2], oa[XR / 2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = 8 * h + (lane >> 3);
    const uint32_t chunk = static_cast<uint32_t>((lane & 7) ^ ((row >> 1) & 7)) * 16;
#pragma unroll
    for (int i = 0; i < NN; ++i)
      ob[i][h] = __umul24(static_cast<uint32_t>(min(i * 16 + row, lim_n)), kpb) + chunk;
  }
#pragma unroll
  for (int h = 0; h < XR / 2; ++h) {
    const int row = 2 * h + (lane >> 5);
    oa[h] = __umul24(static_cast<uint32_t>(min(row, lim_t)), ldb) + static_cast<uint32_t>((lane & 31) ^ (row & 15)) * 16;
  }
  // the scales of a stage, 16 bytes a lane: [block][16 NN outputs]
  const uint8_t *const scale0 = p.sb + lane / NN % 8 * rb + min(n0 + lane % NN * 16, rb - 16);
  f32x4 acc[NN];
#pragma unroll
  for (int i = 0; i < NN; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto load = [&](int u, int block) {
    const int kb = min(block, nkb - 1);
    lds_char *const st = ring + u * kStage;
    auto piece = [&](const uint8_t *src, int at) {
      __builtin_amdgcn_global_load_lds((const void *)src, (__attribute__((address_space(3))) void *)(st + at), 16, 0, 0);
    };
    const uint8_t *const bb = gb + static_cast<int64_t>(kb) * 128, *const ba = ga + static_cast<int64_t>(kb) * 512;
#pragma unroll
    for (int i = 0; i < NN; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) piece(bb + ob[i][h], i * 2048 + h * 1024);
    if (kb == nkb - 1 && chunks % 32 != 0) {
#pragma unroll
      for (int h = 0; h < XR / 2; ++h) {
        const int chunk = kb * 32 + ((lane & 31) ^ ((2 * h + (lane >> 5)) & 15));
        piece(chunk < chunks ? ba + oa[h] : (const uint8_t *)kZeros, kRows + h * 1024);
      }
    } else {
#pragma unroll
      for (int h = 0; h < XR / 2; ++h) piece(ba + oa[h], kRows + h * 1024);
    }
    if (lane < 8 * NN) piece(scale0 + static_cast<int64_t>(kb) * (kQ4Pad / kQ4Block) * rb, kScales);
    __builtin_amdgcn_sched_barrier(0);
  };
  const uint32_t at_b = static_cast<uint32_t>(r16 * 128 + ((g4 ^ (r16 >> 1)) & 7) * 16);
  const int xrow = r16 & (XR - 1);
  u32x4 fb[NN][2], fa[8];
  float s[NN][2];
  auto read = [&](int u) {
    const lds_char *const st = ring + u * kStage;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < NN; ++i) {
        fb[i][h] = *(const lds_u32x4 *)(st + i * 2048 + (h ? at_b ^ 64 : at_b));
        s[i][h] = q4_half_scale(*(const lds_u8 *)(st + kScales + (4 * h + g4) * (16 * NN) + i * 16 + r16));
      }
#pragma unroll
      for (int d = 0; d < 4; ++d)
        fa[4 * h + d] = *(const lds_u32x4 *)(st + kRows + xrow * 512 + (((4 * h + g4) * 4 + d) ^ xrow) * 16);
    }
    // all are in registers before the stage is loaded again
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int i = 0; i < NN; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q4_expand8(fb[i][h][d], s[i][h]),
                                                           __builtin_bit_cast(bf16x8, fa[4 * h + d]), acc[i], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, wave + u * kStreamWaves);
  // each stage takes the block kAhead further on as soon as it has been read; the
  // last kAhead blocks load nothing more
  int k0 = wave;
  for (; k0 + kStreamWaves * kAhead < nkb; k0 += kStreamWaves * kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 1) * kLoads) : "memory");
      read(u);
      load(u, k0 + (kAhead + u) * kStreamWaves);
      multiply();
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (k0 + u * kStreamWaves < nkb) {
      read(u);
      multiply();
    }
  // the waves' sums, each in its own part of the ring
  auto part = [&](int w, int b) { return (lds_f32x4 *)((lds_char *)smem + w * (kAhead * kStage) + b * 1024 + lane * 16); };
  static_assert(NN * 1024 <= kAhead * kStage && NN <= kStreamWaves);
#pragma unroll
  for (int i = 0; i < NN; ++i) *part(wave, i) = acc[i];
  __syncthreads();
  if (wave >= NN) return;
  f32x4 sum = *part(0, wave);
#pragma unroll
  for (int w = 1; w < kStreamWaves; ++w) sum += *part(w, wave);
  const int64_t t = t0 + r16, n = n0 + wave * 16 + 4 * g4;
  if (t >= p.rows) return;
  float v[4] = {2.f * sum[0], 2.f * sum[1], 2.f * sum[2], 2.f * sum[3]};
  finish_run<4>(nullptr, p.out, p.out_dt, t * p.outs + n, p.outs - n, v);
}

// ---- tiles: many rows ----
//
// One work-group of 8 waves (2 x 4) computes TA (128 or 256) outputs of the weight
// by 256 rows, TB below; each wave TA/2 x TB/4 in 16 x 16 blocks.  K advances 64 elements per step: 128
// bytes of a row, and a quarter of the 256 codes (128 bytes) that a stage of the
// weight holds.  Both come into LDS by LDS-bound loads (16 bytes a lane, 128-byte
// rows, the 16-byte chunk XORed with (row / 2) mod 8), in a ring of two stages each: a
// step loads the next step's rows and a quarter of the next stage of the weight.  The
// XOR is the 4-bit product's, where it keeps the fragment reads off each other's banks;
// here, where a lane reads chunks 2 g4 and 2 g4 + 1 of a row, half of the cycles in
// which LDS is active (30% of all) are conflicts.  The two halves of the work-group
// (wm) run in ping-pong: one half's waves read fragments and issue loads while the
// other half's expand and multiply, switching at every barrier.
//
// 2048 rows by 14336 x 4096 take 175 to 180 us, 1.34 to 1.37 PFLOP/s, a large library
// product's rate (1.36).  The matrix instructions, busy 54% of the cycles, and the
// expansions alone, their operands left in registers, take 123 us, everything else
// without them 134, without the loads 158, without the stores 169: neither hides the
// other.  On zeros the whole takes 169, so the clock that power leaves is little of it.
// Expansions placed between the matrix instructions by hand were slower (128 x 256: 65
// -> 70 us of 2048 rows by 4096 x 4096).
//
// A lane's 16 codes of a step are k = 16 g4 + 0 .. 15, eight of them an instruction.
// The order of rows in LDS is that of the 4-bit product's tiles.
constexpr int kTileThreads = 512, kTileRows = 256;
constexpr int kRowBytes = 128;
constexpr int kStep = 64, kStageSteps = kQ4Pad / kStep;
constexpr int kStageBlocks = kQ4Pad / kQ4Block;

template <int TA>
__device__ __forceinline__ void q4_rows_tile(lds_char *const lds, const Q4Product &p, const Rows &x, int64_t n0,
                                             int64_t t0, int kbeg, int kend, f32x4 (&acc)[TA / 32][kTileRows / 64]) {
  constexpr int TB = kTileRows, FM = TA / 32, FN = TB / 64;
  // two stages of the weight with its scales (each half's [block][output]), two
  // of the rows
  constexpr int kScales = TA * kRowBytes, kWeight = kScales + TA * kStageBlocks, kRows = TB * kRowBytes;
  lds_char *const lds_x = lds + 2 * kWeight;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int r16 = lane & 15, g4 = lane >> 4;
  const uint32_t kpb = static_cast<uint32_t>(p.kp / 2), ldb = static_cast<uint32_t>(x.ld * 2);
  const int chunks = static_cast<int>(x.ld / 8);
  const int64_t rb = (p.outs + kQ4ScaleRow - 1) & ~static_cast<int64_t>(kQ4ScaleRow - 1);

  const uint8_t *const gb = p.b + n0 * kpb, *const ga = x.x + t0 * ldb;
  // the last output and row of the tile that exist
  const int lim_n = static_cast<int>(min(p.outs - 1 - n0, static_cast<int64_t>(TA - 1)));
  const int lim_t = static_cast<int>(min(p.rows - 1 - t0, static_cast<int64_t>(TB - 1)));
  // scales: 16 outputs a lane, TA/32 lanes a block
  const uint8_t *const gsb = p.sb + lane / (TA / 32) * rb + min(n0 + wm * (TA / 2) + lane % (TA / 32) * 16, rb - 16);
  // loads: lane l of 1 KB load j of a half fills LDS row (j * 4 + wn) * 8 + l / 8,
  // physical chunk l % 8
  const int q = (wn & 1) * 8 + (lane >> 3);
  const uint32_t chunk = static_cast<uint32_t>((lane & 7) ^ (((wn & 1) * 4 + (lane >> 4)) & 7)) * 16;
  const int base_n = ((q & 3) * 4 + (q >> 2)) * FM + (wn >> 1) + wm * (TA / 2);
  const int base_t = q * FN + (wn >> 1);
  auto piece = [&](const uint8_t *src, lds_char *to) {
    __builtin_amdgcn_global_load_lds((const void *)src, (__attribute__((address_space(3))) void *)to, 16, 0, 0);
  };
  auto load = [&](const uint8_t *src, int row, uint32_t bytes, lds_char *to) {
    piece(src + (__umul24(static_cast<uint32_t>(row), bytes) + chunk), to + wn * 1024);
  };
  // part j (of kStageSteps) of this half's codes of stage kb, and their scales
  auto issue_weight = [&](int kb, int j) {
    lds_char *const st = lds + (kb & 1) * kWeight;
    const int last = static_cast<int>(p.kp / kQ4Pad) - 1;
    const int64_t k = min(kb, last);
    if (j < TA / 64) load(gb + k * kRowBytes, min(base_n + 2 * j, lim_n), kpb, st + wm * (kScales / 2) + j * 4096);
    if (j == kStageSteps - 1 && wn == 3 && lane < TA / 4)
      piece(gsb + k * kStageBlocks * rb, st + kScales + wm * (TA / 2 * kStageBlocks));
  };
  auto issue_rows = [&](int slot, int ks) {
    if (wm != 0) return;
    lds_char *const st = lds_x + slot * kRows;
    int bt = base_t;
    // opaque: the offsets are rebuilt at every issue instead of being kept
    // live across the loop
    asm volatile("" : "+v"(bt));
    const uint8_t *const at = ga + static_cast<int64_t>(ks) * kRowBytes;
    auto each_load = [&](auto go) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < TB / 64; ++j) {
          // row s of the tile's LDS rows: quarter s / (TB / 4), then block and column
          const int s = h * (TB / 2) + j * 32, in_quarter = s % (TB / 4);
          go(min(bt + s / (TB / 4) * (TB / 4) + in_quarter / 16, lim_t), st + s * kRowBytes);
        }
    };
    if ((ks + 1) * 8 > chunks) {
      const bool in = ks * 8 + static_cast<int>(chunk / 16) < chunks;
      each_load([&](int row, lds_char *to) {
        const uint8_t *const src = at + (__umul24(static_cast<uint32_t>(row), ldb) + chunk);
        piece(in ? src : (const uint8_t *)kZeros, to + wn * 1024);
      });
    } else {
      each_load([&](int row, lds_char *to) { load(at, row, ldb, to); });
    }
  };

#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int first = kbeg * kStageSteps;
  const int end = min(kend * kStageSteps, (chunks + 7) / 8);
#pragma unroll
  for (int j = 0; j < kStageSteps; ++j) issue_weight(kbeg, j);
  issue_rows(first & 1, first);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if (wm == 1) barrier();
  for (int ks = first; ks < end; ++ks) {
    const int kb = ks / kStageSteps, part = ks % kStageSteps;
    const lds_char *const st = lds + (kb & 1) * kWeight;
    const lds_char *const opb = st + wm * (kScales / 2);
    const lds_char *const opa = lds_x + (ks & 1) * kRows + wn * (TB / 4 * kRowBytes);
    // the last step loads its own rows again, into the free stage, which keeps the
    // loop free of a branch
    issue_rows((ks + 1) & 1, min(ks + 1, end - 1));
    issue_weight(kb + 1, part);
    u32x2 fb[FM];
    u32x4 fa[FN][2];
    uint32_t sb[FM / 4];
    const int block = 2 * part + (g4 >> 1);
    const lds_char *const ws =
        st + kScales + wm * (TA / 2 * kStageBlocks) + block * (TA / 2) + ((r16 & 3) * 4 + (r16 >> 2)) * FM;
    if constexpr (FM == 8) {
      const u32x2 w = *(const lds_u32x2 *)ws;
      sb[0] = w.x;
      sb[1] = w.y;
    } else {
      sb[0] = *(const lds_u32 *)ws;
    }
    const uint32_t at_b = static_cast<uint32_t>(r16 * kRowBytes + ((block ^ (r16 >> 1)) & 7) * 16 + (g4 & 1) * 8);
#pragma unroll
    for (int i = 0; i < FM; ++i) fb[i] = *(const lds_u32x2 *)(opb + at_b + i * (16 * kRowBytes));
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int d = 0; d < 2; ++d)
        fa[j][d] = *(const lds_u32x4 *)(opa + r16 * kRowBytes + (((2 * g4 + d) ^ (r16 >> 1)) & 7) * 16 + j * (16 * kRowBytes));
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const float s = q4_half_scale(sb[i / 4] >> (8 * (i % 4)) & 0xff);
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const bf16x8 xb = q4_expand8(fb[i][d], s);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, __builtin_bit_cast(bf16x8, fa[j][d]), acc[i][j], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }
  if (wm == 0) barrier();
}

template <int TA>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(2)))
void q4_rows_tile_kernel(Q4Product p, Rows x, TileSplit sp) {
  constexpr int TB = kTileRows, FM = TA / 32, FN = TB / 64;
  __shared__ __attribute__((aligned(1024))) char smem[2 * (TA * (kRowBytes + kStageBlocks) + TB * kRowBytes)];
  const TileWork w = tile_work(sp, blockIdx.x, static_cast<uint32_t>(p.kp / kQ4Pad));
  const int64_t n0 = static_cast<int64_t>(w.a) * TA, t0 = static_cast<int64_t>(w.b) * TB;
  f32x4 acc[FM][FN];
  q4_rows_tile<TA>((lds_char *)smem, p, x, n0, t0, w.begin, w.end, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 2, wn = wave & 3, r16 = lane & 15, g4 = lane >> 4;
  const TileOut o = tile_out(w, TA, TB, nullptr, p.out, p.out_dt, p.rows, p.outs, p.ws);
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int r = wn * (TB / 4) + r16 * FN + j;
    if (r >= o.rows) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int c = wm * (TA / 2) + (v * 4 + g4) * FM;
      float run[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i) run[i] = 2.f * acc[i][j][v];
      finish_run<FM>(nullptr, o.out, o.dt, o.at + r * o.ld + c, o.cols - c, run);
    }
  }
}

// ---- small tiles: a deep ring ----
//
// 128 outputs by TB (64 or 128) rows, one work-group a CU, for launches of few tiles,
// which the latency of a step bounds.  Eight waves: four parts of the tile, of 64 x
// 64 or 32 x 64, and two halves of a step's 128 elements, whose sums are added at the
// end (each code is then expanded by half as many waves).  Two rings, a longer one of
// the weight, which comes from memory, and one of the rows, which come from L2: a
// step waits for the next one's stage, loaded as many steps ago as the ring allows,
// meets the other waves once, loads the stages that all of them have left, reads the
// next step's fragments and multiplies its own.  An output's codes are 64 bytes of a
// stage, their 16-byte chunks XORed with (output / 4) mod 4, a row's elements 256
// bytes, their chunks XORed with the row.
//
// A step of 256 elements takes 1.75 us for 128 x 128 (2.0 with one ring of three
// stages, 2.5 with two and ping-pong) and 0.97 for 128 x 64: about half the matrix
// instructions' alone (0.56 for 128 x 64, expansions 0.03 more), the rest what LDS
// takes in and gives out between barriers.  64 x 64 parts with the sum shared by four
// waves, which read 44% less from LDS, and reads and loads spread between the matrix
// instructions were no faster (64 rows by 14336 x 4096 in these tiles 22.5 us, so
// 24.3 and 25.0).
//
// Block i, row q of a wave's weight part holds output q * FM + i, block j, column r
// of its rows row r * FN + j.
constexpr int kMidThreads = 512, kMidStep = 128;

template <int TB>
__global__ __launch_bounds__(kMidThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void q4_rows_mid_kernel(Q4Product p, Rows x, TileSplit sp) {
  constexpr int TA = 128, WN = TB / 64, WM = 4 / WN;
  constexpr int FM = TA / WM / 16, FN = 4, kBlocks = kMidStep / kQ4Block;
  // stages of the weight (codes, then scales) and of the rows
  constexpr int kWeightStages = 6, kRowStages = TB == 128 ? 3 : 4;
  constexpr int kScales = TA * kMidStep / 2, kWeight = kScales + TA * kBlocks, kRows = TB * kMidStep * 2;
  constexpr int kRowLoads = TB / 32, kLoads = kRowLoads + 2;  // vector loads a wave and step
  __shared__ __attribute__((aligned(1024))) char smem[kRowStages * kRows + kWeightStages * kWeight];
  lds_char *const lds = (lds_char *)smem, *const lds_w = lds + kRowStages * kRows;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave >> 2, wm = (wave & 3) / WN, wn = (wave & 3) % WN, r16 = lane & 15, g4 = lane >> 4;
  const TileWork w = tile_work(sp, blockIdx.x, static_cast<uint32_t>(p.kp / kQ4Pad));
  const int64_t n0 = static_cast<int64_t>(w.a) * TA, t0 = static_cast<int64_t>(w.b) * TB;
  const int begin = w.begin * (kQ4Pad / kMidStep);
  const int chunks = static_cast<int>(x.ld / 8);
  const int end = min(w.end * (kQ4Pad / kMidStep), (chunks + 15) / 16);
  const uint32_t kpb = static_cast<uint32_t>(p.kp / 2), ldb = static_cast<uint32_t>(x.ld * 2);
  const int64_t rb = (p.outs + kQ4ScaleRow - 1) & ~static_cast<int64_t>(kQ4ScaleRow - 1);
  const int lim_n = static_cast<int>(min(p.outs - 1 - n0, static_cast<int64_t>(TA - 1)));
  const int lim_t = static_cast<int>(min(p.rows - 1 - t0, static_cast<int64_t>(TB - 1)));
  // a wave's load of codes fills LDS rows 16 wave + l / 4, physical chunk l % 4; its
  // load j of the rows LDS rows 4 (wave + 8 j) + l / 16, physical chunk l % 16
  uint32_t ob, oa[kRowLoads];
  {
    const int part = wave / FM, i = wave % FM, q = lane >> 2;
    ob = __umul24(static_cast<uint32_t>(min(part * (16 * FM) + q * FM + i, lim_n)), kpb) +
         static_cast<uint32_t>((lane & 3) ^ ((q >> 2) & 3)) * 16;
  }
#pragma unroll
  for (int j = 0; j < kRowLoads; ++j) {
    const int l = 4 * (wave + 8 * j) + (lane >> 4), part = l / (16 * FN), i = l / 16 % FN, q = l % 16;
    oa[j] = __umul24(static_cast<uint32_t>(min(part * (16 * FN) + q * FN + i, lim_t)), ldb) +
            static_cast<uint32_t>((lane & 15) ^ q) * 16;
  }
  const uint8_t *const gb = p.b + n0 * kpb, *const ga = x.x + t0 * ldb;
  // scales, 16 bytes a lane and four lanes a wave: [block][output]
  const int s16 = wave * 4 + (lane & 3);
  const uint8_t *const gs = p.sb + s16 / (TA / 16) * rb + min(n0 + s16 % (TA / 16) * 16, rb - 16);
  auto piece = [&](const uint8_t *src, lds_char *to) {
    __builtin_amdgcn_global_load_lds((const void *)src, (__attribute__((address_space(3))) void *)to, 16, 0, 0);
  };
  auto issue_rows = [&](int ks) {
    lds_char *const st = lds + static_cast<uint32_t>(ks) % kRowStages * kRows;
    const int k = min(ks, end - 1);
    const uint8_t *const at = ga + static_cast<int64_t>(k) * (kMidStep * 2);
    if ((k + 1) * 16 > chunks) {
#pragma unroll
      for (int j = 0; j < kRowLoads; ++j) {
        const int chunk = k * 16 + ((lane & 15) ^ ((4 * (wave + 8 * j) + (lane >> 4)) & 15));
        piece(chunk < chunks ? at + oa[j] : (const uint8_t *)kZeros, st + (wave + 8 * j) * 1024);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kRowLoads; ++j) piece(at + oa[j], st + (wave + 8 * j) * 1024);
    }
  };
  auto issue_weight = [&](int ks) {
    lds_char *const st = lds_w + static_cast<uint32_t>(ks) % kWeightStages * kWeight;
    const int64_t k = min(ks, end - 1);
    piece(gb + k * (kMidStep / 2) + ob, st + wave * 1024);
    if (lane < 4) piece(gs + k * kBlocks * rb, st + kScales + wave * 64);
    __builtin_amdgcn_sched_barrier(0);
  };
  // this lane's sixteen elements of its half: k = 16 g4 + 0 .. 15
  const int block = 2 * half + (g4 >> 1);
  const int at_b = (wm * (16 * FM) + r16) * 64 + ((block ^ (r16 >> 2)) & 3) * 16 + (g4 & 1) * 8;
  const int at_s = kScales + block * TA + wm * (16 * FM) + r16 * FM;
  u32x2 fb[2][FM];
  u32x4 fa[2][FN][2];
  uint32_t sb[2];
  auto read = [&](auto set, int ks) {
    const lds_char *const sw = lds_w + static_cast<uint32_t>(ks) % kWeightStages * kWeight;
    const lds_char *const sx = lds + static_cast<uint32_t>(ks) % kRowStages * kRows + (wn * (16 * FN) + r16) * 256;
    if constexpr (FM == 4)
      sb[set] = *(const lds_u32 *)(sw + at_s);
    else
      sb[set] = *(const lds_u16 *)(sw + at_s);
#pragma unroll
    for (int i = 0; i < FM; ++i) fb[set][i] = *(const lds_u32x2 *)(sw + at_b + i * (16 * 64));
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fa[set][j][d] = *(const lds_u32x4 *)(sx + j * (16 * 256) + (((8 * half + 2 * g4 + d) ^ r16) & 15) * 16);
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](auto set, int ks) {
    // this wave's part of the next stages has landed (the rows' were loaded
    // kRowStages - 2 steps ago, before that step's part of the weight, the weight's
    // earlier); all waves have used the fragments of the stages before
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((kRowStages - 3) * kLoads + 2) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue_rows(ks + kRowStages - 1);
    issue_weight(ks + kWeightStages - 1);
    // the wait for this step's fragments, before the next step's are read
#pragma unroll
    for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(fb[set][i]));
#pragma unroll
    for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(fa[set][j][0]), "+v"(fa[set][j][1]));
    asm volatile("" : "+v"(sb[set]));
    read(std::integral_constant<int, 1 - set>{}, ks + 1);
    float s[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) s[i] = q4_half_scale(sb[set] >> (8 * i) & 0xff);
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const bf16x8 xb = q4_expand8(fb[set][i][d], s[i]);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, __builtin_bit_cast(bf16x8, fa[set][j][d]), acc[i][j], 0, 0, 0);
      }
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> even{};
  constexpr std::integral_constant<int, 1> odd{};
  // the steps' waits count on their order of loads: the last stages as the steps
  // would have loaded them
  constexpr int kFirst = kWeightStages - kRowStages;
#pragma unroll
  for (int u = 0; u < kFirst; ++u) issue_weight(begin + u);
#pragma unroll
  for (int u = 0; u < kRowStages - 1; ++u) {
    issue_rows(begin + u);
    issue_weight(begin + kFirst + u);
  }
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((kRowStages - 2) * kLoads + 2) : "memory");
  read(even, begin);
  for (int ks = begin; ks < end; ks += 2) {
    step(even, ks);
    if (ks + 1 == end) break;
    step(odd, ks + 1);
  }
  // every wave has read its last stage, and the loads that the last steps repeated
  // have landed
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  constexpr int kSlot = FM * FN / 2 * 1024;
  static_assert(8 * kSlot <= sizeof(smem));
  exchange_halves<FM, FN>(acc, half, lds + wave * kSlot, lds + (wave ^ 4) * kSlot);
  const TileOut o = tile_out(w, TA, TB, nullptr, p.out, p.out_dt, p.rows, p.outs, p.ws);
#pragma unroll
  for (int j = 0; j < FN / 2; ++j) {
    const int r = wn * (16 * FN) + r16 * FN + half * (FN / 2) + j;
    if (r >= o.rows) continue;
#pragma unroll
    for (int h = 0; h < FM / 2; ++h) {
      // eight consecutive outputs of the lane's 4 FM
      const int c = wm * (16 * FM) + g4 * (4 * FM) + h * 8;
      float run[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) run[e] = 2.f * acc[(h * 8 + e) % FM][j][(h * 8 + e) / FM];
      finish_run<8>(nullptr, o.out, o.dt, o.at + r * o.ld + c, o.cols - c, run);
    }
  }
}

// A step's time in microseconds with few work-groups on the chip and with all, from
// the slopes of times over the length of the sum.
constexpr std::initializer_list<TileCost> kCosts = {
    {256, 256, 1, 4.6f, 5.9f}, {128, 256, 1, 3.2f, 3.5f}, {128, 128, 1, 1.75f, 2.1f}, {128, 64, 1, 0.97f, 1.15f}};

// How a product runs: streamed (output blocks of a work-group) or in tiles; its
// rows' distance; and the bytes of its workspace's two parts, the padded rows and
// the pieces' results.
struct Plan {
  int nn;  // 0: tiles
  TileSplit split;
  int64_t ld;
  size_t pad_bytes, piece_bytes;
};

// Rows that a streaming work-group loads.
int64_t stream_rows(int64_t rows) { return rows > 8 ? 16 : rows > 4 ? 8 : rows > 2 ? 4 : 2; }

// The weight's time from memory at 4.9 TB/s, in microseconds.
float memory_us(int64_t outs, int64_t kp) { return static_cast<float>(outs * kp) * 0.53f / 4.9e6f; }

// The streaming kernel's time in microseconds: a work-group takes in its weight's
// codes and its rows at 62 GB/s, 256 of them at a time, while the weight comes from
// memory; a quarter of the shorter of the two does not hide.  Beside them the launch,
// of several turns the last work-groups' end and, where LDS does not hold all
// work-groups at once, the first loads' latency of the rest, which the others of a CU
// hide (512 rows of 2048 x 1024, 64 outputs each: 1024 work-groups in four rounds, one
// a CU, 13.3 us, tiles 8.7; one row of 18944 x 3584, 16 outputs each: 1184 in two
// rounds, four a CU, 9.7, 64 outputs each 11.5).
float stream_us(int64_t rows, int64_t outs, int64_t kp, int nn) {
  const int64_t groups = (rows + 15) / 16 * ((outs + 16 * nn - 1) / (16 * nn));
  const int xr = static_cast<int>(stream_rows(rows));
  const int64_t resident = 160 * 1024 / (kStreamWaves * stream_ahead(nn, xr) * stream_stage(nn, xr));  // a CU
  const float work = static_cast<float>(kp) * (16 * nn * 0.53f + 2.f * static_cast<float>(xr)) / 62e3f;
  const int64_t turns = (groups + 255) / 256;
  const float taken = static_cast<float>(turns) * work, memory = memory_us(outs, kp);
  return 1.8f + std::max(taken, memory) + 0.25f * std::min(taken, memory) + (turns > 1 ? 0.3f * work : 0.f) +
         static_cast<float>((groups - 1) / (256 * resident)) * 2.2f / static_cast<float>(resident);
}
// Rows up to which it is considered: 512 of 512 x 512 3.8 us, tiles 6.2; 1000 of 1000
// x 1000 13.4, tiles 9.4.
constexpr int64_t kStreamRows = 1024;

Plan make_plan(int64_t rows, int64_t outs, int64_t inner) {
  Plan pl{};
  if (rows == 0) return pl;
  const int64_t kp = (inner + kQ4Pad - 1) / kQ4Pad * kQ4Pad;
  float us;
  pl.split = choose_split(outs, rows, kp / kQ4Pad, kCosts, &us);
  us += 0.35f * memory_us(outs, kp);  // of which the steps hide the rest
  if (rows <= kStreamRows) {
    for (const int nn : {1, 2, 4}) {
      const float s = stream_us(rows, outs, kp, nn);
      if (s >= us) continue;
      us = s;
      pl.nn = nn;
    }
    if (pl.nn) pl.split = TileSplit{};
  }
  pl.ld = (inner + 7) / 8 * 8;
  if (pl.ld != inner) pl.pad_bytes = (static_cast<size_t>(rows * pl.ld * 2) + 255) & ~static_cast<size_t>(255);
  pl.piece_bytes = pl.split.ws_bytes();
  return pl;
}

// ... kept for the next call, which asks for the same sizes again: the workspace's
// bytes, the check of the workspace and the launch of one product.
Plan plan_of(int64_t rows, int64_t outs, int64_t inner) {
  static thread_local struct {
    int64_t rows, outs, inner;
    Plan plan;  // of no rows, as at first, all zero
  } last;
  if (last.rows != rows || last.outs != outs || last.inner != inner) {
    last.plan = make_plan(rows, outs, inner);
    last.rows = rows;
    last.outs = outs;
    last.inner = inner;
  }
  return last.plan;
}

template <int TA>
hipError_t launch_tiles(const Q4Product &p, const Rows &x, const TileSplit &sp, hipStream_t st) {
  hipLaunchKernelGGL(q4_rows_tile_kernel<TA>, dim3(sp.whole + sp.tail * sp.pieces), dim3(kTileThreads), 0, st, p, x, sp);
  return hipGetLastError();
}

template <int TB>
hipError_t launch_mid(const Q4Product &p, const Rows &x, const TileSplit &sp, hipStream_t st) {
  hipLaunchKernelGGL(q4_rows_mid_kernel<TB>, dim3(sp.whole + sp.tail * sp.pieces), dim3(kMidThreads), 0, st, p, x, sp);
  return hipGetLastError();
}

template <int NN, int XR>
hipError_t launch_stream(const Q4Product &p, const Rows &x, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>((p.outs + 16 * NN - 1) / (16 * NN) * ((p.rows + 15) / 16)));
  hipLaunchKernelGGL((q4_rows_stream_kernel<NN, XR>), grid, dim3(kStreamWaves * 64), 0, st, p, x);
  return hipGetLastError();
}

template <int NN>
hipError_t launch_stream(const Q4Product &p, const Rows &x, hipStream_t st) {
  switch (stream_rows(p.rows)) {
    case 2: return launch_stream<NN, 2>(p, x, st);
    case 4: return launch_stream<NN, 4>(p, x, st);
    case 8: return launch_stream<NN, 8>(p, x, st);
    default: return launch_stream<NN, 16>(p, x, st);
  }
}

}  // namespace

size_t q4_rows_workspace(int64_t rows, int64_t outs, int64_t inner) {
  const Plan pl = plan_of(rows, outs, inner);
  return pl.pad_bytes + pl.piece_bytes;
}

Q4Choice q4_rows_choice(int64_t rows, int64_t outs, int64_t inner) {
  const Plan pl = plan_of(rows, outs, inner);
  if (pl.nn == 0) return Q4Choice{0, 0, 0, 0, pl.split};
  return Q4Choice{1, pl.nn, kStreamWaves, static_cast<int32_t>(stream_rows(rows)), pl.split};
}

hipError_t launch_q4_rows(const Q4Product &args, hipStream_t st) {
  Q4Product p = args;
  const Plan pl = plan_of(p.rows, p.outs, p.inner);
  Rows x{static_cast<const uint8_t *>(p.a), pl.ld};
  if (pl.pad_bytes) {
    const hipError_t e = launch_pad_rows(p.a, p.rows, p.inner, pl.ld, p.ws, st);
    if (e != hipSuccess) return e;
    x.x = static_cast<const uint8_t *>(p.ws);
    p.ws = static_cast<char *>(p.ws) + pl.pad_bytes;
  }
  if (pl.nn == 1) return launch_stream<1>(p, x, st);
  if (pl.nn == 2) return launch_stream<2>(p, x, st);
  if (pl.nn == 4) return launch_stream<4>(p, x, st);
  const TileSplit &sp = pl.split;
  const hipError_t e = sp.ta == 256   ? launch_tiles<256>(p, x, sp, st)
                       : sp.tb == 256 ? launch_tiles<128>(p, x, sp, st)
                       : sp.tb == 128 ? launch_mid<128>(p, x, sp, st)
                                      : launch_mid<64>(p, x, sp, st);
  if (e != hipSuccess || sp.pieces == 1) return e;
  return launch_q8_reduce(static_cast<const float *>(p.ws), sp, p.rows, p.outs, nullptr, p.out, p.out_dt, st);
}

}  // namespace dmuon
