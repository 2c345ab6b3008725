// The weight gradient from an 8-bit checkpoint on gfx950 matrix cores.
//
//   out[n][k] = base[n][k] + sum_t dy[t][n] 2^e[k / 128][t] x[t][k]
//
// The sum runs over t, along which the checkpoint's scales change, so they
// cannot ride on an 8-bit matrix instruction.  Code times half the scale is
// exact in bf16 (four significant bits; 448 * 2^119 is in range, 256 * 2^120, the
// code of the lowest bf16 or fp32 value, would not be, and 2^-9 * 2^-118 is a
// subnormal that expansion and product keep), so x is expanded to bf16 on its way
// into LDS and multiplied with the bf16 gradient; sums are fp32, half of the
// result's.
//
// Bound by LDS reads and the matrix cores in turn: 8192 rows, 14336 x 4096
// outputs, take 766 to 815 us, 1.2 PFLOP/s (a library bf16 product of that size
// 1.38).  With few outputs the fp32 pieces and the reduce launch add to it:
// 4096 rows, 1024 x 4096 outputs, 53 us.

#include <algorithm>

#include "q8_device.h"

namespace dmuon {

namespace {

constexpr int kThreads = 512;
constexpr int kStep = 64;               // rows of t per step
constexpr int kHalfBytes = kStep * 256;  // 128 bf16 columns of a step

// LDS holds dy as halves of 128 columns, a row of a half being one t (256
// bytes).  The 16-byte chunk of a row is XORed with this, so that the
// transposing reads below (16 rows x 32 bytes) touch distinct banks.
__device__ __forceinline__ int swz(int row) { return ((row & 3) | (((row >> 3) & 1) << 2)) << 1; }

// An MFMA operand: eight consecutive t of one column, by two transposing reads
// of four.
struct Fragment {
  u32x2 lo, hi;
  __device__ __forceinline__ bf16x8 get() const {
    return __builtin_bit_cast(bf16x8, u32x4{lo.x, lo.y, hi.x, hi.y});
  }
};

// A step's fragments of FN 16-column blocks, from the blocks' addresses in dy's
// stage.  A read gives four consecutive t of one column: within 16 lanes, lane 4
// e + q names row t0 + e, columns 4 q .. 4 q + 3, and lane j receives rows t0 ..
// t0 + 3 of column j; rows are 256 bytes apart.  Inline assembly, because before
// the builtin the compiler waits for every LDS-bound load in flight (it cannot
// tell the stages apart); one block with its wait, so that no register that a
// read is still to fill is seen outside it.  The wait covers the LDS reads before
// it, too.
__device__ __forceinline__ void read_fragments(const uint32_t (&at)[4], Fragment (&f)[2][4]) {
  asm volatile(
      "ds_read_b64_tr_b16 %0, %16\n\tds_read_b64_tr_b16 %1, %16 offset:1024\n\t"
      "ds_read_b64_tr_b16 %2, %17\n\tds_read_b64_tr_b16 %3, %17 offset:1024\n\t"
      "ds_read_b64_tr_b16 %4, %18\n\tds_read_b64_tr_b16 %5, %18 offset:1024\n\t"
      "ds_read_b64_tr_b16 %6, %19\n\tds_read_b64_tr_b16 %7, %19 offset:1024\n\t"
      "ds_read_b64_tr_b16 %8, %16 offset:8192\n\tds_read_b64_tr_b16 %9, %16 offset:9216\n\t"
      "ds_read_b64_tr_b16 %10, %17 offset:8192\n\tds_read_b64_tr_b16 %11, %17 offset:9216\n\t"
      "ds_read_b64_tr_b16 %12, %18 offset:8192\n\tds_read_b64_tr_b16 %13, %18 offset:9216\n\t"
      "ds_read_b64_tr_b16 %14, %19 offset:8192\n\tds_read_b64_tr_b16 %15, %19 offset:9216\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(f[0][0].lo), "=&v"(f[0][0].hi), "=&v"(f[0][1].lo), "=&v"(f[0][1].hi), "=&v"(f[0][2].lo),
        "=&v"(f[0][2].hi), "=&v"(f[0][3].lo), "=&v"(f[0][3].hi), "=&v"(f[1][0].lo), "=&v"(f[1][0].hi),
        "=&v"(f[1][1].lo), "=&v"(f[1][1].hi), "=&v"(f[1][2].lo), "=&v"(f[1][2].hi), "=&v"(f[1][3].lo),
        "=&v"(f[1][3].hi)
      : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
      : "memory");
}
__device__ __forceinline__ void read_fragments(const uint32_t (&at)[2], Fragment (&f)[2][2]) {
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8\n\tds_read_b64_tr_b16 %1, %8 offset:1024\n\t"
      "ds_read_b64_tr_b16 %2, %9\n\tds_read_b64_tr_b16 %3, %9 offset:1024\n\t"
      "ds_read_b64_tr_b16 %4, %8 offset:8192\n\tds_read_b64_tr_b16 %5, %8 offset:9216\n\t"
      "ds_read_b64_tr_b16 %6, %9 offset:8192\n\tds_read_b64_tr_b16 %7, %9 offset:9216\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(f[0][0].lo), "=&v"(f[0][0].hi), "=&v"(f[0][1].lo), "=&v"(f[0][1].hi), "=&v"(f[1][0].lo),
        "=&v"(f[1][0].hi), "=&v"(f[1][1].lo), "=&v"(f[1][1].hi)
      : "v"(at[0]), "v"(at[1])
      : "memory");
}
// A 16-byte LDS write.  Inline assembly, because before an ordinary one the
// compiler waits for every LDS-bound load in flight; the next lds_barrier()
// waits for it.
template <int OFFSET>
__device__ __forceinline__ void write_lds(uint32_t lds_addr, const u32x4 &v) {
  asm volatile("ds_write_b128 %0, %1 offset:%2" : : "v"(lds_addr), "v"(v), "n"(OFFSET) : "memory");
}

// TK x TN outputs (columns k of x by columns n of dy) per work-group of
// 8 waves (2 x 4), each wave TK/2 k by TN/4 n, in steps of 64 t.  The two
// halves of the work-group (H = 0, 1) run in ping-pong, one reading fragments
// while the other multiplies, switching at every barrier; H = 1 runs one phase
// late.  The halves are separate code, so that the compiler can count each
// one's loads in flight.
//
// dy goes from global memory into LDS by LDS-bound loads, and is turned into
// fragments by transposing reads.  Those run at half the rate of plain 16-byte
// reads (64 against 128 bytes a clock, by the time of the read phase), and with
// both operands read so the read phase was the longer one.  x passes through
// registers anyway, where its codes become bf16: it is transposed there, and
// LDS holds it as rows of one column k, 64 t each, which plain reads take.
//
// x, a ring of two stages: half 0 writes step t + 1 in its product phase of t,
// where the vector unit is idle between matrix instructions, and loads the
// codes of t + 2.  (In the read phase the same work lengthens it past the
// product phase.)  Done by half 0 alone, since half 1's product phase of t
// runs beside half 0's read phase of t + 1.
//
// dy, a ring of three stages: half 1 issues the loads of step t + 2 in its read
// phase of t and waits for them at the end of its read phase of t + 1, before
// either half reads them.  A stage is only written once both halves have read
// it.  Together the rings are all of a CU's 160 KB for 256 x 256.
//
// Row q of x's 16-row block i of a wave's half holds column ((q % 4) * 4 +
// q / 4) * FM + i, so that a lane's results (row 4 g + v of its blocks) are
// FM consecutive columns.  A row's 16-byte chunk (8 t) is XORed with
// (q / 2) ^ (q % 2), which spreads over the banks the 16 rows of a fragment
// read as well as eight neighbouring lanes of a write, FM columns apart.
template <int TK, int TN, int H>
__device__ __forceinline__ void q8_wgrad_tile(lds_char *const lds, const Q8WeightGrad &p, int64_t k0, int64_t n0,
                                              int tbeg, int tend, f32x4 (&acc)[TK / 32][TN / 64]) {
  constexpr int FM = TK / 32, FN = TN / 64, kHalves = TN / 128;
  constexpr int kXBytes = TK / 128 * kHalfBytes, kDyBytes = kHalves * kHalfBytes;  // of a stage
  constexpr int kDyLoads = kDyBytes / 1024 / 4;                // LDS-bound loads of dy per wave of half 1 and step
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 3;
  // dy: 1 KB load j of wave w of half 1 fills rows 16 (j % 4) + 4 w + lane / 16
  // of columns 128 (j / 4) on, one 16-byte chunk a lane; chunks behind the last
  // column are clamped to it
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
  lds_char *const dy_lds = lds + 2 * kXBytes;
  auto issue_dy = [&](int slot, int step) {
    lds_char *const st = dy_lds + slot * kDyBytes + wn * 1024;
    const char *const src = static_cast<const char *>(p.dy) + static_cast<int64_t>(step) * kStep * ld;
    const int left = rows_left(step);
    auto load = [&](const char *from, int j) {
      __builtin_amdgcn_global_load_lds((const void *)from, (__attribute__((address_space(3))) void *)(st + j * 4096), 16,
                                       0, 0);
    };
    if (left == kStep) {
      const uint32_t off = static_cast<uint32_t>(drow) * ld;
#pragma unroll
      for (int j = 0; j < kDyLoads; ++j)
        load(src + static_cast<int64_t>(16 * (j & 3)) * ld + (off + dcol[j >> 2]), j);
    } else {
      // rows behind the last are loaded as copies of it, and zeroed by
      // zero_tail
#pragma unroll
      for (int j = 0; j < kDyLoads; ++j)
        load(src + (static_cast<uint32_t>(min(drow + 16 * (j & 3), left - 1)) * ld + dcol[j >> 2]), j);
    }
  };
  // Zeroes the rows behind the last that this wave loaded, once its loads have
  // landed.
  auto zero_tail = [&](int slot, int step) {
    const int left = rows_left(step);
    if (left == kStep) return;
    // opaque: nothing is kept live across the loop for this
    int l = lane_index();
    asm volatile("" : "+v"(l));
    lds_char *const st = dy_lds + slot * kDyBytes + wn * 1024 + l * 16;
#pragma unroll
    for (int j = 0; j < kDyLoads; ++j)
      if (4 * wn + (l >> 4) + 16 * (j & 3) >= left) *(lds_u32x4 *)(st + j * 4096) = u32x4{0, 0, 0, 0};
  };

  // x: a thread of half 0 takes FM columns (a run) by eight rows of t (a group:
  // one chunk of LDS); columns behind the last block are clamped to it.
  // Offsets from a step's uniform base fit 32 bits: 64 rows of at most 2^22
  // codes, and two scale rows of at most 2^29 bytes.
  constexpr int kWords = FM / 4;
  typedef uint32_t Run __attribute__((ext_vector_type(kWords)));
  typedef __attribute__((address_space(1))) Run g_Run;
  const int64_t t4 = (p.rows + 3) & ~static_cast<int64_t>(3);
  const uint32_t last_col = static_cast<uint32_t>(min(p.kp - FM - k0, static_cast<int64_t>(TK)));
  // made anew where they are used: registers are short
  auto run_and_group = [&](int &run, int &group) {
    int l = lane_index();
    asm volatile("" : "+v"(l));
    run = l & 31;
    group = 2 * wn + (l >> 5);
  };
  Run codes[8];
  uint32_t sword[2];
  auto load_x = [&](int step) {
    int run, group;
    run_and_group(run, group);
    const uint32_t xcol = min(static_cast<uint32_t>(FM * run), last_col);
    const uint32_t scol = xcol / kQ8Block * static_cast<uint32_t>(t4);
    const int64_t t0 = static_cast<int64_t>(step) * kStep;
    const uint8_t *const xs = p.x + t0 * p.kp + k0, *const ss = p.sx + k0 / kQ8Block * t4 + t0;
    // Rows behind the last are loaded as copies of it, with scales of other
    // rows or the table's padding, and zeroed by zero_x_tail.
    const int last_row = rows_left(step) - 1, last_word = static_cast<int>(min(t4 - 4 - t0, static_cast<int64_t>(kStep)));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      codes[j] = *(const g_Run *)(xs + (__umul24(static_cast<uint32_t>(min(group * 8 + j, last_row)),
                                                 static_cast<uint32_t>(p.kp)) + xcol));
#pragma unroll
    for (int h = 0; h < 2; ++h)
      sword[h] = *(const g_u32 *)(ss + (scol + static_cast<uint32_t>(min(group * 8 + 4 * h, last_word))));
  };
  // expands and transposes the loaded codes into stage `slot`: a thread's first
  // column goes to `at`, its others follow 16 rows apart
  auto write_x = [&](int slot) {
    int run, group;
    run_and_group(run, group);
    const int r = run & 15, row = (r & 3) * 4 + (r >> 2);
    const uint32_t at =
        static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds)) + static_cast<uint32_t>(slot * kXBytes) +
        static_cast<uint32_t>(((run >> 4) * (TK / 2) + row) * 128 + ((group ^ (row >> 1) ^ (row & 1)) & 7) * 16);
    // half the scales (the bytes are 10 or more, but for those behind the last
    // row, which are the word's last)
    const uint32_t half[2] = {sword[0] - 0x01010101u, sword[1] - 0x01010101u};
#pragma unroll
    for (int c = 0; c < kWords; ++c) {
      uint32_t lo[8], hi[8];  // columns 4 c, 4 c + 1 and 4 c + 2, 4 c + 3 of row j
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = __uint_as_float(((half[j >> 2] >> (8 * (j & 3))) & 0xff) << 23);
        const int q = static_cast<int>(codes[j][c]);
        lo[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, s, false));
        hi[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, s, true));
      }
      u32x4 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[0][j] = __builtin_amdgcn_perm(lo[2 * j + 1], lo[2 * j], 0x05040100u);
        w[1][j] = __builtin_amdgcn_perm(lo[2 * j + 1], lo[2 * j], 0x07060302u);
        w[2][j] = __builtin_amdgcn_perm(hi[2 * j + 1], hi[2 * j], 0x05040100u);
        w[3][j] = __builtin_amdgcn_perm(hi[2 * j + 1], hi[2 * j], 0x07060302u);
      }
      if (c == 0) {
        write_lds<0>(at, w[0]);
        write_lds<2048>(at, w[1]);
        write_lds<4096>(at, w[2]);
        write_lds<6144>(at, w[3]);
      } else {
        write_lds<8192>(at, w[0]);
        write_lds<10240>(at, w[1]);
        write_lds<12288>(at, w[2]);
        write_lds<14336>(at, w[3]);
      }
    }
  };

  // Zeroes the rows behind the last in stage `slot`, in the two groups that this
  // wave wrote there for every column: a code under another row's scale may
  // exceed bf16's range, and an infinity times dy's zero rows would be NaN.
  const int full_steps = static_cast<int>(p.rows / kStep);
  auto zero_x_tail = [&](int slot, int step) {
    if (step < full_steps) return;
    // opaque: nothing is kept live across the loop for this
    int l = lane_index();
    asm volatile("" : "+v"(l));
    for (int g = 2 * wn; g < 2 * wn + 2; ++g) {
      const int first = max(rows_left(step) - 8 * g, 0);
      if (first >= 8) continue;
      for (int c = l; c < TK; c += 64) {
        lds_char *const chunk = lds + slot * kXBytes + c * 128 + ((g ^ ((c & 15) >> 1) ^ (c & 1)) & 7) * 16;
        if (first == 0)
          *(lds_u32x4 *)chunk = u32x4{0, 0, 0, 0};
        else
          for (int r = first; r < 8; ++r) *(lds_u16 *)(chunk + 2 * r) = 0;
      }
    }
  };

#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // dy's fragments: lane (g4, e, q) names row 32 s + 8 g4 + 4 h + e, columns
  // c + 4 q .. c + 4 q + 3 of its 16-column block, whose bits are XORed into the
  // lane's swizzled chunk
  auto dy_base = [](int l) {
    const int row = 8 * (l >> 4) + ((l >> 2) & 3);
    return static_cast<uint32_t>(row * 256 + (l & 1) * 8 + ((((l & 3) >> 1) ^ swz(row)) * 16));
  };
  static_assert(kHalfBytes == 16384 && 4 * 256 == 1024 && 32 * 256 == 8192, "offsets in read_fragments");
  auto dy_at = [&](const lds_char *op, uint32_t rb, int col) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(op)) + static_cast<uint32_t>((col >> 7) * kHalfBytes) +
           (rb ^ ((col & 127) * 2));
  };
  // x's fragments: row lane % 16 of block i, chunk 4 s + lane / 16
  auto x_base = [](int l) {
    const int r = l & 15;
    return static_cast<uint32_t>(r * 128 + (((l >> 4) ^ (r >> 1) ^ (r & 1)) & 7) * 16);
  };
  auto read_x = [&](const lds_char *op, uint32_t xb, int i, int s) {
    return *(const lds_u32x4 *)(op + (H * (TK / 2) + i * 16) * 128 + (xb ^ (s * 64)));
  };

  const int last = tend - 1;
  int s0 = 0, s1 = 1, s2 = 2;  // stages of dy: of step t, t + 1 and t + 2
  if constexpr (H == 0) {
    load_x(tbeg);
    write_x(tbeg & 1);
    zero_x_tail(tbeg & 1, tbeg);
    load_x(min(tbeg + 1, last));
  } else {
    issue_dy(s0, tbeg);
    issue_dy(s1, min(tbeg + 1, last));
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    zero_tail(s0, tbeg);
    zero_tail(s1, min(tbeg + 1, last));
  }
  lds_barrier();
  if (H == 1) barrier();
  for (int t = tbeg; t < tend; ++t) {
    const lds_char *const xs = lds + (t & 1) * kXBytes, *const ds = dy_lds + s0 * kDyBytes;
    // the last steps load and write the last rows again, into free stages,
    // which keeps the loop free of branches
    if constexpr (H == 1) issue_dy(s2, min(t + 2, last));
    __builtin_amdgcn_sched_barrier(0);
    u32x4 fx[2][FM];
    Fragment fd[2][FN];
    // opaque: the fragments' addresses are rebuilt at every step instead of
    // being kept live across the loop
    int l = lane_index();
    asm volatile("" : "+v"(l));
    const uint32_t xb = x_base(l), rb = dy_base(l);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < FM; ++i) fx[s][i] = read_x(xs, xb, i, s);
    __builtin_amdgcn_sched_barrier(0);
    uint32_t at[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) at[j] = dy_at(ds, rb, wn * (TN / 4) + j * 16);
    read_fragments(at, fd);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (H == 1) {
      // dy of t + 1: all loads but those of t + 2
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kDyLoads) : "memory");
      if (t + 1 < tend) zero_tail(s1, t + 1);
      lds_barrier();
    } else {
      barrier();
    }
    __builtin_amdgcn_sched_barrier(0);
    auto multiply = [&](int s, int i) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fx[s][i]), fd[s][j].get(), acc[i][j], 0, 0, 0);
    };
    // a quarter first: it frees registers, and half 0's codes are used late, to
    // give their loads most of a step
#pragma unroll
    for (int i = 0; i < FM / 2; ++i) multiply(0, i);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (H == 0) {
      write_x((t + 1) & 1);
      load_x(min(t + 2, last));
    }
#pragma unroll
    for (int i = FM / 2; i < FM; ++i) multiply(0, i);
#pragma unroll
    for (int i = 0; i < FM; ++i) multiply(1, i);
    if constexpr (H == 0) {
      // a matrix instruction takes the time of four others: three between two
#pragma unroll
      for (int i = 0; i < FM * FN * 3 / 2; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (H == 0) {
      zero_x_tail((t + 1) & 1, min(t + 1, last));
      lds_barrier();
    } else {
      barrier();
    }
    __builtin_amdgcn_sched_barrier(0);
    const int s = s0;
    s0 = s1;
    s1 = s2;
    s2 = s;
  }
  // no load into LDS is in flight after the loop
  if constexpr (H == 1) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if (H == 0) barrier();
}

template <int TK, int TN>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(TN == 256 ? 2 : 4)))
void q8_wgrad_kernel(Q8WeightGrad p, TileSplit sp) {
  constexpr int FM = TK / 32, FN = TN / 64;
  __shared__ __attribute__((aligned(1024))) char smem[(2 * (TK / 128) + 3 * (TN / 128)) * kHalfBytes];
  const TileWork w = tile_work(sp, blockIdx.x, static_cast<uint32_t>((p.rows + kStep - 1) / kStep));
  const int64_t k0 = static_cast<int64_t>(w.a) * TK, n0 = static_cast<int64_t>(w.b) * TN;
  const uint32_t wave = uniform(threadIdx.x >> 6);
  f32x4 acc[FM][FN];
  if (wave < 4)
    q8_wgrad_tile<TK, TN, 0>((lds_char *)smem, p, k0, n0, w.begin, w.end, acc);
  else
    q8_wgrad_tile<TK, TN, 1>((lds_char *)smem, p, k0, n0, w.begin, w.end, acc);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] *= 2.f;

  const int lane = lane_index(), r16 = lane & 15, g4 = lane >> 4;
  const int wm = static_cast<int>(wave >> 2), wn = static_cast<int>(wave & 3);
  const TileOut o = tile_out(w, TK, TN, p.base, p.out, p.out_dt, p.outs, p.cols, p.ws);
  // Where all of the tile's columns exist, base is added before the first store:
  // a load may not pass a store, since base may be out, and each run of outputs
  // would wait for its own (1000 rows, 8192 x 4096 fp32 outputs: 97 us so, 114 run
  // by run; 272 rows, 11904 x 1603: 54 and 60).
  const bool base_first = o.base && o.cols >= TK;
  if (base_first) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int r = wn * (TN / 4) + j * 16 + r16;
      if (r >= o.rows) continue;
      float b[4][FM];
      load_runs<FM, 4>(o.base, o.dt, o.at + r * o.ld + wm * (TK / 2) + g4 * FM, 4 * FM, b);
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[i][j][v] += b[v][i];
    }
  }
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int r = wn * (TN / 4) + j * 16 + r16;
    if (r >= o.rows) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int c = wm * (TK / 2) + (v * 4 + g4) * FM;
      float run[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i) run[i] = acc[i][j][v];
      finish_run<FM>(base_first ? nullptr : o.base, o.out, o.dt, o.at + r * o.ld + c, o.cols - c, run);
    }
  }
}

// Work-groups of the two kernels below, 2048 elements each at a time: their
// threads stay below 2^32 whatever the size.
uint32_t element_groups(int64_t n) { return static_cast<uint32_t>(std::min<int64_t>((n + 2047) / 2048, 1 << 20)); }

// No rows: out = base, or zero.
__global__ __launch_bounds__(256) void q8_wgrad_empty_kernel(Q8WeightGrad p) {
  const int64_t n = p.outs * p.cols;
  for (int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8; at < n; at += gridDim.x * int64_t(2048)) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    finish_run<8>(p.base, p.out, p.out_dt, at, n - at, v);
  }
}

// A copy of bf16 rows with rows of ld elements, a multiple of 8 (zeros behind the
// last column), for a dy whose rows are no such multiple: the LDS-bound loads take
// 16 bytes.  One pass, bound by HBM: 8192 x 14335 in about 95 us, beside 110 for
// the product with 512 columns.
__global__ __launch_bounds__(256) void q8_pad_rows_kernel(const uint16_t *__restrict__ dy, int64_t rows, int64_t cols,
                                                          int64_t ld, uint16_t *__restrict__ out) {
  for (int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8; at < rows * ld;
       at += gridDim.x * int64_t(2048)) {
    const int64_t t = at / ld, c = at - t * ld;
    const uint16_t *const src = dy + t * cols + c;
    if (c + 8 <= cols) {
      *(g_u32x4 *)(out + at) = *(const g_u32x4_at2 *)src;
      continue;
    }
    uint32_t e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = c + k < cols ? ((const g_u16 *)src)[k] : 0;
    *(g_u32x4 *)(out + at) = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
  }
}

// Microseconds a step of 64 rows, measured on 4096 and 8192 rows: 256 x 256
// tiles 1.5 with few work-groups on the chip and 1.6 with 256, 128 x 256 tiles
// 0.95 and 1.12, 128 x 128 tiles 0.8 alone on their CU and 1.22 for two.  The
// best with each: 8192 rows, 1024 x 4096 outputs 79 us, 86 and 92; 1500 rows,
// 3000 x 1800 outputs 44, 34 and 36; 4096 rows, 256 x 1536 outputs 35, 26 and 19.
constexpr std::initializer_list<TileCost> kCosts = {
    {256, 256, 1, 1.5f, 1.6f}, {128, 256, 1, 0.95f, 1.12f}, {128, 128, 2, 0.8f, 1.22f}};

// How a weight gradient runs: the tiles' split, and the bytes of its
// workspace's two parts, the padded dy and the pieces' results.
struct Plan {
  TileSplit split;
  int64_t dy_ld;
  size_t pad_bytes, piece_bytes;
};

Plan plan_of(int64_t rows, int64_t outs, int64_t cols) {
  Plan pl{};
  if (rows == 0) return pl;
  pl.split = choose_split(cols, outs, (rows + kStep - 1) / kStep, kCosts);
  pl.dy_ld = (outs + 7) & ~static_cast<int64_t>(7);
  if (pl.dy_ld != outs) pl.pad_bytes = (static_cast<size_t>(rows * pl.dy_ld * 2) + 255) & ~static_cast<size_t>(255);
  pl.piece_bytes = pl.split.ws_bytes();
  return pl;
}

}  // namespace

size_t q8_wgrad_workspace(int64_t rows, int64_t outs, int64_t cols) {
  const Plan pl = plan_of(rows, outs, cols);
  return pl.pad_bytes + pl.piece_bytes;
}

hipError_t launch_pad_rows(const void *x, int64_t rows, int64_t cols, int64_t ld, void *out, hipStream_t st) {
  hipLaunchKernelGGL(q8_pad_rows_kernel, dim3(element_groups(rows * ld)), dim3(256), 0, st,
                     static_cast<const uint16_t *>(x), rows, cols, ld, static_cast<uint16_t *>(out));
  return hipGetLastError();
}

hipError_t launch_q8_wgrad(const Q8WeightGrad &args, hipStream_t st) {
  Q8WeightGrad p = args;
  if (p.rows == 0) {
    hipLaunchKernelGGL(q8_wgrad_empty_kernel, dim3(element_groups(p.outs * p.cols)), dim3(256), 0, st, p);
    return hipGetLastError();
  }
  const Plan pl = plan_of(p.rows, p.outs, p.cols);
  p.dy_ld = pl.dy_ld;
  if (pl.pad_bytes) {
    const hipError_t e = launch_pad_rows(p.dy, p.rows, p.outs, pl.dy_ld, p.ws, st);
    if (e != hipSuccess) return e;
    p.dy = p.ws;
    p.ws = static_cast<char *>(p.ws) + pl.pad_bytes;
  }
  const TileSplit &sp = pl.split;
  const dim3 grid(sp.whole + sp.tail * sp.pieces);
  if (sp.ta == 256)
    hipLaunchKernelGGL((q8_wgrad_kernel<256, 256>), grid, dim3(kThreads), 0, st, p, sp);
  else if (sp.tb == 256)
    hipLaunchKernelGGL((q8_wgrad_kernel<128, 256>), grid, dim3(kThreads), 0, st, p, sp);
  else
    hipLaunchKernelGGL((q8_wgrad_kernel<128, 128>), grid, dim3(kThreads), 0, st, p, sp);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.pieces == 1) return e;
  return launch_q8_reduce(static_cast<const float *>(p.ws), sp, p.outs, p.cols, p.base, p.out, p.out_dt, st);
}

}  // namespace dmuon
