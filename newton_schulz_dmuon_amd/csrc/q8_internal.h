// Declarations shared by the 8-bit block products' entry points (q8_api.cpp)
// and kernels (q8_quant.hip, q8_matmul.hip, q8_wgrad.hip, q8_reduce.hip).  Not
// part of the C ABI.
#pragma once

#include <initializer_list>

#include "internal.h"

namespace dmuon {

// Elements that share one scale: along a row, and per side of a weight block.
constexpr int kQ8Block = 128;
// Range of the scale's exponent.  448 * 2^120 exceeds every finite fp32, and so
// do codes of 256 and more at 2^120, which the lowest values of bf16 and fp32
// round to: expansions to bf16 use half the scale.  At 2^-117 the smallest code,
// 2^-9, stands for 2^-126, fp32's and bf16's smallest normal number.
constexpr int kQ8MinExp = -117, kQ8MaxExp = 120;
// Rows of a scale table are a multiple of this many bytes.
constexpr int kQ8ScaleRow = 4;

// Quantising weights: batches of up to kQ8Batch matrices per launch, by value.
constexpr int kQ8Batch = 32;
struct Q8WeightBatch {
  int32_t n;
  int32_t pad_;
  int64_t first_block[kQ8Batch + 1];  // prefix sum of 128 x 128 blocks
  const void *param[kQ8Batch];
  uint8_t *codes[kQ8Batch], *codes_t[kQ8Batch];    // codes_t: nullable
  uint8_t *scales[kQ8Batch], *scales_t[kQ8Batch];
  int64_t rows[kQ8Batch], cols[kQ8Batch];
  int32_t param_dt[kQ8Batch];
};

hipError_t launch_q8_rows(const void *x, int32_t dt, int64_t rows, int64_t cols, uint8_t *codes,
                          uint8_t *scales, hipStream_t st);
hipError_t launch_q8_weights(const Q8WeightBatch &b, hipStream_t st);

// How a product's output tiles (ta columns by tb rows; na across, nb down) are
// shared out: the first `whole` of them one work-group each, the last `tail`
// split into `pieces` along the sum, whose fp32 results go to slots of the
// workspace, [tail tile][piece], and are added by a reduce launch.
struct TileSplit {
  uint32_t ta, tb, na, nb;
  uint32_t whole, tail, pieces;
  size_t ws_bytes() const {
    return pieces > 1 ? size_t(tail) * pieces * ta * tb * sizeof(float) : 0;
  }
};

// A tile that a kernel can take, and what a step of its work-group costs in
// microseconds, as measured (the kernels say where): for one work-group a CU,
// with the chip nearly empty and full; for two, with one and two on each CU.
struct TileCost {
  int64_t ta, tb, per_cu;
  float low, full;
};
// The cheapest tile and split by that measure; steps of the sum.  Tiles are
// listed from the largest down.
TileSplit choose_split(int64_t cols, int64_t rows, int64_t steps, std::initializer_list<TileCost> tiles,
                       float *cost = nullptr);

// out[r][c] = base[r][c] (0 if null) + the sum of the pieces' results, in order,
// rounded once to dt, over the tail tiles of a split.  base may be out.
hipError_t launch_q8_reduce(const float *ws, const TileSplit &sp, int64_t rows, int64_t cols, const void *base,
                            void *out, int32_t dt, hipStream_t st);

// out[t][n] = sum over blocks b of 2^(sa[b][t] + sb[n / 128][b] - 254) *
// sum over k in b of a[t][k] b[n][k]; all strides follow from the sizes.
struct Q8Product {
  const uint8_t *a, *sa;  // codes [rows][kp], scales [kp / 128][rows up to 4]
  const uint8_t *b, *sb;  // codes [outs][kp], scales [outs up to 128 / 128][kp / 128]
  void *out;              // [rows][outs]
  float *ws;              // q8_matmul_workspace bytes
  int64_t rows, outs, kp;
  int32_t out_dt;
  bool fast;              // the 8-bit instruction's sums in place of fp32's
};
size_t q8_matmul_workspace(int64_t rows, int64_t outs, int64_t kp, bool fast);
hipError_t launch_q8_matmul(const Q8Product &p, hipStream_t st);

// out[n][k] = base[n][k] + sum over t of dy[t][n] 2^(sx[k / 128][t] - 127) x[t][k]
struct Q8WeightGrad {
  const void *dy;         // bf16 [rows][outs], rows dy_ld elements apart
  const uint8_t *x, *sx;  // codes [rows][kp], scales [kp / 128][rows up to 4]
  const void *base;       // nullable: [outs][cols], out_dt; may be out
  void *out;              // [outs][cols]
  void *ws;               // q8_wgrad_workspace bytes
  int64_t rows, outs, cols, kp;
  int64_t dy_ld;          // set by the launcher
  int32_t out_dt;
};
// A copy of bf16 rows [rows][cols] as [rows][ld], zeros behind cols; ld is a
// multiple of 8.
hipError_t launch_pad_rows(const void *x, int64_t rows, int64_t cols, int64_t ld, void *out, hipStream_t st);
size_t q8_wgrad_workspace(int64_t rows, int64_t outs, int64_t cols);
hipError_t launch_q8_wgrad(const Q8WeightGrad &p, hipStream_t st);

}  // namespace dmuon
