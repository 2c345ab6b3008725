// Declarations shared by the 4-bit block products' entry points (q4_api.cpp)
// and kernels (q4_quant.hip, q4_matmul.hip, q4_rows.hip).  Not part of the C
// ABI.
#pragma once

#include "q8_internal.h"

namespace dmuon {

// Elements that share one scale, along the direction that a product sums over.
constexpr int kQ4Block = 32;
// Rows of codes are padded to this many: 128 bytes, a cache line and a step of
// the products.
constexpr int kQ4Pad = 256;
// Rows of a scale table are a multiple of this many bytes.
constexpr int kQ4ScaleRow = 16;
// Range of the scale's exponent.  6 * 2^126 exceeds every finite fp32; at 2^-125
// the smallest code, 0.5, stands for 2^-126, fp32's and bf16's smallest normal
// number.
constexpr int kQ4MinExp = -125, kQ4MaxExp = 126;
// The scale byte of a block that holds a NaN or an infinity: the whole block
// is NaN.
constexpr int kQ4Nan = 255;

// Quantising: batches of up to kQ4Batch matrices of one type per launch, by value;
// all of them rounded by random bytes, or none.
constexpr int kQ4Batch = 24;
struct Q4Batch {
  int32_t n;
  int32_t dt;
  int64_t first_tile[kQ4Batch + 1];  // prefix sum of 128 x 128 tiles
  const void *x[kQ4Batch];
  const uint8_t *random[kQ4Batch];                  // nullable
  uint8_t *codes[kQ4Batch], *scales[kQ4Batch];      // both null: not written
  uint8_t *codes_t[kQ4Batch], *scales_t[kQ4Batch];  // both null: not written
  int64_t rows[kQ4Batch], cols[kQ4Batch];
};
// Tiles of 128 x 128 that a matrix takes: over its elements, the padding of its
// codes and that of its scale tables.
int64_t q4_tiles(int64_t rows, int64_t cols, bool plain, bool transposed);
hipError_t launch_q4_quantize(const Q4Batch &b, hipStream_t st);
// The values of codes and scales, rows x cols.
hipError_t launch_q4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *out,
                                int32_t dt, hipStream_t st);
// out[r][c] = src[r * row_step + c * col_step], bytes; cols is a multiple of 16.
hipError_t launch_q4_copy(const uint8_t *src, int64_t rows, int64_t cols, int64_t row_step, int64_t col_step,
                          uint8_t *out, hipStream_t st);

// out[t][n] = base[t][n] + sum over blocks b of 2^(sa[b][t] + sb[b][n] - 254) *
// sum over k in b of a[t][k] b[n][k]; all strides follow from the sizes.
struct Q4Product {
  const void *a;      // codes [rows][kp / 2]; of bf16 rows the elements [rows][inner]
  const uint8_t *sa;  // scales [kp / 32][rows up to 16]; null: a is bf16
  const uint8_t *b, *sb;  // codes [outs][kp / 2], scales [kp / 32][outs up to 16]
  const void *base;   // nullable: [rows][outs], out_dt; may be out
  void *out;          // [rows][outs]
  void *ws;           // the workspace bytes below
  int64_t rows, outs, inner, kp;  // kp: inner up to 256
  int32_t out_dt;
};
// inner = 0: out = base, or zero.
size_t q4_matmul_workspace(int64_t rows, int64_t outs, int64_t kp);
hipError_t launch_q4_matmul(const Q4Product &p, hipStream_t st);
// bf16 rows, without a base.
size_t q4_rows_workspace(int64_t rows, int64_t outs, int64_t inner);
hipError_t launch_q4_rows(const Q4Product &p, hipStream_t st);

// The kernel that a product of these sizes runs in: a streaming work-group's blocks of
// 16 rows and outputs and the rows that it loads (blocks 0: in tiles), or the tiles.
struct Q4Choice {
  int32_t row_blocks, out_blocks, waves, rows;
  TileSplit tiles;
};
Q4Choice q4_matmul_choice(int64_t rows, int64_t outs, int64_t kp);
Q4Choice q4_rows_choice(int64_t rows, int64_t outs, int64_t inner);

}  // namespace dmuon
