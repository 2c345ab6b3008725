// C entry points of the 4-bit block products: argument validation and
// launches.  Every check runs before the first HIP call.

#include <cstring>

#include "../../include/dmuon.h"
#include "host_common.h"
#include "q4_internal.h"

namespace dmuon {
namespace {

// inner = 0 is a sum of nothing.
int check_sizes(int64_t rows, int64_t outs, int64_t inner, int64_t min_inner) {
  if (rows < 0 || rows > kMaxRows) return fail(DMUON_ERR_INVALID_ARG, "rows %lld", (long long)rows);
  if (outs < 1 || outs > kMaxSide) return fail(DMUON_ERR_INVALID_ARG, "outputs %lld", (long long)outs);
  if (inner < min_inner || inner > kMaxSide) return fail(DMUON_ERR_INVALID_ARG, "columns %lld", (long long)inner);
  const int64_t kp = round_up(inner, kQ4Pad), r16 = round_up(rows, kQ4ScaleRow), n16 = round_up(outs, kQ4ScaleRow);
  if (too_large(r16, kp) || too_large(rows, outs) || too_large(n16, kp))
    return fail(DMUON_ERR_INVALID_ARG, "%lld rows, %lld outputs, %lld columns: a buffer exceeds 2^37 elements",
                (long long)rows, (long long)outs, (long long)inner);
  return DMUON_OK;
}

int64_t code_bytes(int64_t rows, int64_t cols) { return rows * (round_up(cols, kQ4Pad) / 2); }
int64_t scale_bytes(int64_t rows, int64_t cols) {
  return round_up(cols, kQ4Pad) / kQ4Block * round_up(rows, kQ4ScaleRow);
}

// Codes and scales as a product or a read back takes them.
int add_codes(Buffers &b, const void *codes, const void *scales, int64_t rows, int64_t cols, const char *what,
              const char *what_scales) {
  const int rc = b.add(codes, code_bytes(rows, cols), false, what);
  return rc ? rc : b.add(scales, scale_bytes(rows, cols), false, what_scales);
}

int add_source(Buffers &b, const dmuon_q4_source &d, int32_t i) {
  if (d.rows < 0 || d.rows > kMaxRows || d.cols < 1 || d.cols > kMaxSide || (d.codes_t && d.rows > kMaxSide) ||
      too_large(round_up(d.rows, kQ4Pad), round_up(d.cols, kQ4Pad)))
    return fail(DMUON_ERR_INVALID_ARG, "matrix %d: bad shape %lld x %lld", i, (long long)d.rows, (long long)d.cols);
  if (!dtype_ok(d.dtype)) return fail(DMUON_ERR_UNSUPPORTED_DTYPE, "matrix %d: dtype code %d", i, d.dtype);
  if (d.reserved != 0) return fail(DMUON_ERR_INVALID_ARG, "matrix %d: reserved != 0", i);
  if (!d.codes != !d.scales || !d.codes_t != !d.scales_t)
    return fail(DMUON_ERR_INVALID_ARG, "matrix %d: codes and scales go together", i);
  if (d.rows == 0) return DMUON_OK;
  if (!d.codes && !d.codes_t) return fail(DMUON_ERR_INVALID_ARG, "matrix %d: no codes to write", i);
  int rc;
  if ((rc = b.add(d.x, d.rows * d.cols * elem_size(d.dtype), false, "x", 16, i))) return rc;
  if (d.random && (rc = b.add(d.random, d.rows * d.cols, false, "random", 16, i))) return rc;
  if (d.codes) {
    if ((rc = b.add(d.codes, code_bytes(d.rows, d.cols), true, "codes", 16, i))) return rc;
    if ((rc = b.add(d.scales, scale_bytes(d.rows, d.cols), true, "scales", 16, i))) return rc;
  }
  if (d.codes_t) {
    if ((rc = b.add(d.codes_t, code_bytes(d.cols, d.rows), true, "codes_t", 16, i))) return rc;
    if ((rc = b.add(d.scales_t, scale_bytes(d.cols, d.rows), true, "scales_t", 16, i))) return rc;
  }
  return DMUON_OK;
}

Q4Product product(const void *a, const void *sa, int64_t rows, const void *b, const void *sb, int64_t outs,
                  int64_t inner, const void *base, void *out, int32_t out_dtype, void *ws) {
  Q4Product p;
  p.a = a;
  p.sa = static_cast<const uint8_t *>(sa);
  p.b = static_cast<const uint8_t *>(b);
  p.sb = static_cast<const uint8_t *>(sb);
  p.base = base;
  p.out = out;
  p.ws = ws;
  p.rows = rows;
  p.outs = outs;
  p.inner = inner;
  p.kp = round_up(inner, kQ4Pad);
  p.out_dt = out_dtype;
  return p;
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_q4_quantize(const dmuon_q4_source *m, int32_t n, void *stream) {
  return guarded([&]() -> int {
    if (n < 0) return fail(DMUON_ERR_INVALID_ARG, "n < 0");
    if (n == 0) return DMUON_OK;
    if (!m) return fail(DMUON_ERR_INVALID_ARG, "m is NULL");
    Buffers b;
    int rc;
    for (int32_t i = 0; i < n; ++i)
      if ((rc = add_source(b, m[i], i))) return rc;
    if ((rc = b.check())) return rc;
    Q4Batch batch;
    std::memset(&batch, 0, sizeof batch);
    auto flush = [&]() -> int {
      const int status = check_launch(launch_q4_quantize(batch, static_cast<hipStream_t>(stream)), "q4 quantise launch");
      std::memset(&batch, 0, sizeof batch);
      return status;
    };
    for (int32_t i = 0; i < n; ++i) {
      const dmuon_q4_source &d = m[i];
      if (d.rows == 0) continue;
      // a matrix has at most 2^37 / 2^14 tiles, so a batch's threads stay below 2^32
      if (batch.n > 0 && (batch.n == kQ4Batch || batch.first_tile[batch.n] > (1 << 22) || batch.dt != d.dtype ||
                          !batch.random[0] != !d.random) &&
          (rc = flush()))
        return rc;
      const int k = batch.n++;
      batch.dt = d.dtype;
      batch.x[k] = d.x;
      batch.random[k] = static_cast<const uint8_t *>(d.random);
      batch.codes[k] = static_cast<uint8_t *>(d.codes);
      batch.scales[k] = static_cast<uint8_t *>(d.scales);
      batch.codes_t[k] = static_cast<uint8_t *>(d.codes_t);
      batch.scales_t[k] = static_cast<uint8_t *>(d.scales_t);
      batch.rows[k] = d.rows;
      batch.cols[k] = d.cols;
      batch.first_tile[k + 1] = batch.first_tile[k] + q4_tiles(d.rows, d.cols, d.codes != nullptr, d.codes_t != nullptr);
    }
    return batch.n > 0 ? flush() : DMUON_OK;
  });
}

int dmuon_q4_dequantize(const void *codes, const void *scales, int64_t rows, int64_t cols, void *out, int32_t dtype,
                        void *stream) {
  return guarded([&]() -> int {
    if (!dtype_ok(dtype)) return fail(DMUON_ERR_UNSUPPORTED_DTYPE, "dtype code %d", dtype);
    int rc = check_sizes(rows, 1, cols, 1);
    if (rc) return rc;
    if (rows == 0) return DMUON_OK;
    Buffers b;
    if ((rc = add_codes(b, codes, scales, rows, cols, "codes", "scales"))) return rc;
    if ((rc = b.add(out, rows * cols * elem_size(dtype), true, "out"))) return rc;
    if ((rc = b.check())) return rc;
    return check_launch(launch_q4_dequantize(static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales),
                                             rows, cols, out, dtype, static_cast<hipStream_t>(stream)),
                        "q4 dequantise launch");
  });
}

int dmuon_q4_copy(const void *src, int64_t rows, int64_t cols, int64_t row_step, int64_t col_step, void *out,
                  void *stream) {
  return guarded([&]() -> int {
    // at most 2^22 + 2^23 tiles of 128 x 128, whose threads stay below 2^32
    if (rows < 0 || rows > kMaxRows) return fail(DMUON_ERR_INVALID_ARG, "rows %lld", (long long)rows);
    if (cols < 0 || cols > kMaxRows || cols % kQ4ScaleRow != 0)
      return fail(DMUON_ERR_INVALID_ARG, "columns %lld", (long long)cols);
    if (too_large(rows, 2 * cols))
      return fail(DMUON_ERR_INVALID_ARG, "%lld x %lld bytes exceed 2^36", (long long)rows, (long long)cols);
    constexpr int64_t kMaxExtent = int64_t(1) << 47;
    if (row_step < 0 || row_step > kMaxExtent || col_step < 0 || col_step > kMaxExtent)
      return fail(DMUON_ERR_INVALID_ARG, "steps %lld, %lld", (long long)row_step, (long long)col_step);
    if (rows == 0 || cols == 0) return DMUON_OK;
    const __int128 extent = static_cast<__int128>(rows - 1) * row_step + static_cast<__int128>(cols - 1) * col_step + 1;
    if (extent > kMaxExtent) return fail(DMUON_ERR_INVALID_ARG, "src spans more than 2^47 bytes");
    Buffers b;
    int rc;
    if ((rc = b.add(src, static_cast<int64_t>(extent), false, "src", 1))) return rc;
    if ((rc = b.add(out, rows * cols, true, "out"))) return rc;
    if ((rc = b.check())) return rc;
    return check_launch(launch_q4_copy(static_cast<const uint8_t *>(src), rows, cols, row_step, col_step,
                                       static_cast<uint8_t *>(out), static_cast<hipStream_t>(stream)),
                        "q4 copy launch");
  });
}

int dmuon_q4_matmul_workspace_bytes(int64_t rows, int64_t outs, int64_t inner, size_t *out_bytes) {
  return guarded([&]() -> int {
    if (!out_bytes) return fail(DMUON_ERR_INVALID_ARG, "out_bytes is NULL");
    const int rc = check_sizes(rows, outs, inner, 0);
    if (rc) return rc;
    *out_bytes = q4_matmul_workspace(rows, outs, round_up(inner, kQ4Pad));
    return DMUON_OK;
  });
}

int dmuon_q4_matmul(const void *codes, const void *scales, int64_t rows, const void *codes_b, const void *scales_b,
                    int64_t outs, int64_t inner, const void *base, void *out, int32_t out_dtype, void *workspace,
                    size_t workspace_bytes, void *stream) {
  return guarded([&]() -> int {
    if (!dtype_ok(out_dtype)) return fail(DMUON_ERR_UNSUPPORTED_DTYPE, "dtype code %d", out_dtype);
    int rc = check_sizes(rows, outs, inner, 0);
    if (rc) return rc;
    if (rows == 0) return DMUON_OK;
    const int64_t out_bytes = rows * outs * elem_size(out_dtype);
    Buffers b;
    if (inner > 0) {
      if ((rc = add_codes(b, codes, scales, rows, inner, "codes", "scales"))) return rc;
      if ((rc = add_codes(b, codes_b, scales_b, outs, inner, "codes_b", "scales_b"))) return rc;
    }
    if ((rc = b.add(out, out_bytes, true, "out"))) return rc;
    // base = out: each element is read and written by the same thread
    if (base && base != out && (rc = b.add(base, out_bytes, false, "base"))) return rc;
    if ((rc = add_workspace(b, workspace, workspace_bytes, q4_matmul_workspace(rows, outs, round_up(inner, kQ4Pad)))))
      return rc;
    if ((rc = b.check())) return rc;
    return check_launch(launch_q4_matmul(product(codes, scales, rows, codes_b, scales_b, outs, inner, base, out,
                                                 out_dtype, workspace),
                                         static_cast<hipStream_t>(stream)),
                        "q4 product launch");
  });
}

int dmuon_q4_rows_matmul_workspace_bytes(int64_t rows, int64_t outs, int64_t inner, size_t *out_bytes) {
  return guarded([&]() -> int {
    if (!out_bytes) return fail(DMUON_ERR_INVALID_ARG, "out_bytes is NULL");
    const int rc = check_sizes(rows, outs, inner, 1);
    if (rc) return rc;
    *out_bytes = q4_rows_workspace(rows, outs, inner);
    return DMUON_OK;
  });
}

int dmuon_q4_rows_matmul(const void *x, int64_t rows, const void *codes_b, const void *scales_b, int64_t outs,
                         int64_t inner, void *out, int32_t out_dtype, void *workspace, size_t workspace_bytes,
                         void *stream) {
  return guarded([&]() -> int {
    if (!dtype_ok(out_dtype)) return fail(DMUON_ERR_UNSUPPORTED_DTYPE, "dtype code %d", out_dtype);
    int rc = check_sizes(rows, outs, inner, 1);
    if (rc) return rc;
    if (rows == 0) return DMUON_OK;
    Buffers b;
    if ((rc = b.add(x, rows * inner * 2, false, "x"))) return rc;
    if ((rc = add_codes(b, codes_b, scales_b, outs, inner, "codes_b", "scales_b"))) return rc;
    if ((rc = b.add(out, rows * outs * elem_size(out_dtype), true, "out"))) return rc;
    if ((rc = add_workspace(b, workspace, workspace_bytes, q4_rows_workspace(rows, outs, inner)))) return rc;
    if ((rc = b.check())) return rc;
    return check_launch(launch_q4_rows(product(x, nullptr, rows, codes_b, scales_b, outs, inner, nullptr, out, out_dtype,
                                               workspace),
                                       static_cast<hipStream_t>(stream)),
                        "q4 rows product launch");
  });
}

// Not part of the public ABI: the tests ask it which kernels their sizes run in.
// choice: Q4Choice's first four numbers, then ta, tb, whole, tail, pieces.
int dmuon_q4_choice(int32_t bf16_rows, int64_t rows, int64_t outs, int64_t inner, int64_t *choice) {
  return guarded([&]() -> int {
    const int rc = check_sizes(rows, outs, inner, 1);
    if (rc) return rc;
    const Q4Choice c = bf16_rows ? q4_rows_choice(rows, outs, inner) : q4_matmul_choice(rows, outs, round_up(inner, kQ4Pad));
    const int64_t out[] = {c.row_blocks, c.out_blocks, c.waves, c.rows, c.tiles.ta, c.tiles.tb, c.tiles.whole, c.tiles.tail, c.tiles.pieces};
    std::memcpy(choice, out, sizeof out);
    return DMUON_OK;
  });
}

}  // extern "C"
