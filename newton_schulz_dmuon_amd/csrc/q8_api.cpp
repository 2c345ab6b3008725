// C entry points of the 8-bit block products: argument validation and
// launches.  Every check runs before the first HIP call.

#include <cstring>
#include <exception>
#include <vector>

#include "../../include/dmuon.h"
#include "host_common.h"
#include "q8_internal.h"

namespace dmuon {
namespace {

// A launch takes fewer than 2^32 threads along its grid.  With these limits the
// products' grids stay below that: at most 2^22 tiles of 128, or with 2^37
// outputs 2^21 whole and as many ragged tiles of 256, of 512 threads each.
constexpr int64_t kMaxRows = int64_t(1) << 29;
constexpr int64_t kMaxSide = int64_t(1) << 22;
constexpr int64_t kMaxElems = int64_t(1) << 37;

// Whether a buffer has more than kMaxElems elements (the factors are within the
// limits above, so the product cannot overflow).
bool too_large(int64_t rows, int64_t cols) { return rows * cols > kMaxElems; }

int check_sizes(int64_t rows, int64_t outs, int64_t cols) {
  if (rows < 0 || rows > kMaxRows) return fail(DMUON_ERR_INVALID_ARG, "rows %lld", (long long)rows);
  if (outs < 1 || outs > kMaxSide) return fail(DMUON_ERR_INVALID_ARG, "outputs %lld", (long long)outs);
  if (cols < 1 || cols > kMaxSide) return fail(DMUON_ERR_INVALID_ARG, "columns %lld", (long long)cols);
  const int64_t kp = round_up(cols, kQ8Block), np = round_up(outs, kQ8Block);
  if (too_large(rows, kp) || too_large(rows, outs) || too_large(np, kp))
    return fail(DMUON_ERR_INVALID_ARG, "%lld rows, %lld outputs, %lld columns: a buffer exceeds 2^37 elements",
                (long long)rows, (long long)outs, (long long)cols);
  return DMUON_OK;
}

// The buffers of one call: alignment as they are added, overlaps at the end.
class Buffers {
 public:
  // index: the matrix the buffer belongs to
  int add(const void *p, int64_t bytes, bool written, const char *what, int align = 16, int32_t index = 0) {
    if (!p) return fail(DMUON_ERR_INVALID_ARG, "%s is NULL", what);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (lo % static_cast<uintptr_t>(align))
      return fail(DMUON_ERR_MISALIGNED, "%s must be %d-byte aligned", what, align);
    iv_.push_back(Interval{lo, lo + static_cast<uintptr_t>(bytes), written, what, index});
    return DMUON_OK;
  }
  int check() { return check_aliasing(iv_); }

 private:
  std::vector<Interval> iv_;
};

int add_workspace(Buffers &b, void *workspace, size_t have, size_t need) {
  if (need == 0) return DMUON_OK;
  if (have < need)
    return fail(DMUON_ERR_WORKSPACE_TOO_SMALL, "workspace needs %zu bytes, got %zu", need, have);
  return b.add(workspace, static_cast<int64_t>(need), true, "workspace", 256);
}

// A product's out_dtype: the result's type, and whether its sums are fast.
struct ProductType {
  int32_t dt;
  bool fast;
};
int product_type(int32_t out_dtype, ProductType &t) {
  t.dt = out_dtype & ~static_cast<int32_t>(DMUON_Q8_FAST_SUMS);
  t.fast = (out_dtype & DMUON_Q8_FAST_SUMS) != 0;
  if (!dtype_ok(t.dt)) return fail(DMUON_ERR_UNSUPPORTED_DTYPE, "dtype code %d", out_dtype);
  if (t.fast && t.dt != DMUON_BF16) return fail(DMUON_ERR_UNSUPPORTED_DTYPE, "fast sums take a bf16 result");
  return DMUON_OK;
}

// No exception leaves a C entry.
template <typename F>
int guarded(F f) {
  clear_error();
  try {
    return f();
  } catch (const std::exception &e) {
    return fail(DMUON_ERR_INVALID_ARG, "internal error: %s", e.what());
  } catch (...) {
    return fail(DMUON_ERR_INVALID_ARG, "internal error");
  }
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_q8_quantize(const void *x, int32_t dtype, int64_t rows, int64_t cols, void *codes, void *scales,
                      void *stream) {
  return guarded([&]() -> int {
    if (!dtype_ok(dtype)) return fail(DMUON_ERR_UNSUPPORTED_DTYPE, "dtype code %d", dtype);
    int rc = check_sizes(rows, 1, cols);
    if (rc) return rc;
    if (rows == 0) return DMUON_OK;
    const int64_t kp = round_up(cols, kQ8Block), t4 = round_up(rows, kQ8ScaleRow);
    Buffers b;
    if ((rc = b.add(x, rows * cols * elem_size(dtype), false, "x"))) return rc;
    if ((rc = b.add(codes, rows * kp, true, "codes"))) return rc;
    if ((rc = b.add(scales, kp / kQ8Block * t4, true, "scales", 4))) return rc;
    if ((rc = b.check())) return rc;
    return check_launch(launch_q8_rows(x, dtype, rows, cols, static_cast<uint8_t *>(codes),
                                       static_cast<uint8_t *>(scales), static_cast<hipStream_t>(stream)),
                        "q8 rows launch");
  });
}

int dmuon_q8_quantize_weights(const dmuon_q8_weight *w, int32_t n, void *stream) {
  return guarded([&]() -> int {
    if (n < 0) return fail(DMUON_ERR_INVALID_ARG, "n < 0");
    if (n == 0) return DMUON_OK;
    if (!w) return fail(DMUON_ERR_INVALID_ARG, "w is NULL");
    Buffers b;
    int rc;
    for (int32_t i = 0; i < n; ++i) {
      const dmuon_q8_weight &d = w[i];
      if (d.rows < 1 || d.rows > kMaxSide || d.cols < 1 || d.cols > kMaxSide || 
          too_large(round_up(d.rows, kQ8Block), round_up(d.cols, kQ8Block)))
        return fail(DMUON_ERR_INVALID_ARG, "matrix %d: bad shape %lld x %lld", i, (long long)d.rows,
                    (long long)d.cols);
      if (!dtype_ok(d.param_dtype))
        return fail(DMUON_ERR_UNSUPPORTED_DTYPE, "matrix %d: dtype code %d", i, d.param_dtype);
      if (d.reserved != 0) return fail(DMUON_ERR_INVALID_ARG, "matrix %d: reserved != 0", i);
      if (!d.codes_t != !d.scales_t)
        return fail(DMUON_ERR_INVALID_ARG, "matrix %d: codes_t and scales_t go together", i);
      const int64_t kp = round_up(d.cols, kQ8Block), np = round_up(d.rows, kQ8Block);
      const int64_t blocks = kp / kQ8Block * (np / kQ8Block);
      if ((rc = b.add(d.param, d.rows * d.cols * elem_size(d.param_dtype), false, "param", 16, i))) return rc;
      if ((rc = b.add(d.codes, d.rows * kp, true, "codes", 16, i))) return rc;
      if ((rc = b.add(d.scales, blocks, true, "scales", 4, i))) return rc;
      if (d.codes_t) {
        if ((rc = b.add(d.codes_t, d.cols * np, true, "codes_t", 16, i))) return rc;
        if ((rc = b.add(d.scales_t, blocks, true, "scales_t", 4, i))) return rc;
      }
    }
    if ((rc = b.check())) return rc;
    Q8WeightBatch batch;
    std::memset(&batch, 0, sizeof batch);
    for (int32_t i = 0; i < n; ++i) {
      const dmuon_q8_weight &d = w[i];
      const int k = batch.n;
      batch.param[k] = d.param;
      batch.codes[k] = static_cast<uint8_t *>(d.codes);
      batch.scales[k] = static_cast<uint8_t *>(d.scales);
      batch.codes_t[k] = static_cast<uint8_t *>(d.codes_t);
      batch.scales_t[k] = static_cast<uint8_t *>(d.scales_t);
      batch.rows[k] = d.rows;
      batch.cols[k] = d.cols;
      batch.param_dt[k] = d.param_dtype;
      // a matrix has at most 2^37 / 2^14 blocks, so a batch's threads stay
      // below 2^32
      batch.first_block[k + 1] = batch.first_block[k] + (round_up(d.rows, kQ8Block) / kQ8Block) *
                                                            (round_up(d.cols, kQ8Block) / kQ8Block);
      batch.n = k + 1;
      if (batch.n == kQ8Batch || i + 1 == n || batch.first_block[batch.n] > (1 << 22)) {
        rc = check_launch(launch_q8_weights(batch, static_cast<hipStream_t>(stream)), "q8 weights launch");
        if (rc) return rc;
        std::memset(&batch, 0, sizeof batch);
      }
    }
    return DMUON_OK;
  });
}

int dmuon_q8_matmul_workspace_bytes(int64_t rows, int64_t outs, int64_t inner, int32_t out_dtype,
                                    size_t *out_bytes) {
  return guarded([&]() -> int {
    if (!out_bytes) return fail(DMUON_ERR_INVALID_ARG, "out_bytes is NULL");
    ProductType type;
    int rc = product_type(out_dtype, type);
    if (rc || (rc = check_sizes(rows, outs, inner))) return rc;
    *out_bytes = q8_matmul_workspace(rows, outs, round_up(inner, kQ8Block), type.fast);
    return DMUON_OK;
  });
}

int dmuon_q8_matmul(const void *codes, const void *scales, int64_t rows, const void *codes_b, const void *scales_b,
                    int64_t outs, int64_t inner, void *out, int32_t out_dtype, void *workspace,
                    size_t workspace_bytes, void *stream) {
  return guarded([&]() -> int {
    ProductType type;
    int rc = product_type(out_dtype, type);
    if (rc || (rc = check_sizes(rows, outs, inner))) return rc;
    if (rows == 0) return DMUON_OK;
    const int64_t kp = round_up(inner, kQ8Block), t4 = round_up(rows, kQ8ScaleRow), nkb = kp / kQ8Block;
    Buffers b;
    if ((rc = b.add(codes, rows * kp, false, "codes"))) return rc;
    if ((rc = b.add(scales, nkb * t4, false, "scales", 4))) return rc;
    if ((rc = b.add(codes_b, outs * kp, false, "codes_b"))) return rc;
    if ((rc = b.add(scales_b, round_up(outs, kQ8Block) / kQ8Block * nkb, false, "scales_b", 4))) return rc;
    if ((rc = b.add(out, rows * outs * elem_size(type.dt), true, "out"))) return rc;
    if ((rc = add_workspace(b, workspace, workspace_bytes, q8_matmul_workspace(rows, outs, kp, type.fast)))) return rc;
    if ((rc = b.check())) return rc;
    Q8Product p;
    p.a = static_cast<const uint8_t *>(codes);
    p.sa = static_cast<const uint8_t *>(scales);
    p.b = static_cast<const uint8_t *>(codes_b);
    p.sb = static_cast<const uint8_t *>(scales_b);
    p.out = out;
    p.ws = static_cast<float *>(workspace);
    p.rows = rows;
    p.outs = outs;
    p.kp = kp;
    p.out_dt = type.dt;
    p.fast = type.fast;
    return check_launch(launch_q8_matmul(p, static_cast<hipStream_t>(stream)), "q8 product launch");
  });
}

int dmuon_q8_weight_grad_workspace_bytes(int64_t rows, int64_t outs, int64_t cols, size_t *out_bytes) {
  return guarded([&]() -> int {
    if (!out_bytes) return fail(DMUON_ERR_INVALID_ARG, "out_bytes is NULL");
    const int rc = check_sizes(rows, outs, cols);
    if (rc) return rc;
    *out_bytes = q8_wgrad_workspace(rows, outs, cols);
    return DMUON_OK;
  });
}

int dmuon_q8_weight_grad(const void *dy, const void *codes, const void *scales, int64_t rows, int64_t outs,
                         int64_t cols, const void *base, void *out, int32_t out_dtype, void *workspace,
                         size_t workspace_bytes, void *stream) {
  return guarded([&]() -> int {
    if (!dtype_ok(out_dtype)) return fail(DMUON_ERR_UNSUPPORTED_DTYPE, "dtype code %d", out_dtype);
    int rc = check_sizes(rows, outs, cols);
    if (rc) return rc;
    const int64_t kp = round_up(cols, kQ8Block), t4 = round_up(rows, kQ8ScaleRow);
    const int64_t out_bytes = outs * cols * elem_size(out_dtype);
    Buffers b;
    if (rows > 0) {
      if ((rc = b.add(dy, rows * outs * 2, false, "dy"))) return rc;
      if ((rc = b.add(codes, rows * kp, false, "codes"))) return rc;
      if ((rc = b.add(scales, kp / kQ8Block * t4, false, "scales", 4))) return rc;
    }
    if ((rc = b.add(out, out_bytes, true, "out"))) return rc;
    // base = out: each element is read and written by the same thread
    if (base && base != out && (rc = b.add(base, out_bytes, false, "base"))) return rc;
    if ((rc = add_workspace(b, workspace, workspace_bytes, q8_wgrad_workspace(rows, outs, cols)))) return rc;
    if ((rc = b.check())) return rc;
    Q8WeightGrad p;
    p.dy = dy;
    p.x = static_cast<const uint8_t *>(codes);
    p.sx = static_cast<const uint8_t *>(scales);
    p.base = base;
    p.out = out;
    p.ws = workspace;
    p.rows = rows;
    p.outs = outs;
    p.cols = cols;
    p.kp = kp;
    p.out_dt = out_dtype;
    return check_launch(launch_q8_wgrad(p, static_cast<hipStream_t>(stream)), "q8 weight gradient launch");
  });
}

}  // extern "C"
