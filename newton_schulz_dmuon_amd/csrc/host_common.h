// Host helpers shared by the C entry points (host_api.cpp, q8_api.cpp,
// q4_api.cpp).
#pragma once

#include <stdint.h>

#include <exception>
#include <vector>

#include "../../include/dmuon.h"
#include "internal.h"

namespace dmuon {

// Records the thread's error message and returns `status`.
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_error();
// DMUON_OK, or the HIP error as a failure of `what`.
int check_launch(hipError_t e, const char *what);

inline int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline int64_t elem_size(int32_t dt) { return dt == DMUON_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t dt) { return dt == DMUON_BF16 || dt == DMUON_F32; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Interval {
  uintptr_t lo, hi;  // [lo, hi)
  bool written;
  const char *what;
  int32_t index;
};

// Fails if a written interval overlaps any other interval.
int check_aliasing(std::vector<Interval> &iv);

// Limits of the block products' entry points.  A launch takes fewer than 2^32
// threads along its grid.  With these limits the products' grids stay below that: at
// most 2^22 tiles of 128, or with 2^37 outputs 2^21 whole and as many ragged tiles of
// 256, of 512 threads each.
constexpr int64_t kMaxRows = int64_t(1) << 29;
constexpr int64_t kMaxSide = int64_t(1) << 22;
constexpr int64_t kMaxElems = int64_t(1) << 37;

// Whether a buffer has more than kMaxElems elements (the factors are within the
// limits above, so the product cannot overflow).
inline bool too_large(int64_t rows, int64_t cols) { return rows * cols > kMaxElems; }

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

inline int add_workspace(Buffers &b, void *workspace, size_t have, size_t need) {
  if (need == 0) return DMUON_OK;
  if (have < need)
    return fail(DMUON_ERR_WORKSPACE_TOO_SMALL, "workspace needs %zu bytes, got %zu", need, have);
  return b.add(workspace, static_cast<int64_t>(need), true, "workspace", 256);
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

}  // namespace dmuon
