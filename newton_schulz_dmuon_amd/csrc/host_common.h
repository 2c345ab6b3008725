// Host helpers shared by the C entry points (host_api.cpp, q8_api.cpp).
#pragma once

#include <stdint.h>

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

}  // namespace dmuon
