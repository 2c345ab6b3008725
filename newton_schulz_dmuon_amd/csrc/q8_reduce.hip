// Sharing out the tiles of the 8-bit products, and adding the fp32 results of
// tiles that were split along their sum.

#include <algorithm>

#include "q8_device.h"

namespace dmuon {

namespace {

constexpr int64_t kCus = 256;

// Adds the pieces of the tail tiles, plus the base of a weight gradient, in a
// fixed order: eight columns of a row per thread.  Bound by the memory that
// holds the pieces' results, each read once: with their writing 6 TB/s.
__global__ __launch_bounds__(256) void q8_reduce_kernel(const float *__restrict__ ws, TileSplit sp, int64_t rows,
                                                        int64_t cols, const void *base, void *out, int32_t dt) {
  const uint32_t size = sp.ta * sp.tb, per = size / 2048;
  const uint32_t place = uniform(blockIdx.x / per), part = blockIdx.x - place * per;
  uint32_t a, b;
  tile_at(sp.whole + place, sp.na, sp.nb, a, b);
  const uint32_t at = (part * 256 + threadIdx.x) * 8;
  const uint32_t shift = sp.ta == 256 ? 8 : 7;
  const int64_t r = static_cast<int64_t>(b) * sp.tb + (at >> shift);
  const int64_t c = static_cast<int64_t>(a) * sp.ta + (at & (sp.ta - 1));
  if (r >= rows || c >= cols) return;
  const float *const src = ws + static_cast<int64_t>(place) * sp.pieces * size + at;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (uint32_t i = 0; i < sp.pieces; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 w = *(const g_f32x4 *)(src + static_cast<int64_t>(i) * size + 4 * h);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * h + k] += w[k];
    }
  finish_run<8>(base, out, dt, r * cols + c, cols - c, v);
}

}  // namespace

TileSplit choose_split(int64_t cols, int64_t rows, int64_t steps, std::initializer_list<TileCost> tiles,
                       float *cost) {
  TileSplit best{};
  float best_us = 0.f;
  for (const TileCost &c : tiles) {
    const int64_t na = (cols + c.ta - 1) / c.ta, nb = (rows + c.tb - 1) / c.tb, count = na * nb;
    const int64_t slots = c.per_cu * kCus;  // work-groups on the chip at once
    // a step's time with this many work-groups on the chip
    auto step_us = [&](int64_t n) {
      if (c.per_cu == 1) return c.low + (c.full - c.low) * static_cast<float>(std::min(n, kCus)) / kCus;
      return n <= kCus ? c.low : c.full;
    };
    // a launch's threads stay below 2^32
    if (best.ta && count > (1 << 22)) continue;
    const int64_t rounds = count / slots, left = count - rounds * slots;
    const float whole_us = static_cast<float>(rounds * steps) * step_us(slots);
    for (const int64_t pieces : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (pieces > steps || (pieces > 1 && left == 0)) break;
      const int64_t groups = left * pieces, piece_steps = (steps + pieces - 1) / pieces;
      float us = whole_us + 4.f;  // launch, first loads, epilogue
      const int64_t full = groups / slots, rest = groups - full * slots;
      us += static_cast<float>(full * piece_steps) * step_us(slots);
      if (rest) us += static_cast<float>(piece_steps) * step_us(rest);
      // the reduce launch: every piece's result written and read at 6 TB/s
      if (pieces > 1) us += 3.5f + static_cast<float>(groups * c.ta * c.tb * 8) / 6e6f;
      if (best.ta == 0 || us < best_us) {
        best_us = us;
        best.ta = static_cast<uint32_t>(c.ta);
        best.tb = static_cast<uint32_t>(c.tb);
        best.na = static_cast<uint32_t>(na);
        best.nb = static_cast<uint32_t>(nb);
        best.whole = static_cast<uint32_t>(pieces > 1 ? rounds * slots : count);
        best.tail = static_cast<uint32_t>(pieces > 1 ? left : 0);
        best.pieces = static_cast<uint32_t>(pieces);
      }
    }
  }
  if (cost) *cost = best_us;
  return best;
}

hipError_t launch_q8_reduce(const float *ws, const TileSplit &sp, int64_t rows, int64_t cols, const void *base,
                            void *out, int32_t dt, hipStream_t st) {
  const uint32_t grid = sp.tail * (sp.ta * sp.tb / 2048);
  hipLaunchKernelGGL(q8_reduce_kernel, dim3(grid), dim3(256), 0, st, ws, sp, rows, cols, base, out, dt);
  return hipGetLastError();
}

}  // namespace dmuon
