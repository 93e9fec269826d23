// score_common.cuh -- device helpers shared by the score-modified attention
// kernels: row intervals, kept blocks and the score function.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace calibatt {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float ld_elem(const float* p) { return *p; }
__device__ __forceinline__ float ld_elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Visible keys [x, y) of row i of batch entry b; (0, 0) where it sees nothing.
__device__ __forceinline__ int2 score_row(const ScoreArgs& a, int b, int i) {
  if (i >= a.Nq) return make_int2(0, 0);
  int2 r = a.row[static_cast<size_t>(b) * a.Nq + i];
  r.x = max(r.x, 0);
  r.y = min(r.y, a.Nk);
  return r.x < r.y ? r : make_int2(0, 0);
}

// Range of a query tile, clamped to the keys: x, y as score_row for the union
// of its rows; keys inside [z, w) are seen by every row.
__device__ __forceinline__ int4 score_tile(const ScoreArgs& a, int b, int qb) {
  int4 t = a.tile[static_cast<size_t>(b) * a.nqb + qb];
  t.x = max(t.x, 0);
  t.y = min(t.y, a.Nk);
  return t;
}

// Whether the calibrated mask keeps block (qb, kb) of head h.
__device__ __forceinline__ bool score_kept(const ScoreArgs& a, int h, int qb, int kb) {
  return a.mask == nullptr ||
         a.mask[(static_cast<size_t>(a.map_offset + h) * a.nqb + qb) * a.nkb + kb] != 0;
}

// Bucket of offset j - p; a map entry outside [0, n_buckets) is reported by
// the caller through *bad and read as bucket 0.
__device__ __forceinline__ int score_bucket(const ScoreArgs& a, int off, bool* bad) {
  const int n = a.buckets[min(max(off, -a.R), a.R) + a.R];
  if (n < 0 || n >= a.n_buckets) {
    *bad = true;
    return 0;
  }
  return n;
}

}  // namespace calibatt
