// score_common.cuh -- device helpers shared by the score-modified attention
// kernels: row intervals, kept blocks and the score function.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace calibatt {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

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

template <int V>
using IntC = std::integral_constant<int, V>;

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t f2u(float x) { return __float_as_uint(x); }
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Warp-collective: one elected lane issues the copy.
__device__ __forceinline__ void tma_load_4d_w(void* dst, const CUtensorMap* tm, int x, int n, int h, int b, uint64_t* bar,
                                              uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;\n\t}\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(n), "r"(h), "r"(b), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
// Untiled copy: both addresses 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_load_w(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}\n" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// One 64-column box row of a 128-byte-swizzled tile: zeroed when it holds a
// NaN or an infinity (an exponent of all ones carries into the sign's place),
// and whether it did.  `at`: the row's address; lanes of consecutive rows read
// different banks.
__device__ __forceinline__ bool clean_box_row(uint8_t* at, int row) {
  uint32_t nf = 0;
#pragma unroll
  for (int ch = 0; ch < 8; ++ch) {
    const uint4 u = *reinterpret_cast<const uint4*>(at + ((ch ^ (row & 7)) << 4));
    nf |= ((u.x & 0x7f807f80u) + 0x00800080u) | ((u.y & 0x7f807f80u) + 0x00800080u) |
          ((u.z & 0x7f807f80u) + 0x00800080u) | ((u.w & 0x7f807f80u) + 0x00800080u);
  }
  const bool bad = (nf & 0x80008000u) != 0;
  if (bad) {
    const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) *reinterpret_cast<uint4*>(at + (ch << 4)) = z;
  }
  return bad;
}

// Walk over the kept key tiles [lo, hi) of one query tile, in order.  Every
// lane of a warp holds the same state; all roles evaluate the same data.
struct KeyWalk {
  int kb, next, hi;      // current and next kept key tile (-1: none), end of the range
  uint32_t word;         // mask: kept tiles after `next` in the 32 tiles from wbase on
  int wbase;
};

__device__ __forceinline__ int key_find(const ScoreArgs& a, int h, int qb, KeyWalk& w) {
  while (w.word == 0) {
    w.wbase += 32;
    if (w.wbase >= w.hi) return -1;
    const int kb = w.wbase + lane_id();
    w.word = __ballot_sync(0xffffffffu, kb < w.hi && score_kept(a, h, qb, kb));
  }
  const int kb = w.wbase + __ffs(w.word) - 1;
  w.word &= w.word - 1;
  return kb;
}

__device__ __forceinline__ void key_next(const ScoreArgs& a, int h, int qb, KeyWalk& w) {
  w.kb = w.next;
  if (a.mask != nullptr) w.next = key_find(a, h, qb, w);
  else w.next = w.kb + 1 < w.hi ? w.kb + 1 : -1;
}

// Starts the walk; returns whether it has a tile.
__device__ __forceinline__ bool key_start(const ScoreArgs& a, int h, int qb, int lo, int hi, KeyWalk& w) {
  w.hi = hi;
  w.word = 0;
  w.wbase = lo - 32;
  w.next = a.mask != nullptr ? key_find(a, h, qb, w) : lo < hi ? lo : -1;
  if (w.next < 0) {
    w.kb = -1;
    return false;
  }
  key_next(a, h, qb, w);
  return true;
}

// The score function on N columns of one thread's row, in log2 units.  DIR =
// 1: the columns are keys, off0 the first one's offset j - p; DIR = -1: the
// columns are queries.  `near`: the table's values for the columns are wr[DIR
// x]; otherwise `far` is added.  With FACTOR, f becomes d c / d s of the cap.
// cap tanh(x) = cap - 2 cap / (1 + e^(2x)) is right at both ends, and the
// MUFU's relative errors stay 1e-7 of the cap.
struct ScoreTerms {
  float sc, capA, kcap;   // scale log2e; cap log2e; 2 log2e scale / cap
};
__device__ __forceinline__ ScoreTerms score_terms(const ScoreArgs& a) {
  ScoreTerms t;
  t.sc = a.scale * kLog2e;
  t.capA = a.cap * kLog2e;
  t.kcap = a.cap > 0.f ? 2.f * kLog2e * a.scale / a.cap : 0.f;
  return t;
}
template <int DIR, bool FACTOR, int N>
__device__ __forceinline__ void score_columns(const ScoreArgs& a, const ScoreTerms& t, uint32_t (&r)[N], float (&f)[N],
                                              float slope, float off0, bool near, const float* wr, float far) {
  if (a.cap > 0.f) {
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const float rc = rcp_approx(1.f + ex2_approx(u2f(r[x]) * t.kcap));
      if (FACTOR) f[x] = 4.f * (rc - rc * rc);
      r[x] = f2u(fmaf(-2.f * t.capA, rc, t.capA));
    }
  } else {
#pragma unroll
    for (int x = 0; x < N; ++x) {
      r[x] = f2u(u2f(r[x]) * t.sc);
      if (FACTOR) f[x] = 1.f;
    }
  }
  if (a.slopes != nullptr) {
#pragma unroll
    for (int x = 0; x < N; ++x) r[x] = f2u(fmaf(-slope, fabsf(off0 + static_cast<float>(DIR * x)), u2f(r[x])));
  }
  if (near) {
#pragma unroll
    for (int x = 0; x < N; ++x) r[x] = f2u(u2f(r[x]) + wr[DIR * x]);
  } else if (a.table != nullptr) {
#pragma unroll
    for (int x = 0; x < N; ++x) r[x] = f2u(u2f(r[x]) + far);
  }
}

}  // namespace calibatt
