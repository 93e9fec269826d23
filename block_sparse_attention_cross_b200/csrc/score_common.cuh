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

// Whether the row at position p sees a key farther away than fp32 counts.
// Positions go up to 2^30, and with rounded distances neighbouring keys would
// get the same one, or jump by many: with a slope such a row becomes NaN
// (through its sum, which costs the walk over the keys nothing) and is
// reported.
constexpr int kMaxSlopeDistance = 1 << 24;
__device__ __forceinline__ bool score_far(int2 vis, int p) {
  return vis.x < vis.y && max(abs(vis.x - p), abs(vis.y - 1 - p)) > kMaxSlopeDistance;
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

// Non-suspending test of a barrier's phase, for a warp that serves several.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
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

// Columns below n of a chunk of 32, as bits.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Columns whose bit is 0 become `value`.
__device__ __forceinline__ void keep_bits(uint32_t (&r)[32], uint32_t bits, float value) {
#pragma unroll
  for (int x = 0; x < 32; ++x)
    if (!(bits & (1u << x))) r[x] = f2u(value);
}

// The boxes of row `row` of a tile of 128 rows: each zeroed where it holds a
// NaN or an infinity; whether one did.  Out of line: only tiles that the mask
// cuts need it.  Called with no TMEM load or store in flight: their registers
// are not safe across a call.
template <int BOXES>
__device__ __noinline__ bool clean_row(uint8_t* tile, int row) {
  bool bad = false;
#pragma unroll 1
  for (int x = 0; x < BOXES; ++x) bad |= clean_box_row(tile + x * 128 * 128 + row * 128, row);
  fence_proxy_async_smem();
  return bad;
}

// ---- the table's values along the offsets of a tile pair ---------------------
// A tile pair meets 255 offsets; entry x of a window is offset o0 + x.  Far
// from zero a logarithmic bucket spans many offsets, so a window often holds
// few buckets: up to four boundaries are listed, and a window of one bucket
// needs no reads at all.
constexpr int kMaxCuts = 4;
struct WindowInfo {
  int cuts;                  // boundaries; kMaxCuts + 1: more, see the per-offset arrays
  int at[kMaxCuts];          // first entry of the next bucket
  int bucket[kMaxCuts + 1];
  int pad[2];
};

// The warp that fills the windows runs up to two windows ahead, and a walk may
// hold many tiles that need none: its waits get this many times the limit.
constexpr uint64_t kWindowPatience = 64;

// Whether the table's value may vary over a tile of keys [k0, k0 + 128) and
// rows at positions p0 ... p1: some offset is nearer than the distance.
__device__ __forceinline__ bool is_near(const ScoreArgs& a, int k0, int p0, int p1) {
  return a.table != nullptr && k0 - p1 < a.R && k0 + 127 - p0 > -a.R;
}

// Warp-collective; `heads` windows of consecutive heads from h0 on, 256 floats apart (log2 units: an entry below
// -2.35e38, as the type's lowest value, becomes -inf).
__device__ __forceinline__ void fill_window(const ScoreArgs& a, int h0, int heads, int o0, float* win, uint8_t* bwin,
                                            WindowInfo* info, bool* bad) {
  const int lane = lane_id();
  int n[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) n[x] = score_bucket(a, o0 + x * 32 + lane, bad);
  int cuts = 0;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    int prev = __shfl_up_sync(0xffffffffu, n[x], 1);
    const int last = __shfl_sync(0xffffffffu, n[x > 0 ? x - 1 : 0], 31);
    if (lane == 0) prev = x > 0 ? last : n[0];
    const bool cut = n[x] != prev && x * 32 + lane < 255;
    const uint32_t m = __ballot_sync(0xffffffffu, cut);
    const int at = cuts + __popc(m & ((1u << lane) - 1u));
    if (cut && at < kMaxCuts) {
      info->at[at] = x * 32 + lane;
      info->bucket[at + 1] = n[x];
    }
    cuts += __popc(m);
  }
  if (lane == 0) {
    info->cuts = min(cuts, kMaxCuts + 1);
    info->bucket[0] = n[0];
  }
  for (int g = 0; g < heads; ++g) {
    const __nv_bfloat16* tab =
        reinterpret_cast<const __nv_bfloat16*>(a.table) + static_cast<size_t>(h0 + g) * a.n_buckets;
#pragma unroll
    for (int x = 0; x < 8; ++x) win[g * 256 + x * 32 + lane] = __bfloat162float(tab[n[x]]) * kLog2e;
  }
  if (bwin != nullptr) {
#pragma unroll
    for (int x = 0; x < 8; ++x) bwin[x * 32 + lane] = static_cast<uint8_t>(n[x]);
  }
}

// ---- the score function on the columns of a thread's row ---------------------
// In log2 units.  cap tanh(x), x = s scale / cap: where |x| is at most 0.45, s
// times a polynomial in x^2 on the FMA pipe, whose error is relative to the
// score; beyond, cap - 2 cap / (1 + e^(2x)), two MUFU operations a score, right
// at both ends, off by up to 3e-7 of the cap, which is 7e-7 of a score of that
// size.  (That form alone is not enough: of scores far below the cap it leaves
// the cap's last bits, 12% of a score at a millionth of it.)  The polynomial
// leaves the MUFU, which bounds the softmax, to the exponentials.  Every score
// chooses by itself, so no other row and no masked place changes a bit of it;
// a row without large ones skips the second form.
struct ScoreTerms {
  float sc;                  // scale log2e
  float capA, kcap, small;   // cap log2e; 2 log2e scale / cap; largest |s| for the polynomial
  float k, ninv2;            // scale / cap; -1 / (cap log2e)^2
  float shift;               // added to the capped score where there is no bias
  float c[4];                // capped score = s (c0 + c1 x^2 + c2 x^4 + c3 x^6), x = k s
};
__device__ __forceinline__ ScoreTerms score_terms(const ScoreArgs& a) {
  ScoreTerms t = {};
  t.sc = a.scale * kLog2e;
  if (a.cap > 0.f) {
    t.k = a.scale / a.cap;
    t.capA = a.cap * kLog2e;
    t.kcap = 2.f * kLog2e * t.k;
    // (1 / cap^2 must stay finite; under smaller caps the second form's error,
    // relative to the cap, is nothing to the scores)
    t.small = a.cap > 1e-18f ? 0.45f / t.k : -1.f;
    t.ninv2 = -(1.f / t.capA) * (1.f / t.capA);
    // tanh(x) / x as a polynomial in x^2, interpolated at the four Chebyshev
    // nodes of [0, 0.2025] (relative error at most 2.6e-7).  The powers of x
    // are formed from x itself: coefficients with powers of scale / cap would
    // underflow under large caps.  (Five terms, right to 8e-8 up to 0.6: 24
    // heads of 8192 tokens, d = 128, 1217 us instead of 1135.)
    t.c[0] = 0.999999762f * t.sc;
    t.c[1] = -0.333294511f * t.sc;
    t.c[2] = 0.132361695f * t.sc;
    t.c[3] = -0.0460216627f * t.sc;
  }
  return t;
}

__device__ __forceinline__ uint64_t pair_of(const uint32_t* r, int x) { return f2pack(u2f(r[x]), u2f(r[x + 1])); }
__device__ __forceinline__ void set_pair(uint32_t* r, int x, uint64_t v) {
  float lo, hi;
  f2unpack(v, lo, hi);
  r[x] = f2u(lo);
  r[x + 1] = f2u(hi);
}

// F: which terms the kernel was built for.  A kernel carries the code of its
// own terms only: code that a call skips costs instruction-cache misses (all
// terms in one kernel ran plain far tiles of a table at half the speed).
enum ScoreForm { kCap = 1, kBias = 2 };

// What a tile pair adds to the scores of one thread's row.
struct ScoreBias {
  float slope, off0;   // distance: -slope |off0 + DIR x| at column x
  int side;            // +1 / -1: every offset of the tile is >= 0 / <= 0, the distance is linear; 0: neither
  bool window;         // the table's value at column x is wr[DIR x], otherwise `flat` everywhere
  const float* wr;
  float flat;          // 0 without a table
};

// Largest |score| of the row.  (A NaN is not seen; every form passes it on.)
template <int N>
__device__ __forceinline__ float score_extent(const uint32_t (&r)[N]) {
  float big0 = 0.f, big1 = 0.f;
#pragma unroll
  for (int x = 0; x < N; x += 4) {
    big0 = fmax3(big0, fabsf(u2f(r[x])), fabsf(u2f(r[x + 1])));
    big1 = fmax3(big1, fabsf(u2f(r[x + 2])), fabsf(u2f(r[x + 3])));
  }
  return fmaxf(big0, big1);
}

// The capped scores s of two columns by the polynomial, plus `shift`; f: the cap's derivative.
template <bool FACTOR, bool BIAS>
__device__ __forceinline__ uint64_t cap_pair(const ScoreTerms& t, uint64_t s, uint64_t shift2, float& f0, float& f1) {
  const uint64_t x = fmul2(s, f2pack(t.k, t.k)), v = fmul2(x, x);
  uint64_t q = f2pack(t.c[3], t.c[3]);
#pragma unroll
  for (int i = 2; i >= 0; --i) q = ffma2(q, v, f2pack(t.c[i], t.c[i]));
  if (!FACTOR) return ffma2(s, q, shift2);
  const uint64_t y = fmul2(s, q);
  f2unpack(ffma2(fmul2(y, f2pack(t.ninv2, t.ninv2)), y, f2pack(1.f, 1.f)), f0, f1);
  return BIAS ? fadd2(y, shift2) : y;   // (the backward has no other shift)
}
template <bool FACTOR, bool BIAS, int N>
__device__ __forceinline__ void cap_polynomial(const ScoreTerms& t, uint32_t (&r)[N], float (&f)[N], float shift) {
  const uint64_t shift2 = f2pack(shift, shift);
#pragma unroll
  for (int x = 0; x < N; x += 2) set_pair(r, x, cap_pair<FACTOR, BIAS>(t, pair_of(r, x), shift2, f[x], f[x + 1]));
}
// Either form, score by score.
template <bool FACTOR, bool BIAS, int N>
__device__ __forceinline__ void cap_mixed(const ScoreTerms& t, uint32_t (&r)[N], float (&f)[N], float shift) {
  const uint64_t shift2 = f2pack(shift, shift);
#pragma unroll
  for (int x = 0; x < N; x += 2) {
    const float s[2] = {u2f(r[x]), u2f(r[x + 1])};
    set_pair(r, x, cap_pair<FACTOR, BIAS>(t, f2pack(s[0], s[1]), shift2, f[x], f[x + 1]));
#pragma unroll
    for (int e = 0; e < 2; ++e) {   // (no branches: the two forms of different scores run beside each other)
      const bool large = fabsf(s[e]) > t.small;
      const float rc = rcp_approx(1.f + ex2_approx(s[e] * t.kcap));
      if (FACTOR) f[x + e] = large ? 4.f * (rc - rc * rc) : f[x + e];
      r[x + e] = large ? f2u(fmaf(-2.f * t.capA, rc, t.capA) + shift) : r[x + e];
    }
  }
}

// The score function.  DIR = 1: the columns are keys; DIR = -1: queries.
// BENT: the distance may pass 0 inside the tile.  live = false: a row whose
// result nobody reads, which must not drag its warp through the cap's second
// form.
template <int F, int DIR, bool FACTOR, bool BENT, int N>
__device__ __forceinline__ void score_columns(const ScoreArgs& a, const ScoreTerms& t, uint32_t (&r)[N], float (&f)[N],
                                              const ScoreBias& b, bool live = true) {
  // The constant part of the biases: the flat table value, and the distance
  // of column 0 where the distance is linear over the tile.
  const bool slopes = (F & kBias) && a.slopes != nullptr, linear = slopes && (!BENT || b.side != 0);
  const float sl = b.side > 0 ? -b.slope : b.slope;   // -slope |off0 + DIR x| = sl (off0 + DIR x)
  const float shift = F & kBias ? (b.window ? 0.f : b.flat) + (linear ? sl * b.off0 : 0.f) : t.shift;
  if (F & kCap) {
    if (live && score_extent(r) > t.small) cap_mixed<FACTOR, (F & kBias) != 0>(t, r, f, shift);
    else cap_polynomial<FACTOR, (F & kBias) != 0>(t, r, f, shift);
    __syncwarp();   // rows of a warp may take either form, and the tensor-memory accesses that follow need all lanes
  } else {
    const uint64_t sc = f2pack(t.sc, t.sc), shift2 = f2pack(shift, shift);
#pragma unroll
    for (int x = 0; x < N; x += 2) set_pair(r, x, ffma2(pair_of(r, x), sc, shift2));
    if (FACTOR) {
#pragma unroll
      for (int x = 0; x < N; ++x) f[x] = 1.f;
    }
  }
  if (!(F & kBias)) return;
  if (linear) {
#pragma unroll
    for (int x = 0; x < N; ++x) r[x] = f2u(fmaf(sl, static_cast<float>(DIR * x), u2f(r[x])));
  } else if (BENT && slopes) {
#pragma unroll
    for (int x = 0; x < N; ++x) r[x] = f2u(fmaf(-b.slope, fabsf(b.off0 + static_cast<float>(DIR * x)), u2f(r[x])));
  }
  if (b.window) {
#pragma unroll
    for (int x = 0; x < N; ++x) r[x] = f2u(u2f(r[x]) + b.wr[DIR * x]);
  }
}

}  // namespace calibatt
