// score_fwd.cu -- score-modified attention forward on the tensor cores (bf16).
//
// The pipeline is the block-sparse forward's: a persistent CTA per SM holds
// two query tiles ("slots") of 128 rows, one thread per query row; the tensor
// core alternates between the slots, so that one slot's softmax runs while the
// other slot's products do.  Warps 0-3 and 4-7: softmax of slots 0 and 1;
// warps 8 and 11: TMA producers, one K/V ring each; warp 9 issues every
// tcgen05.mma; warp 10 fills the table's windows (score_common.cuh).  TMEM:
// slot s owns columns [256 s, 256 s + 256):
// scores at + 0 (the probabilities overwrite their first half as bf16 pairs,
// the A operand of the second product), O at + 128.
//
// What differs:
//  - a tile walks the 128-key tiles of its rows' interval range, restricted to
//    the calibrated mask's kept blocks where one is given, and only tiles
//    that the interval of some row cuts pay for an element mask;
//  - the scores pass through the cap, the distance bias and the table in
//    chunks of 32 columns, kept in TMEM between the pass that finds the maximum
//    and the one that exponentiates; a cap without a bias needs no maximum;
//  - tensors are 4-D maps with their own strides, so lengths need no padding
//    and rows past a length read as zero;
//  - the G query heads of a key head share one tile when their rows fit (few
//    queries: rows g Nq + i), so K and V are read once for all of them;
//  - with at most 32 such rows they are repeated in all four lane quarters of
//    the tile, and each warp takes a quarter of every key tile's columns (a
//    warp reaches only its own TMEM lanes), leaving four partial results;
//  - few tiles against many keys are split along the keys; k_score_join
//    (score_rows.cu) adds the partial results in a fixed order.
//
// What bounds it.  Long queries: per 128 x 128 pair 1024 MUFU cycles of
// exponentials and 1024 tensor cycles (d = 128), but a slot's chain (scores,
// softmax, second product, next scores) is serial, and a softmax warp, mostly
// alone on its sub-partition, runs at its latencies: 2300 cycles of softmax a
// pair for plain scores, 3300 capped or with slopes, 5100 with both, beside
// 1660 of products.  24 heads of 8192 tokens, d = 128: 0.91 ms plain (907
// TFLOP/s), 1.14 capped, 1.13 with slopes, 1.06 with a table.  (Two warpgroups
// a slot, half of the columns each: capped 1.10, but plain 0.96, a table 1.30
// ms.)  Few queries: HBM; 4 tokens of 24 heads read 930 MB of K and V in 0.15
// ms (6.2 TB/s, 96% of the measured copy), 32 sequences of different lengths
// 670 MB in 0.16 ms (the longest sequences last).
#include <algorithm>
#include <atomic>

#include "score_common.cuh"

namespace calibatt {
namespace {

constexpr int TILE = 128;
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;
constexpr uint32_t kSoftmaxRegs = 192;
constexpr uint32_t kControlRegs = 120;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs == kThreads * kLaunchRegs, "register split");
constexpr int kProducer0 = 8, kMma = 9, kWindow = 10, kProducer1 = 11;
constexpr uint32_t kTmemCols = 512;
// The reference maximum is raised, and O rescaled, only when a tile's maximum
// exceeds it by more than this many log2 units: P stays below 2^64, and sums
// over 2^24 keys inside fp32 for |v| < 2^39.
constexpr float kRescaleThreshold = 64.0f;
constexpr int kMaxPackedTable = 4;   // heads of a packed tile with a table (windows in shared memory, two buffers)

template <int D>
struct Layout {
  static constexpr uint32_t BOX = TILE * 64 * 2;         // 128 rows x 64 columns, one swizzle span
  static constexpr uint32_t TBYTES = TILE * D * 2;       // one Q, K or V tile
  static constexpr uint32_t WIN = 2 * kMaxPackedTable * 256 * 4;   // the table's values in a tile pair's offsets, two buffers
  static constexpr int RING = D == 128 ? 2 : 4;          // K/V tiles per slot
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_RING = 2 * TBYTES;
  static constexpr uint32_t OFF_WIN = OFF_RING + 2 * RING * TBYTES;   // [2 slots][2 buffers][WIN / 2]
  static constexpr uint32_t OFF_CTRL = OFF_WIN + 2 * WIN;
  static constexpr uint32_t CTRL = 1024;
  static constexpr uint32_t SMEM = OFF_CTRL + CTRL + 1024;   // + alignment slack
  static_assert(SMEM <= 232448, "shared memory");
};

template <int RING>
struct Ctrl {
  uint64_t ring_full[2][RING], ring_empty[2][RING];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2];
  uint64_t o_full[2], o_free[2];
  uint64_t win_full[2][2], win_empty[2][2];
  WindowInfo win_info[2][2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  uint32_t bad[2][2][4];   // [slot][step & 1]: keys of a V tile that hold a non-finite value
};

struct FwdArgs {
  ScoreArgs a;
  int Hx;       // heads of the tile grid: Hkv where the G heads share a tile, else H
  int nq;       // query tiles per head of the grid
  int hgroup;   // heads walked together, see tile_at
  int T;        // tiles
};

// One tile of the walk and its current key tile.
struct Walk : KeyWalk {
  int b, hx, qb, sp;
};

// Order of the tiles: heads in groups whose K and V fit well into L2, and
// inside a group query tiles from the last to the first, all heads of one
// query tile together: under a causal rule the longest walks come first, so
// the static round-robin over slots stays balanced.  Splits innermost.
__device__ __forceinline__ void tile_at(const FwdArgs& f, int t, Walk& w) {
  w.sp = t % f.a.splits;
  int u = t / f.a.splits;
  const int BH = f.a.B * f.Hx;
  const int g = u / (f.hgroup * f.nq);
  const int base = g * f.hgroup, size = min(f.hgroup, BH - base);
  u -= base * f.nq;
  w.qb = f.nq - 1 - u / size;
  const int bh = base + u % size;
  w.b = bh / f.Hx;
  w.hx = bh % f.Hx;
}

// Starts tile t; returns whether it has a key tile.
__device__ __forceinline__ bool walk_start(const FwdArgs& f, int t, Walk& w) {
  tile_at(f, t, w);
  const int4 r = score_tile(f.a, w.b, w.qb);
  int lo = r.x >> 7;
  w.hi = (r.y + TILE - 1) >> 7;
  if (f.a.splits > 1 && w.hi > lo) {
    const int per = (w.hi - lo + f.a.splits - 1) / f.a.splits;
    lo = min(w.hi, lo + w.sp * per);
    w.hi = min(w.hi, lo + per);
  }
  if (r.x >= r.y) w.hi = lo;
  return key_start(f.a, w.hx, w.qb, lo, w.hi, w);
}

// Tile of slot c in round `round` of n slots: the slots take turns from the
// front and from the back, so that a slot that drew a long walk in one round
// draws a short one in the next.  T or more: none.
__device__ __forceinline__ int tile_of(int round, int c, int n) {
  return round * n + ((round & 1) ? n - 1 - c : c);
}

// A role's position: key tiles of this slot's non-empty tiles, one after the other.
struct Cursor {
  Walk w;
  int round, slot;
  bool first, done;
};

__device__ __forceinline__ void cursor_seek(const FwdArgs& f, Cursor& c) {
  const int n = 2 * gridDim.x;
  for (; c.round * n < f.T; ++c.round) {
    const int t = tile_of(c.round, c.slot, n);
    if (t < f.T && walk_start(f, t, c.w)) {
      c.first = true;
      return;
    }
  }
  c.done = true;
}

__device__ __forceinline__ void cursor_init(const FwdArgs& f, Cursor& c, int s) {
  c.slot = blockIdx.x + s * gridDim.x;
  c.round = 0;
  c.done = false;
  cursor_seek(f, c);
}

__device__ __forceinline__ void cursor_next(const FwdArgs& f, Cursor& c) {
  if (c.w.next >= 0) {
    c.first = false;
    key_next(f.a, c.w.hx, c.w.qb, c.w);
  } else {
    ++c.round;
    cursor_seek(f, c);
  }
}

// Beside the ScoreForm bits: capped scores without a bias and with a cap of
// at most kBoundedCap need no maximum.
constexpr int kBounded = 4;
// At most 32 rows, repeated in the four lane quarters (a kernel of its own, so
// that neither form carries the other's code).
constexpr int kFew = 8;
// Key tiles whose scores the mask leaves whole; that it cuts (or where the
// distance passes 0); and, without a cap, whole ones with one table value and
// no slope, or with a slope and one table value.
enum TileKind { kFullTile, kCutTile, kFlatTile, kLinearTile };
// Largest cap in log2 units that goes without a maximum.  The reference is a
// quarter of the cap: probabilities lie in 2^-100 ... 2^60, so that sums over
// 2^24 keys stay inside fp32 for |v| < 2^43, rows whose scores are all at -cap
// keep full precision down to |v| = 2^-26, and bf16 has fp32's exponents.
constexpr float kBoundedCap = 80.f;

template <int D, int F>
__global__ void __launch_bounds__(kThreads, 1)
    k_score_fwd(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ FwdArgs f) {
  using L = Layout<D>;
  constexpr bool FEW = (F & kFew) != 0;
  constexpr int R = L::RING;
  static_assert(sizeof(Ctrl<R>) <= L::CTRL, "control block");
  const ScoreArgs& a = f.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctrl<R>* c = reinterpret_cast<Ctrl<R>*>(smem + L::OFF_CTRL);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      for (int e = 0; e < R; ++e) {
        mbar_init(&c->ring_full[s][e], 1);
        mbar_init(&c->ring_empty[s][e], 1);
      }
      mbar_init(&c->q_full[s], 1);
      mbar_init(&c->q_empty[s], 1);
      mbar_init(&c->s_full[s], 1);
      mbar_init(&c->p_full[s], 128);
      mbar_init(&c->o_full[s], 1);
      mbar_init(&c->o_free[s], 128);
      for (int e = 0; e < 2; ++e) {
        mbar_init(&c->win_full[s][e], 32);
        mbar_init(&c->win_empty[s][e], 128);
      }
    }
    mbar_init(&c->drain, 1);
    c->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kMma) {
    tmem_alloc(&c->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem_base;

  if (warp >= 8) regs_dec<kControlRegs>();
  if (warp == kProducer0 || warp == kProducer1) {
    // ===================== TMA producer of one slot ===========================
    const int s = warp == kProducer1;
    Cursor cu;
    cursor_init(f, cu, s);
    uint32_t g = 0;
    int qf = 0;
    bool ok = true;
    // (with few queries K and V are read once)
    const uint64_t pol_q = l2_policy_evict_first(), pol = FEW ? pol_q : l2_policy_evict_last();
    uint8_t* ring = smem + L::OFF_RING + s * R * L::TBYTES;
    const int copies = FEW ? 4 : 1;
    const uint32_t q_bytes = a.packed ? static_cast<uint32_t>(copies * a.G * a.Nq * D * 2) : L::TBYTES;
    while (ok && !cu.done) {
      const Walk& w = cu.w;
      if (cu.first) {
        ok = __all_sync(0xffffffffu, mbar_wait(&c->q_empty[s], (qf & 1) ^ 1, &c->abort, a.spin_ns));
        if (!ok) break;
        mbar_arrive_expect_tx_w(&c->q_full[s], q_bytes);
        for (int r = 0; r < copies; ++r)
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tma_load_4d_w(smem + L::OFF_Q + s * L::TBYTES + x * L::BOX + r * 32 * 128, &tmQ, x * 64, w.qb * TILE,
                          a.packed ? w.hx * a.G : w.hx, w.b, &c->q_full[s], pol_q);
        ++qf;
      }
      const int hk = a.packed ? w.hx : w.hx / a.G;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const int e = g % R;
        ok = __all_sync(0xffffffffu, mbar_wait(&c->ring_empty[s][e], ((g / R) & 1) ^ 1, &c->abort, a.spin_ns));
        if (!ok) break;
        mbar_arrive_expect_tx_w(&c->ring_full[s][e], L::TBYTES);
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tma_load_4d_w(ring + e * L::TBYTES + x * L::BOX, kv ? &tmV : &tmK, x * 64, w.kb * TILE, hk, w.b,
                        &c->ring_full[s][e], pol);
        ++g;
      }
      cursor_next(f, cu);
    }
    if (lane == 0) {
      if (!ok) {
        c->abort = 1;
        report_status(a.status, CALIBATT_E_TIMEOUT);
      }
      // Drain: every copy issued must have landed before the CTA may exit.
      for (int e = 0; e < R; ++e) {
        const uint32_t fills = (g > static_cast<uint32_t>(e)) ? (g - 1 - e) / R + 1 : 0;
        if (fills > 0) mbar_wait(&c->ring_full[s][e], (fills - 1) & 1, nullptr, a.spin_ns);
      }
      if (qf > 0) mbar_wait(&c->q_full[s], (qf - 1) & 1, nullptr, a.spin_ns);
    }
  } else if (warp == kMma) {
    // ===================== MMA issuer =========================================
    // Per key tile of a slot: S, then (once the probabilities are stored) the
    // second product and the slot's next S; the slots are served in turn.
    Cursor cu0, cu1;
    cursor_init(f, cu0, 0);
    cursor_init(f, cu1, 1);
    constexpr uint32_t IDESC_S = idesc_bf16_f32(TILE, TILE, false);
    constexpr uint32_t IDESC_O = idesc_bf16_f32(TILE, D, true);
    uint32_t g0 = 0, g1 = 0, gb0 = 0, gb1 = 0;
    int qt0 = 0, qt1 = 0, ot0 = 0, ot1 = 0;
    bool ok = true;
    auto issue_s = [&](auto s_c) {
      constexpr int s = decltype(s_c)::value;
      Cursor& cu = s ? cu1 : cu0;
      uint32_t& g = s ? g1 : g0;
      int& qt = s ? qt1 : qt0;
      const int e = g % R;
      const bool w = (!cu.first || mbar_wait(&c->q_full[s], qt & 1, &c->abort, a.spin_ns)) &&
                     mbar_wait(&c->ring_full[s][e], (g / R) & 1, &c->abort, a.spin_ns);
      if (!__all_sync(0xffffffffu, w)) return false;
      tc_fence_after();
      const uint32_t sQ = smem_u32(smem + L::OFF_Q + s * L::TBYTES);
      const uint32_t sK = smem_u32(smem + L::OFF_RING + (s * R + e) * L::TBYTES);
      const uint32_t tS = tmem + s * 256;
      if (D == 128) {
        mma_ss_k128_w(tS, sdesc_sw128(sQ, 16, 1024), sdesc_sw128(sK, 16, 1024), IDESC_S, L::BOX >> 4);
      } else {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16_ss_w(tS, sdesc_sw128(sQ + kk * 32, 16, 1024), sdesc_sw128(sK + kk * 32, 16, 1024), IDESC_S,
                        kk > 0 ? 1u : 0u);
      }
      mma_commit_w(&c->s_full[s]);
      mma_commit_w(&c->ring_empty[s][e]);
      if (cu.first) ++qt;
      if (cu.w.next < 0) mma_commit_w(&c->q_empty[s]);
      ++g;
      return true;
    };
    auto issue_pv = [&](auto s_c) {
      constexpr int s = decltype(s_c)::value;
      Cursor& cu = s ? cu1 : cu0;
      uint32_t& g = s ? g1 : g0;
      uint32_t& gb = s ? gb1 : gb0;
      int& ot = s ? ot1 : ot0;
      const int e = g % R;
      const uint32_t tS = tmem + s * 256;
      const uint64_t vd = sdesc_sw128(smem_u32(smem + L::OFF_RING + (s * R + e) * L::TBYTES), L::BOX, 1024);
      mma_ts_k128_w(tS + 128, tS, vd, IDESC_O, cu.first ? 0u : 1u);
      mma_commit_w(&c->ring_empty[s][e]);
      if (cu.first) ++ot;
      if (cu.w.next < 0) mma_commit_w(&c->o_full[s]);
      ++g;
      ++gb;
      cursor_next(f, cu);
      return cu.done ? true : issue_s(s_c);
    };
    bool due0 = false, due1 = false;
    if (!cu0.done) ok = due0 = issue_s(IntC<0>{});
    if (ok && !cu1.done) ok = due1 = issue_s(IntC<1>{});
    int turn = 0;
    while (ok && (due0 || due1)) {
      const int s = (due0 && (turn == 0 || !due1)) ? 0 : 1;
      const Cursor& cu = s ? cu1 : cu0;
      const uint32_t g = s ? g1 : g0;
      const bool w = mbar_wait(&c->ring_full[s][g % R], (g / R) & 1, &c->abort, a.spin_ns) &&
                     (!cu.first || mbar_wait(&c->o_free[s], ((s ? ot1 : ot0) & 1) ^ 1, &c->abort, a.spin_ns)) &&
                     mbar_wait(&c->p_full[s], (s ? gb1 : gb0) & 1, &c->abort, a.spin_ns);
      if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
      tc_fence_after();
      if (s == 0) {
        ok = issue_pv(IntC<0>{});
        due0 = !cu0.done;
      } else {
        ok = issue_pv(IntC<1>{});
        due1 = !cu1.done;
      }
      turn = s ^ 1;
    }
    if (!ok && lane == 0) {
      c->abort = 1;
      report_status(a.status, CALIBATT_E_TIMEOUT);
    }
    __syncwarp();
    mma_commit_w(&c->drain);
    mbar_wait(&c->drain, 0, nullptr, a.spin_ns);
  } else if (warp == kWindow) {
    // ===================== the table's windows ================================
    // The windows of both slots' tiles near the diagonal, each filled as soon as
    // its buffer is free (polled, so that no slot waits for the other).
    if ((F & kBias) && a.table != nullptr) {
      Cursor cu[2];
      uint32_t n[2] = {0, 0};
      cursor_init(f, cu[0], 0);
      cursor_init(f, cu[1], 1);
      bool ok = true, corrupt = false;
      uint64_t since = globaltimer_ns();
      while (ok && !(cu[0].done && cu[1].done)) {
        bool moved = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (cu[s].done) continue;
          const Walk& w = cu[s].w;
          const int p0 = a.q_start[w.b] + (a.packed ? 0 : w.qb * TILE), p1 = p0 + (a.packed ? a.Nq : TILE) - 1;
          const uint32_t e = n[s] & 1;
          if (is_near(a, w.kb * TILE, p0, p1)) {
            if (!__all_sync(0xffffffffu, mbar_test_wait(&c->win_empty[s][e], ((n[s] >> 1) & 1) ^ 1))) continue;
            fill_window(a, a.packed ? w.hx * a.G : w.hx, a.packed ? a.G : 1, w.kb * TILE - p1,
                        reinterpret_cast<float*>(smem + L::OFF_WIN + s * L::WIN + e * (L::WIN / 2)), nullptr,
                        &c->win_info[s][e], &corrupt);
            mbar_arrive(&c->win_full[s][e]);
            ++n[s];
          }
          cursor_next(f, cu[s]);
          moved = true;
        }
        const uint64_t now = globaltimer_ns();
        if (moved) since = now;
        else __nanosleep(200);   // leave the issue slots to the softmax warps
        ok = moved || __all_sync(0xffffffffu, now - since <= kWindowPatience * a.spin_ns && *static_cast<volatile int*>(&c->abort) == 0);
      }
      if (!ok) {
        c->abort = 1;
        report_status(a.status, CALIBATT_E_TIMEOUT);
      }
      if (corrupt) report_status(a.status, CALIBATT_E_CORRUPT);
    }
  } else if (warp < 8) {
    // ===================== softmax warpgroups =================================
    regs_inc<kSoftmaxRegs>();
    const int slot = warp >> 2, w4 = warp & 3;
    const int row = w4 * 32 + lane;
    const uint32_t t_s = tmem + (static_cast<uint32_t>(w4 * 32) << 16) + slot * 256;
    const uint32_t t_o = t_s + 128;
    // Scores are in log2 units.
    ScoreTerms terms = score_terms(a);
    if (F & kBounded) terms.shift = -0.25f * terms.capA;
    uint32_t gb = 0, nw = 0;   // key tiles and windows consumed
    int tiles = 0;
    bool ok = true, corrupt = false;
    const int slots = 2 * gridDim.x;
    for (int round = 0; ok && round * slots < f.T; ++round) {
      const int t = tile_of(round, blockIdx.x + slot * gridDim.x, slots);
      if (t >= f.T) continue;
      Walk w;
      const bool any = walk_start(f, t, w);
      // this thread's row
      int h, i;
      bool live;
      if (a.packed) {
        const int r = FEW ? lane : row, g = r / a.Nq;
        i = r - g * a.Nq;
        live = g < a.G;
        h = w.hx * a.G + min(g, a.G - 1);
      } else {
        i = w.qb * TILE + row;
        live = i < a.Nq;
        h = w.hx;
      }
      const size_t orow = (static_cast<size_t>(w.b) * a.H + h) * a.Nq + i;   // of lse and the partial results
      __nv_bfloat16* op = reinterpret_cast<__nv_bfloat16*>(a.o.p) + w.b * a.o.sb + h * a.o.sh + i * a.o.sn;
      const size_t part = orow * a.parts + (FEW ? w.sp * 4 + w4 : w.sp);
      if (!any) {
        if (live) {
          if (a.parts > 1) {
            a.part_lse[part] = -INFINITY;
          } else {
            const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int x = 0; x < D / 8; ++x) reinterpret_cast<uint4*>(op)[x] = z;
            if (a.lse != nullptr) a.lse[orow] = -INFINITY;
          }
        }
        continue;
      }
      const int4 tr = score_tile(a, w.b, w.qb);
      const int2 vis = live ? score_row(a, w.b, i) : make_int2(0, 0);
      const int p0 = a.q_start[w.b] + (a.packed ? 0 : w.qb * TILE);   // positions of the tile's rows: p0 ... p1
      const int p1 = p0 + (a.packed ? a.Nq : TILE) - 1;
      const int p = a.q_start[w.b] + i;
      const float slope = a.slopes != nullptr ? a.slopes[h] * kLog2e : 0.f;
      const __nv_bfloat16* tab =
          reinterpret_cast<const __nv_bfloat16*>(a.table) + static_cast<size_t>(h) * a.n_buckets;
      float far_lo = 0.f, far_hi = 0.f;
      if ((F & kBias) && a.table != nullptr) {
        far_lo = __bfloat162float(tab[score_bucket(a, -a.R, &corrupt)]) * kLog2e;
        far_hi = __bfloat162float(tab[score_bucket(a, a.R, &corrupt)]) * kLog2e;
      }
      float m = F & kBounded ? 0.25f * terms.capA : -INFINITY, l = 0.f;
      float best = F & kBounded ? 0.f : -INFINITY;   // kBounded: largest probability; else largest score
      bool row_bad = false;
      bool scanned = false;      // the step before this one listed bad keys
      int seen0 = 0, seen1 = 0;  // and the row saw these columns of it
      auto see_bad = [&](uint32_t step) {
        if (!scanned) return;
        scanned = false;
#pragma unroll 1
        for (int q = 0; q < 4; ++q)
          row_bad |= (c->bad[slot][(step & 1) ^ 1][q] & bits_below(seen1 - 32 * q) & ~bits_below(seen0 - 32 * q)) != 0;
      };
      const bool work = __any_sync(0xffffffffu, live);   // few queries: warps without a row only keep the pace
      for (bool first = true;; first = false, ++gb) {
        const int k0 = w.kb * TILE;
        const bool edge = k0 < tr.z || k0 + TILE > tr.w;
        const bool near = (F & kBias) && is_near(a, k0, p0, p1);
        bool got = mbar_wait(&c->s_full[slot], gb & 1, &c->abort, a.spin_ns);
        if (near && got) got = mbar_wait(&c->win_full[slot][nw & 1], (nw >> 1) & 1, &c->abort, a.spin_ns);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        tc_fence_after();
        const int e0 = vis.x - k0, e1 = vis.y - k0;   // columns of the row's interval
        see_bad(gb);
        if (edge) {
          // A probability of 0 does not silence a NaN or infinity in V: rows of
          // the V tile that hold one are zeroed before the second product, and
          // the query rows that see such a key become NaN: the list of the
          // keys is read at the next step, when every thread has written.
          const uint32_t ge = 2 * gb + 1;
          ok = __all_sync(0xffffffffu,
                          mbar_wait(&c->ring_full[slot][ge % R], (ge / R) & 1, &c->abort, a.spin_ns));
          if (!ok) break;
          const bool bad = clean_row<D / 64>(smem + L::OFF_RING + (slot * R + ge % R) * L::TBYTES, row);
          const uint32_t bw = __ballot_sync(0xffffffffu, bad);
          if (lane == 0) c->bad[slot][gb & 1][w4] = bw;
          scanned = true;
          seen0 = e0;
          seen1 = e1;
        }
        if (work) {
        // Both passes go over the tile in chunks of 32 columns, in loops that
        // are not unrolled, and a tile that the mask cuts or where the distance
        // passes 0 has loops of its own: a warp is mostly alone on its
        // sub-partition, so instruction fetch bounds it, and instructions that
        // the ordinary tiles skip cost them (masks inside their loops: plain
        // scores 932 -> 1003 us, capped 1127 -> 1351 us at 24 heads of 8192
        // tokens, d = 128; all 128 columns unrolled: 1573 us capped).
        ScoreBias bias = {};
        if (F & kBias) {
          bias.wr = reinterpret_cast<const float*>(smem + L::OFF_WIN + slot * L::WIN + (nw & 1) * (L::WIN / 2)) +
                    (a.packed ? min((FEW ? lane : row) / a.Nq, a.G - 1) * 256 : 0) + (p1 - (live ? p : p1));
          bias.window = near && c->win_info[slot][nw & 1].cuts > 0;
          bias.flat = near ? (bias.window ? 0.f : bias.wr[0]) : k0 > p1 ? far_hi : far_lo;
          bias.side = k0 >= p1 ? 1 : k0 + TILE - 1 <= p0 ? -1 : 0;
          bias.slope = slope;
          bias.off0 = static_cast<float>(k0 - p);
        }
        float alpha = 1.f;
        bool rescale = false;
        uint64_t acc0 = f2pack(0.f, 0.f), acc1 = acc0;
        auto softmax = [&](auto cut_c) {
          constexpr bool CUT = decltype(cut_c)::value == kCutTile;
          // raw scores in both passes: no terms, one table value for the whole
          // tile, or a distance that is linear over it (per column slope x,
          // added in the scale's FFMA, and a constant per chunk)
          constexpr bool LINEAR = decltype(cut_c)::value == kLinearTile;
          constexpr bool RAW = (F & 3) == 0 || decltype(cut_c)::value == kFlatTile || LINEAR;
          // columns of a chunk: 64 where the code is short (plain 904 against 925
          // us), else 32 (capped 1137 against 1207 us, a table 1199 against 1342)
          constexpr int W = RAW && !LINEAR && !CUT && !FEW ? 64 : 32;
          const float scale = RAW ? terms.sc : 1.f, offset = RAW && (F & 3) ? bias.flat : 0.f;
          const float sl = bias.side > 0 ? -slope : slope;   // LINEAR: the distance's part is sl (off0 + x)
          const uint64_t sc2 = f2pack(terms.sc, terms.sc);
          uint64_t ramp[LINEAR ? 16 : 1];
          if (LINEAR) {
#pragma unroll
            for (int x = 0; x < 16; ++x) ramp[x] = f2pack(sl * (2 * x), sl * (2 * x + 1));
          }
          auto chunk_shift = [&](int ch) { return fmaf(sl, bias.off0 + static_cast<float>(32 * ch), bias.flat); };
          uint32_t r[W];
          uint32_t dead = 0;   // chunks that no row of the warp sees
          auto load = [&](int ch) {
#pragma unroll
            for (int x = 0; x < W; x += 32) tmem_ld32(t_s + ch * W + x, *reinterpret_cast<uint32_t(*)[32]>(&r[x]));
            tmem_ld_wait();
            reg_fence(r);
          };
          // log2 units, -inf where masked; false: no row of the warp sees the chunk
          auto transform = [&](int ch) {
            const uint32_t bits = CUT ? bits_below(e1 - 32 * ch) & ~bits_below(e0 - 32 * ch) : 0xffffffffu;
            if (CUT && !__any_sync(0xffffffffu, bits != 0)) return false;
            if (!RAW) {
              ScoreBias at = bias;
              at.off0 += static_cast<float>(W * ch);
              at.wr += W * ch;
              float none[W];
              score_columns<F & 3, 1, false, CUT>(a, terms, r, none, at, live);
            }
            if constexpr (CUT) keep_bits(r, bits, -INFINITY);
            return true;
          };
          if (!(F & kBounded)) {
            // First pass: (transformed) scores and the tile's maximum.
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll 1
            for (int ch = FEW ? w4 : 0; ch < (FEW ? w4 + 1 : TILE / W); ++ch) {
              load(ch);
              if (!transform(ch)) {
                dead |= 1u << ch;
                continue;
              }
              if constexpr (LINEAR) {   // (r keeps the raw scores for the second pass)
                float c0 = -INFINITY, c1 = -INFINITY;
#pragma unroll
                for (int x = 0; x < W; x += 4) {
                  float y0, y1, y2, y3;
                  f2unpack(ffma2(pair_of(r, x), sc2, ramp[x / 2]), y0, y1);
                  f2unpack(ffma2(pair_of(r, x + 2), sc2, ramp[x / 2 + 1]), y2, y3);
                  c0 = fmax3(c0, y0, y1);
                  c1 = fmax3(c1, y2, y3);
                }
                mx0 = fmaxf(mx0, fmaxf(c0, c1) + chunk_shift(ch));
              } else {
#pragma unroll
                for (int x = 0; x < W; x += 4) {
                  mx0 = fmax3(mx0, u2f(r[x]), u2f(r[x + 1]));
                  mx1 = fmax3(mx1, u2f(r[x + 2]), u2f(r[x + 3]));
                }
              }
              if ((!RAW || CUT) && !FEW) {   // one chunk stays in registers
#pragma unroll
                for (int x = 0; x < W; x += 32) tmem_st32(t_s + ch * W + x, *reinterpret_cast<uint32_t(*)[32]>(&r[x]));
              }
            }
            const float m_cand = LINEAR ? mx0 : fmaf(fmaxf(mx0, mx1), scale, offset);
            best = fmaxf(best, m_cand);
            // The reference: the first tile's maximum, raised (and O and l
            // rescaled) only by more than the threshold.  While a row has seen
            // nothing it is -inf and the exponent's shift 0.
            if (first) {
              m = m_cand;
            } else {
              const bool raise = m_cand > m + kRescaleThreshold;
              rescale = __any_sync(0xffffffffu, raise);
              if (raise) {
                alpha = ex2_approx(m - m_cand);
                m = m_cand;
              }
            }
            if ((!RAW || CUT) && !FEW) tmem_st_wait();
          }
          // Second pass: probabilities, stored as bf16 pairs over the scores
          // already read, and their fp32 sum.
          const float neg = (m == -INFINITY ? 0.f : -m) + (LINEAR ? 0.f : offset);
          const uint64_t negm = f2pack(neg, neg), scale2 = f2pack(scale, scale);
          float pm0 = 0.f, pm1 = 0.f;
#pragma unroll 1
          for (int ch = FEW ? w4 : 0; ch < (FEW ? w4 + 1 : TILE / W); ++ch) {
            uint32_t pk[W / 2];
            bool some = true;
            if (!CUT || !((dead >> ch) & 1u)) {
              if ((F & kBounded) || !FEW) load(ch);
              if (F & kBounded) some = transform(ch);
            } else {
              some = false;
            }
            if constexpr (CUT) {
              if (!some) {
#pragma unroll
                for (int x = 0; x < 16; ++x) pk[x] = 0;
                tmem_st16(t_s + ch * 16, pk);
                continue;
              }
            }
            const float shift = LINEAR ? neg + chunk_shift(ch) : 0.f;
            const uint64_t shift2 = f2pack(shift, shift);
#pragma unroll
            for (int x = 0; x < W / 2; ++x) {
              uint64_t y = pair_of(r, 2 * x);
              if (LINEAR) y = fadd2(ffma2(y, sc2, ramp[LINEAR ? x : 0]), shift2);
              else if (!(F & kBounded)) y = ffma2(y, scale2, negm);
              float xl, xh;
              f2unpack(y, xl, xh);
              xl = ex2_approx(xl);
              xh = ex2_approx(xh);
              const uint64_t pv = f2pack(xl, xh);
              if (x & 1) acc1 = fadd2(acc1, pv); else acc0 = fadd2(acc0, pv);
              if (F & kBounded) {
                if (x & 1) pm1 = fmax3(pm1, xl, xh); else pm0 = fmax3(pm0, xl, xh);
              }
              pk[x] = pack_bf16x2(xl, xh);
            }
#pragma unroll
            for (int x = 0; x < W / 2; x += 16)
              tmem_st16(t_s + ch * (W / 2) + x, *reinterpret_cast<uint32_t(*)[16]>(&pk[x]));
          }
          if (F & kBounded) best = fmaxf(best, fmaxf(pm0, pm1));
        };
        if (edge || ((F & kBias) && a.slopes != nullptr && bias.side == 0)) softmax(IntC<kCutTile>{});
        else if (!FEW && (F & 3) == kBias && !bias.window && a.slopes == nullptr) softmax(IntC<kFlatTile>{});
        else if (!FEW && (F & 3) == kBias && !bias.window) softmax(IntC<kLinearTile>{});
        else softmax(IntC<kFullTile>{});
        if (FEW) {   // the other warps' columns are 0 in these lanes
          uint32_t pk[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) pk[x] = 0;
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch)
            if (ch != w4) tmem_st16(t_s + ch * 16, pk);
        }
        if (rescale) {
#pragma unroll 1
          for (int q4 = 0; q4 < D / 32; ++q4) {
            uint32_t ro[32];
            tmem_ld32(t_o + q4 * 32, ro);
            tmem_ld_wait();
            reg_fence(ro);
#pragma unroll
            for (int x = 0; x < 32; ++x) ro[x] = f2u(u2f(ro[x]) * alpha);
            tmem_st32(t_o + q4 * 32, ro);
          }
        }
        float a0, a1, b0, b1;
        f2unpack(acc0, a0, a1);
        f2unpack(acc1, b0, b1);
        l = l * alpha + ((a0 + a1) + (b0 + b1));
        tmem_st_wait();
        }
        if (near) {
          mbar_arrive(&c->win_empty[slot][nw & 1]);
          ++nw;
        }
        tc_fence_before();
        mbar_arrive(&c->p_full[slot]);
        if (w.next < 0) { ++gb; break; }
        key_next(a, w.hx, w.qb, w);
      }
      if (!ok) break;
      // ---- epilogue: O / l, LSE.  As in the block-sparse forward, the
      // rounding error of the row's largest probability moves into the
      // normaliser, so that a row with one dominant key returns its value.
      const float p_best = F & kBounded ? best : ex2_approx(best - m);
      const float corr = __uint_as_float(pack_bf16x2(p_best, 0.f) << 16) - p_best;
      ok = __all_sync(0xffffffffu, mbar_wait(&c->o_full[slot], tiles & 1, &c->abort, a.spin_ns));
      if (!ok) break;
      ++tiles;
      tc_fence_after();
      see_bad(gb);
      if ((F & kBias) && slope != 0.f && l != 0.f && score_far(vis, p)) {
        l = NAN;
        report_status(a.status, CALIBATT_E_UNSUPPORTED);
      }
      const float inv_l = row_bad ? NAN : l == 0.f ? 0.f : 1.f / (l + corr);
      const float row_lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      if (a.parts > 1) {
        float* po = a.part_o + part * D;
#pragma unroll 1
        for (int q4 = 0; q4 < D / 32; ++q4) {
          uint32_t ro[32];
          tmem_ld32(t_o + q4 * 32, ro);
          tmem_ld_wait();
          reg_fence(ro);
          if (live) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              reinterpret_cast<float4*>(po + q4 * 32)[x] =
                  make_float4(u2f(ro[4 * x]) * inv_l, u2f(ro[4 * x + 1]) * inv_l, u2f(ro[4 * x + 2]) * inv_l,
                              u2f(ro[4 * x + 3]) * inv_l);
          }
        }
        if (live) a.part_lse[part] = row_lse;
      } else {
#pragma unroll 1
        for (int q4 = 0; q4 < D / 32; ++q4) {
          uint32_t ro[32];
          tmem_ld32(t_o + q4 * 32, ro);
          tmem_ld_wait();
          reg_fence(ro);
          if (live) {
            uint4* dst = reinterpret_cast<uint4*>(op + q4 * 32);
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
              dst[v4] = make_uint4(pack_bf16x2(u2f(ro[8 * v4 + 0]) * inv_l, u2f(ro[8 * v4 + 1]) * inv_l),
                                   pack_bf16x2(u2f(ro[8 * v4 + 2]) * inv_l, u2f(ro[8 * v4 + 3]) * inv_l),
                                   pack_bf16x2(u2f(ro[8 * v4 + 4]) * inv_l, u2f(ro[8 * v4 + 5]) * inv_l),
                                   pack_bf16x2(u2f(ro[8 * v4 + 6]) * inv_l, u2f(ro[8 * v4 + 7]) * inv_l));
          }
        }
        if (live && a.lse != nullptr) a.lse[orow] = row_lse;
      }
      tc_fence_before();
      mbar_arrive(&c->o_free[slot]);
    }
    if (!ok) {
      c->abort = 1;
      report_status(a.status, CALIBATT_E_TIMEOUT);
    }
    if (corrupt) report_status(a.status, CALIBATT_E_CORRUPT);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, kTmemCols);
}

template <int D, int F>
int launch(const ScoreArgs& a, int sms, cudaStream_t s) {
  FwdArgs f;
  f.a = a;
  f.Hx = a.packed ? a.Hkv : a.H;
  f.nq = a.packed ? 1 : a.nqb;
  // K and V of a group of heads: up to 64 MB of the 126 MB L2
  const long long head_bytes = 4ll * a.Nk * D;
  const long long per = a.packed ? 1 : a.G;   // grid heads of one key head
  f.hgroup = static_cast<int>(std::min<long long>(std::max<long long>(1, (64ll << 20) / head_bytes) * per,
                                                  static_cast<long long>(a.B) * f.Hx));
  const long long T = static_cast<long long>(a.B) * f.Hx * f.nq * a.splits;
  if (T >= (1ll << 31)) return set_error(CALIBATT_E_UNSUPPORTED, "too many query tiles");
  f.T = static_cast<int>(T);
  CUtensorMap tq, tk, tv;
  int rc;
  if ((rc = make_tmap4_bf16(&tq, a.q, a.B, a.H, a.Nq, D, a.packed ? a.Nq : TILE, a.packed ? a.G : 1))) return rc;
  if ((rc = make_tmap4_bf16(&tk, a.k, a.B, a.Hkv, a.Nk, D, TILE, 1))) return rc;
  if ((rc = make_tmap4_bf16(&tv, a.v, a.B, a.Hkv, a.Nk, D, TILE, 1))) return rc;
  auto kern = k_score_fwd<D, F>;
  static std::atomic<bool> done[kMaxDevices];
  if ((rc = configure_kernel(reinterpret_cast<const void*>(kern), done, Layout<D>::SMEM, kLaunchRegs, "k_score_fwd")))
    return rc;
  const int grid = static_cast<int>(std::min<long long>(sms, T));
  kern<<<grid, kThreads, Layout<D>::SMEM, s>>>(tq, tk, tv, f);
  count_launch();
  if ((rc = check_launch("k_score_fwd"))) return rc;
  return a.parts > 1 ? launch_score_join(a, D, CALIBATT_BF16, s) : CALIBATT_OK;
}

}  // namespace

// Whether the G query heads of a key head share a tile: their rows fit, no
// mask (it may differ between the heads) and the table's windows fit.
bool score_packs(int G, int Nq, bool mask, bool table) {
  return static_cast<long long>(G) * Nq <= TILE && !mask && (!table || G <= kMaxPackedTable);
}

// Splits of the key axis, at least two key tiles each, for 296 slots (two on
// each of 148 SMs) of one unit (query tile and split) at a time: as many as
// still fit one round of the slots.  A unit costs about as much as a key tile
// (its last product, its partial results), so finer splits, which would even
// out sequences of different lengths, lose more than they win: 4 tokens, 24
// heads, 75 600 keys 150 us in one round, 165 in two, 180 in four; 32
// sequences of 2500 ... 8191 keys 162, 174, 160; 8 of 4800 ... 16 000 76, 70, 82.
// Only equal splits were compared, not ones in proportion to the lengths, and
// 149 to 296 units get one split whatever slots that leaves idle.
int score_splits(int B, int heads, int nq_tiles, int nkb) {
  const long long tiles = static_cast<long long>(B) * heads * nq_tiles;
  return static_cast<int>(std::max<long long>(1, std::min<long long>(296 / tiles, nkb / 2)));
}

int launch_score_fwd_tc(const ScoreArgs& a, int d, cudaStream_t s) {
  int sms = 0;
  if (int rc = device_sms(&sms)) return rc;
  const bool bias = a.slopes != nullptr || a.table != nullptr;
  const int form = (a.cap > 0.f ? kCap : 0) | (bias ? kBias : 0) |
                   (a.cap > 0.f && !bias && a.cap * kLog2e <= kBoundedCap ? kBounded : 0);
  auto go = [&](auto form_c) {
    constexpr int F = decltype(form_c)::value;
    if (a.few) return d == 128 ? launch<128, F | kFew>(a, sms, s) : launch<64, F | kFew>(a, sms, s);
    return d == 128 ? launch<128, F>(a, sms, s) : launch<64, F>(a, sms, s);
  };
  switch (form) {
    case 0: return go(IntC<0>{});
    case kCap: return go(IntC<kCap>{});
    case kCap | kBounded: return go(IntC<kCap | kBounded>{});
    case kBias: return go(IntC<kBias>{});
    default: return go(IntC<kCap | kBias>{});
  }
}

}  // namespace calibatt
