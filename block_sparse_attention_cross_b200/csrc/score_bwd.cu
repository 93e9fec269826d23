// score_bwd.cu -- score-modified attention backward on the tensor cores (bf16).
//
// Two kernels, each recomputing the scores, so that every gradient is summed
// by one CTA in a fixed order, without atomics and without an fp32 buffer for
// dQ:
//   k_score_dq   one 128-query tile (TMEM lanes are queries), two sweeps over
//                the key tiles that it sees.  The first forms S = Q K^T and
//                dP = dO V^T and sums D = sum_j P dP of every row in fp32.  (D
//                could be had as dO . O, but O is rounded to bf16, and that
//                error, common to a whole row of dZ = P (dP - D), would double
//                the error of dQ and of the table's gradient.)  The second
//                forms S and dP again, then dQ += dS K and the sums of dZ by
//                bucket.
//   k_score_dkv  one 128-key tile of a key head (TMEM lanes are keys), after
//                k_score_dq: for every query tile that sees it (all G query
//                heads) S^T = K Q^T and dP^T = V dO^T, then dV += P^T dO and
//                dK += dS^T Q.
// Both products that read a probability or dS take it as the A operand from
// TMEM, where the softmax warps leave it as bf16 in place of the scores; the
// other operand is the input tile as it lies in shared memory (128-byte
// swizzle, read K-major by the first products and MN-major by the second).
// Nine 128 x 128 x d products a tile pair (2 + 3 + 4) instead of the five of
// one kernel with atomics on dQ and D from the rounded O.
//
// A CTA (one per SM): warps 0-3 and 4-7 softmax, the lanes' columns split in
// halves of 64 between the warpgroups; warp 8 TMA producer; warp 9 MMA issuer;
// warp 10 fills the table's windows one tile ahead.  With P = exp(z - LSE)
// known from the forward's LSE no running maximum is needed.
//
// What bounds it: the arithmetic between the products.  Two softmax warps a
// sub-partition work at the same time, so a pair costs 1024 MUFU cycles a
// sweep at least, against 1024 (first sweep), 1536 and 2048 (dK/dV) tensor
// cycles at d = 128.  24 heads of 8192 tokens, d = 128: dQ 1.71 ms, dK/dV 1.30
// ms, together 0.5 PFLOP/s of the products that the gradients need and 0.9 of
// those that run; with a cap 2.18 and 1.68.  The tensor pipe is 38% busy
// (capped), the issue slots 43%; the rest is the latency of dependent
// instructions (1.8 stalled warps an issue).
#include <algorithm>
#include <atomic>

#include "score_common.cuh"

namespace calibatt {
namespace {

constexpr int TILE = 128;
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;
constexpr uint32_t kSoftmaxRegs = 208;
constexpr uint32_t kControlRegs = 88;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs == kThreads * kLaunchRegs, "register split");
constexpr int kProducer = 8, kMma = 9, kWindow = 10;
// Beside the ScoreForm bits: the dQ kernel sums the table's gradient.
constexpr int kGrad = 4;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kCtrlBytes = 2048;              // barriers and small state, checked against its size below
constexpr uint32_t kRowBytes = 512 + 512 + 1024;   // -LSE, -D and interval of a tile's rows

template <int D>
__device__ __forceinline__ void mma_scores(uint32_t t, uint32_t sA, uint32_t sB, uint32_t idesc) {
  constexpr uint32_t BOX = TILE * 64 * 2;
  if (D == 128) {
    mma_ss_k128_w(t, sdesc_sw128(sA, 16, 1024), sdesc_sw128(sB, 16, 1024), idesc, BOX >> 4);
  } else {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      mma_bf16_ss_w(t, sdesc_sw128(sA + kk * 32, 16, 1024), sdesc_sw128(sB + kk * 32, 16, 1024), idesc, kk > 0 ? 1u : 0u);
  }
}

// D[t] (+)= A B with A the bf16 pairs at columns [ta, ta + 32) and [ta + 64, ta + 96)
// (the two halves of 64 columns) and B the MN-major tile at sB.
__device__ __forceinline__ void mma_from_tmem(uint32_t t, uint32_t ta, uint32_t sB, uint32_t idesc, uint32_t accumulate) {
  const uint64_t bd = sdesc_sw128(sB, TILE * 64 * 2, 1024);
  mma_ts_k64_w(t, ta, bd, idesc, accumulate);
  mma_ts_k64_w(t, ta + 64, bd + 512, idesc, 1u);
}

// ===========================================================================
// dK, dV
// ===========================================================================

template <int D>
struct DkvLayout {
  static constexpr uint32_t BOX = TILE * 64 * 2;
  static constexpr uint32_t TB = TILE * D * 2;
  static constexpr int RING = D == 128 ? 2 : 4;   // stages of a query tile's Q, dO and row terms
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = TB;
  static constexpr uint32_t OFF_Q = 2 * TB;
  static constexpr uint32_t OFF_DO = OFF_Q + RING * TB;
  static constexpr uint32_t OFF_ROWS = OFF_DO + RING * TB;
  static constexpr uint32_t OFF_WIN = OFF_ROWS + RING * kRowBytes;   // float [2][256]
  static constexpr uint32_t OFF_CTRL = OFF_WIN + 2048;
  static constexpr uint32_t SMEM = OFF_CTRL + kCtrlBytes + 1024;   // + alignment slack
  static_assert(SMEM <= 232448, "shared memory");
};

template <int RING>
struct DkvCtrl {
  uint64_t kv_full, ring_full[RING], ring_empty[RING];
  uint64_t s_full, p_full, dp_full, ds_full, o_full, drain;
  uint64_t win_full[2], win_empty[2];
  WindowInfo win_info[2];
  uint32_t tmem_base;
  int abort;
};

// Walk over the (query head, query tile) pairs that see key tile kb, of the
// pairs g nqb + qb in [u0, u1).
struct QueryWalk {
  int g, qb;
  uint32_t word;
  int wbase;
};
struct QueryRange {
  int b, hk, kb, u0, u1;
};

__device__ __forceinline__ uint32_t query_word(const ScoreArgs& a, const QueryRange& q, int g, int wbase) {
  const int qb = wbase + lane_id(), u = g * a.nqb + qb;
  bool on = false;
  if (qb < a.nqb && u >= q.u0 && u < q.u1) {
    const int4 r = score_tile(a, q.b, qb);
    on = r.x < r.y && r.x < (q.kb + 1) * TILE && r.y > q.kb * TILE && score_kept(a, q.hk * a.G + g, qb, q.kb);
  }
  return __ballot_sync(0xffffffffu, on);
}

// Next pair; false at the end.
__device__ __forceinline__ bool query_next(const ScoreArgs& a, const QueryRange& q, QueryWalk& w) {
  while (w.word == 0) {
    w.wbase += 32;
    if (w.wbase >= a.nqb) {
      w.wbase = 0;
      ++w.g;
    }
    if (w.g * a.nqb + w.wbase >= q.u1) return false;
    w.word = query_word(a, q, w.g, w.wbase);
  }
  w.qb = w.wbase + __ffs(w.word) - 1;
  w.word &= w.word - 1;
  return true;
}

__device__ __forceinline__ bool query_start(const ScoreArgs& a, const QueryRange& q, QueryWalk& w) {
  w.g = q.u0 / a.nqb;
  w.wbase = (q.u0 - w.g * a.nqb) / 32 * 32 - 32;
  w.word = 0;
  return query_next(a, q, w);
}

// Rounds 64 fp32 values of a lane to bf16 pairs in TMEM columns [t, t + 32).
__device__ __forceinline__ void store_half(uint32_t t, const float (&x)[64]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(x[c * 32 + 2 * i], x[c * 32 + 2 * i + 1]);
    tmem_st16(t + c * 16, pk);
  }
}

// Writes D TMEM columns of this lane, times `mul`, as one bf16 row.
template <int COLS>
__device__ __forceinline__ void store_row(uint32_t t, __nv_bfloat16* dst, float mul, bool live) {
#pragma unroll
  for (int q = 0; q < COLS / 32; ++q) {
    uint32_t r[32];
    tmem_ld32(t + q * 32, r);
    tmem_ld_wait();
    reg_fence(r);
    if (live) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        reinterpret_cast<uint4*>(dst + q * 32)[v] =
            make_uint4(pack_bf16x2(u2f(r[8 * v + 0]) * mul, u2f(r[8 * v + 1]) * mul),
                       pack_bf16x2(u2f(r[8 * v + 2]) * mul, u2f(r[8 * v + 3]) * mul),
                       pack_bf16x2(u2f(r[8 * v + 4]) * mul, u2f(r[8 * v + 5]) * mul),
                       pack_bf16x2(u2f(r[8 * v + 6]) * mul, u2f(r[8 * v + 7]) * mul));
    }
  }
}

template <int COLS>
__device__ __forceinline__ void zero_row(__nv_bfloat16* dst, bool live) {
  if (!live) return;
#pragma unroll
  for (int x = 0; x < COLS / 8; ++x) reinterpret_cast<uint4*>(dst)[x] = make_uint4(0, 0, 0, 0);
}

// TMEM: S^T (P^T in place) [0, 128), dP^T (dS^T in place) [128, 256), dV at
// 256, dK at 384.  Issue order: S(0), dP(0); then per pair t, once P(t) is
// stored, dV(t) and S(t + 1), and once dS(t) is stored, dK(t) and dP(t + 1):
// the exponentials of pair t + 1 run while dK(t) and dP(t + 1) do, the
// products' second half of the softmax (dS) while dV and S of the next do.
template <int D, int F>
__global__ void __launch_bounds__(kThreads, 1)
    k_score_dkv(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                const __grid_constant__ ScoreArgs a) {
  using L = DkvLayout<D>;
  constexpr int R = L::RING;
  static_assert(sizeof(DkvCtrl<R>) <= kCtrlBytes, "control block");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DkvCtrl<R>* c = reinterpret_cast<DkvCtrl<R>*>(smem + L::OFF_CTRL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // key tiles of a head side by side: they read the same Q and dO; under a
  // causal rule the first ones, which most queries see, start first
  const int part = blockIdx.x % a.kv_parts, tile = blockIdx.x / a.kv_parts;
  const int kb = tile % a.nkb, bh = tile / a.nkb;
  const int b = bh / a.Hkv, hk = bh % a.Hkv;
  const int k0 = kb * TILE;
  const long long units = static_cast<long long>(a.G) * a.nqb;
  const QueryRange range{b, hk, kb, static_cast<int>(units * part / a.kv_parts),
                         static_cast<int>(units * (part + 1) / a.kv_parts)};

  if (threadIdx.x == 0) {
    mbar_init(&c->kv_full, 1);
    for (int e = 0; e < R; ++e) {
      mbar_init(&c->ring_full[e], 1);
      mbar_init(&c->ring_empty[e], 1);
    }
    mbar_init(&c->s_full, 1);
    mbar_init(&c->p_full, 256);
    mbar_init(&c->dp_full, 1);
    mbar_init(&c->ds_full, 256);
    mbar_init(&c->o_full, 1);
    mbar_init(&c->drain, 1);
    for (int e = 0; e < 2; ++e) {
      mbar_init(&c->win_full[e], 32);
      mbar_init(&c->win_empty[e], 256);
    }
    c->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmDO);
  }
  if (warp == kMma) {
    tmem_alloc(&c->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem_base;
  const uint32_t tS = tmem, tP = tmem + 128, tV = tmem + 256, tK = tmem + 384;

  if (warp >= 8) regs_dec<kControlRegs>();
  if (warp == kProducer) {
    QueryWalk w;
    bool more = query_start(a, range, w), ok = true;
    const bool any = more;
    uint32_t t = 0;
    const uint64_t pol = l2_policy_evict_last(), pol_kv = l2_policy_evict_first();
    if (any) {
      mbar_arrive_expect_tx_w(&c->kv_full, 2 * L::TB);
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        tma_load_4d_w(smem + L::OFF_K + x * L::BOX, &tmK, x * 64, k0, hk, b, &c->kv_full, pol_kv);
        tma_load_4d_w(smem + L::OFF_V + x * L::BOX, &tmV, x * 64, k0, hk, b, &c->kv_full, pol_kv);
      }
    }
    while (more) {
      const int e = t % R;
      ok = __all_sync(0xffffffffu, mbar_wait(&c->ring_empty[e], ((t / R) & 1) ^ 1, &c->abort, a.spin_ns));
      if (!ok) break;
      mbar_arrive_expect_tx_w(&c->ring_full[e], 2 * L::TB + kRowBytes);
      const int h = hk * a.G + w.g;
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        tma_load_4d_w(smem + L::OFF_Q + e * L::TB + x * L::BOX, &tmQ, x * 64, w.qb * TILE, h, b, &c->ring_full[e], pol);
        tma_load_4d_w(smem + L::OFF_DO + e * L::TB + x * L::BOX, &tmDO, x * 64, w.qb * TILE, h, b, &c->ring_full[e], pol);
      }
      uint8_t* rows = smem + L::OFF_ROWS + e * kRowBytes;
      const size_t r0 = ((static_cast<size_t>(b) * a.H + h) * a.nqb + w.qb) * TILE;
      bulk_load_w(rows, a.row_lse + r0, 512, &c->ring_full[e]);
      bulk_load_w(rows + 512, a.row_d + r0, 512, &c->ring_full[e]);
      bulk_load_w(rows + 1024, a.row_span + (static_cast<size_t>(b) * a.nqb + w.qb) * TILE, 1024, &c->ring_full[e]);
      ++t;
      more = query_next(a, range, w);
    }
    if (lane == 0) {
      if (!ok) {
        c->abort = 1;
        report_status(a.status, CALIBATT_E_TIMEOUT);
      }
      // Drain: every copy issued must have landed before the CTA may exit.
      if (any) mbar_wait(&c->kv_full, 0, nullptr, a.spin_ns);
      for (int e = 0; e < R; ++e) {
        const uint32_t fills = (t > static_cast<uint32_t>(e)) ? (t - 1 - e) / R + 1 : 0;
        if (fills > 0) mbar_wait(&c->ring_full[e], (fills - 1) & 1, nullptr, a.spin_ns);
      }
    }
  } else if (warp == kMma) {
    uint32_t n = 0;
    for (int g = range.u0 / a.nqb; g * a.nqb < range.u1; ++g)
      for (int w = 0; w < a.nqb; w += 32) n += __popc(query_word(a, range, g, w));
    constexpr uint32_t IDESC_S = idesc_bf16_f32(TILE, TILE, false);
    constexpr uint32_t IDESC_O = idesc_bf16_f32(TILE, D, true);
    const uint32_t sK = smem_u32(smem + L::OFF_K), sV = smem_u32(smem + L::OFF_V);
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, &c->abort, a.spin_ns));
      tc_fence_after();
      return ok;
    };
    auto sQ = [&](uint32_t t) { return smem_u32(smem + L::OFF_Q + (t % R) * L::TB); };
    auto sO = [&](uint32_t t) { return smem_u32(smem + L::OFF_DO + (t % R) * L::TB); };
    if (n > 0 && wait(&c->kv_full, 0) && wait(&c->ring_full[0], 0)) {
      mma_scores<D>(tS, sK, sQ(0), IDESC_S);
      mma_commit_w(&c->s_full);
      mma_scores<D>(tP, sV, sO(0), IDESC_S);
      mma_commit_w(&c->dp_full);
      for (uint32_t t = 0; t < n; ++t) {
        if (!wait(&c->p_full, t & 1)) break;
        mma_from_tmem(tV, tS, sO(t), IDESC_O, t > 0 ? 1u : 0u);
        if (t + 1 < n) {
          if (!wait(&c->ring_full[(t + 1) % R], ((t + 1) / R) & 1)) break;
          mma_scores<D>(tS, sK, sQ(t + 1), IDESC_S);
          mma_commit_w(&c->s_full);
        }
        if (!wait(&c->ds_full, t & 1)) break;
        mma_from_tmem(tK, tP, sQ(t), IDESC_O, t > 0 ? 1u : 0u);
        mma_commit_w(&c->ring_empty[t % R]);
        if (t + 1 < n) {
          mma_scores<D>(tP, sV, sO(t + 1), IDESC_S);
          mma_commit_w(&c->dp_full);
        } else {
          mma_commit_w(&c->o_full);
        }
      }
    }
    if (!ok && lane == 0) {
      c->abort = 1;
      report_status(a.status, CALIBATT_E_TIMEOUT);
    }
    __syncwarp();
    mma_commit_w(&c->drain);
    mbar_wait(&c->drain, 0, nullptr, a.spin_ns);
  } else if (warp == kWindow) {
    if ((F & kBias) && a.table != nullptr) {
      QueryWalk w;
      bool bad = false, ok = true;
      uint32_t t = 0;
      for (bool more = query_start(a, range, w); more; more = query_next(a, range, w)) {
        const int p0 = a.q_start[b] + w.qb * TILE;
        if (!is_near(a, k0, p0, p0 + TILE - 1)) continue;
        const int e = t & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&c->win_empty[e], ((t >> 1) & 1) ^ 1, &c->abort,
                                                  kWindowPatience * a.spin_ns));
        if (!ok) break;
        ++t;
        fill_window(a, hk * a.G + w.g, 1, k0 - p0 - (TILE - 1), reinterpret_cast<float*>(smem + L::OFF_WIN) + e * 256, nullptr,
                      &c->win_info[e], &bad);
        mbar_arrive(&c->win_full[e]);
      }
      if (!ok) {
        c->abort = 1;
        report_status(a.status, CALIBATT_E_TIMEOUT);
      }
      if (bad) report_status(a.status, CALIBATT_E_CORRUPT);
    }
  } else if (warp < 8) {
    regs_inc<kSoftmaxRegs>();
    const int half = warp >> 2, w4 = warp & 3, row = w4 * 32 + lane;   // row: key of the tile
    const uint32_t lanes = static_cast<uint32_t>(w4 * 32) << 16;
    const uint32_t tSh = tS + lanes + half * 64, tPh = tP + lanes + half * 64;
    const ScoreTerms terms = score_terms(a);
    constexpr bool xform = F != 0;
    const uint64_t c2x2 = f2pack(xform ? 1.f : terms.sc, xform ? 1.f : terms.sc);
    const int j = k0 + row;
    bool ok = true;
    uint32_t t = 0, nw = 0;   // pairs and windows consumed
    QueryWalk w;
    for (bool more = query_start(a, range, w); more; more = query_next(a, range, w), ++t) {
      const int e = t % R, h = hk * a.G + w.g;
      const int p0 = a.q_start[b] + w.qb * TILE;
      const int4 tr = score_tile(a, b, w.qb);
      const bool edge = k0 < tr.z || k0 + TILE > tr.w;
      const bool near = (F & kBias) && is_near(a, k0, p0, p0 + TILE - 1);
      const uint8_t* rows = smem + L::OFF_ROWS + e * kRowBytes;
      const float4* nlse = reinterpret_cast<const float4*>(rows) + half * 16;
      const float4* nd = reinterpret_cast<const float4*>(rows + 512) + half * 16;
      float slope = 0.f, far = 0.f;
      if ((F & kBias) && a.slopes != nullptr) slope = a.slopes[h] * kLog2e;
      if ((F & kBias) && a.table != nullptr && !near) {
        bool bad = false;
        const int n = score_bucket(a, k0 > p0 ? a.R : -a.R, &bad);
        far = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.table)[static_cast<size_t>(h) * a.n_buckets + n]) * kLog2e;
        if (bad) report_status(a.status, CALIBATT_E_CORRUPT);
      }
      // The row terms of the first 32 queries are read before the wait for the
      // scores, those of the next 32 a chunk ahead: the tensor core's operand
      // reads keep shared memory busy, and a read between two exponentials
      // stalls them (1950 against 1400 cycles a tile pair).
      bool got = mbar_wait(&c->ring_full[e], (t / R) & 1, &c->abort, a.spin_ns);
      float4 nl[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) nl[x] = nlse[x];
      got = got && mbar_wait(&c->s_full, t & 1, &c->abort, a.spin_ns);
      if (got && near) got = mbar_wait(&c->win_full[nw & 1], (nw >> 1) & 1, &c->abort, a.spin_ns);
      if (got && edge) got = mbar_wait(&c->dp_full, t & 1, &c->abort, a.spin_ns);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      tc_fence_after();
      // column x: query 64 half + x, offset j - p falls with x
      ScoreBias bias = {};
      if (F & kBias) {
        bias.wr = reinterpret_cast<const float*>(smem + L::OFF_WIN) + (nw & 1) * 256 + row + TILE - 1 - half * 64;
        bias.window = near && c->win_info[nw & 1].cuts > 0;
        bias.flat = near ? (bias.window ? 0.f : bias.wr[0]) : far;
        bias.side = k0 >= p0 + TILE - 1 ? 1 : k0 + TILE - 1 <= p0 ? -1 : 0;
        bias.slope = slope;
        bias.off0 = static_cast<float>(j - p0 - half * 64);
      }
      // A tile that the mask cuts, or where the distance passes 0, has code of
      // its own: the ordinary tiles are bound by instruction fetch as much as
      // by arithmetic.
      auto pair = [&](auto cut_c) {
        constexpr bool CUT = decltype(cut_c)::value != 0;
        uint32_t seen0 = 0xffffffffu, seen1 = 0xffffffffu;
        if (CUT) {
          const int2* span = reinterpret_cast<const int2*>(rows + 1024) + half * 64;
          seen0 = seen1 = 0;
#pragma unroll 4
          for (int x = 0; x < 32; ++x) {
            const int2 u = span[x], v = span[x + 32];
            if (j >= u.x && j < u.y) seen0 |= 1u << x;
            if (j >= v.x && j < v.y) seen1 |= 1u << x;
          }
          // Queries with a NaN or an infinity would leave it in every key's
          // sums through a probability of 0: their rows of Q (read by S, which
          // is complete) and of dO (read by dP, awaited above) are zeroed
          // before the second products.  Keys that are seen get it from P or
          // dS, which are NaN then.
          if (edge) clean_row<D / 64>(smem + (half == 0 ? L::OFF_Q : L::OFF_DO) + e * L::TB, row);
        }
        uint32_t r[64];
        tmem_ld32(tSh, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
        tmem_ld32(tSh + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
        tmem_ld_wait();
        reg_fence(r);
        float pf[64];   // first the cap's factor, then P times it
        // P, rounded to bf16 for dV, and P times the cap's factor kept for dS.
        // Half of the columns at a time: the two warps of a sub-partition then
        // alternate between the FMA and the MUFU pipe.
#pragma unroll
        for (int c32 = 0; c32 < 2; ++c32) {
          const uint32_t seen = c32 ? seen1 : seen0;
          if (F != 0) {
            ScoreBias at = bias;
            at.off0 -= static_cast<float>(32 * c32);
            at.wr -= 32 * c32;
            score_columns<F, -1, true, CUT>(a, terms, *reinterpret_cast<uint32_t(*)[32]>(&r[c32 * 32]),
                                            *reinterpret_cast<float(*)[32]>(&pf[c32 * 32]), at);
            if (c32 == 1 && near) mbar_arrive(&c->win_empty[nw & 1]);
          }
          float pv[32];
          float4 ahead[8];
          if (c32 == 0) {
#pragma unroll
            for (int x = 0; x < 8; ++x) ahead[x] = nlse[8 + x];
          }
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const float4 n4 = nl[x / 4];
            const int o = c32 * 32 + x;
            f2unpack(ffma2(pair_of(r, o), c2x2, f2pack(n4.x, n4.y)), pv[x], pv[x + 1]);
            f2unpack(ffma2(pair_of(r, o + 2), c2x2, f2pack(n4.z, n4.w)), pv[x + 2], pv[x + 3]);
          }
          if (c32 == 0) {
#pragma unroll
            for (int x = 0; x < 8; ++x) nl[x] = ahead[x];
          }
          uint32_t pk[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            pv[x] = ex2_approx(pv[x]);
            pv[x + 1] = ex2_approx(pv[x + 1]);
            if (CUT) {
              if (!(seen & (1u << x))) pv[x] = 0.f;
              if (!(seen & (2u << x))) pv[x + 1] = 0.f;
            }
            pk[x / 2] = pack_bf16x2(pv[x], pv[x + 1]);
            const int o = c32 * 32 + x;
            if (F & kCap) {
              f2unpack(fmul2(f2pack(pf[o], pf[o + 1]), f2pack(pv[x], pv[x + 1])), pf[o], pf[o + 1]);
            } else {
              pf[o] = pv[x];
              pf[o + 1] = pv[x + 1];
            }
          }
          tmem_st16(tSh + c32 * 16, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&c->p_full);
#pragma unroll
        for (int x = 0; x < 8; ++x) nl[x] = nd[x];
        ok = __all_sync(0xffffffffu, mbar_wait(&c->dp_full, t & 1, &c->abort, a.spin_ns));
        if (!ok) return;
        tc_fence_after();
        tmem_ld32(tPh, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
        tmem_ld32(tPh + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
        tmem_ld_wait();
        reg_fence(r);
#pragma unroll
        for (int c32 = 0; c32 < 2; ++c32) {
          const uint32_t seen = c32 ? seen1 : seen0;
          uint32_t pk[16];
          float4 ahead[8];
          if (c32 == 0) {
#pragma unroll
            for (int x = 0; x < 8; ++x) ahead[x] = nd[8 + x];
          }
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const float4 d4 = nl[x / 4];
            const int o = c32 * 32 + x;
            float y0, y1, y2, y3;
            f2unpack(fmul2(fadd2(pair_of(r, o), f2pack(d4.x, d4.y)), f2pack(pf[o], pf[o + 1])), y0, y1);
            f2unpack(fmul2(fadd2(pair_of(r, o + 2), f2pack(d4.z, d4.w)), f2pack(pf[o + 2], pf[o + 3])), y2, y3);
            if (CUT) {   // dP of a masked pair may be NaN
              if (!(seen & (1u << x))) y0 = 0.f;
              if (!(seen & (2u << x))) y1 = 0.f;
              if (!(seen & (4u << x))) y2 = 0.f;
              if (!(seen & (8u << x))) y3 = 0.f;
            }
            pk[x / 2] = pack_bf16x2(y0, y1);
            pk[x / 2 + 1] = pack_bf16x2(y2, y3);
          }
          tmem_st16(tPh + c32 * 16, pk);
          if (c32 == 0) {
#pragma unroll
            for (int x = 0; x < 8; ++x) nl[x] = ahead[x];
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&c->ds_full);
      };
      if (edge || ((F & kBias) && a.slopes != nullptr && bias.side == 0)) pair(IntC<1>{});
      else pair(IntC<0>{});
      if (!ok) break;
      if (near) ++nw;
    }
    // ---- epilogue: warpgroup 0 writes dV, warpgroup 1 dK ---------------------
    const bool live = j < a.Nk;
    const Tensor4& ot = half == 0 ? a.dv : a.dk;
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(ot.p) + b * ot.sb + hk * ot.sh + static_cast<long long>(j) * ot.sn;
    const uint32_t src = (half == 0 ? tV : tK) + lanes;
    const float mul = half == 0 ? 1.f : a.scale;
    if (ok && t > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(&c->o_full, 0, &c->abort, a.spin_ns));
      tc_fence_after();
    }
    if (ok && a.kv_parts > 1) {   // fp32 partial sums, added up by k_score_sum_parts
      float* po = a.part_kv + (((static_cast<size_t>(part) * 2 + half) * a.B + b) * a.Hkv + hk) * a.Nk * D +
                  static_cast<size_t>(j) * D;
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t r[32];
        if (t > 0) {
          tmem_ld32(src + q * 32, r);
          tmem_ld_wait();
          reg_fence(r);
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) r[x] = 0;
        }
        if (live) {
#pragma unroll
          for (int x = 0; x < 32; x += 4)
            *reinterpret_cast<float4*>(po + q * 32 + x) =
                make_float4(u2f(r[x]) * mul, u2f(r[x + 1]) * mul, u2f(r[x + 2]) * mul, u2f(r[x + 3]) * mul);
        }
      }
    } else if (ok && t > 0) {
      store_row<D>(src, dst, mul, live);
    } else if (ok) {
      zero_row<D>(dst, live);
    }
    if (!ok) {
      c->abort = 1;
      report_status(a.status, CALIBATT_E_TIMEOUT);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, kTmemCols);
}

// ===========================================================================
// dQ and the table's gradient
// ===========================================================================

template <int D>
struct DqLayout {
  static constexpr uint32_t BOX = TILE * 64 * 2;
  static constexpr uint32_t TB = TILE * D * 2;
  static constexpr int RK = D == 128 ? 3 : 4;   // K tiles: read by S(t) and by dQ(t), two pairs later
  static constexpr int RV = D == 128 ? 1 : 2;   // V tiles: read by dP(t) alone
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_DO = TB;
  static constexpr uint32_t OFF_K = 2 * TB;
  static constexpr uint32_t OFF_V = OFF_K + RK * TB;
  static constexpr uint32_t OFF_WIN = OFF_V + RV * TB;      // float [2][256]
  static constexpr uint32_t OFF_BWIN = OFF_WIN + 2048;      // uint8 [2][256]
  static constexpr uint32_t OFF_HIST = OFF_BWIN + 512;      // float [8 warps][256]
  static constexpr uint32_t OFF_CTRL = OFF_HIST + 8192;
  static constexpr uint32_t SMEM = OFF_CTRL + kCtrlBytes + 1024;   // + alignment slack
  static_assert(SMEM <= 232448, "shared memory");
};

template <int RK, int RV>
struct DqCtrl {
  uint64_t q_full, k_full[RK], k_empty[RK], v_full[RV], v_empty[RV];
  uint64_t a_full[2], a_free[2], mid;   // first sweep
  uint64_t s_full[2], dp_full, dp_free, ds_full[2], o_full, drain;
  uint64_t win_full[2], win_empty[2];
  WindowInfo win_info[2];
  uint32_t tmem_base;
  int abort;
  float d_part[2][TILE];   // the column halves' sums of P dP
};

// First sweep: S and dP of key tile t in the column pairs [128 (t & 1), + 128)
// and [256 + 128 (t & 1), + 128), issued two tiles ahead of the softmax warps.
// Second sweep: S of key tile t in [128 (t & 1), + 128), dS in place; dP [256, 384);
// dQ at 384.  Issue order: S(0), dP(0), S(1); then per tile t, once dP(t) is
// read, dP(t + 1), and once dS(t) is stored, dQ(t) and S(t + 2): the scores are
// a tile ahead and dP(t + 1) is formed during the second half of tile t's
// arithmetic.  A warp may therefore store dS(t + 1) before a slower one has
// stored dS(t) (the table's gradient takes longer near the diagonal): tiles
// alternate between two ds_full barriers.  It gets no further ahead, since
// S(t + 2) waits for dS(t).
// Adds the warp's sum of v to *acc, in a fixed order.
__device__ __forceinline__ void add_to_bucket(float* acc, float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if (lane_id() == 0) *acc += v;
  __syncwarp();
}

// dZ of 32 columns whose offsets meet boundaries k ... k1 - 1 of a window:
// column x is entry `entry` + x.  Per segment the row's sum, added up over the
// warp.  (Each segment from its own columns: as a difference of running sums a
// small bucket behind a large one kept only the large one's rounding.)
__device__ __forceinline__ void sum_by_cuts(const uint32_t (&g)[32], const WindowInfo& info, int k, int k1, int entry,
                                         float* acc) {
  int from = 0;
  for (; k <= k1; ++k) {
    const int cut = k < k1 ? min(max(info.at[k] - entry, from), 32) : 32;
    const unsigned len = cut - from;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int x = 0; x < 32; x += 2) {
      if (static_cast<unsigned>(x - from) < len) s0 += u2f(g[x]);
      if (static_cast<unsigned>(x + 1 - from) < len) s1 += u2f(g[x + 1]);
    }
    add_to_bucket(acc + info.bucket[k], s0 + s1);
    from = cut;
  }
}

// dZ of 32 rows and 32 columns summed along the diagonals (one offset each) by
// passing a running sum from row to row: after column x lane 31 holds the sum
// of the diagonal that ends in it, with bucket b[x]; 31 more steps drain the
// others.  Runs of offsets of one bucket are added up before the accumulators
// are touched.
__device__ __forceinline__ void sum_by_diagonals(const uint32_t (&g)[32], const uint8_t* b, float* acc) {
  const int lane = lane_id();
  float diag = 0.f, run = 0.f;
  int cur = b[0];
  auto add = [&](int x) {
    const int n = b[x];
    if (n != cur) {
      if (lane == 31) acc[cur] += run;
      run = 0.f;
      cur = n;
    }
    run += diag;
  };
#pragma unroll
  for (int x = 0; x < 32; ++x) {
    const float up = __shfl_up_sync(0xffffffffu, diag, 1);
    diag = u2f(g[x]) + (lane == 0 ? 0.f : up);
    add(x);
  }
#pragma unroll 1
  for (int x = 32; x < 63; ++x) {
    const float up = __shfl_up_sync(0xffffffffu, diag, 1);
    diag = lane == 0 ? 0.f : up;
    add(x);
  }
  if (lane == 31) acc[cur] += run;
  __syncwarp();
}

template <int D, int F>
__global__ void __launch_bounds__(kThreads, 1)
    k_score_dq(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
               const __grid_constant__ ScoreArgs a) {
  using L = DqLayout<D>;
  constexpr int RK = L::RK, RV = L::RV;
  static_assert(sizeof(DqCtrl<RK, RV>) <= kCtrlBytes, "control block");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DqCtrl<RK, RV>* c = reinterpret_cast<DqCtrl<RK, RV>*>(smem + L::OFF_CTRL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // query tiles of a head side by side (they read the same K and V), the last
  // ones, which see most keys under a causal rule, first
  const int qb = a.nqb - 1 - blockIdx.x % a.nqb, bh = blockIdx.x / a.nqb;
  const int b = bh / a.H, h = bh % a.H, hk = h / a.G;
  const int4 tr = score_tile(a, b, qb);
  const int lo = tr.x >> 7, hi = tr.x < tr.y ? (tr.y + TILE - 1) >> 7 : lo;
  const int p0 = a.q_start[b] + qb * TILE;
  float* hist = reinterpret_cast<float*>(smem + L::OFF_HIST);

  if (threadIdx.x == 0) {
    mbar_init(&c->q_full, 1);
    for (int e = 0; e < RK; ++e) {
      mbar_init(&c->k_full[e], 1);
      mbar_init(&c->k_empty[e], 1);
    }
    for (int e = 0; e < RV; ++e) {
      mbar_init(&c->v_full[e], 1);
      mbar_init(&c->v_empty[e], 1);
    }
    for (int e = 0; e < 2; ++e) {
      mbar_init(&c->a_full[e], 1);
      mbar_init(&c->a_free[e], 256);
      mbar_init(&c->s_full[e], 1);
      mbar_init(&c->ds_full[e], 256);
      mbar_init(&c->win_full[e], 32);
      mbar_init(&c->win_empty[e], 256);
    }
    mbar_init(&c->mid, 256);
    mbar_init(&c->dp_full, 1);
    mbar_init(&c->dp_free, 256);
    mbar_init(&c->o_full, 1);
    mbar_init(&c->drain, 1);
    c->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmDO);
  }
  if ((F & kGrad))
    for (int x = threadIdx.x; x < 8 * 256; x += kThreads) hist[x] = 0.f;
  if (warp == kMma) {
    tmem_alloc(&c->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem_base;
  const uint32_t tP = tmem + 256, tQ = tmem + 384;

  if (warp >= 8) regs_dec<kControlRegs>();
  if (warp == kProducer) {
    KeyWalk w;
    bool ok = true;
    const bool any = key_start(a, h, qb, lo, hi, w);
    uint32_t t = 0;
    int sweep = 0;
    bool loaded_v = true;   // the last tile's V copy was issued too
    const uint64_t pol = l2_policy_evict_last(), pol_q = l2_policy_evict_first();
    if (any) {
      mbar_arrive_expect_tx_w(&c->q_full, 2 * L::TB);
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        tma_load_4d_w(smem + L::OFF_Q + x * L::BOX, &tmQ, x * 64, qb * TILE, h, b, &c->q_full, pol_q);
        tma_load_4d_w(smem + L::OFF_DO + x * L::BOX, &tmDO, x * 64, qb * TILE, h, b, &c->q_full, pol_q);
      }
    }
    while (any) {
      const int e = t % RK, v = t % RV;
      ok = __all_sync(0xffffffffu, mbar_wait(&c->k_empty[e], ((t / RK) & 1) ^ 1, &c->abort, a.spin_ns));
      if (!ok) break;
      mbar_arrive_expect_tx_w(&c->k_full[e], L::TB);
#pragma unroll
      for (int x = 0; x < D / 64; ++x)
        tma_load_4d_w(smem + L::OFF_K + e * L::TB + x * L::BOX, &tmK, x * 64, w.kb * TILE, hk, b, &c->k_full[e], pol);
      ++t;
      loaded_v = false;
      ok = __all_sync(0xffffffffu, mbar_wait(&c->v_empty[v], (((t - 1) / RV) & 1) ^ 1, &c->abort, a.spin_ns));
      if (!ok) break;
      mbar_arrive_expect_tx_w(&c->v_full[v], L::TB);
#pragma unroll
      for (int x = 0; x < D / 64; ++x)
        tma_load_4d_w(smem + L::OFF_V + v * L::TB + x * L::BOX, &tmV, x * 64, w.kb * TILE, hk, b, &c->v_full[v], pol);
      loaded_v = true;
      if (w.next >= 0) key_next(a, h, qb, w);
      else if (sweep++ == 0) key_start(a, h, qb, lo, hi, w);
      else break;
    }
    if (lane == 0) {
      if (!ok) {
        c->abort = 1;
        report_status(a.status, CALIBATT_E_TIMEOUT);
      }
      // Drain: every copy issued must have landed before the CTA may exit.
      if (any) mbar_wait(&c->q_full, 0, nullptr, a.spin_ns);
      const uint32_t tv = loaded_v ? t : t - 1;
      for (int e = 0; e < RK; ++e) {
        const uint32_t fills = (t > static_cast<uint32_t>(e)) ? (t - 1 - e) / RK + 1 : 0;
        if (fills > 0) mbar_wait(&c->k_full[e], (fills - 1) & 1, nullptr, a.spin_ns);
      }
      for (int e = 0; e < RV; ++e) {
        const uint32_t fills = (tv > static_cast<uint32_t>(e)) ? (tv - 1 - e) / RV + 1 : 0;
        if (fills > 0) mbar_wait(&c->v_full[e], (fills - 1) & 1, nullptr, a.spin_ns);
      }
    }
  } else if (warp == kMma) {
    uint32_t n = 0;
    if (a.mask == nullptr) {
      n = max(0, hi - lo);
    } else {
      for (int w = lo; w < hi; w += 32) n += __popc(__ballot_sync(0xffffffffu, w + lane < hi && score_kept(a, h, qb, w + lane)));
    }
    constexpr uint32_t IDESC_S = idesc_bf16_f32(TILE, TILE, false);
    constexpr uint32_t IDESC_O = idesc_bf16_f32(TILE, D, true);
    const uint32_t sQ = smem_u32(smem + L::OFF_Q), sO = smem_u32(smem + L::OFF_DO);
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, &c->abort, a.spin_ns));
      tc_fence_after();
      return ok;
    };
    // u: position in the rings, which go on from the first sweep to the second
    auto sK = [&](uint32_t u) { return smem_u32(smem + L::OFF_K + (u % RK) * L::TB); };
    auto qk = [&](uint32_t u, uint32_t dst) {
      if (!wait(&c->k_full[u % RK], (u / RK) & 1)) return false;
      mma_scores<D>(dst, sQ, sK(u), IDESC_S);
      return true;
    };
    auto ov = [&](uint32_t u, uint32_t dst) {
      if (!wait(&c->v_full[u % RV], (u / RV) & 1)) return false;
      mma_scores<D>(dst, sO, smem_u32(smem + L::OFF_V + (u % RV) * L::TB), IDESC_S);
      mma_commit_w(&c->v_empty[u % RV]);
      return true;
    };
    auto scores = [&](uint32_t t) {
      if (!qk(n + t, tmem + (t & 1) * 128)) return false;
      mma_commit_w(&c->s_full[t & 1]);
      return true;
    };
    auto grads = [&](uint32_t t) {
      if (!ov(n + t, tP)) return false;
      mma_commit_w(&c->dp_full);
      return true;
    };
    if (n > 0 && wait(&c->q_full, 0)) {
      for (uint32_t t = 0; t < n; ++t) {
        if (!wait(&c->a_free[t & 1], ((t >> 1) & 1) ^ 1)) break;
        if (!qk(t, tmem + (t & 1) * 128)) break;
        mma_commit_w(&c->k_empty[t % RK]);
        if (!ov(t, tP + (t & 1) * 128)) break;
        mma_commit_w(&c->a_full[t & 1]);
      }
    }
    if (n > 0 && ok && wait(&c->mid, 0) && scores(0) && grads(0) && (n == 1 || scores(1))) {
      for (uint32_t t = 0; t < n; ++t) {
        if (!wait(&c->dp_free, t & 1)) break;
        if (t + 1 < n && !grads(t + 1)) break;
        if (!wait(&c->ds_full[t & 1], (t >> 1) & 1)) break;
        mma_from_tmem(tQ, tmem + (t & 1) * 128, sK(n + t), IDESC_O, t > 0 ? 1u : 0u);
        mma_commit_w(&c->k_empty[(n + t) % RK]);
        if (t + 1 == n) mma_commit_w(&c->o_full);
        if (t + 2 < n && !scores(t + 2)) break;
      }
    }
    if (!ok && lane == 0) {
      c->abort = 1;
      report_status(a.status, CALIBATT_E_TIMEOUT);
    }
    __syncwarp();
    mma_commit_w(&c->drain);
    mbar_wait(&c->drain, 0, nullptr, a.spin_ns);
  } else if (warp == kWindow) {
    if ((F & kBias) && a.table != nullptr) {
      KeyWalk w;
      bool bad = false, ok = true;
      uint32_t t = 0;
      int sweep = 0;
      for (bool more = key_start(a, h, qb, lo, hi, w); more;) {
        if (is_near(a, w.kb * TILE, p0, p0 + TILE - 1)) {
          const int e = t & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&c->win_empty[e], ((t >> 1) & 1) ^ 1, &c->abort,
                                                  kWindowPatience * a.spin_ns));
          if (!ok) break;
          fill_window(a, h, 1, w.kb * TILE - p0 - (TILE - 1), reinterpret_cast<float*>(smem + L::OFF_WIN) + e * 256,
                      smem + L::OFF_BWIN + e * 256, &c->win_info[e], &bad);
          mbar_arrive(&c->win_full[e]);
          ++t;
        }
        if (w.next >= 0) key_next(a, h, qb, w);
        else more = sweep++ == 0 && key_start(a, h, qb, lo, hi, w);
      }
      if (!ok) {
        c->abort = 1;
        report_status(a.status, CALIBATT_E_TIMEOUT);
      }
      if (bad) report_status(a.status, CALIBATT_E_CORRUPT);
    }
  } else if (warp < 8) {
    regs_inc<kSoftmaxRegs>();
    const int half = warp >> 2, w4 = warp & 3, row = w4 * 32 + lane;   // row: query of the tile
    const int i = qb * TILE + row;
    const uint32_t lanes = static_cast<uint32_t>(w4 * 32) << 16;
    const uint32_t tPh = tP + lanes + half * 64;
    const ScoreTerms terms = score_terms(a);
    constexpr bool xform = F != 0;
    const uint64_t c2x2 = f2pack(xform ? 1.f : terms.sc, xform ? 1.f : terms.sc);
    const int2 vis = score_row(a, b, i);
    // -log2(e) LSE; -inf (P = 0) where the row sees nothing
    float nlse = -INFINITY;
    if (vis.x < vis.y) {
      const float x = a.lse[(static_cast<size_t>(b) * a.H + h) * a.Nq + i];
      if (x != -INFINITY) nlse = -kLog2e * x;
    }
    uint64_t nlse2 = f2pack(nlse, nlse);
    const float slope = (F & kBias) && a.slopes != nullptr ? a.slopes[h] * kLog2e : 0.f;
    float far_lo = 0.f, far_hi = 0.f;
    int n_lo = 0, n_hi = 0;
    if ((F & kBias) && a.table != nullptr) {
      bool bad = false;
      const __nv_bfloat16* tab = reinterpret_cast<const __nv_bfloat16*>(a.table) + static_cast<size_t>(h) * a.n_buckets;
      n_lo = score_bucket(a, -a.R, &bad);
      n_hi = score_bucket(a, a.R, &bad);
      far_lo = __bfloat162float(tab[n_lo]) * kLog2e;
      far_hi = __bfloat162float(tab[n_hi]) * kLog2e;
      if (bad) report_status(a.status, CALIBATT_E_CORRUPT);
    }
    // What key tile k0 adds to this thread's 64 columns' scores (`near`: from window wt & 1).
    auto bias_of = [&](int k0, bool near, uint32_t wt) {
      ScoreBias bias = {};
      if (F & kBias) {
        bias.wr = reinterpret_cast<const float*>(smem + L::OFF_WIN) + (wt & 1) * 256 + TILE - 1 - row + half * 64;
        bias.window = near && c->win_info[wt & 1].cuts > 0;
        bias.flat = near ? (bias.window ? 0.f : bias.wr[0]) : k0 > p0 ? far_hi : far_lo;
        bias.side = k0 >= p0 + TILE - 1 ? 1 : k0 + TILE - 1 <= p0 ? -1 : 0;
        bias.slope = slope;
        bias.off0 = static_cast<float>(k0 + half * 64 - p0 - row);
      }
      return bias;
    };
    // The table's gradient: 32 columns of dZ, the first at column c0 of the
    // tile, go to the buckets of their offsets.  While a warp's chunks stay in
    // one bucket their sums stay in registers; it is added up over the warp
    // when the bucket changes.  The order is fixed throughout.
    int cur = 0;
    float cur_sum = 0.f;
    auto flush = [&](int next) {
      if (next != cur) {
        add_to_bucket(hist + warp * 256 + cur, cur_sum);
        cur_sum = 0.f;
        cur = next;
      }
    };
    auto add_buckets = [&](const uint32_t (&g)[32], bool near, int k0, uint32_t wt, int c0) {
      int bucket = k0 > p0 ? n_hi : n_lo;
      if (near) {
        // entries of the window that this warp's 32 rows and 32 columns meet
        const WindowInfo& info = c->win_info[wt & 1];
        const int first = TILE - 1 - (w4 * 32 + 31) + c0, last = first + 62;
        int k = 0, k1 = 0;
        if (info.cuts <= kMaxCuts) {
          while (k < info.cuts && info.at[k] <= first) ++k;
          k1 = k;
          while (k1 < info.cuts && info.at[k1] <= last) ++k1;
          bucket = info.bucket[k];
        }
        if (info.cuts > kMaxCuts || k != k1) {
          if (info.cuts <= kMaxCuts) sum_by_cuts(g, info, k, k1, TILE - 1 - row + c0, hist + warp * 256);
          else sum_by_diagonals(g, smem + L::OFF_BWIN + (wt & 1) * 256 + first, hist + warp * 256);
          return;
        }
      }
      flush(bucket);
      uint64_t s = f2pack(0.f, 0.f);
#pragma unroll
      for (int x = 0; x < 32; x += 2) s = fadd2(s, pair_of(g, x));
      float lo_, hi_;
      f2unpack(s, lo_, hi_);
      cur_sum += lo_ + hi_;
    };
    bool ok = true;
    uint32_t t = 0, wt = 0, nw = 0;   // wt, nw: tiles and windows consumed, over both sweeps
    KeyWalk w;
    // ---- first sweep: D = sum over the visible keys of P dP ------------------
    float d_sum = 0.f;
    for (bool more = key_start(a, h, qb, lo, hi, w); more; ++t, ++wt) {
      const int k0 = w.kb * TILE;
      const uint32_t tSh = tmem + (t & 1) * 128 + lanes + half * 64;
      const bool edge = k0 < tr.z || k0 + TILE > tr.w;
      const bool near = (F & kBias) && is_near(a, k0, p0, p0 + TILE - 1);
      bool got = mbar_wait(&c->a_full[t & 1], (t >> 1) & 1, &c->abort, a.spin_ns);
      if (got && near) got = mbar_wait(&c->win_full[nw & 1], (nw >> 1) & 1, &c->abort, a.spin_ns);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      tc_fence_after();
      const int e0 = vis.x - k0 - half * 64, e1 = vis.y - k0 - half * 64;   // columns of the row's interval
      const ScoreBias bias = bias_of(k0, near, nw);
      auto tile = [&](auto cut_c) {
        constexpr bool CUT = decltype(cut_c)::value != 0;
        uint64_t s0 = f2pack(0.f, 0.f), s1 = s0;
#pragma unroll 1
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t r[32], g[32];
          tmem_ld32(tSh + ch * 32, r);
          tmem_ld32(tSh + 256 + ch * 32, g);
          tmem_ld_wait();
          reg_fence(r);
          reg_fence(g);
          if (ch == 1) {
            tc_fence_before();
            mbar_arrive(&c->a_free[t & 1]);
          }
          const uint32_t bits = CUT ? bits_below(e1 - 32 * ch) & ~bits_below(e0 - 32 * ch) : 0xffffffffu;
          if (F != 0) {
            ScoreBias at = bias;
            at.off0 += static_cast<float>(32 * ch);
            at.wr += 32 * ch;
            float none[32];
            score_columns<F & 3, 1, false, CUT>(a, terms, r, none, at);
          }
          if (CUT) {
            keep_bits(r, bits, -INFINITY);
            keep_bits(g, bits, 0.f);
          }
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            float y0, y1;
            f2unpack(ffma2(pair_of(r, x), c2x2, nlse2), y0, y1);
            const uint64_t pp = f2pack(ex2_approx(y0), ex2_approx(y1));
            if (x & 2) s1 = ffma2(pp, pair_of(g, x), s1); else s0 = ffma2(pp, pair_of(g, x), s0);
          }
        }
        float u0, u1, v0, v1;
        f2unpack(s0, u0, u1);
        f2unpack(s1, v0, v1);
        d_sum += (u0 + u1) + (v0 + v1);
      };
      if (edge || ((F & kBias) && a.slopes != nullptr && bias.side == 0)) tile(IntC<1>{});
      else tile(IntC<0>{});
      if (near) {
        mbar_arrive(&c->win_empty[nw & 1]);
        ++nw;
      }
      more = w.next >= 0;
      if (more) key_next(a, h, qb, w);
    }
    float nd = 0.f;
    if (ok) {
      c->d_part[half][row] = d_sum;
      mbar_arrive(&c->mid);
      ok = __all_sync(0xffffffffu, mbar_wait(&c->mid, 0, &c->abort, a.spin_ns));
      nd = -(c->d_part[0][row] + c->d_part[1][row]);
      // A row with a non-finite dO (or V that it sees) marks every gradient it
      // enters: its probabilities become NaN.
      if (!isfinite(nd)) nlse = NAN;
      nlse2 = f2pack(nlse, nlse);
      if (half == 0) {
        const size_t r0 = (static_cast<size_t>(b) * a.H + h) * a.nqb * TILE + i;
        a.row_lse[r0] = nlse;
        a.row_d[r0] = nd;
        if (h == 0) a.row_span[static_cast<size_t>(b) * a.nqb * TILE + i] = vis;
      }
    }
    const uint64_t nd2 = f2pack(nd, nd);
    // ---- second sweep ----------------------------------------------------------
    t = 0;
    for (bool more = ok && key_start(a, h, qb, lo, hi, w); more; ++t, ++wt) {
      const int k0 = w.kb * TILE;
      const uint32_t tSh = tmem + (t & 1) * 128 + lanes + half * 64;
      const bool edge = k0 < tr.z || k0 + TILE > tr.w;
      const bool near = (F & kBias) && is_near(a, k0, p0, p0 + TILE - 1);
      const uint32_t u = wt;   // position in the K ring
      bool got = mbar_wait(&c->s_full[t & 1], (t >> 1) & 1, &c->abort, a.spin_ns);
      if (got && near) got = mbar_wait(&c->win_full[nw & 1], (nw >> 1) & 1, &c->abort, a.spin_ns);
      if (got && edge) got = mbar_wait(&c->k_full[u % RK], (u / RK) & 1, &c->abort, a.spin_ns);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      tc_fence_after();
      const int e0 = vis.x - k0 - half * 64, e1 = vis.y - k0 - half * 64;   // columns of the row's interval
      const ScoreBias bias = bias_of(k0, near, nw);
      auto tile = [&](auto cut_c) {
        constexpr bool CUT = decltype(cut_c)::value != 0;
        // Keys with a NaN or an infinity: zeroed before dQ reads them (S, which
        // is complete, has made a visible one's dS NaN).
        if (CUT && edge && half < D / 64) clean_row<1>(smem + L::OFF_K + (u % RK) * L::TB + half * L::BOX, row);
        ok = __all_sync(0xffffffffu, mbar_wait(&c->dp_full, t & 1, &c->abort, a.spin_ns));
        if (!ok) return;
        tc_fence_after();
#pragma unroll 1
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t r[32], g[32];
          tmem_ld32(tSh + ch * 32, r);
          tmem_ld32(tPh + ch * 32, g);
          tmem_ld_wait();
          reg_fence(r);
          reg_fence(g);
          if (ch == 1) {
            tc_fence_before();
            mbar_arrive(&c->dp_free);
          }
          const uint32_t bits = CUT ? bits_below(e1 - 32 * ch) & ~bits_below(e0 - 32 * ch) : 0xffffffffu;
          float f[32];
          if (F != 0) {
            ScoreBias at = bias;
            at.off0 += static_cast<float>(32 * ch);
            at.wr += 32 * ch;
            score_columns<F & 3, 1, (F & kCap) != 0, CUT>(a, terms, r, f, at);
          }
          // dZ = P (dP - D) in place of dP
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            float y0, y1;
            f2unpack(ffma2(pair_of(r, x), c2x2, nlse2), y0, y1);
            set_pair(g, x, fmul2(fadd2(pair_of(g, x), nd2), f2pack(ex2_approx(y0), ex2_approx(y1))));
          }
          if (CUT) {
            keep_bits(g, bits, 0.f);
            if (F & kCap) {   // the factor of a masked score may be NaN
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (!(bits & (1u << x))) f[x] = 0.f;
            }
          }
          if (F & kGrad) add_buckets(g, near, k0, nw, half * 64 + ch * 32);
          uint32_t pk[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            float y0, y1;
            uint64_t v = pair_of(g, x);
            if (F & kCap) v = fmul2(v, f2pack(f[x], f[x + 1]));
            f2unpack(v, y0, y1);
            pk[x / 2] = pack_bf16x2(y0, y1);
          }
          tmem_st16(tSh + ch * 16, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&c->ds_full[t & 1]);
      };
      if (edge || ((F & kBias) && a.slopes != nullptr && bias.side == 0)) tile(IntC<1>{});
      else tile(IntC<0>{});
      if (!ok) break;
      if (near) {
        mbar_arrive(&c->win_empty[nw & 1]);
        ++nw;
      }
      more = w.next >= 0;
      if (more) key_next(a, h, qb, w);
    }
    // ---- epilogue: each warpgroup writes half of dQ's columns ----------------
    const bool live = i < a.Nq;
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.dq.p) + b * a.dq.sb + h * a.dq.sh +
                         static_cast<long long>(i) * a.dq.sn + half * (D / 2);
    if (ok && t > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(&c->o_full, 0, &c->abort, a.spin_ns));
      tc_fence_after();
      if (ok) store_row<D / 2>(tQ + lanes + half * (D / 2), dst, a.scale, live);
    } else if (ok) {
      zero_row<D / 2>(dst, live);
    }
    if (!ok) {
      c->abort = 1;
      report_status(a.status, CALIBATT_E_TIMEOUT);
    }
    if ((F & kGrad)) {
      flush(-1);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if ((F & kGrad)) {
    float* dst = a.part_table + ((static_cast<size_t>(b) * a.H + h) * a.table_tiles + qb) * a.n_buckets;
    for (int n = threadIdx.x; n < a.n_buckets; n += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x) s += hist[x * 256 + n];
      dst[n] = s;
    }
  }
  if (warp == kMma) tmem_dealloc(tmem, kTmemCols);
}

template <int D, int F>
int launch(const ScoreArgs& a, cudaStream_t s) {
  CUtensorMap tq, tk, tv, to;
  int rc;
  if ((rc = make_tmap4_bf16(&tq, a.q, a.B, a.H, a.Nq, D, TILE, 1))) return rc;
  if ((rc = make_tmap4_bf16(&tk, a.k, a.B, a.Hkv, a.Nk, D, TILE, 1))) return rc;
  if ((rc = make_tmap4_bf16(&tv, a.v, a.B, a.Hkv, a.Nk, D, TILE, 1))) return rc;
  if ((rc = make_tmap4_bf16(&to, a.dout, a.B, a.H, a.Nq, D, TILE, 1))) return rc;
  const long long nk = static_cast<long long>(a.B) * a.Hkv * a.nkb * a.kv_parts, nq = static_cast<long long>(a.B) * a.H * a.nqb;
  if (nk >= (1ll << 31) || nq >= (1ll << 31)) return set_error(CALIBATT_E_UNSUPPORTED, "too many tiles");
  static std::atomic<bool> done_kv[kMaxDevices], done_q[2][kMaxDevices];
  auto dkv = k_score_dkv<D, F>;
  auto dq = k_score_dq<D, F>;
  if ((F & kBias) && a.dtable != nullptr) dq = k_score_dq<D, F & kBias ? F | kGrad : F>;
  if ((rc = configure_kernel(reinterpret_cast<const void*>(dkv), done_kv, DkvLayout<D>::SMEM, kLaunchRegs, "k_score_dkv")))
    return rc;
  if ((rc = configure_kernel(reinterpret_cast<const void*>(dq), done_q[a.dtable != nullptr], DqLayout<D>::SMEM, kLaunchRegs, "k_score_dq")))
    return rc;
  dq<<<static_cast<unsigned>(nq), kThreads, DqLayout<D>::SMEM, s>>>(tq, tk, tv, to, a);
  dkv<<<static_cast<unsigned>(nk), kThreads, DkvLayout<D>::SMEM, s>>>(tq, tk, tv, to, a);
  count_launch(2);
  if (int rc2 = check_launch("k_score_bwd")) return rc2;
  return launch_score_sum_parts(a, D, CALIBATT_BF16, s);
}

}  // namespace

// Parts of the (query head, query tile) pairs of a key tile: with fewer key
// tiles than SMs the pairs are divided, at least two to a part (five query
// heads on one key head at 1264 tokens, d = 64: 20 CTAs of 50 pairs otherwise).
int score_kv_parts(int B, int Hkv, int G, int nqb, int nkb) {
  const long long tiles = static_cast<long long>(B) * Hkv * nkb;
  return static_cast<int>(std::max<long long>(1, std::min<long long>(148 / tiles, static_cast<long long>(G) * nqb / 2)));
}

int launch_score_bwd_tc(const ScoreArgs& a, int d, cudaStream_t s) {
  switch ((a.cap > 0.f ? kCap : 0) | (a.slopes != nullptr || a.table != nullptr ? kBias : 0)) {
    case 0: return d == 128 ? launch<128, 0>(a, s) : launch<64, 0>(a, s);
    case kCap: return d == 128 ? launch<128, kCap>(a, s) : launch<64, kCap>(a, s);
    case kBias: return d == 128 ? launch<128, kBias>(a, s) : launch<64, kBias>(a, s);
    default: return d == 128 ? launch<128, kCap | kBias>(a, s) : launch<64, kCap | kBias>(a, s);
  }
}

}  // namespace calibatt
