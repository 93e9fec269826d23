// score_simt.cu -- score-modified attention on the CUDA cores (FFMA), forward
// and backward, for fp32 inputs (tensor cores would round them to tf32).
//
// 64 x 64 score tiles, 256 threads as 16 x 16; a thread owns rows 4 ty .. 4 ty
// + 3 and score columns tx, tx + 16, tx + 32, tx + 48 (so that the rows of the
// second operand read by a quarter warp fall into different banks), and for
// the products with a D-wide result the same rows and columns 4 tx + 64 c ..
// + 3.  Every product reads its operands from shared memory as float4: 8 reads
// for 64 FFMAs of a score step, bound by the FFMA pipe and shared memory
// together.  Softmax over one pass of the keys with running maximum and sum;
// the backward recomputes the scores in both of its passes (keys outer for dK
// and dV, queries outer for dQ and the table's gradient), so every gradient is
// summed in a fixed order, without atomics; with few tiles the walks are
// divided into parts, whose sums are added in part order.
#include <algorithm>

#include "score_common.cuh"

namespace calibatt {
namespace {

constexpr int BT = 64;          // rows and columns of a score tile
constexpr int kThreads = 256;
constexpr int PS = BT + 4;      // row pitch of a stored score tile
template <int D>
constexpr int PD = D + 4;       // row pitch of a stored input tile (16-byte aligned rows)

__device__ __forceinline__ void store4(float* p, float x, float y, float z, float w) {
  *reinterpret_cast<float4*>(p) = make_float4(x, y, z, w);
}

// Rows [r0, r0 + 64) of one head into shared memory, zero past n.
template <int D>
__device__ __forceinline__ void load_tile(float* dst, const Tensor4& t, int b, int h, int r0, int n) {
  const float* src = reinterpret_cast<const float*>(t.p) + b * t.sb + h * t.sh;
  for (int x = threadIdx.x; x < BT * D / 4; x += kThreads) {
    const int r = x / (D / 4), c = x % (D / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < n) v = *reinterpret_cast<const float4*>(src + (r0 + r) * t.sn + c);
    *reinterpret_cast<float4*>(dst + r * PD<D> + c) = v;
  }
}

// acc[i][j] += sum over d of A[4 ty + i][d] Bm[tx + 16 j][d]
template <int D>
__device__ __forceinline__ void dot_tile(float (&acc)[4][4], const float* A, const float* Bm, int ty, int tx) {
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(A + (ty * 4 + i) * PD<D> + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(Bm + (tx + 16 * j) * PD<D> + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
  }
}

// acc[i][4 c + e] += sum over k of P[4 ty + i][k] X[k][4 tx + 64 c + e]
template <int D>
__device__ __forceinline__ void mul_tile(float (&acc)[4][D / 16], const float* P, const float* X, int ty, int tx) {
#pragma unroll 2
  for (int k = 0; k < BT; k += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty * 4 + i) * PS + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float4 x = *reinterpret_cast<const float4*>(X + (k + kk) * PD<D> + tx * 4 + 64 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
          acc[i][c * 4 + 0] = fmaf(w, x.x, acc[i][c * 4 + 0]);
          acc[i][c * 4 + 1] = fmaf(w, x.y, acc[i][c * 4 + 1]);
          acc[i][c * 4 + 2] = fmaf(w, x.z, acc[i][c * 4 + 2]);
          acc[i][c * 4 + 3] = fmaf(w, x.w, acc[i][c * 4 + 3]);
        }
      }
  }
}

// Transposed form: acc[i][..] += sum over q of P[q][4 ty + i] X[q][4 tx + 64 c + e]
template <int D>
__device__ __forceinline__ void mul_tile_t(float (&acc)[4][D / 16], const float* P, const float* X, int ty, int tx) {
#pragma unroll 4
  for (int q = 0; q < BT; ++q) {
    const float4 p = *reinterpret_cast<const float4*>(P + q * PS + ty * 4);
    const float w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const float4 x = *reinterpret_cast<const float4*>(X + q * PD<D> + tx * 4 + 64 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][c * 4 + 0] = fmaf(w[i], x.x, acc[i][c * 4 + 0]);
        acc[i][c * 4 + 1] = fmaf(w[i], x.y, acc[i][c * 4 + 1]);
        acc[i][c * 4 + 2] = fmaf(w[i], x.z, acc[i][c * 4 + 2]);
        acc[i][c * 4 + 3] = fmaf(w[i], x.w, acc[i][c * 4 + 3]);
      }
    }
  }
}

// Rows of X that hold a non-finite value are zeroed and marked: a probability
// of 0 of a masked pair would turn them into NaN.
template <int D>
__device__ __forceinline__ void clean_rows(float* X, int* bad) {
  const int r = threadIdx.x >> 2, part = threadIdx.x & 3;   // four threads a row
  float* at = X + r * PD<D> + part * (D / 4);
  bool ok = true;
#pragma unroll
  for (int c = 0; c < D / 4; c += 4) {
    const float4 v = *reinterpret_cast<const float4*>(at + c);
    ok = ok && isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w);
  }
  ok = (__ballot_sync(0xffffffffu, !ok) >> (threadIdx.x & 28) & 15u) == 0;
  if (!ok) {
#pragma unroll
    for (int c = 0; c < D / 4; c += 4) *reinterpret_cast<float4*>(at + c) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (part == 0) bad[r] = !ok;
}

// The table along the 127 offsets of a 64 x 64 tile: entry x is offset o0 + x.
// (Read pair by pair from global memory these were the longest part of small
// training steps.)
struct Window {
  float value[2 * BT];
  int bucket[2 * BT];
};
__device__ __forceinline__ void fill_window(const ScoreArgs& a, int h, int o0, Window* w, bool* bad) {
  if (a.table == nullptr) return;
  const int x = threadIdx.x;
  if (x < 2 * BT - 1) {
    const int n = score_bucket(a, o0 + x, bad);
    w->bucket[x] = n;
    // An entry that log2(e) takes below fp32's range (the lowest value, as a
    // mask) is -inf, as in the kernels that work in log2 units.  Kept finite it
    // would absorb the scores, and a row that sees nothing else would have an
    // LSE without its logarithm.
    const float v = reinterpret_cast<const float*>(a.table)[static_cast<size_t>(h) * a.n_buckets + n];
    w->value[x] = v * kLog2e == -INFINITY ? -INFINITY : v;
  }
}

// z of the pair (row, col) of the tile with offset `off`, and the cap's tanh in *th (0 without a cap).
__device__ __forceinline__ float score_of(const ScoreArgs& a, float slope, const Window& w, float dot, int row, int col,
                                          int off, float* th) {
  float z = dot * a.scale;
  *th = 0.f;
  if (a.cap > 0.f) {
    *th = tanhf(z / a.cap);
    z = a.cap * *th;
  }
  if (a.slopes != nullptr) z -= slope * fabsf(static_cast<float>(off));
  if (a.table != nullptr) z += w.value[col - row + BT - 1];
  return z;
}

template <int D>
struct SimtSmem {
  static constexpr int IN = BT * PD<D>;   // floats of an input tile
  static constexpr int SC = BT * PS;      // floats of a score tile
};

template <int D>
__global__ void __launch_bounds__(kThreads) k_score_fwd_simt(const ScoreArgs a) {
  using S = SimtSmem<D>;
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm, *sK = sQ + S::IN, *sV = sK + S::IN, *sP = sV + S::IN;
  __shared__ int bad_row[BT];
  __shared__ Window win;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int q0 = blockIdx.x / a.splits * BT, sp = blockIdx.x % a.splits, h = blockIdx.y, b = blockIdx.z, hk = h / a.G;
  const int qb = q0 >> 7;
  const int4 t = score_tile(a, b, qb);
  const int qs = a.q_start[b];
  const float slope = a.slopes != nullptr ? a.slopes[h] : 0.f;
  int2 vis[4];
  float m[4], l[4], o[4][D / 16];
  bool nan_row[4], bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    vis[i] = score_row(a, b, q0 + ty * 4 + i);
    m[i] = -INFINITY;
    l[i] = 0.f;
    nan_row[i] = false;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
  }
  load_tile<D>(sQ, a.q, b, h, q0, a.Nq);
  // this split's key tiles
  const int first = t.x / BT, tiles = max(0, (t.y + BT - 1) / BT - first), per = (tiles + a.splits - 1) / a.splits;
  const int end = min(t.y, (first + min(tiles, (sp + 1) * per)) * BT);
  for (int k0 = (first + sp * per) * BT; k0 < end; k0 += BT) {
    if (!score_kept(a, h, qb, k0 >> 7)) continue;
    const bool edge = k0 < t.z || k0 + BT > t.w;
    __syncthreads();
    load_tile<D>(sK, a.k, b, hk, k0, a.Nk);
    load_tile<D>(sV, a.v, b, hk, k0, a.Nk);
    fill_window(a, h, k0 - (qs + q0) - (BT - 1), &win, &bad);
    __syncthreads();
    if (edge) clean_rows<D>(sV, bad_row);
    float s[4][4] = {};
    dot_tile<D>(s, sQ, sK, ty, tx);
    if (edge) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = k0 + tx + 16 * j;
        float th;
        const bool see = col >= vis[i].x && col < vis[i].y;
        s[i][j] = see ? score_of(a, slope, win, s[i][j], ty * 4 + i, tx + 16 * j, col - (qs + q0 + ty * 4 + i), &th)
                      : -INFINITY;
        if (edge && see && bad_row[tx + 16 * j]) nan_row[i] = true;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      mx = fmaxf(mx, m[i]);
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float alpha = expf(m[i] - ref);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = expf(s[i][j] - ref);
        sum += s[i][j];
        sP[(ty * 4 + i) * PS + tx + 16 * j] = s[i][j];
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[i] = l[i] * alpha + sum;
      m[i] = mx;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[i][c] *= alpha;
    }
    __syncthreads();
    mul_tile<D>(o, sP, sV, ty, tx);
  }
  if (bad) report_status(a.status, CALIBATT_E_CORRUPT);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned any = __ballot_sync(0xffffffffu, nan_row[i]) >> (threadIdx.x & 16);
    const int r = q0 + ty * 4 + i;
    if (r >= a.Nq) continue;
    if (slope != 0.f && l[i] != 0.f && score_far(vis[i], qs + r)) {
      l[i] = NAN;
      report_status(a.status, CALIBATT_E_UNSUPPORTED);
    }
    const float inv = (any & 0xffffu) ? NAN : l[i] == 0.f ? 0.f : 1.f / l[i];
    const float row_lse = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
    const size_t at = (static_cast<size_t>(b) * a.H + h) * a.Nq + r;
    if (a.parts > 1) {
      float* dst = a.part_o + (at * a.parts + sp) * D;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        store4(dst + tx * 4 + 64 * c, o[i][c * 4] * inv, o[i][c * 4 + 1] * inv, o[i][c * 4 + 2] * inv, o[i][c * 4 + 3] * inv);
      if (tx == 0) a.part_lse[at * a.parts + sp] = row_lse;
      continue;
    }
    float* dst = reinterpret_cast<float*>(a.o.p) + b * a.o.sb + h * a.o.sh + r * a.o.sn;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store4(dst + tx * 4 + 64 * c, o[i][c * 4] * inv, o[i][c * 4 + 1] * inv, o[i][c * 4 + 2] * inv, o[i][c * 4 + 3] * inv);
    if (tx == 0 && a.lse != nullptr)
      a.lse[at] = row_lse;
  }
}

// P and the two forms of dS of one score tile: dZ = P (dP - D) (what the bias
// gets) and dS = dZ (1 - tanh^2) scale (what the dot product gets).
template <int D>
__device__ __forceinline__ void grad_tile(const ScoreArgs& a, float slope, const Window& win, int q0, int k0, int qs,
                                          const int2 (&vis)[4],
                                          const float (&lse)[4], const float (&dd)[4], const float (&s)[4][4],
                                          const float (&dp)[4][4], int ty, int tx, float* sP, float* sZ, float* sS) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = k0 + tx + 16 * j, at = (ty * 4 + i) * PS + tx + 16 * j;
      float th, p = 0.f, dz = 0.f;
      if (col >= vis[i].x && col < vis[i].y) {
        const float z = score_of(a, slope, win, s[i][j], ty * 4 + i, tx + 16 * j, col - (qs + q0 + ty * 4 + i), &th);
        p = expf(z - lse[i]);
        dz = p * (dp[i][j] - dd[i]);
      } else {
        th = 0.f;
      }
      if (sP != nullptr) sP[at] = p;
      if (sZ != nullptr) sZ[at] = dz;
      sS[at] = dz * (1.f - th * th) * a.scale;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) k_score_dq_simt(const ScoreArgs a) {
  using S = SimtSmem<D>;
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm, *sO = sQ + S::IN, *sK = sO + S::IN, *sV = sK + S::IN, *sS = sV + S::IN, *sZ = sS + S::SC;
  float* diag = sZ + S::SC;        // [2 BT] sums of dZ over the diagonals of a tile
  float* acc_t = diag + 2 * BT;    // [n_buckets]
  __shared__ int bad_row[BT];
  __shared__ Window win;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int q0 = blockIdx.x / a.q_parts * BT, part = blockIdx.x % a.q_parts, h = blockIdx.y, b = blockIdx.z, hk = h / a.G;
  const int qb = q0 >> 7;
  const int4 t = score_tile(a, b, qb);
  const int qs = a.q_start[b];
  const float slope = a.slopes != nullptr ? a.slopes[h] : 0.f;
  int2 vis[4];
  float lse[4], dd[4], dq[4][D / 16] = {};
  bool bad = false;
  const size_t r0 = (static_cast<size_t>(b) * a.H + h) * a.nqb * 128 + q0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    vis[i] = score_row(a, b, q0 + ty * 4 + i);
    lse[i] = a.row_lse[r0 + ty * 4 + i];
    dd[i] = a.row_d[r0 + ty * 4 + i];
  }
  if (a.dtable != nullptr)
    for (int n = threadIdx.x; n < a.n_buckets; n += kThreads) acc_t[n] = 0.f;
  load_tile<D>(sQ, a.q, b, h, q0, a.Nq);
  load_tile<D>(sO, a.dout, b, h, q0, a.Nq);
  // this part's key tiles
  const int first = t.x / BT, tiles = max(0, (t.y + BT - 1) / BT - first), per = (tiles + a.q_parts - 1) / a.q_parts;
  const int end = min(t.y, (first + min(tiles, (part + 1) * per)) * BT);
  for (int k0 = (first + part * per) * BT; k0 < end; k0 += BT) {
    if (!score_kept(a, h, qb, k0 >> 7)) continue;
    const bool edge = k0 < t.z || k0 + BT > t.w;
    __syncthreads();
    load_tile<D>(sK, a.k, b, hk, k0, a.Nk);
    load_tile<D>(sV, a.v, b, hk, k0, a.Nk);
    fill_window(a, h, k0 - (qs + q0) - (BT - 1), &win, &bad);
    __syncthreads();
    float s[4][4] = {}, dp[4][4] = {};
    dot_tile<D>(s, sQ, sK, ty, tx);
    dot_tile<D>(dp, sO, sV, ty, tx);
    grad_tile<D>(a, slope, win, q0, k0, qs, vis, lse, dd, s, dp, ty, tx, nullptr, a.dtable ? sZ : nullptr, sS);
    __syncthreads();
    if (edge) {
      clean_rows<D>(sK, bad_row);   // the scores that read them are formed: a visible one is in dS as NaN
      __syncthreads();
    }
    mul_tile<D>(dq, sS, sK, ty, tx);
    if (a.dtable != nullptr) {
      // offset j - p of diagonal x: column - row = x - (BT - 1)
      // (two threads a diagonal: its upper and lower half, added in that order)
      const int x = threadIdx.x >> 1, low = threadIdx.x & 1;
      float v = 0.f;
      if (x < 2 * BT - 1) {
        const int r0 = max(0, BT - 1 - x), r1 = min(BT, 2 * BT - 1 - x), mid = (r0 + r1) / 2;
        for (int r = low ? mid : r0; r < (low ? r1 : mid); ++r) v += sZ[r * PS + r + x - (BT - 1)];
      }
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      if (x < 2 * BT - 1 && !low) diag[x] = v;
      __syncthreads();
      for (int n = threadIdx.x; n < a.n_buckets; n += kThreads) {
        float sum = 0.f;
#pragma unroll 8
        for (int d = 0; d < 2 * BT - 1; ++d) sum += win.bucket[d] == n ? diag[d] : 0.f;
        acc_t[n] += sum;
      }
    }
  }
  if (bad) report_status(a.status, CALIBATT_E_CORRUPT);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = q0 + ty * 4 + i;
    if (r >= a.Nq) continue;
    float* dst = a.q_parts > 1 ? a.part_q + (((static_cast<size_t>(part) * a.B + b) * a.H + h) * a.Nq + r) * D
                               : reinterpret_cast<float*>(a.dq.p) + b * a.dq.sb + h * a.dq.sh + r * a.dq.sn;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store4(dst + tx * 4 + 64 * c, dq[i][c * 4], dq[i][c * 4 + 1], dq[i][c * 4 + 2], dq[i][c * 4 + 3]);
  }
  if (a.dtable != nullptr) {
    __syncthreads();
    float* dst = a.part_table + ((static_cast<size_t>(b) * a.H + h) * a.table_tiles + blockIdx.x) * a.n_buckets;
    for (int n = threadIdx.x; n < a.n_buckets; n += kThreads) dst[n] = acc_t[n];
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) k_score_dkv_simt(const ScoreArgs a) {
  using S = SimtSmem<D>;
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm, *sO = sQ + S::IN, *sK = sO + S::IN, *sV = sK + S::IN, *sS = sV + S::IN, *sP = sS + S::SC;
  __shared__ int bad_row[BT];
  __shared__ Window win;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int k0 = blockIdx.x / a.kv_parts * BT, part = blockIdx.x % a.kv_parts, hk = blockIdx.y, b = blockIdx.z;
  const int qs = a.q_start[b];
  float dk[4][D / 16] = {}, dv[4][D / 16] = {};
  bool bad = false;
  load_tile<D>(sK, a.k, b, hk, k0, a.Nk);
  load_tile<D>(sV, a.v, b, hk, k0, a.Nk);
  // this part's (query head, query tile) pairs g nqt + q0 / 64
  const int nqt = (a.Nq + BT - 1) / BT;
  const long long units = static_cast<long long>(a.G) * nqt;
  const int u0 = static_cast<int>(units * part / a.kv_parts), u1 = static_cast<int>(units * (part + 1) / a.kv_parts);
  for (int g = u0 / nqt; g < a.G && g * nqt < u1; ++g) {
    const int h = hk * a.G + g;
    const float slope = a.slopes != nullptr ? a.slopes[h] : 0.f;
    for (int q0 = max(0, u0 - g * nqt) * BT; q0 < a.Nq && g * nqt + q0 / BT < u1; q0 += BT) {
      const int qb = q0 >> 7;
      const int4 t = score_tile(a, b, qb);
      if (t.x >= k0 + BT || t.y <= k0 || !score_kept(a, h, qb, k0 >> 7)) continue;
      const bool edge = k0 < t.z || k0 + BT > t.w;
      __syncthreads();
      load_tile<D>(sQ, a.q, b, h, q0, a.Nq);
      load_tile<D>(sO, a.dout, b, h, q0, a.Nq);
      fill_window(a, h, k0 - (qs + q0) - (BT - 1), &win, &bad);
      int2 vis[4];
      float lse[4], dd[4];
      const size_t r0 = (static_cast<size_t>(b) * a.H + h) * a.nqb * 128 + q0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vis[i] = score_row(a, b, q0 + ty * 4 + i);
        lse[i] = a.row_lse[r0 + ty * 4 + i];
        dd[i] = a.row_d[r0 + ty * 4 + i];
      }
      __syncthreads();
      float s[4][4] = {}, dp[4][4] = {};
      dot_tile<D>(s, sQ, sK, ty, tx);
      dot_tile<D>(dp, sO, sV, ty, tx);
      grad_tile<D>(a, slope, win, q0, k0, qs, vis, lse, dd, s, dp, ty, tx, sP, nullptr, sS);
      __syncthreads();
      if (edge) {
        clean_rows<D>(sQ, bad_row);
        clean_rows<D>(sO, bad_row);
        __syncthreads();
      }
      mul_tile_t<D>(dv, sP, sO, ty, tx);
      mul_tile_t<D>(dk, sS, sQ, ty, tx);
    }
  }
  if (bad) report_status(a.status, CALIBATT_E_CORRUPT);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = k0 + ty * 4 + i;
    if (r >= a.Nk) continue;
    float* pk = reinterpret_cast<float*>(a.dk.p) + b * a.dk.sb + hk * a.dk.sh + r * a.dk.sn;
    float* pv = reinterpret_cast<float*>(a.dv.p) + b * a.dv.sb + hk * a.dv.sh + r * a.dv.sn;
    if (a.kv_parts > 1) {
      const size_t one = static_cast<size_t>(a.B) * a.Hkv * a.Nk * D;
      pv = a.part_kv + 2 * part * one + ((static_cast<size_t>(b) * a.Hkv + hk) * a.Nk + r) * D;
      pk = pv + one;
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      store4(pk + tx * 4 + 64 * c, dk[i][c * 4], dk[i][c * 4 + 1], dk[i][c * 4 + 2], dk[i][c * 4 + 3]);
      store4(pv + tx * 4 + 64 * c, dv[i][c * 4], dv[i][c * 4 + 1], dv[i][c * 4 + 2], dv[i][c * 4 + 3]);
    }
  }
}

// The dynamic shared-memory limit is a per-device function attribute; setting
// it again is cheap against these kernels and needs no state.
template <typename K>
int set_smem(K kern, size_t bytes) {
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess)
    return check_launch("cudaFuncSetAttribute(score_simt)");
  return CALIBATT_OK;
}

template <int D>
int fwd(const ScoreArgs& a, cudaStream_t s) {
  using S = SimtSmem<D>;
  const size_t smem = (3 * S::IN + S::SC) * sizeof(float);
  if (int rc = set_smem(k_score_fwd_simt<D>, smem)) return rc;
  k_score_fwd_simt<D><<<dim3((a.Nq + BT - 1) / BT * a.splits, a.H, a.B), kThreads, smem, s>>>(a);
  count_launch();
  if (int rc = check_launch("k_score_fwd_simt")) return rc;
  return a.parts > 1 ? launch_score_join(a, D, CALIBATT_FP32, s) : CALIBATT_OK;
}

template <int D>
int bwd(const ScoreArgs& a, cudaStream_t s) {
  using S = SimtSmem<D>;
  const size_t smem_q = (4 * S::IN + 2 * S::SC + 2 * BT + a.n_buckets) * sizeof(float);
  const size_t smem_k = (4 * S::IN + 2 * S::SC) * sizeof(float);
  if (int rc = set_smem(k_score_dq_simt<D>, smem_q)) return rc;
  if (int rc = set_smem(k_score_dkv_simt<D>, smem_k)) return rc;
  k_score_dq_simt<D><<<dim3((a.Nq + BT - 1) / BT * a.q_parts, a.H, a.B), kThreads, smem_q, s>>>(a);
  k_score_dkv_simt<D><<<dim3((a.Nk + BT - 1) / BT * a.kv_parts, a.Hkv, a.B), kThreads, smem_k, s>>>(a);
  count_launch(2);
  if (int rc = check_launch("k_score_bwd_simt")) return rc;
  return launch_score_sum_parts(a, D, CALIBATT_FP32, s);
}

}  // namespace

// Splits of the key axis: two CTAs on each of 148 SMs, at least one key tile a split.
int score_splits_simt(int B, int H, int Nq, int Nk) {
  const long long tiles = static_cast<long long>(B) * H * ((Nq + BT - 1) / BT);
  return static_cast<int>(std::max<long long>(1, std::min<long long>(296 / tiles, (Nk + BT - 1) / BT)));
}

// Parts of the backward's walks: one CTA (by its shared memory) on each of 148
// SMs, at least one tile a part.
int score_q_parts_simt(int B, int H, int Nq, int Nk) {
  const long long tiles = static_cast<long long>(B) * H * ((Nq + BT - 1) / BT);
  return static_cast<int>(std::max<long long>(1, std::min<long long>(148 / tiles, (Nk + BT - 1) / BT)));
}
int score_kv_parts_simt(int B, int Hkv, int G, int Nq, int Nk) {
  const long long tiles = static_cast<long long>(B) * Hkv * ((Nk + BT - 1) / BT);
  return static_cast<int>(std::max<long long>(1, std::min<long long>(148 / tiles, static_cast<long long>(G) * ((Nq + BT - 1) / BT))));
}

int launch_score_fwd_simt(const ScoreArgs& a, int d, cudaStream_t s) { return d == 128 ? fwd<128>(a, s) : fwd<64>(a, s); }
int launch_score_bwd_simt(const ScoreArgs& a, int d, cudaStream_t s) { return d == 128 ? bwd<128>(a, s) : bwd<64>(a, s); }

}  // namespace calibatt
