// score_plan.cu -- visible key intervals of the score-modified attention.
//
// Packed documents, a causal rule, a prefix that everybody of the document
// sees and padded lengths all leave every query row one interval of keys, so
// a mask is two integers a row instead of a matrix, and a tile of rows knows
// from four integers which key tiles it can skip (outside [min lo, max hi))
// and which need no element mask (inside [max lo, min hi)).
#include <climits>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace calibatt {
namespace {

constexpr int kTile = 128;

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// One CTA per (query tile, batch entry), one thread per row; latency-bound
// (a few integer loads and a binary search a row), made once per batch layout.
__global__ void __launch_bounds__(kTile)
    k_attn_spans(int Nq, int Nk, int nqb, int causal, const int32_t* docs, int n_docs, const int32_t* prefix,
                 const int32_t* kv_len, const int32_t* q_len, const int32_t* q_start, int2* row, int4* tile,
                 int32_t* q_start_out) {
  const int b = blockIdx.y;
  const int i = blockIdx.x * kTile + threadIdx.x;
  // Lengths and positions from device memory are clamped, so that no content
  // can lead outside [0, Nk).
  const int kv = kv_len ? clampi(kv_len[b], 0, Nk) : Nk;
  const int nq = q_len ? clampi(q_len[b], 0, Nq) : Nq;
  const int qs = q_start ? clampi(q_start[b], -(1 << 30), 1 << 30) : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) q_start_out[b] = qs;
  int lo = 0, hi = 0;
  if (i < nq) {
    const int p = qs + i;
    int s = 0, e = kv, m = 0;
    bool in = true;
    if (docs != nullptr) {
      const int32_t* bd = docs + static_cast<size_t>(b) * (n_docs + 1);
      int l = 0, r = n_docs + 1;   // first bound above p
      while (l < r) {
        const int mid = (l + r) >> 1;
        if (bd[mid] <= p) l = mid + 1; else r = mid;
      }
      m = l - 1;
      in = m >= 0 && m < n_docs;
      if (in) {
        s = clampi(bd[m], 0, Nk);
        e = min(clampi(bd[m + 1], 0, Nk), kv);
      }
      m = clampi(m, 0, n_docs - 1);
    }
    if (in) {
      if (causal) {
        const int pre = prefix ? clampi(prefix[static_cast<size_t>(b) * max(n_docs, 1) + m], 0, Nk) : 0;
        e = min(e, max(p + 1, s + pre));
      }
      if (e > s) { lo = s; hi = e; }
    }
  }
  if (i < Nq) row[static_cast<size_t>(b) * Nq + i] = make_int2(lo, hi);
  // Rows past Nq do not count; a row that sees nothing makes every key tile
  // of its query tile one that needs the element mask (max lo = Nk).
  const bool some = hi > lo;
  __shared__ int red[4][4];
  int v0 = some ? lo : INT_MAX, v1 = some ? hi : 0;
  int v2 = i >= Nq ? 0 : some ? lo : Nk, v3 = i >= Nq ? INT_MAX : some ? hi : 0;
  v0 = __reduce_min_sync(0xffffffffu, v0);
  v1 = __reduce_max_sync(0xffffffffu, v1);
  v2 = __reduce_max_sync(0xffffffffu, v2);
  v3 = __reduce_min_sync(0xffffffffu, v3);
  if ((threadIdx.x & 31) == 0) {
    const int w = threadIdx.x >> 5;
    red[w][0] = v0; red[w][1] = v1; red[w][2] = v2; red[w][3] = v3;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int4 t = make_int4(red[0][0], red[0][1], red[0][2], red[0][3]);
    for (int w = 1; w < 4; ++w) {
      t.x = min(t.x, red[w][0]);
      t.y = max(t.y, red[w][1]);
      t.z = max(t.z, red[w][2]);
      t.w = min(t.w, red[w][3]);
    }
    if (t.y <= 0) t.x = 0;   // no row of the tile sees a key: an empty range
    tile[static_cast<size_t>(b) * nqb + blockIdx.x] = t;
  }
}

}  // namespace

int launch_attn_spans(int B, int Nq, int Nk, int causal, const int32_t* docs, int n_docs, const int32_t* prefix,
                      const int32_t* kv_len, const int32_t* q_len, const int32_t* q_start, int2* row, int4* tile,
                      int32_t* q_start_out, cudaStream_t s) {
  const int nqb = (Nq + kTile - 1) / kTile;
  k_attn_spans<<<dim3(nqb, B), kTile, 0, s>>>(Nq, Nk, nqb, causal, docs, n_docs, prefix, kv_len, q_len, q_start, row,
                                              tile, q_start_out);
  count_launch();
  return check_launch("k_attn_spans");
}

}  // namespace calibatt
