// score_api.cu -- the extern "C" entry points of the score-modified attention:
// argument checks, workspace layout and dispatch.  Nothing here allocates
// device memory.
#include <algorithm>
#include <cmath>
#include <utility>

#include "common.cuh"
#include "internal.h"

using namespace calibatt;

namespace {

constexpr int kMaxBuckets = 256;
constexpr int kMaxDistance = 1 << 20;
constexpr long long kMaxLen = 1ll << 24;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// A [B, heads, N, d] tensor: 16-byte aligned rows, positive strides wherever a
// dimension has more than one entry (strides of single entries are not used).
int check_tensor(const char* name, const calibatt_tensor4* t, int B, int heads, int N, int d, int esz) {
  if (t == nullptr || t->ptr == nullptr) return set_error(CALIBATT_E_INVALID, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(t->ptr) & 15u) != 0)
    return set_error(CALIBATT_E_INVALID, "%s must be 16-byte aligned", name);
  const int64_t st[3] = {t->stride_b, t->stride_h, t->stride_n};
  const int len[3] = {B, heads, N};
  for (int i = 0; i < 3; ++i) {
    if (len[i] == 1) continue;
    if (st[i] <= 0 || (st[i] * esz) % 16 != 0 || st[i] >= (1ll << 38))
      return set_error(CALIBATT_E_INVALID, "%s: strides must be positive multiples of 16 bytes", name);
  }
  if (N > 1 && t->stride_n < d) return set_error(CALIBATT_E_INVALID, "%s: rows overlap", name);
  return CALIBATT_OK;
}

// An output: its rows may not overlap one another either.
int check_output(const char* name, const calibatt_tensor4* t, int B, int heads, int N, int d, int esz) {
  if (int rc = check_tensor(name, t, B, heads, N, d, esz)) return rc;
  std::pair<int64_t, int> dims[3] = {{t->stride_b, B}, {t->stride_h, heads}, {t->stride_n, N}};
  std::sort(dims, dims + 3);
  int64_t extent = d;
  for (const auto& x : dims) {
    if (x.second == 1) continue;
    if (x.first < extent) return set_error(CALIBATT_E_INVALID, "%s: output rows overlap", name);
    extent = x.first * x.second;
  }
  return CALIBATT_OK;
}

Tensor4 to_tensor(const calibatt_tensor4* t, int B, int heads, int N, int d) {
  Tensor4 r;
  r.p = t->ptr;
  r.sn = N == 1 ? d : t->stride_n;
  r.sh = heads == 1 ? r.sn * N : t->stride_h;
  r.sb = B == 1 ? r.sh * heads : t->stride_b;
  return r;
}

// Sizes, spans and score terms, shared by the forward and the backward and by
// their workspace queries; fills the fields of `a` that do not depend on tensors.
int check_sizes(int B, int H, int Hkv, int Nq, int Nk, int d, int dtype) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || Nq <= 0 || Nk <= 0 || H % Hkv != 0)
    return set_error(CALIBATT_E_INVALID, "bad sizes B=%d H=%d Hkv=%d Nq=%d Nk=%d", B, H, Hkv, Nq, Nk);
  if (dtype != CALIBATT_BF16 && dtype != CALIBATT_FP32)
    return set_error(CALIBATT_E_UNSUPPORTED, "unknown dtype %d", dtype);
  if (d != 64 && d != 128) return set_error(CALIBATT_E_UNSUPPORTED, "d must be 64 or 128");
  if (B > 65535 || H > 65535 || Nq > kMaxLen || Nk > kMaxLen)
    return set_error(CALIBATT_E_UNSUPPORTED, "B and H up to 65535, Nq and Nk up to 2^24");
  if (static_cast<long long>(B) * H * (std::max(Nq, Nk) + 128ll) >= (1ll << 31))
    return set_error(CALIBATT_E_UNSUPPORTED, "B * H * N must be below 2^31 rows");
  return CALIBATT_OK;
}

int check_score(ScoreArgs& a, int B, int H, int Hkv, int Nq, int Nk, int d, int dtype, const calibatt_spans* sp,
                const calibatt_score* sc) {
  if (int rc = check_sizes(B, H, Hkv, Nq, Nk, d, dtype)) return rc;
  if (sp == nullptr || sp->row == nullptr || sp->tile == nullptr || sp->q_start == nullptr)
    return set_error(CALIBATT_E_INVALID, "spans are NULL");
  if (sp->B != B || sp->Nq != Nq || sp->Nk != Nk)
    return set_error(CALIBATT_E_INVALID, "spans of B=%d Nq=%d Nk=%d do not match B=%d Nq=%d Nk=%d", sp->B, sp->Nq,
                     sp->Nk, B, Nq, Nk);
  if (((reinterpret_cast<uintptr_t>(sp->row) & 7u) | (reinterpret_cast<uintptr_t>(sp->tile) & 15u)) != 0)
    return set_error(CALIBATT_E_INVALID, "spans are not aligned (row 8 bytes, tile 16 bytes)");
  if (sc == nullptr) return set_error(CALIBATT_E_INVALID, "score is NULL");
  if (!(sc->scale > 0.f) || !std::isfinite(sc->scale))
    return set_error(CALIBATT_E_INVALID, "scale must be finite and > 0");
  if (!(sc->cap >= 0.f) || !std::isfinite(sc->cap))
    return set_error(CALIBATT_E_INVALID, "cap must be finite and >= 0 (0: no cap)");
  if (!std::isfinite(sc->scale * 4.f) || (sc->cap > 0.f && (!std::isfinite(sc->cap * 4.f) || !std::isfinite(4.f * sc->scale / sc->cap))))
    return set_error(CALIBATT_E_INVALID, "scale, cap and scale / cap must stay below a quarter of the fp32 range");
  if ((sc->table == nullptr) != (sc->buckets == nullptr))
    return set_error(CALIBATT_E_INVALID, "table and buckets come together");
  if (sc->table != nullptr) {
    if (sc->n_buckets < 1 || sc->max_distance < 0) return set_error(CALIBATT_E_INVALID, "bad bucket sizes");
    if (sc->n_buckets > kMaxBuckets || sc->max_distance > kMaxDistance)
      return set_error(CALIBATT_E_UNSUPPORTED, "at most %d buckets and a distance of 2^20", kMaxBuckets);
  }
  a = ScoreArgs{};
  a.B = B; a.H = H; a.Hkv = Hkv; a.G = H / Hkv; a.Nq = Nq; a.Nk = Nk;
  a.nqb = (Nq + 127) / 128;
  a.nkb = (Nk + 127) / 128;
  if (sc->mask != nullptr && (sc->map_offset < 0 || static_cast<long long>(sc->map_offset) + H > sc->n_maps))
    return set_error(CALIBATT_E_INVALID, "map_offset %d + H %d exceeds n_maps %d", sc->map_offset, H, sc->n_maps);
  a.scale = sc->scale; a.cap = sc->cap; a.slopes = sc->slopes;
  a.table = sc->table; a.buckets = sc->buckets; a.n_buckets = sc->n_buckets; a.R = sc->max_distance;
  a.mask = sc->mask; a.map_offset = sc->map_offset;
  a.row = reinterpret_cast<const int2*>(sp->row);
  a.tile = reinterpret_cast<const int4*>(sp->tile);
  a.q_start = sp->q_start;
  a.spin_ns = std::min<uint64_t>(spin_limit_ns(), 1ull << 57);   // the window warps' waits take a multiple of it
  return CALIBATT_OK;
}

// Forward workspace: [part_o][part_lse].
size_t fwd_layout(ScoreArgs& a, int d, void* ws) {
  if (a.parts <= 1) return 0;
  char* p = static_cast<char*>(ws);
  const size_t rows = static_cast<size_t>(a.B) * a.H * a.Nq * a.parts;
  a.part_o = reinterpret_cast<float*>(p);
  const size_t off = align256(rows * d * 4);
  a.part_lse = reinterpret_cast<float*>(p + off);
  return off + align256(rows * 4);
}

void fwd_plan(ScoreArgs& a, bool packed) {
  a.packed = packed;
  a.few = packed && a.G * a.Nq <= 32;
  a.splits = score_splits(a.B, packed ? a.Hkv : a.H, packed ? 1 : a.nqb, a.nkb);
  a.parts = a.few ? 4 * a.splits : a.splits;
}

// Backward workspace: [row_lse][row_d][row_span][part_kv][part_q][part_table], 256-byte aligned pieces.
size_t bwd_layout(ScoreArgs& a, int d, int dtype, void* ws) {
  char* p = static_cast<char*>(ws);
  size_t off = 0;
  const size_t rows = static_cast<size_t>(a.B) * a.H * a.nqb * 128;
  a.row_lse = reinterpret_cast<float*>(p + off);
  off += align256(rows * 4);
  a.row_d = reinterpret_cast<float*>(p + off);
  off += align256(rows * 4);
  if (dtype == CALIBATT_BF16) {
    a.row_span = reinterpret_cast<int2*>(p + off);
    off += align256(static_cast<size_t>(a.B) * a.nqb * 128 * 8);
    a.kv_parts = score_kv_parts(a.B, a.Hkv, a.G, a.nqb, a.nkb);
    a.q_parts = 1;
  } else {
    a.kv_parts = score_kv_parts_simt(a.B, a.Hkv, a.G, a.Nq, a.Nk);
    a.q_parts = score_q_parts_simt(a.B, a.H, a.Nq, a.Nk);
  }
  if (a.kv_parts > 1) {
    a.part_kv = reinterpret_cast<float*>(p + off);
    off += align256(static_cast<size_t>(a.kv_parts) * 2 * a.B * a.Hkv * a.Nk * d * 4);
  }
  if (a.q_parts > 1) {
    a.part_q = reinterpret_cast<float*>(p + off);
    off += align256(static_cast<size_t>(a.q_parts) * a.B * a.H * a.Nq * d * 4);
  }
  if (a.dtable != nullptr) {
    a.table_tiles = dtype == CALIBATT_BF16 ? a.nqb : (a.Nq + 63) / 64 * a.q_parts;
    a.part_table = reinterpret_cast<float*>(p + off);
    off += align256(static_cast<size_t>(a.B) * a.H * a.table_tiles * a.n_buckets * 4);
  }
  return off;
}

}  // namespace

extern "C" {

int calibatt_relative_buckets(int n_buckets, int max_distance, int bidirectional, int32_t* out) {
  if (out == nullptr) return set_error(CALIBATT_E_INVALID, "out is NULL");
  const int half = bidirectional ? n_buckets / 2 : n_buckets;
  const int exact = half / 2;
  if (n_buckets > kMaxBuckets || max_distance > kMaxDistance)
    return set_error(CALIBATT_E_UNSUPPORTED, "at most %d buckets and a distance of 2^20", kMaxBuckets);
  if ((bidirectional && n_buckets % 2 != 0) || exact < 1 || max_distance <= exact)
    return set_error(CALIBATT_E_INVALID, "n_buckets=%d (bidirectional: even) must leave exact buckets and max_distance=%d"
                     " must exceed them", n_buckets, max_distance);
  // The logarithm is nudged up by less than the distance of any other integer
  // from a bucket border, so that a distance exactly on a border (a power of
  // the ratio) belongs to the upper bucket whatever the rounding of log.
  const double ratio = std::log(static_cast<double>(max_distance) / exact);
  for (int off = -max_distance; off <= max_distance; ++off) {
    const int dist = off < 0 ? -off : off;
    int n = dist;
    if (dist >= exact)
      n = exact + static_cast<int>(std::floor((half - exact) * std::log(static_cast<double>(dist) / exact) / ratio + 1e-9));
    n = std::min(n, half - 1);
    if (bidirectional) n += off > 0 ? half : 0;
    else if (off > 0) n = 0;
    out[off + max_distance] = n;
  }
  return CALIBATT_OK;
}

int calibatt_attn_spans(int B, int Nq, int Nk, int causal, const int32_t* docs, int n_docs, const int32_t* prefix,
                        const int32_t* kv_len, const int32_t* q_len, const int32_t* q_start, int32_t* row_out,
                        int32_t* tile_out, int32_t* q_start_out, calibatt_stream_t stream) {
  if (B <= 0 || Nq <= 0 || Nk <= 0 || B > 65535 || Nq > kMaxLen || Nk > kMaxLen)
    return set_error(CALIBATT_E_INVALID, "bad sizes B=%d Nq=%d Nk=%d", B, Nq, Nk);
  if ((docs == nullptr) != (n_docs == 0) || n_docs < 0 || n_docs > (1 << 24))
    return set_error(CALIBATT_E_INVALID, "docs and n_docs come together");
  if (prefix != nullptr && !causal) return set_error(CALIBATT_E_INVALID, "a prefix needs the causal rule");
  if (row_out == nullptr || tile_out == nullptr || q_start_out == nullptr)
    return set_error(CALIBATT_E_INVALID, "outputs are NULL");
  if (((reinterpret_cast<uintptr_t>(row_out) & 7u) | (reinterpret_cast<uintptr_t>(tile_out) & 15u)) != 0)
    return set_error(CALIBATT_E_INVALID, "outputs are not aligned (row 8 bytes, tile 16 bytes)");
  return launch_attn_spans(B, Nq, Nk, causal != 0, docs, n_docs, prefix, kv_len, q_len, q_start,
                           reinterpret_cast<int2*>(row_out), reinterpret_cast<int4*>(tile_out), q_start_out,
                           reinterpret_cast<cudaStream_t>(stream));
}

int calibatt_score_attn_fwd_workspace_size(int B, int H, int Hkv, int Nq, int Nk, int d, int dtype, size_t* bytes) {
  if (bytes == nullptr) return set_error(CALIBATT_E_INVALID, "bytes is NULL");
  if (int rc = check_sizes(B, H, Hkv, Nq, Nk, d, dtype)) return rc;
  *bytes = 0;
  // enough for every score function and mask of these sizes
  ScoreArgs a{};
  a.B = B; a.H = H; a.Hkv = Hkv; a.G = H / Hkv; a.Nq = Nq; a.nqb = (Nq + 127) / 128; a.nkb = (Nk + 127) / 128;
  if (dtype == CALIBATT_FP32) {
    a.splits = a.parts = score_splits_simt(B, H, Nq, Nk);
    *bytes = fwd_layout(a, d, nullptr);
    return CALIBATT_OK;
  }
  for (int packed = 0; packed < 2; ++packed) {
    if (packed && !score_packs(a.G, Nq, false, false)) continue;
    fwd_plan(a, packed != 0);
    *bytes = std::max(*bytes, fwd_layout(a, d, nullptr));
  }
  return CALIBATT_OK;
}

int calibatt_score_attn_fwd(const calibatt_tensor4* q, const calibatt_tensor4* k, const calibatt_tensor4* v,
                            const calibatt_tensor4* o, float* lse, int B, int H, int Hkv, int Nq, int Nk, int d,
                            int dtype, const calibatt_spans* spans, const calibatt_score* score, void* workspace,
                            size_t workspace_bytes, int32_t* dev_status, calibatt_stream_t stream) {
  ScoreArgs a;
  if (int rc = check_score(a, B, H, Hkv, Nq, Nk, d, dtype, spans, score)) return rc;
  const int esz = dtype == CALIBATT_BF16 ? 2 : 4;
  int rc;
  if ((rc = check_tensor("q", q, B, H, Nq, d, esz)) || (rc = check_tensor("k", k, B, Hkv, Nk, d, esz)) ||
      (rc = check_tensor("v", v, B, Hkv, Nk, d, esz)) || (rc = check_output("o", o, B, H, Nq, d, esz)))
    return rc;
  a.q = to_tensor(q, B, H, Nq, d);
  a.k = to_tensor(k, B, Hkv, Nk, d);
  a.v = to_tensor(v, B, Hkv, Nk, d);
  a.o = to_tensor(o, B, H, Nq, d);
  a.lse = lse;
  a.status = dev_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == CALIBATT_FP32) a.splits = a.parts = score_splits_simt(B, H, Nq, Nk);
  else fwd_plan(a, score_packs(a.G, Nq, a.mask != nullptr, a.table != nullptr));
  const size_t need = fwd_layout(a, d, workspace);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
    return set_error(CALIBATT_E_WORKSPACE, "workspace of %zu bytes (256-byte aligned) needed, %zu given", need,
                     workspace_bytes);
  return dtype == CALIBATT_FP32 ? launch_score_fwd_simt(a, d, s) : launch_score_fwd_tc(a, d, s);
}

int calibatt_score_attn_bwd_workspace_size(int B, int H, int Hkv, int Nq, int Nk, int d, int dtype, int n_buckets,
                                           size_t* bytes) {
  if (bytes == nullptr) return set_error(CALIBATT_E_INVALID, "bytes is NULL");
  if (int rc = check_sizes(B, H, Hkv, Nq, Nk, d, dtype)) return rc;
  if (n_buckets < 0 || n_buckets > kMaxBuckets) return set_error(CALIBATT_E_INVALID, "bad n_buckets %d", n_buckets);
  ScoreArgs a{};
  a.B = B; a.H = H; a.Hkv = Hkv; a.G = H / Hkv; a.Nq = Nq; a.Nk = Nk;
  a.nqb = (Nq + 127) / 128; a.nkb = (Nk + 127) / 128; a.n_buckets = n_buckets;
  a.dtable = n_buckets > 0 ? bytes : nullptr;   // only whether it is set matters here
  *bytes = bwd_layout(a, d, dtype, nullptr);
  return CALIBATT_OK;
}

int calibatt_score_attn_bwd(const calibatt_tensor4* dout, const calibatt_tensor4* q, const calibatt_tensor4* k,
                            const calibatt_tensor4* v, const calibatt_tensor4* o, const float* lse,
                            const calibatt_tensor4* dq, const calibatt_tensor4* dk, const calibatt_tensor4* dv,
                            void* dtable, int B, int H, int Hkv, int Nq, int Nk, int d, int dtype,
                            const calibatt_spans* spans, const calibatt_score* score, void* workspace,
                            size_t workspace_bytes, int32_t* dev_status, calibatt_stream_t stream) {
  ScoreArgs a;
  if (int rc = check_score(a, B, H, Hkv, Nq, Nk, d, dtype, spans, score)) return rc;
  const int esz = dtype == CALIBATT_BF16 ? 2 : 4;
  int rc;
  if ((rc = check_tensor("dout", dout, B, H, Nq, d, esz)) || (rc = check_tensor("q", q, B, H, Nq, d, esz)) ||
      (rc = check_tensor("k", k, B, Hkv, Nk, d, esz)) || (rc = check_tensor("v", v, B, Hkv, Nk, d, esz)) ||
      (rc = check_tensor("o", o, B, H, Nq, d, esz)) || (rc = check_output("dq", dq, B, H, Nq, d, esz)) ||
      (rc = check_output("dk", dk, B, Hkv, Nk, d, esz)) || (rc = check_output("dv", dv, B, Hkv, Nk, d, esz)))
    return rc;
  if (lse == nullptr) return set_error(CALIBATT_E_INVALID, "lse is NULL");
  if (dtable != nullptr && a.table == nullptr)
    return set_error(CALIBATT_E_INVALID, "the gradient of a table needs the table");
  a.dout = to_tensor(dout, B, H, Nq, d);
  a.q = to_tensor(q, B, H, Nq, d);
  a.k = to_tensor(k, B, Hkv, Nk, d);
  a.v = to_tensor(v, B, Hkv, Nk, d);
  a.o = to_tensor(o, B, H, Nq, d);
  a.dq = to_tensor(dq, B, H, Nq, d);
  a.dk = to_tensor(dk, B, Hkv, Nk, d);
  a.dv = to_tensor(dv, B, Hkv, Nk, d);
  a.lse = const_cast<float*>(lse);
  a.dtable = dtable;
  a.status = dev_status;
  const size_t need = bwd_layout(a, d, dtype, workspace);
  if (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return set_error(CALIBATT_E_WORKSPACE, "workspace of %zu bytes (256-byte aligned) needed, %zu given", need,
                     workspace_bytes);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == CALIBATT_BF16) rc = launch_score_bwd_tc(a, d, s);
  else if ((rc = launch_score_rows(a, d, s)) == CALIBATT_OK) rc = launch_score_bwd_simt(a, d, s);
  if (rc) return rc;
  return dtable != nullptr ? launch_score_table_sum(a, dtype, s) : CALIBATT_OK;
}

}  // extern "C"
