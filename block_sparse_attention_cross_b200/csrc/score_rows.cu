// score_rows.cu -- the small kernels around the score-modified attention: the
// join of the forward's key splits, the sums of the backward's parts, the fp32
// backward's row terms, the sum of the table's gradient.
#include "score_common.cuh"

namespace calibatt {
namespace {

// Joins the partial results of a row: weights e^(lse_s - max), a lane D / 32
// columns.  WARPS = 4 (many parts): one CTA a row, warp w adds up the parts w,
// w + 4, ..., then the warps' sums are added in warp order; WARPS = 1 (up to 8
// parts): a warp a row (a CTA a row took longer than the forward for two parts
// of 12 640 rows).  A fixed order either way; reads the parts once.
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(128) k_score_join(const ScoreArgs a) {
  constexpr int C = D / 32;
  __shared__ float sums[WARPS == 4 ? 4 : 1][D], norm[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = WARPS == 4 ? warp : 0;
  const long long r = WARPS == 4 ? blockIdx.x : static_cast<long long>(blockIdx.x) * 4 + warp;
  if (r >= static_cast<long long>(a.B) * a.H * a.Nq) return;
  const float* pl = a.part_lse + r * a.parts;
  float mx = -INFINITY;
  for (int s = lane; s < a.parts; s += 32) mx = fmaxf(mx, pl[s]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  float acc[C] = {}, l = 0.f;
  // eight parts' loads in flight; a part that saw nothing has no partial O
  for (int s0 = w; s0 < a.parts; s0 += 8 * WARPS) {
    float x[8], po[8][C];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int s = min(s0 + WARPS * k, a.parts - 1);
      x[k] = s0 + WARPS * k < a.parts ? pl[s] : -INFINITY;
#pragma unroll
      for (int e = 0; e < C; ++e) po[k][e] = a.part_o[(r * a.parts + s) * D + lane * C + e];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (x[k] == -INFINITY) continue;
      const float wgt = expf(x[k] - mx);   // NaN stays NaN
      l += wgt;
#pragma unroll
      for (int e = 0; e < C; ++e) acc[e] = fmaf(wgt, po[k][e], acc[e]);
    }
  }
  if constexpr (WARPS == 4) {
#pragma unroll
    for (int e = 0; e < C; ++e) sums[w][lane * C + e] = acc[e];
    if (lane == 0) norm[w] = l;
    __syncthreads();
    if (w != 0) return;
    l = (norm[0] + norm[1]) + (norm[2] + norm[3]);
#pragma unroll
    for (int e = 0; e < C; ++e) {
      const int at = lane * C + e;
      acc[e] = (sums[0][at] + sums[1][at]) + (sums[2][at] + sums[3][at]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int i = static_cast<int>(r % a.Nq);
  const int bh = static_cast<int>(r / a.Nq), b = bh / a.H, h = bh % a.H;
  T* op = reinterpret_cast<T*>(a.o.p) + b * a.o.sb + h * a.o.sh + i * a.o.sn + lane * C;
#pragma unroll
  for (int e = 0; e < C; e += 2) {
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t*>(op + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    else *reinterpret_cast<float2*>(op + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
  }
  if (lane == 0 && a.lse != nullptr) a.lse[r] = l == 0.f ? -INFINITY : mx + logf(l);
}

template <typename T, int D>
void launch_join(const ScoreArgs& a, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.B) * a.H * a.Nq;   // below 2^31
  if (a.parts > 8) k_score_join<T, D, 4><<<static_cast<unsigned>(rows), 128, 0, s>>>(a);
  else k_score_join<T, D, 1><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, s>>>(a);
}

// fp32: D_i = sum over d of dO_i O_i, and the row's LSE as the backward
// kernels read it: +inf where the row sees nothing (every probability becomes
// 0), NaN where D is not finite (so that a row with a non-finite dO or O marks
// every gradient it enters).  One warp a row: reads dO and O once, DRAM-bound.
template <int D>
__global__ void __launch_bounds__(256) k_score_rows(const ScoreArgs a) {
  const long long rows = 128ll * a.nqb;
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (w >= rows * a.B * a.H) return;
  const int lane = threadIdx.x & 31;
  const int bh = static_cast<int>(w / rows), i = static_cast<int>(w % rows);
  const int b = bh / a.H, h = bh % a.H;
  float sum = 0.f, lse = INFINITY;
  const int2 r = score_row(a, b, i);
  if (r.x < r.y) {
    const float* po = reinterpret_cast<const float*>(a.o.p) + b * a.o.sb + h * a.o.sh + i * a.o.sn;
    const float* pd = reinterpret_cast<const float*>(a.dout.p) + b * a.dout.sb + h * a.dout.sh + i * a.dout.sn;
#pragma unroll
    for (int x = lane; x < D; x += 32) sum = fmaf(po[x], pd[x], sum);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    lse = a.lse[static_cast<size_t>(bh) * a.Nq + i];
    if (lse == -INFINITY) { lse = INFINITY; sum = 0.f; }
    else if (!isfinite(sum)) lse = NAN;
  }
  if (lane == 0) {
    a.row_lse[w] = lse;
    a.row_d[w] = sum;
  }
}

// A gradient from its parts' fp32 sums [parts, B, heads, N, d], added in part
// order; a thread four columns of a row.  Reads the parts once.
template <typename T, int D>
__global__ void __launch_bounds__(256)
    k_score_sum_parts(const float* part, int parts, long long stride, Tensor4 out, int B, int heads, int N) {
  const long long x = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long row = x / (D / 4);
  const int col = static_cast<int>(x % (D / 4)) * 4;
  if (row >= static_cast<long long>(B) * heads * N) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < parts; ++p) {
    const float4 v = *reinterpret_cast<const float4*>(part + p * stride + row * D + col);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  const int j = static_cast<int>(row % N);
  const int bh = static_cast<int>(row / N), b = bh / heads, h = bh % heads;
  T* dst = reinterpret_cast<T*>(out.p) + b * out.sb + h * out.sh + static_cast<long long>(j) * out.sn + col;
  if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  else *reinterpret_cast<float4*>(dst) = s;
}

template <typename T, int D>
void sum_parts(const float* part, int parts, long long stride, const Tensor4& out, int B, int heads, int N, cudaStream_t s) {
  const long long quads = static_cast<long long>(B) * heads * N * (D / 4);
  k_score_sum_parts<T, D><<<static_cast<unsigned>((quads + 255) / 256), 256, 0, s>>>(part, parts, stride, out, B, heads, N);
  count_launch();
}

template <typename T, int D>
void sum_all(const ScoreArgs& a, cudaStream_t s) {
  if (a.q_parts > 1)
    sum_parts<T, D>(a.part_q, a.q_parts, static_cast<long long>(a.B) * a.H * a.Nq * D, a.dq, a.B, a.H, a.Nq, s);
  if (a.kv_parts > 1) {
    const long long one = static_cast<long long>(a.B) * a.Hkv * a.Nk * D;   // [parts, 2 (dV, dK), ...]
    sum_parts<T, D>(a.part_kv, a.kv_parts, 2 * one, a.dv, a.B, a.Hkv, a.Nk, s);
    sum_parts<T, D>(a.part_kv + one, a.kv_parts, 2 * one, a.dk, a.B, a.Hkv, a.Nk, s);
  }
}

// Gradient of the bias table: the partial sums of every (batch entry, query
// tile) of a head, added in a fixed order in double.  One CTA per (head,
// bucket).
template <typename T>
__global__ void __launch_bounds__(128) k_score_table_sum(const ScoreArgs a) {
  const int h = blockIdx.y, n = blockIdx.x;
  const int tiles = a.B * a.table_tiles;
  double s = 0.0;
  for (int t = threadIdx.x; t < tiles; t += 128) {
    const int b = t / a.table_tiles, q = t % a.table_tiles;
    s += a.part_table[((static_cast<size_t>(b) * a.H + h) * a.table_tiles + q) * a.n_buckets + n];
  }
  __shared__ double red[128];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int m = 64; m > 0; m >>= 1) {
    if (threadIdx.x < m) red[threadIdx.x] += red[threadIdx.x + m];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const float r = static_cast<float>(red[0]);
    if constexpr (sizeof(T) == 2) reinterpret_cast<__nv_bfloat16*>(a.dtable)[h * a.n_buckets + n] = __float2bfloat16(r);
    else reinterpret_cast<float*>(a.dtable)[h * a.n_buckets + n] = r;
  }
}

}  // namespace

int launch_score_join(const ScoreArgs& a, int d, int dtype, cudaStream_t s) {
  if (dtype == CALIBATT_BF16) d == 128 ? launch_join<__nv_bfloat16, 128>(a, s) : launch_join<__nv_bfloat16, 64>(a, s);
  else d == 128 ? launch_join<float, 128>(a, s) : launch_join<float, 64>(a, s);
  count_launch();
  return check_launch("k_score_join");
}

int launch_score_sum_parts(const ScoreArgs& a, int d, int dtype, cudaStream_t s) {
  if (dtype == CALIBATT_BF16) d == 128 ? sum_all<__nv_bfloat16, 128>(a, s) : sum_all<__nv_bfloat16, 64>(a, s);
  else d == 128 ? sum_all<float, 128>(a, s) : sum_all<float, 64>(a, s);
  return check_launch("k_score_sum_parts");
}

int launch_score_rows(const ScoreArgs& a, int d, cudaStream_t s) {
  const long long rows = 128ll * a.nqb * a.B * a.H;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (d == 128) k_score_rows<128><<<grid, 256, 0, s>>>(a);
  else k_score_rows<64><<<grid, 256, 0, s>>>(a);
  count_launch();
  return check_launch("k_score_rows");
}

int launch_score_table_sum(const ScoreArgs& a, int dtype, cudaStream_t s) {
  const dim3 grid(a.n_buckets, a.H);
  if (dtype == CALIBATT_BF16) k_score_table_sum<__nv_bfloat16><<<grid, 128, 0, s>>>(a);
  else k_score_table_sum<float><<<grid, 128, 0, s>>>(a);
  count_launch();
  return check_launch("k_score_table_sum");
}

}  // namespace calibatt
