// score_rows.cu -- the small kernels around the score-modified attention: the
// join of the forward's key splits, the fp32 backward's row terms, the sum of
// the table's gradient.
#include "score_common.cuh"

namespace calibatt {
namespace {

// Joins the partial results of a row: weights e^(lse_s - max).  One CTA a row;
// warp w adds up the parts w, w + 4, ... (a lane D / 32 columns), then the
// warps' sums are added in warp order: a fixed order.  Reads the partial
// results once.
template <typename T, int D>
__global__ void __launch_bounds__(128) k_score_join(const ScoreArgs a) {
  constexpr int C = D / 32;
  __shared__ float sums[4][D], norm[4];
  const long long r = blockIdx.x;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const float* pl = a.part_lse + r * a.parts;
  float mx = -INFINITY;
  for (int s = lane; s < a.parts; s += 32) mx = fmaxf(mx, pl[s]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  float acc[C] = {}, l = 0.f;
  // eight parts' loads in flight; a part that saw nothing has no partial O
  for (int s0 = w; s0 < a.parts; s0 += 32) {
    float x[8], po[8][C];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int s = min(s0 + 4 * k, a.parts - 1);
      x[k] = s0 + 4 * k < a.parts ? pl[s] : -INFINITY;
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
#pragma unroll
  for (int e = 0; e < C; ++e) sums[w][lane * C + e] = acc[e];
  if (lane == 0) norm[w] = l;
  __syncthreads();
  l = (norm[0] + norm[1]) + (norm[2] + norm[3]);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int i = static_cast<int>(r % a.Nq);
  const int bh = static_cast<int>(r / a.Nq), b = bh / a.H, h = bh % a.H;
  T* op = reinterpret_cast<T*>(a.o.p) + b * a.o.sb + h * a.o.sh + i * a.o.sn;
  if (threadIdx.x < D / 2) {
    const int e = threadIdx.x * 2;
    const float x = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
    const float y = (sums[0][e + 1] + sums[1][e + 1]) + (sums[2][e + 1] + sums[3][e + 1]);
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t*>(op + e) = pack_bf16x2(x * inv, y * inv);
    else *reinterpret_cast<float2*>(op + e) = make_float2(x * inv, y * inv);
  }
  if (threadIdx.x == 0 && a.lse != nullptr) a.lse[r] = l == 0.f ? -INFINITY : mx + logf(l);
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
  const unsigned rows = static_cast<unsigned>(static_cast<long long>(a.B) * a.H * a.Nq);   // below 2^31
  if (dtype == CALIBATT_BF16) {
    if (d == 128) k_score_join<__nv_bfloat16, 128><<<rows, 128, 0, s>>>(a);
    else k_score_join<__nv_bfloat16, 64><<<rows, 128, 0, s>>>(a);
  } else {
    if (d == 128) k_score_join<float, 128><<<rows, 128, 0, s>>>(a);
    else k_score_join<float, 64><<<rows, 128, 0, s>>>(a);
  }
  count_launch();
  return check_launch("k_score_join");
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
