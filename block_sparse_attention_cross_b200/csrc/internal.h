// internal.h -- host-side declarations shared by the calibatt translation units.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "calibatt.h"

namespace calibatt {

// Error reporting (thread-local text behind calibatt_last_error).
int set_error(int code, const char* fmt, ...);
int check_launch(const char* what);   // cudaGetLastError -> status
void count_launch(int n = 1);
uint64_t spin_limit_ns();

// One-time launch set-up (dynamic shared-memory limits, SM counts, symbol
// addresses) is a per-device property: it is kept per device ordinal.
constexpr int kMaxDevices = 64;
// The current device's ordinal, checked against kMaxDevices.
int current_device(int* dev);

// Kernel arguments of the tensor-core attention kernels.
struct TcArgs {
  int B, H, N, Np, nqb, nkb;   // N, Np: query rows (real, padded)
  int Nk, Npk;                 // forward: key rows (real, padded); equal to N, Np unless queries are gathered
  float scale_log2;
  const int32_t* row_base;
  const int32_t* row_pat;
  const int32_t* pat_ptr;
  const int16_t* pat_off;
  int n_pat, nnz_pat, map_offset;
  int block_k;             // key-block size (64, 80, 96, 128 or 144)
  int nke;                 // energies: key blocks of block_k keys, ceil(N / block_k)
  void* o;                 // bf16 [B, H, Np, d]
  float* lse;              // [B, H, Np] natural-log LSE or nullptr
  float* lse2;             // calibration: per-row log2-domain LSE [H * Np]
  float* energy;           // calibration: [H, nqb, nkb]
  int32_t* status;
  unsigned long long spin_ns;
};

struct SimtArgs {
  int B, H, N, Np, block_q, block_k, nqb, nkb;
  float scale;
  const int32_t* row_base;
  const int32_t* row_pat;
  const int32_t* pat_ptr;
  const int16_t* pat_off;
  int n_pat, nnz_pat, map_offset;
  float* lse;        // fwd: [B,H,Np] or nullptr; calibration: per-row LSE [H*Np]
  float* energy;     // calibration: [H, nqb, nkb]
  int32_t* status;
};

// Argument checks and launch of the block energies, shared by
// calibatt_block_energy, calibatt_calibrate and calibatt_block_energy_noalloc
// (api.cu).  lse_ws: per-row scratch of H * Np floats.
int check_energy_args(const void* q, const void* k, int H, int N, int Np, int d, int dtype, int block_q,
                      int block_k, float scale);
int energy_impl(const void* q, const void* k, int H, int N, int Np, int d, int dtype, int block_q, int block_k,
                float scale, float* energy_out, float* lse_ws, int32_t* dev_status, cudaStream_t s);

// attn_tc.cu (bf16, tcgen05)
int launch_tc_fwd(const void* q, const void* k, const void* v, int d, const TcArgs& a, cudaStream_t s);
int launch_tc_energy(const void* q, const void* k, int d, const TcArgs& a, cudaStream_t s);
// The STATS pass alone: a.lse2[h * Np + row] = log2-domain LSE of every row over the real keys.
int launch_tc_stats(const void* q, const void* k, int d, const TcArgs& a, cudaStream_t s);

// attn_simt.cu (fp32, FFMA)
int launch_simt_fwd(const void* q, const void* k, const void* v, void* o, int d, const SimtArgs& a,
                    cudaStream_t s);
int launch_simt_energy(const void* q, const void* k, int d, const SimtArgs& a, cudaStream_t s);

// Kernel arguments of the score-modified attention (score_*.cu).
struct Tensor4 {            // [B, heads, N, d], d contiguous; strides in elements
  void* p;
  long long sb, sh, sn;
};
struct ScoreArgs {
  int B, H, Hkv, G;         // G = H / Hkv query heads per key head
  int Nq, Nk, nqb, nkb;     // nqb, nkb: 128-row query tiles, 128-key tiles
  float scale, cap;         // cap = 0: scores are not capped
  const float* slopes;      // [H] or nullptr
  const void* table;        // [H, n_buckets] of the inputs' type or nullptr
  const int32_t* buckets;   // [2 R + 1]
  int n_buckets, R;
  const uint8_t* mask;      // [maps, nqb, nkb] kept 128 x 128 blocks or nullptr
  int map_offset;
  const int2* row;          // [B, Nq] visible keys [x, y) of every query row
  const int4* tile;         // [B, nqb] min x, max y, max x, min y over a tile's rows
  const int32_t* q_start;   // [B] key position of query row 0
  Tensor4 q, k, v, o, dout, dq, dk, dv;
  float* lse;               // [B, H, Nq] (forward: written, may be nullptr; backward: read)
  void* dtable;             // [H, n_buckets] or nullptr
  // workspace
  int splits, packed, few;  // forward: splits of the key axis; packed: the G heads of a key head share a tile;
                            // few: packed, at most 32 rows, repeated in the tile's four lane quarters
  int parts;                // partial results per row: splits, four times as many with `few`
  float* part_o;            // [B, H, Nq, parts, d]
  float* part_lse;          // [B, H, Nq, parts]
  float* row_lse;           // backward: [B, H, 128 nqb]; fp32: LSE, +inf where a row sees nothing; bf16: -log2(e) of it
  float* row_d;             // backward: [B, H, 128 nqb]; fp32: D; bf16: -D
  int2* row_span;           // backward, bf16: [B, 128 nqb] the rows' intervals, padded to whole tiles
  int kv_parts;             // backward: parts of a key tile's query tiles
  float* part_kv;           // backward: [kv_parts, 2, B, Hkv, Nk, d] dV and dK
  int q_parts;              // backward, fp32: parts of a query tile's key tiles
  float* part_q;            // backward, fp32: [q_parts, B, H, Nq, d] dQ
  float* part_table;        // backward: [B, H, table tiles, n_buckets]
  int table_tiles;          // query tiles per head that write part_table
  int32_t* status;
  unsigned long long spin_ns;
};

// score_simt.cu (fp32, FFMA)
int score_splits_simt(int B, int H, int Nq, int Nk);
int score_q_parts_simt(int B, int H, int Nq, int Nk);
int score_kv_parts_simt(int B, int Hkv, int G, int Nq, int Nk);
int launch_score_fwd_simt(const ScoreArgs& a, int d, cudaStream_t s);
int launch_score_bwd_simt(const ScoreArgs& a, int d, cudaStream_t s);
// score_fwd.cu (bf16, tcgen05)
bool score_packs(int G, int Nq, bool mask, bool table);
int score_splits(int B, int heads, int nq_tiles, int nkb);
int score_kv_parts(int B, int Hkv, int G, int nqb, int nkb);   // score_bwd.cu
int launch_score_bwd_tc(const ScoreArgs& a, int d, cudaStream_t s);
int launch_score_fwd_tc(const ScoreArgs& a, int d, cudaStream_t s);
// score_plan.cu
int launch_attn_spans(int B, int Nq, int Nk, int causal, const int32_t* docs, int n_docs, const int32_t* prefix,
                      const int32_t* kv_len, const int32_t* q_len, const int32_t* q_start, int2* row, int4* tile,
                      int32_t* q_start_out, cudaStream_t s);
// score_rows.cu: the join of partial results, per-row terms of the fp32 backward pass, the sum of the table's partial gradients
int launch_score_join(const ScoreArgs& a, int d, int dtype, cudaStream_t s);
int launch_score_sum_parts(const ScoreArgs& a, int d, int dtype, cudaStream_t s);
int launch_score_rows(const ScoreArgs& a, int d, cudaStream_t s);
int launch_score_table_sum(const ScoreArgs& a, int dtype, cudaStream_t s);

// select_vote.cu
int launch_select_vote(const float* energy, int rows, int nkb, int mode, int topk, double eps,
                       int32_t* votes, float* esum, cudaStream_t s);
int launch_finalize(const int32_t* votes, const float* esum, int rows, int nkb, int min_votes,
                    uint8_t* mask, cudaStream_t s);

// compile.cu
size_t compile_workspace_bytes(long long rows, int nkb);
int run_compile(const uint8_t* masks, int n_maps, int nqb, int nkb, int dedup, void* ws, size_t ws_bytes,
                calibatt_blocklist* out, int64_t totals[3], cudaStream_t s);

// selftest
int launch_selftest_timeout(uint64_t limit_ns, int32_t* status, cudaStream_t s);

// TMA descriptor for a row-major bf16 matrix [rows, cols]; box 64 cols x box_rows rows, 128-byte swizzle.
int make_tmap_bf16(CUtensorMap* tm, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows = 128);

// TMA descriptor of a bf16 [B, heads, N, d] tensor; box 64 cols x box_n rows x box_h heads, 128-byte swizzle.
// Rows past N read as zero.
int make_tmap4_bf16(CUtensorMap* tm, const Tensor4& t, int B, int heads, int N, int d, int box_n, int box_h);
// Dynamic shared-memory limit of a kernel, set once per device (done[kMaxDevices]), and its launch register count (the register
// re-split inside the kernel is sized for exactly `regs`).
int configure_kernel(const void* kern, std::atomic<bool>* done, size_t smem, int regs, const char* what);
int device_sms(int* sms);

}  // namespace calibatt
