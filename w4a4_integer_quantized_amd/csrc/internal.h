// internal.h -- declarations shared by the HIP translation units of libconvrot.so.
// Not part of the public ABI (see include/convrot.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convrot {

enum InDtype { kF32 = 0, kF16 = 1, kBF16 = 2 };

// Weight-scale rules (values of rq_qconfig.w_scale_mode).
enum WScaleMode { kWScaleAbsmax = 0, kWScaleMse = 1, kWScaleTensor = 2 };

// Code layouts written by the quantizers (convrot.h): row-major int8 / packed int4, the tiled
// int layout (256-row panels), and FP6 tiles of 4-bit codes in 256-row (activation) or 128-row
// (weight) panels.
enum CodeLayout { kCodeRows = 0, kCodeTiled = 1, kCodeFp6X = 2, kCodeFp6W = 3 };

// Rotate + quantize `rows` rows of length K (dtype `dt`) into codes Q in `layout` (a CodeLayout;
// the FP6 layouts need bits == 4) and one fp32 scale per row. Arguments are pre-validated.
hipError_t launch_rotate_quant(const void* X, int dt, int64_t rows, int64_t K, int bits,
                               int layout, void* Q, float* S, hipStream_t stream);

// The norm with the residual's addition, rotated and quantized (norm_quant.hip). Strides in bytes,
// below 2^27; pre-validated, fewer than 2^32 threads.
struct NormQuantArgs {
  const uint8_t *x, *res;      // [M, K]; res null: none
  const uint8_t* weight;       // [K], binary32 (weight_f32) or the rows' type; null: ones
  uint8_t* h;                  // out: x + res; null: not kept
  uint8_t* codes;
  float* scales;
  int64_t x_stride, res_stride, h_stride, M;
  int K, weight_f32, layout;   // layout: a CodeLayout
  int lanes;                   // of a row (set by the launcher)
  float eps;
};
int64_t norm_quant_threads(int64_t M, int64_t K);   // of the launch
hipError_t launch_norm_quant(const NormQuantArgs& a, int dt, int bits, hipStream_t stream);

// The weight quantizer's MSE-clipped (kWScaleMse) or tensor-wise (kWScaleTensor) scale rule:
// codes Wq (row-major int8 / packed int4, or FP6 tiles of 128-row panels when fp6) and one fp32
// scale per row. Arguments are pre-validated; N < 2^31.
hipError_t launch_weight_quant(int mode, const void* W, int dt, int64_t N, int64_t K, int bits,
                               bool fp6, void* Wq, float* S, hipStream_t stream);

// acc = Xq * Wq^T over K (codes of `bits` bits; Xq row-major or tiled when x_tiled, Wq
// row-major), then either the dequantizing epilogue into Y (out_dt kF16 / kBF16), with the
// activation `act` (gemm::ActKind) applied before the rounding, or, when acc32 != nullptr, the
// raw int32 accumulators (act ignored).
hipError_t launch_gemm(const void* Xq, const float* sx, const void* Wq, const float* sw,
                       const float* bias, int64_t M, int64_t N, int64_t K, int bits,
                       bool x_tiled, void* Y, int out_dt, int32_t* acc32, int act,
                       hipStream_t stream);

// 4-bit codes on the FP6 matrix cores: Xt and Wt in the FP6 tile layout of convrot.h (256-row
// and 128-row panels). K % 128 == 0. `act` as for launch_gemm.
hipError_t launch_gemm_fp6(const void* Xt, const float* sx, const void* Wt, const float* sw,
                           const float* bias, int64_t M, int64_t N, int64_t K, void* Y,
                           int out_dt, int32_t* acc32, int act, hipStream_t stream);

// Y[m, n] = act(g) * u, g and u the dequantized values of gate row n and up row n of Wq: 2 N rows, 16 gate
// rows and 16 up rows in turn (as are sw and bias). act: any gemm::ActKind.
hipError_t launch_gemm_gated(const void* Xq, const float* sx, const void* Wq, const float* sw, const float* bias, int64_t M,
                             int64_t N, int64_t K, int bits, bool x_tiled, void* Y, int out_dt, int act, hipStream_t stream);
hipError_t launch_gemm_gated_fp6(const void* Xt, const float* sx, const void* Wt, const float* sw, const float* bias, int64_t M,
                                 int64_t N, int64_t K, void* Y, int out_dt, int act, hipStream_t stream);

// The gated product for few tokens (gemm_skinny.hip); launch_gemm_gated takes it where
// gated_skinny_supported() holds.
bool gated_skinny_supported(int64_t M, int64_t N);
hipError_t launch_gated_skinny(const void* Xq, const float* sx, const void* Wq, const float* sw, const float* bias, int64_t M,
                               int64_t N, int64_t Kb, int bits, bool x_tiled, void* Y, int out_dt, int act, hipStream_t stream);

hipError_t launch_gated_skinny6(const void* Xt, const float* sx, const void* Wt, const float* sw, const float* bias, int64_t M, int64_t N,
                                int64_t K, void* Y, int out_dt, int act, hipStream_t st);

// The same GEMM with each CU's weight tile resident in LDS and eight independent waves
// (int8 codes in the tiled layout, K = 1024; gemm_rw.hip). launch_gemm takes it where
// gemm_rw_supported() holds.
bool gemm_rw_supported(int64_t M, int64_t N, int64_t Kb, int bits, bool x_tiled);
hipError_t launch_gemm_rw(const void* Xq, const float* sx, const void* Wq, const float* sw,
                          const float* bias, int64_t M, int64_t N, void* Y, int out_dt,
                          int32_t* acc32, int act, hipStream_t stream);

// The same GEMM on 256 x 256 tiles with 128-byte k steps (launch_gemm picks it for long K);
// it needs Kb (K in bytes of codes) to be a multiple of 128 and at least 256.
bool wide_gemm_supported(int64_t Kb);
hipError_t launch_gemm_wide(const void* Xq, const float* sx, const void* Wq, const float* sw,
                            const float* bias, int64_t M, int64_t N, int64_t K, int bits,
                            void* Y, int out_dt, int32_t* acc32, hipStream_t stream);

// The cache operators (layout and arithmetic in convrot.h). Strides in elements; pre-validated.
struct KvCacheArgs {
  uint8_t* cache;
  const int64_t* slots;                       // [tokens]
  const uint8_t *k, *v;                       // write: rows in
  uint8_t *k_out, *v_out;                     // read: rows out
  int64_t k_token, k_head, v_token, v_head;   // strides of the rows
  int64_t tokens, num_pages, head_bytes;      // head_bytes: one head's block of a page
  int heads, lps, dt;                         // lps: log2 of the page size; dt: the rows' type
};
hipError_t launch_kv_cache(const KvCacheArgs& a, int head_dim, int bits, bool write, hipStream_t stream);

struct KvAttentionArgs {
  const uint8_t* cache;
  const uint8_t* q;
  uint8_t* out;
  float* lse;                 // [total_q, q_heads] or null
  const int32_t* q_start;     // [seqs + 1], or null: every sequence has total_q / seqs rows
  const int32_t* kv_len;      // [seqs]
  const int32_t* pages;       // [seqs, max_pages]
  float* part_out;            // [total_q, q_heads, splits, head_dim] when splits > 1
  float* part_stat;           // [total_q, q_heads, splits, 2]
  int64_t q_token, q_head, out_token, out_head;
  int64_t total_q, num_pages, head_bytes;
  int seqs, q_heads, heads, group, max_pages, lps, dt, causal, window, splits, row_tiles;
  int chunk;                  // keys of a split, unless the split count makes it more
  int block;                  // 1: the kernel for many query rows
  int max_q;                  // rows of a sequence that are computed
  int even_q;                 // rows of every sequence where q_start is null
  uint32_t group_mul;         // n / group = (mulhi(n, group_mul) + n) >> group_shift for n < 2^31
  int group_shift;
  float scale;
};
// How a call is split: see kv_attention.hip.
struct KvAttentionPlan {
  int splits, row_tiles, chunk, block;
  size_t workspace_bytes;
};
KvAttentionPlan plan_kv_attention(int64_t total_q, int seqs, int q_heads, int heads, int head_dim,
                                  int64_t max_q_len, int64_t max_kv_len, int window);
hipError_t launch_kv_attention(const KvAttentionArgs& a, int head_dim, int bits, hipStream_t stream);

// Attention weights added up for each cached token (kv_weigh.hip). `a` as for attention, without `out` and
// parts, lse read; a.splits: ranges of tokens, a.row_tiles: shares of the query rows.
struct KvWeighArgs {
  KvAttentionArgs a;
  float* weights;             // [seqs, heads, max_pages << lps]
  float* parts;               // [row_tiles][seqs, heads, part_span], where row_tiles > 1
  uint8_t* queries;           // rotated queries (many)
  int64_t part_span;          // tokens, from a sequence's first on, whose rows are shared out
  int64_t part_stride;        // elements of one share
  int64_t query_tiles_seq;    // tiles of 16 rows of the longest sequence
  int join_blocks;
  float keep;
};
struct KvWeighPlan {
  int64_t splits, row_splits, query_tiles_seq, query_bytes, part_bytes, part_span;
  int kt;                     // 16-token steps of a wave
  bool many;                  // queries are rotated by a kernel of their own
};
KvWeighPlan plan_kv_weigh(int64_t total_q, int seqs, int q_heads, int heads, int head_dim, int64_t max_q_len, int64_t max_kv_len);
hipError_t launch_kv_weigh(const KvWeighArgs& w, int head_dim, int bits, int kt, bool many, hipStream_t stream);

// A cache brought down to a budget (kv_evict.hip). Pre-validated: first + recent <= budget <= new_max_pages << lps.
struct KvEvictArgs {
  uint8_t* cache;
  const int32_t *kv_len, *pages, *new_pages;   // [seqs], [seqs, max_pages], [seqs, new_max_pages]
  const float* weights;                        // [seqs, heads, max_pages << lps]
  float* new_weights;                          // [seqs, heads, new_max_pages << lps], or null
  int32_t *new_kv_len, *kept;                  // [seqs], [seqs, heads, budget]
  int64_t num_pages, head_bytes;
  int seqs, heads, max_pages, new_max_pages, lps, budget, first, recent;
  int chunks;                                  // kv_evict_chunks(budget)
  int parts;                                   // workgroups that choose for a (sequence, head)
  uint32_t* scratch;                           // their workspace
};
struct KvEvictPlan {
  int parts;
  size_t workspace_bytes;
};
int64_t kv_evict_chunks(int budget);           // workgroups that move a (sequence, head)
KvEvictPlan plan_kv_evict(int64_t groups, int64_t span);   // groups: (sequence, head) pairs
hipError_t launch_kv_evict(const KvEvictArgs& a, int row_bytes, hipStream_t stream);

}  // namespace convrot
