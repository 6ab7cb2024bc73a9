// dsa_internal.h -- parameter blocks and launchers shared by the kernels and the
// C-ABI layer of libdsa.so.  Not part of the public interface (include/dsa.h is).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <utility>

namespace dsa {

// Launches a kernel with programmatic stream serialization: it may be scheduled
// while the previous kernel in the stream finishes, and waits for it inside
// (griddep_wait) before touching global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---------------------------------------------------------------- indexer
struct IndexerParams {
  int B, Lq, Lk, q_offset;
  int H_I, d_I;
  int qb;                 // queries per MMA (N = qb * H_I <= 256)
  int nsub;               // query sub-blocks resident per unit
  int queries_per_unit;   // qb * nsub
  int n_qblocks;          // ceil(Lq / queries_per_unit)
  int kchunks;            // key-tile ranges per query block (>1 splits long rows across CTAs)
  int n_units;            // n_qblocks * B * kchunks
  int fill_upper;         // write -inf for s > t (full-matrix output)
  int scale_ring;         // key scales staged per tile by TMA (k_scale set, Lk % 4 == 0)
  const float* q_scale;   // [B, Lq] or null
  const __nv_bfloat16* w; // [B, Lq, H_I]
  const float* k_scale;   // [B, Lk] or null
  float* scores;          // [B, Lq, Lk] (scores mode)
  // ---- fused top-k mode (scores == nullptr): every row's k largest scores are
  // selected on chip; no score reaches global memory except the selected ones.
  int k;                  // positions selected per row
  int cap;                // candidate-list capacity per row (multiple of 32, >= k + 128)
  int n_stage;            // staging slots (one per accumulator use) in shared memory
  int rows_per_unit;      // queries_per_unit
  int32_t* indices;       // [B, Lq, k]
  float* sel_scores;      // [B, Lq, k] or null
  uint32_t* xkey;         // kchunks > 1: each unit's top-k per row, keys:  [unit][rows_per_unit][cap]
  uint32_t* xpos;         // kchunks > 1: the same, positions
  uint4* xmeta;           // kchunks > 1: per (unit, row) {count, min key, max key, 0}
  uint32_t* done;         // kchunks > 1: per row, chunks finished (zeroed before the launch)
};
// Shared-memory bytes of the indexer kernel for a query block of q_rows (query,
// head) rows, `stages` key stages and, in the fused mode, the staging and
// selection areas.
size_t indexer_smem_bytes(int q_rows, int d_I, int w_floats, int sq_floats, int stages, bool scale_ring,
                          bool fused, int qb, int n_stage, int rows_per_unit, int cap);
cudaError_t launch_indexer(const IndexerParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& ts, int grid, cudaStream_t stream);
int indexer_fused_max_rows();    // rows per unit the fused mode supports
int indexer_fused_max_stage();   // staging slots the fused mode supports

// ---------------------------------------------------------------- top-k
struct TopkParams {
  const float* scores;    // [B, Lq, Lk]
  int B, Lq, Lk, q_offset, k;
  int32_t* indices;       // [B, Lq, k]
  float* sel_scores;      // [B, Lq, k] or null: score of each selected position (-0.0 as +0.0), -inf padding
  int cache_cap;          // row elements cached in shared memory (0 = re-read from global); multiple of 4
  int bit_words;          // 32-bit words of each position bitmap (>= ceil(row length / 32)); multiple of 4
  int cand_cap;           // candidate (key, position) pairs held in shared memory
  int vec4;               // rows start 16-byte aligned (scores aligned, Lk % 4 == 0): 16-byte loads
  int cluster;            // each row spread over a cluster of kTopkClusterCtas CTAs (few long rows);
                          // bit_words then covers one CTA's segment
  int warp_rows;          // one warp per row (many rows): no block-wide steps, rows streamed from L2
  int sampled;            // long rows: try the single-pass selection above a sampled threshold first
};
constexpr int kTopkClusterCtas = 4;
size_t topk_smem_bytes(int cache_cap, int bit_words, int cand_cap, bool cluster);
cudaError_t launch_topk(const TopkParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- sparse attention
struct AttnParams {
  int B, Lq, Lk, H, k;
  int n_tiles;            // ceil(k / 128)
  int splits;             // key-tile ranges per query (split-k); 1 = direct output
  int tiles_per_split;
  int n_units;            // B * Lq * splits
  int compact;            // indices are valid-first (top-k output): skip all-padding tiles
  int dense;              // short sequence (q_offset + Lq <= k): row t attends to keys 0..t, read as
                          // contiguous tiles; the kernel writes those positions to idx_out
  int q_offset;           // only used when compact or dense
  int32_t* idx_out;       // dense: [B, Lq, k] receives 0..t then -1
  float scale_log2;       // softmax scale * log2(e)
  const int32_t* indices; // [B, Lq, k]
  __nv_bfloat16* out;     // [B, Lq, H, d_v] (splits == 1)
  float* lse;             // [B, Lq, H] or null (splits == 1)
  float* part_o;          // [B*Lq, splits, H, d_v] fp32 (splits > 1)
  float* part_lse;        // [B*Lq, splits, H] fp32 (splits > 1)
  // ---- sliding window (window > 0): row (b, i) at t = (start ? start[b] : q_offset) + i sees
  // keys (t - window, t] and [0, sinks); no index lists
  int window, sinks;
  const int32_t* start;   // [B] or null
  // ---- lists over rows with one row of zeros behind them: the row that masked slots gather
  // (0: they gather the sequence's first row)
  int zero_row;
  // ---- 4-bit cache (codes set): indices (or dense) pick its rows
  const uint8_t* codes;   // [B, Lk, d_v / 2]
  const __nv_bfloat16* scales;   // [B, Lk, d_v / 32]
  const __nv_bfloat16* tail;     // [B, Lk, d_qk - d_v]
};
cudaError_t launch_sparse_attn(const AttnParams& p, int d_qk, int d_v, const CUtensorMap& tq,
                               const CUtensorMap& tkv, const CUtensorMap& tkv_tile, int grid_clusters,
                               cudaStream_t stream);
cudaError_t launch_attn_combine(const AttnParams& p, int d_v, cudaStream_t stream);

// ---------------------------------------------------------------- indexer training loss
struct KlParams {
  int B, Lq, Lk, H, k;
  int n_rows;             // B * Lq
  int n_tiles;            // ceil(k / 128)
  float scale_log2;       // softmax scale * log2(e)
  const int32_t* indices; // [B, Lq, k]
  const float* lse;       // [B, Lq, H], natural log
  const float* scores;    // [B, Lq, Lk], or null when sel_scores is given
  const float* sel_scores;  // [B, Lq, k]: the score of each index slot (or null)
  float* target;          // [B, Lq, k] or null
  float* kl;              // [B, Lq]
};
size_t indexer_kl_smem_bytes(int d_qk);
cudaError_t launch_indexer_kl(const KlParams& p, int d_qk, const CUtensorMap& tq, const CUtensorMap& tkv,
                              int grid_clusters, cudaStream_t stream);

// ---------------------------------------------------------------- norm and rotation of heads
// n / d for 0 <= n < 2^31: with s = ceil(log2 d) and mul = ceil(2^(31+s) / d) the product
// n * mul exceeds n * 2^(31+s) / d by less than n * d / d * 2^s / d, too little to reach the
// next multiple of 2^(31+s).
struct FastDiv {
  uint32_t d, mul, shift;   // d == 1: n itself
#ifdef __CUDACC__
  __device__ __forceinline__ int operator()(int n) const {
    return d == 1 ? n : (int)(__umulhi((uint32_t)n, mul) >> shift);
  }
#endif
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  uint32_t s = 0;
  while (s < 31 && (1u << s) < d) ++s;
  if (d > 1) {
    f.mul = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
    f.shift = s - 1;
  }
  return f;
}
struct NormRopeParams {
  FastDiv div_h, div_l, div_parts;   // by H, L and parts
  float inv_norm_dim;
  // Set by the launcher: blocks walk spans of span_tokens tokens (whose angles are filled in
  // together) in steps of tokens_per_step tokens, or of one of `parts` parts of a token's heads.
  int n_spans, span_tokens, tokens_per_step, parts;
  int L, H, D;            // tokens are (b, l) pairs, b = token / L
  int n_tokens;           // B * L
  int norm, norm_dim;     // dsa_norm; columns [0, norm_dim) are normalised
  float eps;
  int w_bf16;             // w and b in bf16 instead of fp32
  int rot_start, n_freq;  // rotated columns [rot_start, rot_start + 2 n_freq)
  int interleaved, q_offset;
  long long stride_b, stride_l, stride_h;   // of x, in elements
  const __nv_bfloat16* x;
  const void* w;          // [norm_dim]
  const void* b;          // [norm_dim] or null
  const float* inv_freq;  // [n_freq]
  const int32_t* positions;   // [B, L] or null: q_offset + l
  __nv_bfloat16* out;     // [B, L, H, D] bf16 ...
  uint8_t* codes;         // ... or e4m3 [B, L, H, D]
  float* scale;           // and [B, L]
  const __nv_bfloat16* dy;    // gradient: [B, L, H, D]
  __nv_bfloat16* dx;      // [B, L, H, D]
  float* part;            // [2 (w, b)][blocks][norm_dim]
  float* dw;              // [norm_dim]
  float* db;              // [norm_dim] (when b is given)
};
constexpr int kNormRopeBwdBlocksPerSm = 2;
int norm_rope_bwd_blocks(int sms);   // most partial rows the gradient leaves
cudaError_t launch_norm_rope(NormRopeParams p, int sms, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(NormRopeParams p, int sms, cudaStream_t stream);

// ---------------------------------------------------------------- 4-bit latent cache
struct Kv4Params {
  FastDiv div_l;          // by L
  int B, L, Lk, d_qk, d_v;
  int zero_rows;          // read: rows of zeros written behind the last
  int offset;             // cache row of row 0 when start is null
  const int32_t* start;   // [B] or null
  const __nv_bfloat16* in;    // write: [B, L, d_qk]
  __nv_bfloat16* out;     // read: [B, L, d_qk]
  uint8_t* codes;         // [B, Lk, d_v / 2]
  __nv_bfloat16* scales;  // [B, Lk, d_v / 32]
  __nv_bfloat16* tail;    // [B, Lk, d_qk - d_v]
};
cudaError_t launch_kv4_write(const Kv4Params& p, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4Params& p, cudaStream_t stream);

// ---------------------------------------------------------------- misc
// Error words of the kernel units (one per translation unit), and their union.
cudaError_t read_indexer_error(uint32_t* value, bool clear);
cudaError_t read_topk_error(uint32_t* value, bool clear);
cudaError_t read_attn_error(uint32_t* value, bool clear);
cudaError_t read_kl_error(uint32_t* value, bool clear);
cudaError_t read_device_error(uint32_t* value, bool clear);
cudaError_t launch_wait_selftest(uint32_t spin_limit, cudaStream_t stream);

}  // namespace dsa
