// Internal launcher interface between the C ABI layer (abi.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fast_divide.cuh"

namespace pkv {

cudaError_t launch_kv_write(void* k_cache, void* v_cache, const void* k, const void* v,
                            const int32_t* slots, int64_t num_tokens, int64_t num_slots,
                            int64_t row_k_bytes, int64_t row_v_bytes, int* dev_status,
                            cudaStream_t stream, int num_sms);
cudaError_t launch_kv_write_fp8(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                const void* k, const void* v, const int32_t* slots,
                                int64_t num_tokens, int64_t num_blocks, int block_size, int hkv,
                                int* dev_status, cudaStream_t stream, int num_sms);
cudaError_t launch_copy_blocks(void* cache, int64_t num_blocks, int64_t block_bytes,
                               const int32_t* src, const int32_t* dst, int64_t n, int* dev_status,
                               cudaStream_t stream, int num_sms);
cudaError_t launch_mla_rmsnorm_rope_write(void* cache_nope, void* cache_rope, void* k_nope_out,
                                          void* k_rope_out, const void* latent, const void* gamma,
                                          const float* cosv, const float* sinv,
                                          const int32_t* slots, int64_t num_tokens,
                                          int64_t num_slots, float eps, int* dev_status,
                                          cudaStream_t stream, int num_sms);

// Arguments of the fused rotary embedding + paged write (rope_write.cu). Strides are in
// elements, between tokens; the heads of a token are contiguous.
constexpr int kRopeMaxAxes = 4;
constexpr int kRopeMaxDim = 256;
struct RopeArgs {
  const uint16_t *q, *k, *v;   // [T, H, d], [T, Hkv, d], [T, Hkv, d] bf16
  uint16_t* q_out;             // [T, H, d] bf16
  uint8_t *k_cache, *v_cache;  // [nb, bs, Hkv, d] bf16, or E4M3 codes
  float *k_scale, *v_scale;    // FP8 cache only: [nb, Hkv, bs]
  const float* table;          // [max_pos, rope_dim]: cosines, then sines
  const int32_t* positions;    // [num_axes, T]
  const int32_t* slots;        // [T]
  int* dev_status;
  int64_t num_tokens, num_slots, max_pos;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int H, Hkv, head_dim, rope_dim, num_axes, block_size;
  uint8_t pair_axis[kRopeMaxDim / 2];   // position axis of each pair
  int8_t chunk_axis[kRopeMaxDim / 16];  // axis of 8 pairs at a time, -1 where they differ
};
cudaError_t launch_rope_write(const RopeArgs& a, bool fp8, bool interleaved, cudaStream_t stream,
                              int num_sms);
// Rows of an FP8 cache widened to bf16 (kv_read.cu).
cudaError_t launch_kv_read_fp8(void* k, void* v, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, const int32_t* slots,
                               int64_t num_tokens, int64_t num_blocks, int block_size, int hkv,
                               int* dev_status, cudaStream_t stream, int num_sms);

// The 4-bit cache's write and read (kv_fp4.cu).
struct KvFp4Args {
  uint8_t *k_cache, *v_cache;  // [nb, Hkv, bs, 64] codes
  uint8_t *k_scale, *v_scale;  // [nb, Hkv, bs, 8]
  const int32_t* slots;        // [T]
  int* dev_status;
  int64_t num_tokens, num_blocks;
  int block_size, hkv;
  uint32_t items;              // rows of k and v together, set by the launch, as the divisors are
  FastDivide heads, block;
};
// Strides in elements, between tokens; the heads of a token are contiguous.
cudaError_t launch_kv_write_fp4(KvFp4Args a, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, cudaStream_t stream, int num_sms);
cudaError_t launch_kv_read_fp4(KvFp4Args a, void* k, void* v, cudaStream_t stream, int num_sms);

// Block summaries and block selection (block_select.cu).
constexpr int kSelectMaxBlocks = 8192;  // widest table of a selection: a million tokens
struct SummaryArgs {
  uint8_t* summaries;         // [nb, Hkv, 2, 128] bf16: minima, maxima
  const uint8_t* k_cache;     // [nb, 128, Hkv, 128] bf16
  const int32_t* block_table; // [B, max_blocks]
  const int32_t* seq_lens;    // [B]
  const int32_t* num_new;     // [B]
  int* dev_status;
  int64_t num_blocks;
  int B, Hkv, max_blocks, max_new;
  int span;                   // blocks that max_new new rows can touch
};
cudaError_t launch_block_summaries(const SummaryArgs& a, cudaStream_t stream, int num_sms);
struct SelectArgs {
  const uint16_t* q;          // [B, q_len, H, 128] bf16
  const uint8_t* summaries;
  const int32_t* block_table; // [B, max_blocks]
  const int32_t* seq_lens;    // [B]
  int32_t* out;               // [B, q_len, Hkv, num_selected]
  int* dev_status;
  int64_t num_blocks;
  int B, q_len, H, Hkv, n_rep, max_blocks, num_selected, num_sink, num_recent;
};
cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t stream, int num_sms);

// Attention weights summed per cached row (attn_weights.cu).
constexpr int kKeysBf16 = 0, kKeysFp8 = 1, kKeysFp4 = 2;  // PKV_KEYS_*
constexpr int kWeightsMaxRows = 128;                       // query rows of one launch
struct WeightsArgs {
  float* weights;             // [nb, Hkv, 128]
  const uint16_t* q;          // [B, q_len, H, 128] bf16
  const float* lse;           // [B, q_len, H]
  const uint8_t* k_cache;     // bf16 or E4M3 [nb, 128, Hkv, 128], or codes [nb, Hkv, 128, 64]
  const uint8_t* k_scale;     // null, fp32 [nb, Hkv, 128], or bytes [nb, Hkv, 128, 8]
  const int32_t* block_table; // [B, max_blocks]
  const int32_t* seq_lens;    // [B]
  const int32_t* num_fresh;   // [B]
  int* dev_status;
  int64_t num_blocks;
  int B, q_len, H, Hkv, n_rep, max_blocks;
  int row0, rows, start;      // query tokens of this launch; whether it is the first
  float scale_log2, decay;
};
cudaError_t launch_attn_weights(WeightsArgs a, int format, cudaStream_t stream, int num_sms);

// Eviction (select_rows.cu, compact_rows.cu).
constexpr int kMaxKept = 1 << 30;  // entries of a list: the kernels' strides past its end stay below 2^31
constexpr int kSelectRowsMaxBlocks = 32768;  // widest table of a choice of rows: four million tokens
struct SelectRowsArgs {
  const float* weights;       // [nb, Hkv, bs]
  const int32_t* block_table; // [B, max_blocks]
  const int32_t* seq_lens;    // [B]
  int32_t* out;               // [B, Hkv, num_keep]
  int* dev_status;
  int64_t num_blocks;
  int B, Hkv, block_size, max_blocks, num_keep, num_sink, num_recent;
};
cudaError_t launch_select_rows(const SelectRowsArgs& a, cudaStream_t stream, int num_sms);
constexpr int kCompactMaxCaches = 16;
struct CompactCache {
  uint8_t* data;
  int64_t block_stride, row_stride, head_stride;  // bytes
  int row_bytes, vec, slice_bytes, slices;
};
struct CompactArgs {
  CompactCache cache[kCompactMaxCaches];
  const int32_t* kept;        // [B, Hkv, num_keep]
  const int32_t* block_table; // [B, max_blocks]
  const int32_t* new_table;   // [B, new_max_blocks]: block_table itself in place
  int* dev_status;
  int64_t num_blocks;
  int B, Hkv, block_size, max_blocks, new_max_blocks, num_keep, num_caches;
  int slices, part_rows;      // of a row's bytes at most; rows of the list that one CTA moves
};
cudaError_t launch_compact_rows(CompactArgs a, cudaStream_t stream, int num_sms);

// Arguments of the split-KV decode kernels and their LSE merge.
struct DecodeArgs {
  const uint16_t* q;          // [B, q_len, H, D] bf16
  const uint8_t* k_cache;     // [nb, bs, Hkv, D] bf16
  const uint8_t* v_cache;
  const int32_t* block_table; // [B, max_blocks]
  const int32_t* seq_lens;    // [B]
  void* out;                  // [B, q_len, H, D] bf16 or f32
  float* lse;                 // [B, q_len, H] or null
  float* ws_o;                // [(B*Hkv + G) * q_len * n_rep * D] partial outputs
  float* ws_lse;              // [(B*Hkv + G) * q_len * n_rep] partial log2-sum-exp
  int* dev_status;
  int64_t num_blocks;
  int B, H, Hkv, n_rep, max_blocks, out_f32;
  int q_len;                  // new query rows per sequence (1 = plain decode)
  int row_window;             // window of one query row (0 = full attention)
  int window;                 // live-block span: row_window + q_len - 1 (0 = all)
  int num_ctas;               // G: CTAs of the attention kernel (one per SM)
  float scale_log2;           // scale * log2(e)
  const float* k_scale;       // FP8 cache only: [nb, Hkv, bs] per-row scales
  const float* v_scale;
  // Sparse decode only: B counts query rows, rows_per_seq of each sequence.
  const int32_t* block_indices;  // [B, Hkv, num_selected] blocks of the sequence, or null
  int num_selected, rows_per_seq;
};
// The 4-bit cache's: codes [nb, Hkv, bs, 64].
struct DecodeFp4Args : DecodeArgs {
  const uint8_t* k_scale4;    // [nb, Hkv, bs, 8]
  const uint8_t* v_scale4;
  int q_total, row0;          // the launch's q_len rows are row0 .. row0 + q_len - 1 of q and out's q_total
  bool whole;                 // a CTA for every (sequence, kv head), and no merge
};

size_t decode_workspace_bytes(int B, int H, int Hkv, int D, int G);
void decode_workspace_carve(DecodeArgs& a, void* ws);

// CUDA-core split-KV decode (any group size 1..16) followed by the LSE merge.
cudaError_t launch_decode_simt(const DecodeArgs& a, cudaStream_t stream);
cudaError_t launch_decode_merge(const DecodeArgs& a, cudaStream_t stream);
cudaError_t launch_decode_merge(const DecodeFp4Args& a, cudaStream_t stream);
// tcgen05 split-KV decode for head groups (n_rep 1..16), same partials as above.
cudaError_t launch_decode_tc(const DecodeArgs& a, cudaStream_t stream);
// The same kernel for q_len 1..4 query rows per sequence (q_len * n_rep <= 32).
cudaError_t launch_decode_spec(const DecodeArgs& a, cudaStream_t stream);
// The same kernel over the blocks that each query row lists (a.block_indices), and its merge.
cudaError_t launch_decode_sparse(const DecodeArgs& a, cudaStream_t stream);
// tcgen05 split-KV decode over an FP8 (E4M3) cache with per-row scales; same
// partials and merge as above.
cudaError_t launch_decode_fp8(const DecodeArgs& a, cudaStream_t stream);
// Split-KV decode over the 4-bit cache for q_len 1..4 query rows per sequence, same partials as
// above, and its merge.
cudaError_t launch_decode_fp4(DecodeFp4Args a, cudaStream_t stream);

// Absorbed MLA decode (tcgen05) plus its merge, q_len query rows per sequence
// (1 for plain decode). Workspace: mla_workspace_bytes(B * q_len, num_sms / 2).
size_t mla_workspace_bytes(int rows, int g_half);
cudaError_t launch_mla_decode(const void* q_nope, const void* q_rope, const void* cache_nope,
                              const void* cache_rope, const int32_t* block_table, int max_blocks,
                              const int32_t* seq_lens, void* out, int out_f32, float* lse, int B,
                              int q_len, int H, int64_t num_blocks, float scale, void* ws,
                              int* dev_status, int num_sms, cudaStream_t stream);

// Causal paged prefill (tcgen05, stream-K) plus its merge.
size_t prefill_workspace_bytes(int G);
cudaError_t launch_prefill(const void* q, const int32_t* cu_q, const void* k_cache,
                           const void* v_cache, const int32_t* block_table, int max_blocks,
                           const int32_t* seq_lens, void* out, int out_f32, float* lse, int T,
                           int B, int H, int Hkv, int64_t num_blocks, float scale, int causal,
                           void* ws, int* dev_status, int num_sms, cudaStream_t stream);

// Self-test: a bounded wait that runs out (selftest.cu).
cudaError_t launch_bounded_wait(int* dev_status, cudaStream_t stream);
// And the selection's bf16 matrix products, n of them.
cudaError_t launch_bf16_products(float* d, const void* a, const void* b, int n, cudaStream_t stream);

}  // namespace pkv
