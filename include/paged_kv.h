/*
 * paged_kv.h -- C ABI of the GB300 paged KV cache library (libpaged_kv.so).
 *
 * The problem these calls solve is the one stated by the pages:
 *   - the physical KV cache is laid out [num_blocks, block_size, H_kv, d]
 *     ("KVCache 优化技能" skill note, 模式二 and §3.1);
 *   - new K/V rows are written through slot_mapping, one slot per new token,
 *     slot = block_table[b, pos / block_size] * block_size + pos % block_size
 *     (same note §3.1 / §3.3; "KV Cache 管理设计文档" §4.2.2 prepare_slot_mapping);
 *   - attention reads each sequence's keys through block_table with per-sequence
 *     lengths (actual_seq_lengths_kv), for GQA, sliding windows whose expired
 *     table entries hold a null block, causal prefill, and the absorbed MLA form.
 *
 * Conventions shared by every call:
 *   - Return value: PKV_OK (0) or a negative PKV_ERR_* code. On error nothing was
 *     launched and pkv_last_error() (thread-local) holds a one-line reason.
 *   - Device calls take device pointers owned by the caller and run
 *     asynchronously on `stream` (a cudaStream_t; NULL = legacy default stream).
 *     The library never allocates, frees or synchronises device memory; scratch
 *     space is a caller-provided `workspace` of at least the size the matching
 *     *_workspace_size() call returns, 256-byte aligned.
 *   - Element types: q, caches and new rows are bf16 (raw 16-bit storage);
 *     block tables, slot mappings and lengths are int32. `out_dtype` selects a
 *     bf16 (PKV_BF16, round-to-nearest-even) or fp32 (PKV_F32) output.
 *   - `scale` has no default: callers pass it (the pages warn that a softmax
 *     scale silently falling back to 1.0 ruins accuracy, standalone guide FA
 *     v1/v2 parameter table).
 *   - `dev_status` (nullable) is a device int the kernels set to a nonzero
 *     PKV_DEV_* bit mask when they meet a bad table entry, slot or length; the
 *     offending access is skipped (never performed). The caller zeroes it.
 *   - Tensor-memory-accelerator (TMA) reads need 16-byte aligned base pointers
 *     and row strides; every pointer below must be 16-byte aligned.
 */
#ifndef PAGED_KV_H
#define PAGED_KV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes -------------------------------------------------------- */
#define PKV_OK 0
#define PKV_ERR_INVALID_ARG (-1)   /* null pointer, bad size, misaligned pointer   */
#define PKV_ERR_UNSUPPORTED (-2)   /* a shape this build does not implement        */
#define PKV_ERR_WORKSPACE (-3)     /* workspace missing or too small               */
#define PKV_ERR_LAUNCH (-4)        /* CUDA launch or driver call failed             */
#define PKV_ERR_OUT_OF_BLOCKS (-5) /* pool cannot satisfy an all-or-nothing request */
#define PKV_ERR_DOUBLE_FREE (-6)   /* freeing a free block or the null block        */

/* bits of *dev_status */
#define PKV_DEV_BAD_SLOT 1         /* slot_mapping entry >= num_blocks * block_size  */
#define PKV_DEV_BAD_BLOCK 2        /* block_table entry outside [0, num_blocks)      */
#define PKV_DEV_BAD_LENGTH 4       /* length > max_blocks_per_seq * block_size, < 0  */
#define PKV_DEV_TIMEOUT 8          /* a bounded wait inside a kernel gave up         */
#define PKV_DEV_BAD_POSITION 16    /* rotary position outside [0, max_pos)           */

#define PKV_BF16 0
#define PKV_F32 1

/* One-line reason for the last non-OK return on this thread ("" if none). */
const char* pkv_last_error(void);
/* Library ABI version (major * 100 + minor). */
int pkv_version(void);

/* ==========================================================================
 * Host-side block management (no device pointers)
 * ========================================================================== */

/* Opaque BlockPool: FIFO free queue plus a set that catches double frees
 * ("KV Cache 管理设计文档" §2.4). The queue starts as `initial_order` (a
 * permutation of 0..num_blocks-1; NULL = 0,1,2,...); the first id popped becomes
 * the null block, which is never handed out. Seeded shuffles are expressed by
 * passing a shuffled order. The pool is owned by the caller: destroy it with
 * pkv_pool_destroy. Not thread-safe. */
typedef struct pkv_pool pkv_pool;
int pkv_pool_create(int64_t num_blocks, const int32_t* initial_order, pkv_pool** out);
void pkv_pool_destroy(pkv_pool* pool);
int32_t pkv_pool_null_block(const pkv_pool* pool);
int64_t pkv_pool_num_free(const pkv_pool* pool);
/* Pop n ids from the head of the queue into ids_out[n]; all-or-nothing
 * (PKV_ERR_OUT_OF_BLOCKS leaves the pool unchanged). */
int pkv_pool_alloc(pkv_pool* pool, int64_t n, int32_t* ids_out);
/* Drop one reference per listed id; an id whose count reaches zero goes back to
 * the queue tail, in the listed order. PKV_ERR_DOUBLE_FREE (pool unchanged) if an
 * id is out of range, is the null block, or is listed more often than it is
 * referenced (an unshared block: free already, or listed twice). */
int pkv_pool_free(pkv_pool* pool, const int32_t* ids, int64_t n);
/* One more reference to each of ids[n], all currently held (a block shared by a
 * forked request, "KV Cache 笔记" fork_blocks). PKV_ERR_INVALID_ARG (pool
 * unchanged) if an id is free, out of range or the null block. */
int pkv_pool_share(pkv_pool* pool, const int32_t* ids, int64_t n);
/* Reference count of one block (0 = free or the null block; -1 = bad id). */
int32_t pkv_pool_ref_count(const pkv_pool* pool, int32_t id);

/* Skipped tokens of a manager after n computed tokens: 0 for full attention
 * (window <= 0), max(0, n - window + 1) for a sliding window
 * ("KV Cache 管理设计文档" §2.3 get_num_skipped_tokens). */
int64_t pkv_num_skipped_tokens(int64_t num_computed_tokens, int64_t window);

/* Batch block table [B, max_blocks_per_seq] (row-major, host memory) for sequences
 * of total length seq_lens[b] (including the newest token). Row b holds
 * ceil(len/bs) logical entries; with window > 0 the leading
 * floor(skipped(len - 1) / bs) entries, wholly outside the window, are the null
 * block and take nothing from the pool (§2.3.2); the others are popped from the
 * pool in FIFO order, sequence by sequence. Unused entries hold the null block.
 * All-or-nothing: PKV_ERR_OUT_OF_BLOCKS leaves the pool unchanged. */
int pkv_build_block_table(pkv_pool* pool, const int32_t* seq_lens, int32_t B, int32_t block_size,
                          int32_t window, int32_t max_blocks_per_seq, int32_t* table_out);
/* Static table arange(B * blocks_per_seq).reshape(B, -1) ("KVCache 优化技能" §3.2). */
int pkv_build_block_table_arange(int32_t B, int32_t blocks_per_seq, int32_t* table_out);
/* slot_mapping for num_new[b] tokens at positions start_pos[b].. of each sequence,
 * concatenated in sequence order (host memory). slot = table[b][pos / bs] * bs +
 * pos % bs ("KVCache 优化技能" §3.1; "KV Cache 管理设计文档" §4.2.2). Returns the
 * number of slots written (>= 0) or an error code. */
int64_t pkv_build_slot_mapping(const int32_t* block_table, int32_t max_blocks_per_seq,
                               const int32_t* start_pos, const int32_t* num_new, int32_t B,
                               int32_t block_size, int32_t* slots_out, int64_t slots_capacity);

/* Pool sizing ("KV Cache 管理设计文档" §4.2.1 calculate_block_num); each "+1" is
 * the null block. */
int64_t pkv_block_num_fixed(int64_t max_concurrency, int64_t sliding_window, int64_t next_n,
                            int64_t block_size);
int64_t pkv_block_num_full_offline(int64_t max_len, int64_t block_size, int64_t max_concurrency);
int64_t pkv_block_num_full_online(int64_t available_bytes, int64_t per_token_bytes,
                                  int64_t block_size);

/* ==========================================================================
 * Request-level allocator ("KV Cache 管理设计文档" §2-§3; prefix sharing and
 * fork from "KV Cache 笔记", HF continuous batching). Host memory only.
 * ========================================================================== */

/* KVCacheManager over one manager per attention type (§2.2-§2.3). Type i has
 * window windows[i] (0 = full attention, > 0 = sliding window of that many
 * tokens), its own BlockPool of num_blocks[i] ids whose queue starts as
 * initial_orders[i] (NULL, or a NULL entry = 0,1,2,...), and group id i in block
 * fingerprints. At most one full-attention and one sliding-window type
 * (PKV_ERR_INVALID_ARG otherwise). prefix_caching != 0 turns on prefix sharing for
 * full-attention types. Owned by the caller (pkv_manager_destroy). Not
 * thread-safe. Request ids are any int64 values. */
typedef struct pkv_kv_manager pkv_kv_manager;
int pkv_manager_create(int32_t num_types, const int32_t* windows, const int64_t* num_blocks,
                       const int32_t* const* initial_orders, int32_t block_size,
                       int64_t max_model_len, int32_t prefix_caching, pkv_kv_manager** out);
void pkv_manager_destroy(pkv_kv_manager* mgr);

/* allocate_slots (§3): the request will hold K/V for positions
 * [0, min(computed + num_new + lookahead, max_model_len)). Phase 1, type by type:
 * give back the blocks of a sliding window that no query from position
 * min(computed, max_model_len) on can see (remove_skipped_blocks: they become the
 * null block), then count the new blocks the type needs; return 0 at the first
 * type whose pool cannot supply them, with nothing allocated. Phase 2: append the
 * new entries in every type (leading entries wholly before position
 * computed - W + 1 are the null block, the rest come from the pool in FIFO order).
 * Returns 1 (allocated), 0 (not enough blocks) or a negative error. */
int pkv_manager_allocate_slots(pkv_kv_manager* mgr, int64_t request_id, int64_t computed_tokens,
                               int64_t num_new_tokens, int64_t lookahead_tokens);
/* Logical block list of a request in type `type` (get_block_ids): writes up to
 * `capacity` ids and returns the list's length (0 for an unknown request). */
int64_t pkv_manager_get_block_ids(const pkv_kv_manager* mgr, int64_t request_id, int32_t type,
                                  int32_t* ids_out, int64_t capacity);
/* Release every block of the request in every type (free); unknown ids are a no-op. */
int pkv_manager_free(pkv_kv_manager* mgr, int64_t request_id);
int64_t pkv_manager_num_free(const pkv_kv_manager* mgr, int32_t type);
int32_t pkv_manager_null_block(const pkv_kv_manager* mgr, int32_t type);
int32_t pkv_manager_ref_count(const pkv_kv_manager* mgr, int32_t type, int32_t block);
/* format_usage: "full:used/total,sliding:used/total" in type order; used = blocks
 * handed out (the null block not counted), total = the pool's size. Writes a
 * NUL-terminated string (truncated to capacity) and returns its full length. */
int64_t pkv_manager_format_usage(const pkv_kv_manager* mgr, char* buf, int64_t capacity);
/* prepare_block_tables (§4.2.2) for type `type`: row b is request_ids[b]'s list,
 * padded with the null block, into table_out[B, max_blocks_per_seq].
 * PKV_ERR_INVALID_ARG if a list is longer than max_blocks_per_seq. */
int pkv_manager_block_table(const pkv_kv_manager* mgr, int32_t type, const int64_t* request_ids,
                            int32_t B, int32_t max_blocks_per_seq, int32_t* table_out);

/* Block fingerprint: BLAKE2b (RFC 7693) with an 8-byte digest, read little-endian,
 * over [parent_hash as 8 little-endian bytes, only when has_parent] + tokens as
 * int32 little-endian + group_id as int32 little-endian. The same in every process
 * (the pages' reason for not using a salted built-in hash). */
uint64_t pkv_block_hash(uint64_t parent_hash, int32_t has_parent, const int32_t* tokens,
                        int32_t num_tokens, int32_t group_id);
/* Prefix match for a new request (search_prefix_match): the longest run of
 * leading full blocks of tokens[num_tokens] whose fingerprint chain is held by a
 * live request in every type, never including the block of the last token, is
 * attached to request_id (one more reference per block). Returns the number of
 * cached tokens (a multiple of block_size; 0 with prefix caching off or a
 * sliding-window type present), or a negative error if request_id already holds
 * blocks. Follow with allocate_slots(request_id, cached, num_tokens - cached). */
int64_t pkv_manager_match_prefix(pkv_kv_manager* mgr, int64_t request_id, const int32_t* tokens,
                                 int64_t num_tokens);
/* Fingerprint the request's full blocks that are not fingerprinted yet, from its
 * tokens (call after their K/V is computed). A fingerprint already taken by
 * another block keeps that block. Fingerprints are forgotten when their block's
 * last reference is released. No-op without prefix caching. */
int pkv_manager_cache_blocks(pkv_kv_manager* mgr, int64_t request_id, const int32_t* tokens,
                             int64_t num_tokens);
/* fork_blocks: each of child_ids[num_children] (new requests) gets the first
 * ceil(num_tokens / block_size) entries of the parent's list. shareable != 0:
 * full blocks are shared (one more reference per child) and only an incomplete
 * last block is replaced by a new block to be copied; shareable == 0: every real
 * block is replaced by a new one to be copied. Null entries stay null. The copies
 * (source, destination) are written type by type, child by child, to
 * copy_src/copy_dst (capacity entries), and copies_per_type[num_types] gets each
 * type's count; run pkv_copy_blocks on every cache of a type with its pairs.
 * All-or-nothing: PKV_ERR_OUT_OF_BLOCKS or a too-small capacity
 * (PKV_ERR_INVALID_ARG) leaves everything unchanged. Returns the total copies. */
int64_t pkv_manager_fork(pkv_kv_manager* mgr, int64_t parent_id, const int64_t* child_ids,
                         int32_t num_children, int64_t num_tokens, int32_t shareable,
                         int32_t* copy_src, int32_t* copy_dst, int64_t capacity,
                         int64_t* copies_per_type);

/* ==========================================================================
 * Device calls
 * ========================================================================== */

/* Cache write through slot_mapping (standalone guide 模式二: the cache viewed as
 * [num_blocks * block_size, H_kv, d] takes row t at index slot_mapping[t]).
 *   k_cache [num_blocks, block_size, num_kv_heads, head_dim_k]  written
 *   v_cache [num_blocks, block_size, num_kv_heads, head_dim_v]  written; NULL
 *           (with v = NULL) writes the k side only
 *   k [num_tokens, num_kv_heads, head_dim_k], v [num_tokens, num_kv_heads, head_dim_v]
 *   slot_mapping [num_tokens] int32 (device)
 * The MLA latent write passes cache_nope as k (H_kv 1, 512) and cache_rope as v
 * (H_kv 1, 64). A bit-exact copy; slot < 0 skips the row; slot >= num_blocks *
 * block_size skips it and sets PKV_DEV_BAD_SLOT. Duplicate slots in one call are
 * undefined (one of the rows wins). Row sizes must be multiples of 16 bytes. With
 * num_tokens = 0 nothing is launched and k, v and slot_mapping may be NULL. */
int pkv_kv_cache_write(void* k_cache, void* v_cache, const void* k, const void* v,
                       const int32_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
                       int32_t block_size, int32_t num_kv_heads, int32_t head_dim_k,
                       int32_t head_dim_v, int* dev_status, void* stream);

/* Block copy for a fork ("KV Cache 笔记", fork_blocks: the incomplete last block
 * of a forked request is copied, full blocks are shared). cache is one device
 * cache tensor whose blocks are contiguous rows of block_bytes (any
 * [num_blocks, block_size, heads, dim] cache: block_bytes = block_size * heads *
 * dim * element size). For i in [0, n): block dst[i] becomes a bit copy of block
 * src[i]; src and dst are device int32 arrays. Sources must not be destinations of
 * the same call (pkv_manager_fork's pairs never are). A pair with an id outside
 * [0, num_blocks) is skipped and sets PKV_DEV_BAD_BLOCK. block_bytes must be a
 * positive multiple of 16 and cache 16-byte aligned (PKV_ERR_INVALID_ARG). */
int pkv_copy_blocks(void* cache, int64_t num_blocks, int64_t block_bytes, const int32_t* src,
                    const int32_t* dst, int64_t n, int* dev_status, void* stream);

/* Fused MLA cache write (standalone guide 模式三: the kv_a projection output goes
 * through kv_a_layernorm RMSNorm and RoPE and into nope_cache / rope_cache in one
 * step, optionally returning k_nope / k_rope). For each token t:
 *   k_nope[t] = bf16(x[0:512] / sqrt(mean(x[0:512]^2) + epsilon) * gamma)
 *   k_rope[t] = bf16(x[512:576] * cos[t] + rotate_half(x[512:576]) * sin[t]),
 *   rotate_half(r) = [-r[32:64], r[0:32]] (the Llama forward's RoPE, "KV Cache 笔记"),
 * with x = latent[t], arithmetic in fp32 and round-to-nearest-even results;
 * k_nope[t] goes to cache_nope row slot_mapping[t] and k_rope[t] to cache_rope.
 *   cache_nope [num_blocks, block_size, 1, 512] bf16, cache_rope [.., 1, 64] bf16
 *   k_nope_out [T, 512], k_rope_out [T, 64] bf16: optional copies (NULL = none)
 *   latent [T, 576] bf16 (512 latent + 64 rope), gamma [512] bf16
 *   cos, sin [T, 64] fp32 (per token, every rope element)
 *   slot_mapping [T] int32: negative skips the cache write of the row; a slot
 *   >= num_blocks * block_size is skipped and sets PKV_DEV_BAD_SLOT.
 * kv_lora_rank must be 512 and rope_dim 64 (PKV_ERR_UNSUPPORTED). All pointers
 * 16-byte aligned. Device pointers; asynchronous on `stream`. */
int pkv_mla_rmsnorm_rope_write(void* cache_nope, void* cache_rope, void* k_nope_out,
                               void* k_rope_out, const void* latent, const void* gamma,
                               const float* cos, const float* sin, const int32_t* slot_mapping,
                               int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                               int32_t kv_lora_rank, int32_t rope_dim, float epsilon,
                               int* dev_status, void* stream);

/* Fused rotary embedding and cache write for GQA / MHA caches, with positions of one
 * or several axes (the Llama forward's RoPE, "KV Cache 笔记", and its write through
 * slot_mapping in one pass; several axes serve image and video tokens, whose time,
 * height and width turn different pairs of a head). For token t, each q and k head x
 * and pair i < rope_dim / 2, with p = positions[pair_axis[i]][t]:
 *   c = rope_table[p][i], s = rope_table[p][rope_dim / 2 + i]
 *   (x1, x2) -> (x1 c - x2 s, x2 c + x1 s)
 * x1, x2 are elements i and i + rope_dim / 2 (interleaved = 0: rotate_half) or 2i and
 * 2i + 1 (interleaved = 1); elements from rope_dim on are copied. fp32 arithmetic, one
 * rounding to nearest even. The rotated q row goes to q_out[t], the rotated k row and
 * the v row to cache row slot_mapping[t].
 *   k_cache, v_cache [num_blocks, block_size, H_kv, head_dim] bf16
 *   q, q_out [T, H, head_dim], k, v [T, H_kv, head_dim] bf16; *_stride: elements from
 *     one token to the next (a multiple of 8; heads of a token are contiguous), so q, k
 *     and v can be slices of one projection's output
 *   rope_table [max_pos, rope_dim] fp32: rope_dim / 2 cosines, then the sines
 *   positions [num_axes, T] int32; pair_axis: HOST array of rope_dim / 2 entries in
 *     [0, num_axes), or NULL (every pair axis 0)
 *   slot_mapping [T] int32: a negative slot skips the cache write of the row (q_out is
 *     still written); a slot >= num_blocks * block_size also sets PKV_DEV_BAD_SLOT.
 * A token with a position outside [0, max_pos) on any axis is skipped altogether and
 * sets PKV_DEV_BAD_POSITION. q_out may be q itself (same pointer and stride); any other
 * overlap of q_out's rows with those of q, k or v is refused (PKV_ERR_INVALID_ARG).
 * Supported: head_dim a multiple of 16 up to 256, rope_dim a multiple of 16 up to
 * head_dim, num_axes 1..4 (PKV_ERR_UNSUPPORTED otherwise). All pointers 16-byte aligned
 * (positions and slot_mapping 4). Duplicate slots as for pkv_kv_cache_write. */
int pkv_rope_kv_cache_write(void* k_cache, void* v_cache, void* q_out, int64_t q_out_stride,
                            const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, const float* rope_table,
                            int64_t max_pos, int32_t rope_dim, const int32_t* positions,
                            int32_t num_axes, const int32_t* pair_axis, int32_t interleaved,
                            const int32_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
                            int32_t block_size, int32_t H, int32_t H_kv, int32_t head_dim,
                            int* dev_status, void* stream);

/* Decode attention, one query token per sequence (sparse_mode 0 / band 4).
 * For each b, h: o = softmax(scale * q[b,h] . K^T) V over positions
 * [max(0, len_b - window), len_b) (window <= 0: [0, len_b)) of sequence b, read
 * through block_table; query head h uses kv head h / (H / H_kv) ("KV Cache 笔记",
 * MHA -> MQA -> GQA, repeat_kv). seq_lens counts every visible position including
 * the token just written (the FA reads up to the new token: skill note §3.6).
 *   out  [B, H, head_dim] (bf16 or fp32), lse [B, H] fp32 natural log (nullable);
 *        len_b = 0 gives o = 0, lse = -inf
 *   q    [B, H, head_dim] bf16
 *   k_cache, v_cache [num_blocks, block_size, H_kv, head_dim] bf16
 *   block_table [B, max_blocks_per_seq] int32; seq_lens [B] int32 (device)
 * Supported: head_dim 128, block_size 128, H % H_kv == 0, H / H_kv <= 16.
 * Entries of block_table outside the visible range are never read. */
size_t pkv_decode_workspace_size(int32_t B, int32_t H, int32_t H_kv, int32_t head_dim);

/* Kernel used by pkv_paged_attention_decode, process-wide (not thread-safe to change
 * while calls are in flight). PKV_KERNEL_AUTO picks the tcgen05 tensor-core kernel
 * for every group size; PKV_KERNEL_CUDA_CORE forces the CUDA-core kernel. Both
 * produce the same partial results up to fp32 rounding. */
#define PKV_KERNEL_AUTO 0
#define PKV_KERNEL_CUDA_CORE 1
#define PKV_KERNEL_TENSOR_CORE 2
int pkv_set_decode_kernel(int32_t kernel);
int32_t pkv_get_decode_kernel(void);
int pkv_paged_attention_decode(void* out, int32_t out_dtype, float* lse, const void* q,
                               const void* k_cache, const void* v_cache,
                               const int32_t* block_table, int32_t max_blocks_per_seq,
                               const int32_t* seq_lens, int32_t B, int32_t H, int32_t H_kv,
                               int32_t head_dim, int32_t block_size, int64_t num_blocks,
                               float scale, int32_t window, void* workspace,
                               size_t workspace_bytes, int* dev_status, void* stream);

/* Speculative (multi-token) decode: q_len new query rows per sequence, all already
 * written to the cache (MTP verification; standalone guide appendix C: a decode
 * step with q_len > 1 takes the prefill branch, sparse_mode 3, the bottom-right
 * causal mask; design doc: allocate_slots' lookahead_tokens reserve the slots of
 * the draft rows). Query row i of sequence b sits at position len_b - q_len + i
 * and, for each head h (kv head h / (H / H_kv)), attends to the keys at positions
 * p <= len_b - q_len + i, and with window > 0 only to p > len_b - q_len + i - window:
 * each row is the decode step of the prefix that ends at its own position. A row
 * whose position is negative (len_b < q_len) returns o = 0, lse = -inf. With a
 * window, block_table must keep the blocks from position len_b - q_len + 1 - window
 * on (the generator's window is window + q_len - 1).
 *   out [B, q_len, H, head_dim] (bf16 or fp32), lse [B, q_len, H] fp32 (nullable)
 *   q   [B, q_len, H, head_dim] bf16
 *   k_cache, v_cache [num_blocks, block_size, H_kv, head_dim] bf16
 *   block_table [B, max_blocks_per_seq] int32; seq_lens [B] int32 totals (device)
 * Supported: head_dim 128, block_size 128, q_len 1..4, q_len * H / H_kv <= 32
 * (PKV_ERR_UNSUPPORTED otherwise). q_len = 1 is pkv_paged_attention_decode.
 * Workspace: pkv_decode_spec_workspace_size(B, q_len, H, H_kv, head_dim) bytes,
 * 256-byte aligned. Device pointers; asynchronous on `stream`. */
size_t pkv_decode_spec_workspace_size(int32_t B, int32_t q_len, int32_t H, int32_t H_kv,
                                      int32_t head_dim);
int pkv_paged_attention_decode_spec(void* out, int32_t out_dtype, float* lse, const void* q,
                                    const void* k_cache, const void* v_cache,
                                    const int32_t* block_table, int32_t max_blocks_per_seq,
                                    const int32_t* seq_lens, int32_t B, int32_t q_len, int32_t H,
                                    int32_t H_kv, int32_t head_dim, int32_t block_size,
                                    int64_t num_blocks, float scale, int32_t window,
                                    void* workspace, size_t workspace_bytes, int* dev_status,
                                    void* stream);

/* Sparse decode: attention over a few blocks of each sequence, chosen per query row and
 * kv head by a cheap score. The pages bound a decode step's reads by dropping positions
 * (the sliding window, "KV Cache 管理设计文档" §2.3); here the whole cache stays and each
 * step reads the part of it that matters most to its queries. Three calls, after the
 * step's rows are written: update the summaries, select, attend.
 *
 * Summaries [num_blocks, H_kv, 2, head_dim] bf16: per kv head and channel the smallest
 * (index 0) and the largest (index 1) key value of a block's rows. A cache tensor like
 * any other, in the blocks' order: pkv_copy_blocks copies it for a fork.
 *
 * pkv_update_block_summaries: for each sequence b, the rows at positions
 * [seq_lens[b] - num_new[b], seq_lens[b]), already in k_cache, enter the summaries of the
 * blocks that hold them. A block whose first row is among them starts over; any other
 * keeps what its summary says of its earlier rows. A NaN key makes its channel NaN. Rows
 * that are overwritten later (rejected drafts) go on counting until their block starts
 * over: the bounds stay bounds, only looser.
 *   max_new: at least every num_new[b] (host value; the launch is sized by it)
 * num_new 0 leaves a sequence as it is. num_new outside [0, max_new] or above seq_lens[b],
 * or seq_lens[b] > max_blocks_per_seq * block_size, skips the sequence and sets
 * PKV_DEV_BAD_LENGTH; a table entry outside [0, num_blocks) skips the block
 * (PKV_DEV_BAD_BLOCK). A block that two sequences of one call both update must not be.
 * summaries may not overlap anything the call reads (PKV_ERR_INVALID_ARG).
 * Supported: head_dim 128, block_size 128 (PKV_ERR_UNSUPPORTED otherwise). */
int pkv_update_block_summaries(void* summaries, const void* k_cache, const int32_t* block_table,
                               int32_t max_blocks_per_seq, const int32_t* seq_lens,
                               const int32_t* num_new, int32_t max_new, int32_t B, int32_t H_kv,
                               int32_t head_dim, int32_t block_size, int64_t num_blocks,
                               int* dev_status, void* stream);

/* pkv_select_blocks: for each query row (b, i) and kv head g, the num_selected blocks of the
 * sequence with the largest scores, ascending, -1 behind the last one. Row i of q_len sits
 * at position len_b - q_len + i and sees n = ceil((len_b - q_len + 1 + i) / block_size)
 * blocks (none if that is negative). Block j's score is
 *   sum_d (P_d max_jd + N_d min_jd), P_d = sum_h max(q_hd, 0), N_d = sum_h min(q_hd, 0)
 * over the H / H_kv heads h of g (sums past fp32's range count as infinite): no key of the
 * block has a larger summed dot product with them. Scores decide as they would in 64 bits, whatever the order of the sums; equal ones
 * in favour of the lower block; a NaN score ranks above all. Blocks [0, num_sink) and the
 * last num_recent that the row sees are always among the selected. A row with
 * n <= num_selected takes every block, and no summary is read for it. A summary also
 * covers the rows of a sequence behind the query row's own position.
 *   block_indices [B, q_len, H_kv, num_selected] int32 (written)
 *   q [B, q_len, H, head_dim] bf16; block_table, seq_lens as for decode
 * Table entries outside [0, num_blocks) rank below every block and set
 * PKV_DEV_BAD_BLOCK; a length past the table is clamped (PKV_DEV_BAD_LENGTH). Every block
 * that a row sees competes: a table whose expired entries hold the null block (a sliding
 * window's) does not go with it.
 * block_indices may not overlap anything the call reads (PKV_ERR_INVALID_ARG).
 * Supported: head_dim 128, block_size 128, H % H_kv == 0, H / H_kv <= 16 (lists of groups
 * that pkv_paged_attention_decode_sparse does not take are for the caller's own attention),
 * num_sink + num_recent <= num_selected, max_blocks_per_seq <= 8192 (1,048,576 tokens).
 * No workspace. */
int pkv_select_blocks(int32_t* block_indices, const void* q, const void* summaries,
                      const int32_t* block_table, int32_t max_blocks_per_seq,
                      const int32_t* seq_lens, int32_t B, int32_t q_len, int32_t H, int32_t H_kv,
                      int32_t head_dim, int32_t block_size, int64_t num_blocks,
                      int32_t num_selected, int32_t num_sink, int32_t num_recent, int* dev_status,
                      void* stream);

/* pkv_paged_attention_decode_sparse: decode attention of q_len query rows per sequence (any
 * number; row i as in pkv_paged_attention_decode_spec, without a window) in which row (b, i)
 * and kv head g attend only to the positions, up to the row's own, that lie in the blocks
 * block_indices[b][i][g] (in any order). A negative entry is an empty place. Only the first
 * min(num_selected, n) entries are read, n being the number of blocks that the row sees;
 * an entry of n or more is skipped and sets PKV_DEV_BAD_BLOCK. A block listed twice counts
 * twice. A row without a single position to attend to returns o = 0, lse = -inf; a head
 * with a NaN score (a NaN in its query or in a key that it attends to) o = lse = NaN.
 *   out, q, lse, caches, block_table, seq_lens as for pkv_paged_attention_decode_spec
 *   block_indices [B, q_len, H_kv, num_selected] int32 (device)
 * Always the tensor-core kernel, whatever pkv_set_decode_kernel chose: the weights enter the
 * value product rounded to bf16, and the same rounded weights divide it.
 * Supported: head_dim 128, block_size 128, H / H_kv in {1, 2, 4, 8, 16}.
 * Workspace: pkv_decode_sparse_workspace_size() bytes, 256-byte aligned. */
size_t pkv_decode_sparse_workspace_size(int32_t B, int32_t q_len, int32_t H, int32_t H_kv,
                                        int32_t head_dim);
int pkv_paged_attention_decode_sparse(void* out, int32_t out_dtype, float* lse, const void* q,
                                      const void* k_cache, const void* v_cache,
                                      const int32_t* block_table, int32_t max_blocks_per_seq,
                                      const int32_t* seq_lens, const int32_t* block_indices,
                                      int32_t num_selected, int32_t B, int32_t q_len, int32_t H,
                                      int32_t H_kv, int32_t head_dim, int32_t block_size,
                                      int64_t num_blocks, float scale, void* workspace,
                                      size_t workspace_bytes, int* dev_status, void* stream);

/* Prefill attention over TND-packed queries (standalone guide: sparse_mode 3 for
 * TND paged prefill, q in cumulative form, kv in direct form; "KV Cache 笔记"
 * "手写40行": the causal mask is bottom-right aligned when a cache precedes the new
 * rows). Sequence b owns query rows [cu[b-1], cu[b]) (cu[-1] = 0), q_b rows, and
 * c_b = seq_lens_kv[b] - q_b cached positions before them; its new K/V rows must
 * already be in the cache (pkv_kv_cache_write). Query row r (0-based in the
 * sequence) of head h attends, with kv head h / (H / H_kv), to keys
 * j <= c_b + r when causal = 1, to all seq_lens_kv[b] keys when causal = 0.
 * q_len = 1 rows are decode rows and mix freely with prefill rows.
 *   out [num_tokens, H, head_dim] (bf16 or fp32), lse [num_tokens, H] fp32 (nullable)
 *   q [num_tokens, H, head_dim] bf16; cu_seqlens_q [B] int32 cumulative ends (no
 *   leading zero), seq_lens_kv [B] int32 direct totals, q_b <= seq_lens_kv[b]
 *   k_cache, v_cache [num_blocks, block_size, H_kv, head_dim] bf16
 * Supported: head_dim 128, block_size 128, H / H_kv in {1, 2, 4, 8, 16}.
 * Workspace: pkv_prefill_workspace_size() bytes (depends only on the device). */
size_t pkv_prefill_workspace_size(void);
int pkv_paged_attention_prefill(void* out, int32_t out_dtype, float* lse, const void* q,
                                const int32_t* cu_seqlens_q, int32_t num_tokens,
                                const void* k_cache, const void* v_cache,
                                const int32_t* block_table, int32_t max_blocks_per_seq,
                                const int32_t* seq_lens_kv, int32_t B, int32_t H, int32_t H_kv,
                                int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                float scale, int32_t causal, void* workspace,
                                size_t workspace_bytes, int* dev_status, void* stream);

/* Absorbed MLA decode ("KVCache 优化技能" 模式三; standalone guide 模式三 FA absorb
 * call: key = value = cache_nope, query_rope / key_rope passed separately, one
 * latent kv head). For each b and query head h, over positions [0, len_b):
 *   s_j = scale * (q_nope[b,h] . nope_j + q_rope[b,h] . rope_j),  o = softmax(s) . nope
 *   out [B, H, kv_lora_rank] (bf16 or fp32), lse [B, H] fp32 natural log (nullable)
 *   q_nope [B, H, kv_lora_rank] bf16, q_rope [B, H, rope_dim] bf16
 *   cache_nope [num_blocks, block_size, 1, kv_lora_rank] bf16
 *   cache_rope [num_blocks, block_size, 1, rope_dim] bf16
 *   block_table [B, max_blocks_per_seq] int32, seq_lens [B] int32 (device)
 * New latent rows are written beforehand with pkv_kv_cache_write (k = nope,
 * v = rope). Supported: kv_lora_rank 512, rope_dim 64, block_size 128, H <= 128.
 * Workspace: pkv_mla_decode_workspace_size(B, H) bytes. */
size_t pkv_mla_decode_workspace_size(int32_t B, int32_t H);
int pkv_mla_paged_decode(void* out, int32_t out_dtype, float* lse, const void* q_nope,
                         const void* q_rope, const void* cache_nope, const void* cache_rope,
                         const int32_t* block_table, int32_t max_blocks_per_seq,
                         const int32_t* seq_lens, int32_t B, int32_t H, int32_t kv_lora_rank,
                         int32_t rope_dim, int32_t block_size, int64_t num_blocks, float scale,
                         void* workspace, size_t workspace_bytes, int* dev_status, void* stream);

/* Absorbed MLA decode of q_len new query rows per sequence (multi-token prediction
 * over an MLA cache: standalone guide appendix C, a decode step with q_len > 1 takes
 * sparse_mode 3, the bottom-right causal mask; scores as in pkv_mla_paged_decode).
 * All q_len new latent rows are already in the cache. Query row i of sequence b sits
 * at position len_b - q_len + i and attends to the positions p <= len_b - q_len + i;
 * a row whose position is negative (len_b < q_len) returns o = 0, lse = -inf.
 *   out [B, q_len, H, kv_lora_rank] (bf16 or fp32), lse [B, q_len, H] fp32 (nullable)
 *   q_nope [B, q_len, H, kv_lora_rank] bf16, q_rope [B, q_len, H, rope_dim] bf16
 *   caches, block_table as for pkv_mla_paged_decode; seq_lens [B] int32 totals
 * Supported: q_len 1..4 and the shapes of pkv_mla_paged_decode (PKV_ERR_UNSUPPORTED
 * otherwise); q_len = 1 is pkv_mla_paged_decode. Each row is its own problem: the
 * rows of one sequence run on different CTA pairs at the same time, so their reads
 * of a latent tile meet in L2 rather than each coming from HBM.
 * Workspace: pkv_mla_decode_spec_workspace_size(B, q_len, H) bytes, 256-byte
 * aligned. Device pointers; asynchronous on `stream`. */
size_t pkv_mla_decode_spec_workspace_size(int32_t B, int32_t q_len, int32_t H);
int pkv_mla_paged_decode_spec(void* out, int32_t out_dtype, float* lse, const void* q_nope,
                              const void* q_rope, const void* cache_nope, const void* cache_rope,
                              const int32_t* block_table, int32_t max_blocks_per_seq,
                              const int32_t* seq_lens, int32_t B, int32_t q_len, int32_t H,
                              int32_t kv_lora_rank, int32_t rope_dim, int32_t block_size,
                              int64_t num_blocks, float scale, void* workspace,
                              size_t workspace_bytes, int* dev_status, void* stream);

/* FP8 (E4M3) KV cache: write and decode. A quantised cache halves the bytes a decode
 * step reads. The pages list KV quantisation (skill note 高阶特性: INT8 / W8A8C8;
 * "KV Cache 笔记": KIVI-style grouped quantisation) and warn that dequantising into
 * temporary tensors every step eats the saving; here the decode kernel widens the
 * codes on chip and nothing is materialised.
 * Format: one fp32 scale per (token, kv head) row of head_dim values,
 * scale = amax / 448 (IEEE fp32 division), code = E4M3(x / scale) rounded to nearest
 * even with saturation to +-448 (the "fn" variant: no infinities, S.1111.111 =
 * NaN); an all-zero row has scale 0 and zero codes. value = code * scale. A row with an
 * infinite value has an infinite scale, and every value of it reads back as NaN.
 *   k_cache, v_cache [num_blocks, block_size, H_kv, head_dim] uint8 codes
 *   k_scale, v_scale [num_blocks, H_kv, block_size] fp32 (a block's scales of one
 *                    kv head are contiguous)
 * head_dim must be 128 (PKV_ERR_UNSUPPORTED). */

/* Quantise new rows k, v [num_tokens, H_kv, head_dim] bf16 and write codes and
 * scales through slot_mapping (negative slot: skipped; slot >= num_blocks *
 * block_size: skipped and PKV_DEV_BAD_SLOT). Caches 16-byte aligned, scales 4. NaN values
 * do not count in amax: they keep NaN codes under the scale of the row's other values, and
 * a row of nothing but NaN and zeros is written as zeros. */
int pkv_kv_cache_write_fp8(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                           const void* k, const void* v, const int32_t* slot_mapping,
                           int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                           int32_t num_kv_heads, int32_t head_dim, int* dev_status, void* stream);
/* pkv_rope_kv_cache_write into an FP8 cache: the rotated k row (fp32, not rounded to
 * bf16 first) and the v row are quantised as above, but for NaN: a row with a NaN has the
 * scale NaN and NaN codes, so that all of it reads back as NaN. head_dim must be 128
 * (PKV_ERR_UNSUPPORTED); scales 4-byte aligned. */
int pkv_rope_kv_cache_write_fp8(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                void* q_out, int64_t q_out_stride, const void* q,
                                int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const float* rope_table, int64_t max_pos,
                                int32_t rope_dim, const int32_t* positions, int32_t num_axes,
                                const int32_t* pair_axis, int32_t interleaved,
                                const int32_t* slot_mapping, int64_t num_tokens,
                                int64_t num_blocks, int32_t block_size, int32_t H, int32_t H_kv,
                                int32_t head_dim, int* dev_status, void* stream);
/* Rows of an FP8 cache widened to bf16: k[t], v[t] = code * scale of cache row
 * slot_mapping[t] (one fp32 product, rounded to nearest even), the way a quantised
 * prefix reaches pkv_paged_attention_prefill, which reads bf16 caches. A negative slot
 * gives a row of zeros, a slot >= num_blocks * block_size too and sets
 * PKV_DEV_BAD_SLOT. k, v [num_tokens, H_kv, head_dim] bf16; head_dim must be 128
 * (PKV_ERR_UNSUPPORTED). Rows and caches 16-byte aligned, scales 4. k and v may overlap
 * neither each other nor anything the call reads (PKV_ERR_INVALID_ARG). */
int pkv_kv_cache_read_fp8(void* k, void* v, const void* k_cache, const void* v_cache,
                          const float* k_scale, const float* v_scale, const int32_t* slot_mapping,
                          int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                          int32_t num_kv_heads, int32_t head_dim, int* dev_status, void* stream);
/* pkv_paged_attention_decode over an FP8 cache: same arguments, result, workspace
 * (pkv_decode_workspace_size) and error behaviour, plus the two scale arrays
 * (16-byte aligned). The attention is that of the dequantised cache; q stays bf16.
 * Rows of positions outside [max(0, len - window), len) are never used, whatever
 * bytes they hold. Always runs on the tensor cores. */
int pkv_paged_attention_decode_fp8(void* out, int32_t out_dtype, float* lse, const void* q,
                                   const void* k_cache, const void* v_cache, const float* k_scale,
                                   const float* v_scale, const int32_t* block_table,
                                   int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t B,
                                   int32_t H, int32_t H_kv, int32_t head_dim, int32_t block_size,
                                   int64_t num_blocks, float scale, int32_t window,
                                   void* workspace, size_t workspace_bytes, int* dev_status,
                                   void* stream);

/* 4-bit KV cache: write, read and decode. 72 bytes per row of 128 values where bf16 takes
 * 256 and FP8 132 (the pages' QuantizedCache: 4-bit grouped quantisation, "KV Cache 笔记").
 * Format: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), element 2i in the low
 * half of byte i and 2i + 1 in the high half, and one scale byte per 16 consecutive values:
 * the upper 8 of the 15 magnitude bits of an fp16 (5 bits of exponent, 3 of fraction).
 *   scale = the scale nearest to amax / 6, ties to the even byte, 10240 (0xE2) at most
 *   code  = the code nearest to x / scale, ties to the even one, magnitudes past 6 to 6
 *   value = code * scale (6 significant bits: exact in bf16 and fp16)
 * decided as in exact arithmetic. 16 values of which none reaches 6 * 2^-18 have scale 0 and
 * codes 0; magnitudes past 61440 are held as 61440; 16 values with an infinity or a NaN among
 * them have the scale 0xFF and read back as NaN. Scale bytes 0xE3 to 0xFE are never written, and
 * what they stand for is left open.
 *   k_cache, v_cache [num_blocks, H_kv, block_size, 64] uint8: head-major, so that what the
 *                    decode reads of a block for one kv head is one piece
 *   k_scale, v_scale [num_blocks, H_kv, block_size, 8] uint8
 * Cache tensors like any other: pkv_copy_blocks copies them for a fork. head_dim must be 128
 * (PKV_ERR_UNSUPPORTED). All pointers 16-byte aligned, slot_mapping 4. */

/* Quantise new rows and write them through slot_mapping (negative slot: skipped; slot >=
 * num_blocks * block_size: skipped and PKV_DEV_BAD_SLOT). k, v [num_tokens, H_kv, 128] bf16;
 * *_stride: elements from one token to the next (a multiple of 8; the heads of a token are
 * contiguous). k, v and slot_mapping may not overlap the caches (PKV_ERR_INVALID_ARG).
 * Duplicate slots as for pkv_kv_cache_write. */
int pkv_kv_cache_write_fp4(void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                           const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const int32_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
                           int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                           int* dev_status, void* stream);
/* Rows of a 4-bit cache widened to bf16, as pkv_kv_cache_read_fp8 does for an FP8 cache: a
 * negative slot gives a row of zeros, a slot >= num_blocks * block_size too and sets
 * PKV_DEV_BAD_SLOT. k, v [num_tokens, H_kv, 128] bf16, which may overlap neither each other
 * nor anything the call reads (PKV_ERR_INVALID_ARG). */
int pkv_kv_cache_read_fp4(void* k, void* v, const void* k_cache, const void* v_cache,
                          const void* k_scale, const void* v_scale, const int32_t* slot_mapping,
                          int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                          int32_t num_kv_heads, int32_t head_dim, int* dev_status, void* stream);
/* pkv_paged_attention_decode_spec over a 4-bit cache, q_len 1..4 rows per sequence (1: plain
 * decode): same arguments, result, workspace (pkv_decode_spec_workspace_size) and limits, plus
 * the two scale arrays. The attention is that of the dequantised cache; q stays bf16 (elements
 * smaller than 2^-22 of their row's largest lose bits), the weights enter the value product
 * rounded to fp16, and the same rounded weights divide it. Rows of positions that no query row
 * sees are never used, whatever bytes they hold. A head with a NaN score has o = lse = NaN; a
 * NaN among 16 values of V makes those 16 outputs NaN in the rows that see it. A block of the
 * table outside [0, num_blocks) is skipped (PKV_DEV_BAD_BLOCK). */
int pkv_paged_attention_decode_fp4(void* out, int32_t out_dtype, float* lse, const void* q,
                                   const void* k_cache, const void* v_cache, const void* k_scale,
                                   const void* v_scale, const int32_t* block_table,
                                   int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t B,
                                   int32_t q_len, int32_t H, int32_t H_kv, int32_t head_dim,
                                   int32_t block_size, int64_t num_blocks, float scale,
                                   int32_t window, void* workspace, size_t workspace_bytes,
                                   int* dev_status, void* stream);

/* Eviction by accumulated attention weight: rows that the queries pay little attention to
 * leave the cache (the pages drop positions by a window only, "KV Cache 管理设计文档" §2.3).
 * Three calls: after a step's attention, add its weights; now and then, select the rows that
 * stay and move them to the front. Each kv head keeps rows of its own, all heads of a sequence
 * equally many, so its block table goes on serving every head; keys carry their rotary
 * position, so a row's place in the cache does not matter to the attention.
 *
 * pkv_accumulate_attention_weights: for every position p < seq_lens[b] of sequence b, and kv
 * head g,
 *   weights[p] = (p is fresh ? 0 : decay weights[p]) +
 *                sum_i sum_h exp(scale q[b,i,h] . k[p,g] - lse[b,i,h])
 * over the query rows i with p <= seq_lens[b] - q_len + i and the H / H_kv heads h of g. lse is
 * what the step's attention returned for these rows (fp32, natural log; of any of the decode
 * calls, or the last rows of a prefill), so the terms of a head and row sum to 1. That holds for
 * attention over every visible position: what a window or a selection of blocks leaves out has
 * no part in its lse, but gets its terms here. The
 * num_fresh[b] newest positions are fresh (none if that is negative, all if it exceeds the
 * length): rows that the step wrote, whose places may hold another request's sums.
 *   weights [num_blocks, H_kv, block_size] fp32: a cache tensor like any other, in the blocks'
 *     order (pkv_copy_blocks copies it for a fork, pkv_compact_rows moves it with its rows)
 *   q [B, q_len, H, head_dim] bf16, lse [B, q_len, H] fp32, any q_len
 *   k_cache, k_scale by key_format: PKV_KEYS_BF16 [num_blocks, block_size, H_kv, head_dim] bf16
 *     and NULL; PKV_KEYS_FP8 the FP8 cache's codes and scales; PKV_KEYS_FP4 the 4-bit cache's
 * Positions that no row sees hold any bytes; a NaN score makes the position's sum NaN. fp32
 * sums in a fixed order: the same call gives the same bits. No block may be there twice in a
 * call, in two sequences (their sums would race: call once per sequence) or in one (the null
 * blocks in front of a sliding window's table). Table entries
 * outside [0, num_blocks) are skipped (PKV_DEV_BAD_BLOCK), lengths past the table clamped
 * (PKV_DEV_BAD_LENGTH). weights may not overlap anything the call reads
 * (PKV_ERR_INVALID_ARG). Supported: head_dim 128, block_size 128, H % H_kv == 0,
 * H / H_kv <= 16 (PKV_ERR_UNSUPPORTED otherwise). No workspace. */
#define PKV_KEYS_BF16 0
#define PKV_KEYS_FP8 1
#define PKV_KEYS_FP4 2
int pkv_accumulate_attention_weights(float* weights, const void* q, const float* lse,
                                     const void* k_cache, const void* k_scale, int32_t key_format,
                                     const int32_t* block_table, int32_t max_blocks_per_seq,
                                     const int32_t* seq_lens, const int32_t* num_fresh, int32_t B,
                                     int32_t q_len, int32_t H, int32_t H_kv, int32_t head_dim,
                                     int32_t block_size, int64_t num_blocks, float scale,
                                     float decay, int* dev_status, void* stream);

/* pkv_select_rows: for each sequence and kv head the num_keep positions with the largest
 * weights, ascending, -1 behind the last one. Positions [0, num_sink) and the last num_recent
 * are always among them; equal weights are taken lowest position first (-0 equals 0), a NaN
 * ranks above all. A sequence with no more than num_keep positions keeps every one, and no
 * weight of it is read. Rows of a table entry outside [0, num_blocks) rank below all
 * (PKV_DEV_BAD_BLOCK); lengths past the table are clamped (PKV_DEV_BAD_LENGTH).
 *   kept [B, H_kv, num_keep] int32 (written, 16-byte aligned), which may not overlap anything the
 *     call reads
 * max_blocks_per_seq chooses how many CTAs share a row, so the same sequences take longer behind a
 * wider table: give it the width that the longest sequence needs.
 * Supported: block_size 128, num_sink + num_recent <= num_keep <= 2^30, max_blocks_per_seq
 * <= 32768 (4,194,304 tokens). No workspace. */
int pkv_select_rows(int32_t* kept, const float* weights, const int32_t* block_table,
                    int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t B, int32_t H_kv,
                    int32_t block_size, int64_t num_blocks, int32_t num_keep, int32_t num_sink,
                    int32_t num_recent, int* dev_status, void* stream);

/* pkv_compact_rows: in each of num_caches caches, row i of sequence b and kv head g becomes
 * what row kept[b][g][i] was, for i up to the first negative entry; afterwards the sequence has
 * that many rows and its blocks behind them can go back to the pool. Rows behind stay as they
 * were. kept[b][g] must ascend, every entry above the one before, the negative ones behind the last
 * (pkv_select_rows' does).
 *   caches, row_bytes, head_major: HOST arrays. A cache is [num_blocks, block_size, H_kv] rows
 *     of row_bytes (head_major 0: the bf16 and FP8 caches), or [num_blocks, H_kv, block_size]
 *     (head_major 1: the 4-bit cache, scales, weights). Caches may not overlap one another,
 *     kept or the tables (PKV_ERR_INVALID_ARG).
 *   new_block_table [B, new_max_blocks_per_seq] int32, or NULL (or block_table itself): in place.
 *     With a table, rows are read through block_table and written through the new one (for blocks
 *     that other requests share); the new one's blocks for the kept rows must be none of those
 *     that the call reads. No block that one sequence writes may be read or written by another.
 * Entries past block_table set PKV_DEV_BAD_LENGTH, rows of a block outside [0, num_blocks)
 * PKV_DEV_BAD_BLOCK; neither is moved. Supported: row_bytes a multiple of 4 up to 65536, up to 16 caches,
 * num_keep <= 2^30 (PKV_ERR_UNSUPPORTED otherwise). Caches 16-byte aligned. No workspace. */
int pkv_compact_rows(void* const* caches, const int32_t* row_bytes, const int32_t* head_major,
                     int32_t num_caches, const int32_t* kept, int32_t num_keep,
                     const int32_t* block_table, int32_t max_blocks_per_seq,
                     const int32_t* new_block_table, int32_t new_max_blocks_per_seq, int32_t B,
                     int32_t H_kv, int32_t block_size, int64_t num_blocks, int* dev_status,
                     void* stream);

/* Decode without any caller-provided scratch. The paper has no counterpart for
 * this call; it exists for callers that cannot allocate device memory (a plugin
 * inside a runtime that owns the allocator, a serving loop whose HBM is already
 * fully partitioned, code that must not risk the device synchronisation a
 * cudaMalloc can cause). Same arguments and result as pkv_paged_attention_decode
 * minus the workspace: the split-KV partials live in a file-scope device array of
 * PKV_DECODE_STATIC_SCRATCH_BYTES that every GPU loading the library keeps until
 * the process exits.
 *   - Rejects (PKV_ERR_WORKSPACE) any problem whose workspace would exceed that
 *     size (pkv_decode_workspace_size(B, H, H_kv, head_dim) tells).
 *   - Allocates nothing and calls no allocating routine.
 *   - The first call on a device, with that device current, looks up the array's
 *     device address (cudaGetSymbolAddress) and caches it for the process; make
 *     that first call before any stream capture. The cached address belongs to the
 *     device's primary context: it is not valid across cudaDeviceReset or in a
 *     non-primary driver context.
 *   - Runs on the current device, with its copy of the array: the pointers and
 *     `stream` must belong to that device.
 *   - All calls share the one array, which keeps the last call's contents. No part
 *     of it needs to start at zero. Calls that overlap on the GPU (other streams,
 *     other host threads) race on it: serialise them. */
#define PKV_DECODE_STATIC_SCRATCH_BYTES (8 * 1024 * 1024)
int pkv_paged_attention_decode_static(void* out, int32_t out_dtype, float* lse, const void* q,
                                      const void* k_cache, const void* v_cache,
                                      const int32_t* block_table, int32_t max_blocks_per_seq,
                                      const int32_t* seq_lens, int32_t B, int32_t H, int32_t H_kv,
                                      int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                      float scale, int32_t window, int* dev_status, void* stream);

/* ==========================================================================
 * Self-tests (no counterpart in the pages: checks of the kernels' failure path and
 * of what the block selection takes its products to be)
 * ========================================================================== */

/* Launches one small kernel that waits, with the bounded wait routines every
 * attention kernel uses, on an mbarrier that nothing completes. Each wait gives up
 * after its cycle limit (about a second at full clock) and the kernel sets
 * PKV_DEV_TIMEOUT in *dev_status (device memory, caller-owned; other bits are left
 * as they are), then returns: the CUDA context stays usable. Asynchronous on
 * `stream`. Errors: PKV_ERR_INVALID_ARG for a null dev_status; PKV_ERR_LAUNCH if
 * the launch fails. */
int pkv_selftest_bounded_wait(int* dev_status, void* stream);

/* n products d = a b of 16 x 16 and 16 x 8 bf16 matrices with fp32 sums, by the matrix
 * instruction that scores blocks: a [n, 16, 16] by rows, b [n, 8, 16] by columns,
 * d [n, 16, 8] by rows, device memory, 16-byte aligned. The selection is exact as long
 * as a product is off by at most 32 2^-24 of the sum of its terms' magnitudes. */
int pkv_selftest_bf16_products(float* d, const void* a, const void* b, int32_t n, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PAGED_KV_H */
