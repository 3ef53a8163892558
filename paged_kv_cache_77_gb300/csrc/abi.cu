// C ABI entry points for the device calls: argument validation, workspace
// carving and kernel dispatch onto the caller's stream. Nothing here allocates,
// frees or synchronises device memory.
#include <cuda_runtime.h>

#include <cmath>

#include "abi_common.h"
#include "launch.h"

namespace pkv {

// SM count of the current device (queried once per device).
static int current_num_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  static int cached[64] = {0};
  if (dev >= 0 && dev < 64 && cached[dev]) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) cached[dev] = n;
  return n;
}

// Decode kernel choice (process-wide): 0 = automatic, 1 = CUDA cores, 2 = tensor cores.
static int g_decode_kernel = 0;

static int launch_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return PKV_OK;
  set_error("%s: %s", what, cudaGetErrorString(e));
  return PKV_ERR_LAUNCH;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_kv_cache_write(void* k_cache, void* v_cache, const void* k, const void* v,
                       const int32_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
                       int32_t block_size, int32_t num_kv_heads, int32_t head_dim_k,
                       int32_t head_dim_v, int* dev_status, void* stream) {
  PKV_REQUIRE(num_tokens >= 0 && num_blocks > 0 && block_size > 0 && num_kv_heads > 0 &&
                  head_dim_k > 0,
              PKV_ERR_INVALID_ARG, "pkv_kv_cache_write: non-positive size");
  PKV_REQUIRE(k_cache && (num_tokens == 0 || (k && slot_mapping)), PKV_ERR_INVALID_ARG,
              "pkv_kv_cache_write: null pointer");
  // v goes with v_cache; with no rows to write, v may be NULL (an empty tensor's
  // storage) either way.
  PKV_REQUIRE(v_cache ? (num_tokens == 0 || v != nullptr) : (v == nullptr), PKV_ERR_INVALID_ARG,
              "pkv_kv_cache_write: v_cache and v must both be set or both be NULL");
  const int64_t row_k = (int64_t)num_kv_heads * head_dim_k * 2;
  const int64_t row_v = v_cache ? (int64_t)num_kv_heads * head_dim_v * 2 : 0;
  PKV_REQUIRE(row_k % 16 == 0 && row_v % 16 == 0, PKV_ERR_UNSUPPORTED,
              "pkv_kv_cache_write: row sizes must be multiples of 16 bytes");
  PKV_REQUIRE(aligned16(k_cache) && aligned16(k) && aligned16(v_cache) && aligned16(v),
              PKV_ERR_INVALID_ARG, "pkv_kv_cache_write: pointers must be 16-byte aligned");
  const int64_t num_slots = num_blocks * block_size;
  clear_error();
  return launch_status(launch_kv_write(k_cache, v_cache, k, v, slot_mapping, num_tokens, num_slots,
                                       row_k, row_v, dev_status, (cudaStream_t)stream,
                                       current_num_sms()),
                       "pkv_kv_cache_write");
}

int pkv_copy_blocks(void* cache, int64_t num_blocks, int64_t block_bytes, const int32_t* src,
                    const int32_t* dst, int64_t n, int* dev_status, void* stream) {
  PKV_REQUIRE(num_blocks > 0 && n >= 0 && block_bytes > 0 && block_bytes % 16 == 0,
              PKV_ERR_INVALID_ARG, "pkv_copy_blocks: bad sizes");
  PKV_REQUIRE(cache && aligned16(cache) && (n == 0 || (src && dst)), PKV_ERR_INVALID_ARG,
              "pkv_copy_blocks: null or misaligned pointer");
  clear_error();
  return launch_status(launch_copy_blocks(cache, num_blocks, block_bytes, src, dst, n, dev_status,
                                          (cudaStream_t)stream, current_num_sms()),
                       "pkv_copy_blocks");
}

int pkv_mla_rmsnorm_rope_write(void* cache_nope, void* cache_rope, void* k_nope_out,
                               void* k_rope_out, const void* latent, const void* gamma,
                               const float* cos, const float* sin, const int32_t* slot_mapping,
                               int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                               int32_t kv_lora_rank, int32_t rope_dim, float epsilon,
                               int* dev_status, void* stream) {
  PKV_REQUIRE(num_tokens >= 0 && num_blocks > 0 && block_size > 0, PKV_ERR_INVALID_ARG,
              "pkv_mla_rmsnorm_rope_write: bad sizes");
  PKV_REQUIRE(kv_lora_rank == 512 && rope_dim == 64, PKV_ERR_UNSUPPORTED,
              "pkv_mla_rmsnorm_rope_write: only kv_lora_rank 512 and rope_dim 64 are implemented");
  PKV_REQUIRE(std::isfinite(epsilon) && epsilon >= 0.f, PKV_ERR_INVALID_ARG,
              "pkv_mla_rmsnorm_rope_write: epsilon must be finite and >= 0");
  PKV_REQUIRE(cache_nope && cache_rope && gamma &&
                  (num_tokens == 0 || (latent && cos && sin && slot_mapping)),
              PKV_ERR_INVALID_ARG, "pkv_mla_rmsnorm_rope_write: null pointer");
  PKV_REQUIRE(aligned16(cache_nope) && aligned16(cache_rope) && aligned16(k_nope_out) &&
                  aligned16(k_rope_out) && aligned16(latent) && aligned16(gamma) && aligned16(cos) &&
                  aligned16(sin),
              PKV_ERR_INVALID_ARG, "pkv_mla_rmsnorm_rope_write: pointers must be 16-byte aligned");
  clear_error();
  return launch_status(
      launch_mla_rmsnorm_rope_write(cache_nope, cache_rope, k_nope_out, k_rope_out, latent, gamma,
                                    cos, sin, slot_mapping, num_tokens, num_blocks * block_size,
                                    epsilon, dev_status, (cudaStream_t)stream, current_num_sms()),
      "pkv_mla_rmsnorm_rope_write");
}

int pkv_set_decode_kernel(int32_t kernel) {
  PKV_REQUIRE(kernel >= PKV_KERNEL_AUTO && kernel <= PKV_KERNEL_TENSOR_CORE, PKV_ERR_INVALID_ARG,
              "pkv_set_decode_kernel: unknown kernel %d", kernel);
  g_decode_kernel = kernel;
  return PKV_OK;
}

int32_t pkv_get_decode_kernel(void) { return g_decode_kernel; }

size_t pkv_decode_workspace_size(int32_t B, int32_t H, int32_t H_kv, int32_t head_dim) {
  if (B < 0 || H <= 0 || H_kv <= 0 || H % H_kv || head_dim <= 0) return 0;
  return decode_workspace_bytes(B, H, H_kv, head_dim, current_num_sms());
}

}  // extern "C"

namespace {

// Validation and argument set-up shared by the decode entry points. `what` names
// the caller in error messages; *empty is set when B == 0 (nothing to launch).
int decode_setup(pkv::DecodeArgs& a, bool* empty, const char* what, void* out, int32_t out_dtype,
                 float* lse, const void* q, const void* k_cache, const void* v_cache,
                 const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                 int32_t B, int32_t H, int32_t H_kv, int32_t head_dim, int32_t block_size,
                 int64_t num_blocks, float scale, int32_t window, void* workspace,
                 size_t workspace_bytes, int* dev_status, int32_t q_len = 1) {
  using namespace pkv;
  *empty = false;
  PKV_REQUIRE(B >= 0 && H > 0 && H_kv > 0 && max_blocks_per_seq > 0 && num_blocks > 0,
              PKV_ERR_INVALID_ARG, "%s: bad sizes", what);
  PKV_REQUIRE(H % H_kv == 0, PKV_ERR_INVALID_ARG, "%s: H (%d) not a multiple of H_kv (%d)", what,
              H, H_kv);
  const int n_rep = H / H_kv;
  PKV_REQUIRE(head_dim == 128 && block_size == 128, PKV_ERR_UNSUPPORTED,
              "%s: only head_dim 128 and block_size 128 are implemented", what);
  PKV_REQUIRE(n_rep == 1 || n_rep == 2 || n_rep == 4 || n_rep == 8 || n_rep == 16,
              PKV_ERR_UNSUPPORTED, "%s: H / H_kv = %d unsupported", what, n_rep);
  PKV_REQUIRE(out_dtype == PKV_BF16 || out_dtype == PKV_F32, PKV_ERR_INVALID_ARG,
              "%s: bad out_dtype", what);
  PKV_REQUIRE(std::isfinite(scale) && scale > 0.f, PKV_ERR_INVALID_ARG,
              "%s: scale must be a positive finite number", what);
  PKV_REQUIRE(window >= 0, PKV_ERR_INVALID_ARG, "%s: negative window", what);
  PKV_REQUIRE(q_len >= 1 && q_len <= 4, PKV_ERR_UNSUPPORTED, "%s: q_len %d outside 1..4", what,
              q_len);
  PKV_REQUIRE(q_len * n_rep <= 32, PKV_ERR_UNSUPPORTED,
              "%s: q_len * H / H_kv = %d exceeds 32 query rows per kv head", what, q_len * n_rep);
  PKV_REQUIRE(window <= INT32_MAX - 4, PKV_ERR_INVALID_ARG, "%s: window too large", what);
  PKV_REQUIRE(num_blocks * block_size <= INT32_MAX, PKV_ERR_UNSUPPORTED,
              "%s: num_blocks * block_size must fit in int32", what);
  if (B == 0) {
    *empty = true;
    return PKV_OK;
  }
  PKV_REQUIRE(out && q && k_cache && v_cache && block_table && seq_lens, PKV_ERR_INVALID_ARG,
              "%s: null pointer", what);
  PKV_REQUIRE(aligned16(out) && aligned16(q) && aligned16(k_cache) && aligned16(v_cache),
              PKV_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", what);
  const int G = current_num_sms();
  PKV_REQUIRE(G > 0, PKV_ERR_LAUNCH, "%s: no CUDA device", what);
  const size_t need = decode_workspace_bytes(B, H * q_len, H_kv, head_dim, G);
  PKV_REQUIRE(workspace && workspace_bytes >= need && (((uintptr_t)workspace) & 255) == 0,
              PKV_ERR_WORKSPACE, "%s: workspace needs %zu bytes, 256-aligned", what, need);
  a = DecodeArgs{};
  a.q = (const uint16_t*)q;
  a.k_cache = (const uint8_t*)k_cache;
  a.v_cache = (const uint8_t*)v_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.dev_status = dev_status;
  a.num_blocks = num_blocks;
  a.B = B;
  a.H = H;
  a.Hkv = H_kv;
  a.n_rep = n_rep;
  a.max_blocks = max_blocks_per_seq;
  a.q_len = q_len;
  a.row_window = window;
  a.window = window > 0 ? window + q_len - 1 : 0;
  a.out_f32 = out_dtype == PKV_F32;
  a.num_ctas = G;
  a.scale_log2 = scale * 1.4426950408889634f;
  decode_workspace_carve(a, workspace);
  return PKV_OK;
}

}  // namespace

extern "C" {

int pkv_paged_attention_decode(void* out, int32_t out_dtype, float* lse, const void* q,
                               const void* k_cache, const void* v_cache,
                               const int32_t* block_table, int32_t max_blocks_per_seq,
                               const int32_t* seq_lens, int32_t B, int32_t H, int32_t H_kv,
                               int32_t head_dim, int32_t block_size, int64_t num_blocks,
                               float scale, int32_t window, void* workspace,
                               size_t workspace_bytes, int* dev_status, void* stream) {
  DecodeArgs a;
  bool empty;
  const int rc0 = decode_setup(a, &empty, "pkv_paged_attention_decode", out, out_dtype, lse, q,
                               k_cache, v_cache, block_table, max_blocks_per_seq, seq_lens, B, H,
                               H_kv, head_dim, block_size, num_blocks, scale, window, workspace,
                               workspace_bytes, dev_status);
  if (rc0 != PKV_OK || empty) return rc0;
  clear_error();
  cudaStream_t s = (cudaStream_t)stream;
  // Automatic choice: the tcgen05 kernel for every group size (also faster for n_rep 1:
  // 21.7 against 25.1 us on the tiny MHA workload).
  const bool tensor_cores = g_decode_kernel != PKV_KERNEL_CUDA_CORE;
  int rc = launch_status(tensor_cores ? launch_decode_tc(a, s) : launch_decode_simt(a, s),
                         "pkv_paged_attention_decode (attention)");
  if (rc != PKV_OK) return rc;
  return launch_status(launch_decode_merge(a, s), "pkv_paged_attention_decode (merge)");
}

size_t pkv_decode_spec_workspace_size(int32_t B, int32_t q_len, int32_t H, int32_t H_kv,
                                      int32_t head_dim) {
  if (B < 0 || q_len < 1 || H <= 0 || H_kv <= 0 || H % H_kv || head_dim <= 0) return 0;
  return decode_workspace_bytes(B, H * q_len, H_kv, head_dim, current_num_sms());
}

int pkv_paged_attention_decode_spec(void* out, int32_t out_dtype, float* lse, const void* q,
                                    const void* k_cache, const void* v_cache,
                                    const int32_t* block_table, int32_t max_blocks_per_seq,
                                    const int32_t* seq_lens, int32_t B, int32_t q_len, int32_t H,
                                    int32_t H_kv, int32_t head_dim, int32_t block_size,
                                    int64_t num_blocks, float scale, int32_t window,
                                    void* workspace, size_t workspace_bytes, int* dev_status,
                                    void* stream) {
  DecodeArgs a;
  bool empty;
  const int rc0 = decode_setup(a, &empty, "pkv_paged_attention_decode_spec", out, out_dtype, lse,
                               q, k_cache, v_cache, block_table, max_blocks_per_seq, seq_lens, B,
                               H, H_kv, head_dim, block_size, num_blocks, scale, window, workspace,
                               workspace_bytes, dev_status, q_len);
  if (rc0 != PKV_OK || empty) return rc0;
  clear_error();
  cudaStream_t s = (cudaStream_t)stream;
  int rc = launch_status(launch_decode_spec(a, s), "pkv_paged_attention_decode_spec (attention)");
  if (rc != PKV_OK) return rc;
  return launch_status(launch_decode_merge(a, s), "pkv_paged_attention_decode_spec (merge)");
}

int pkv_kv_cache_write_fp8(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                           const void* k, const void* v, const int32_t* slot_mapping,
                           int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                           int32_t num_kv_heads, int32_t head_dim, int* dev_status, void* stream) {
  PKV_REQUIRE(num_tokens >= 0 && num_blocks > 0 && block_size > 0 && num_kv_heads > 0,
              PKV_ERR_INVALID_ARG, "pkv_kv_cache_write_fp8: bad sizes");
  PKV_REQUIRE(head_dim == 128, PKV_ERR_UNSUPPORTED,
              "pkv_kv_cache_write_fp8: only head_dim 128 is implemented");
  PKV_REQUIRE(k_cache && v_cache && k_scale && v_scale && (num_tokens == 0 || (k && v && slot_mapping)),
              PKV_ERR_INVALID_ARG, "pkv_kv_cache_write_fp8: null pointer");
  PKV_REQUIRE(aligned16(k_cache) && aligned16(v_cache) && aligned16(k) && aligned16(v) &&
                  (((uintptr_t)k_scale) & 3) == 0 && (((uintptr_t)v_scale) & 3) == 0,
              PKV_ERR_INVALID_ARG, "pkv_kv_cache_write_fp8: misaligned pointer");
  clear_error();
  return launch_status(launch_kv_write_fp8(k_cache, v_cache, k_scale, v_scale, k, v, slot_mapping,
                                           num_tokens, num_blocks, block_size, num_kv_heads,
                                           dev_status, (cudaStream_t)stream, current_num_sms()),
                       "pkv_kv_cache_write_fp8");
}

}  // extern "C"

namespace {

// Whether [a, a + a_bytes) and [b, b + b_bytes) share a byte.
bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t pa = (uintptr_t)a, pb = (uintptr_t)b;
  return a_bytes > 0 && b_bytes > 0 && pa < pb + (uint64_t)b_bytes && pb < pa + (uint64_t)a_bytes;
}

// Whether rows of `width` elements at a + t * a_stride and b + t * b_stride (t < tokens, 2-byte
// elements) can share an element. Rows that run through one buffer at a common stride, as
// slices of a projection's output do, are apart when their columns are.
bool rows_overlap(const void* a, int64_t a_stride, int64_t a_width, const void* b, int64_t b_stride,
                  int64_t b_width, int64_t tokens) {
  const int64_t pa = (int64_t)((uintptr_t)a / 2), pb = (int64_t)((uintptr_t)b / 2);
  const int64_t end_a = pa + (tokens - 1) * a_stride + a_width;
  const int64_t end_b = pb + (tokens - 1) * b_stride + b_width;
  if (end_a <= pb || end_b <= pa) return false;
  if (a_stride != b_stride || a_stride <= 0) return true;
  const int64_t off = (((pb - pa) % a_stride) + a_stride) % a_stride;  // b's first column after a's
  return !(off >= a_width && off + b_width <= a_stride);
}

// Validation and argument set-up shared by the 4-bit write and read.
int fp4_setup(pkv::KvFp4Args& a, const char* what, const void* k_cache, const void* v_cache,
              const void* k_scale, const void* v_scale, const void* k, const void* v,
              const int32_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
              int32_t block_size, int32_t num_kv_heads, int32_t head_dim, int* dev_status) {
  using namespace pkv;
  PKV_REQUIRE(num_tokens >= 0 && num_blocks > 0 && block_size > 0 && num_kv_heads > 0,
              PKV_ERR_INVALID_ARG, "%s: bad sizes", what);
  PKV_REQUIRE(head_dim == 128, PKV_ERR_UNSUPPORTED, "%s: only head_dim 128 is implemented", what);
  PKV_REQUIRE(num_blocks * block_size <= INT32_MAX, PKV_ERR_UNSUPPORTED,
              "%s: num_blocks * block_size must fit in int32", what);
  PKV_REQUIRE(num_tokens <= INT32_MAX / 2 / num_kv_heads, PKV_ERR_UNSUPPORTED,
              "%s: too many rows (2 num_tokens * H_kv must fit in int32)", what);
  PKV_REQUIRE(k_cache && v_cache && k_scale && v_scale && (num_tokens == 0 || (k && v && slot_mapping)),
              PKV_ERR_INVALID_ARG, "%s: null pointer", what);
  PKV_REQUIRE(aligned16(k_cache) && aligned16(v_cache) && aligned16(k_scale) && aligned16(v_scale) &&
                  aligned16(k) && aligned16(v) && (((uintptr_t)slot_mapping) & 3) == 0,
              PKV_ERR_INVALID_ARG, "%s: misaligned pointer", what);
  a = KvFp4Args{(uint8_t*)k_cache, (uint8_t*)v_cache, (uint8_t*)k_scale, (uint8_t*)v_scale, slot_mapping,
                dev_status, num_tokens, num_blocks, block_size, num_kv_heads, 0, {}, {}};
  return PKV_OK;
}

// Whether [p, p + bytes) shares a byte with a 4-bit cache's codes or scales.
bool fp4_overlaps(const pkv::KvFp4Args& a, const void* p, int64_t bytes) {
  const int64_t rows = a.num_blocks * a.block_size * a.hkv;
  return overlap(p, bytes, a.k_cache, rows * 64) || overlap(p, bytes, a.v_cache, rows * 64) ||
         overlap(p, bytes, a.k_scale, rows * 8) || overlap(p, bytes, a.v_scale, rows * 8);
}

// Validation and argument set-up shared by the two rotary writes.
int rope_setup(pkv::RopeArgs& a, const char* what, void* k_cache, void* v_cache, void* q_out,
               int64_t q_out_stride, const void* q, int64_t q_stride, const void* k,
               int64_t k_stride, const void* v, int64_t v_stride, const float* rope_table,
               int64_t max_pos, int32_t rope_dim, const int32_t* positions, int32_t num_axes,
               const int32_t* pair_axis, const int32_t* slot_mapping, int64_t num_tokens,
               int64_t num_blocks, int32_t block_size, int32_t H, int32_t H_kv, int32_t head_dim,
               int* dev_status) {
  using namespace pkv;
  PKV_REQUIRE(num_tokens >= 0 && num_blocks > 0 && block_size > 0 && H > 0 && H_kv > 0 &&
                  head_dim > 0 && rope_dim > 0 && max_pos > 0,
              PKV_ERR_INVALID_ARG, "%s: non-positive size", what);
  PKV_REQUIRE(head_dim % 16 == 0 && head_dim <= kRopeMaxDim, PKV_ERR_UNSUPPORTED,
              "%s: head_dim must be a multiple of 16 up to %d", what, kRopeMaxDim);
  PKV_REQUIRE(rope_dim % 16 == 0 && rope_dim <= head_dim, PKV_ERR_UNSUPPORTED,
              "%s: rope_dim must be a multiple of 16 up to head_dim", what);
  PKV_REQUIRE(num_axes >= 1 && num_axes <= kRopeMaxAxes, PKV_ERR_UNSUPPORTED,
              "%s: 1 to %d position axes are implemented", what, kRopeMaxAxes);
  // The kernel counts the heads of a token in 32 bits, and a row's elements from them.
  PKV_REQUIRE((int64_t)H + 2 * (int64_t)H_kv <= (1 << 20), PKV_ERR_UNSUPPORTED,
              "%s: too many heads", what);
  PKV_REQUIRE(num_blocks * block_size <= INT32_MAX, PKV_ERR_UNSUPPORTED,
              "%s: num_blocks * block_size must fit in int32", what);
  PKV_REQUIRE(k_cache && v_cache && rope_table &&
                  (num_tokens == 0 || (q && k && v && q_out && positions && slot_mapping)),
              PKV_ERR_INVALID_ARG, "%s: null pointer", what);
  PKV_REQUIRE(aligned16(k_cache) && aligned16(v_cache) && aligned16(q) && aligned16(k) &&
                  aligned16(v) && aligned16(q_out) && aligned16(rope_table),
              PKV_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", what);
  const int64_t q_width = (int64_t)H * head_dim, kv_width = (int64_t)H_kv * head_dim;
  PKV_REQUIRE(q_stride >= 0 && k_stride >= 0 && v_stride >= 0 && q_stride % 8 == 0 &&
                  k_stride % 8 == 0 && v_stride % 8 == 0 && q_out_stride % 8 == 0 &&
                  (num_tokens <= 1 || q_out_stride >= q_width),
              PKV_ERR_INVALID_ARG, "%s: bad token stride", what);
  if (num_tokens > 0) {
    const bool in_place = q_out == q && (q_out_stride == q_stride || num_tokens == 1);
    PKV_REQUIRE((in_place ||
                 !rows_overlap(q_out, q_out_stride, q_width, q, q_stride, q_width, num_tokens)) &&
                    !rows_overlap(q_out, q_out_stride, q_width, k, k_stride, kv_width, num_tokens) &&
                    !rows_overlap(q_out, q_out_stride, q_width, v, v_stride, kv_width, num_tokens),
                PKV_ERR_INVALID_ARG, "%s: q_out overlaps q, k or v", what);
  }
  a = RopeArgs{};
  for (int i = 0; i < rope_dim / 2; ++i) {
    const int32_t axis = pair_axis ? pair_axis[i] : 0;
    PKV_REQUIRE(axis >= 0 && axis < num_axes, PKV_ERR_INVALID_ARG,
                "%s: pair_axis[%d] = %d outside the %d axes", what, i, axis, num_axes);
    a.pair_axis[i] = (uint8_t)axis;
    a.chunk_axis[i / 8] = (i % 8 == 0 || a.chunk_axis[i / 8] == axis) ? (int8_t)axis : (int8_t)-1;
  }
  a.q = (const uint16_t*)q;
  a.k = (const uint16_t*)k;
  a.v = (const uint16_t*)v;
  a.q_out = (uint16_t*)q_out;
  a.k_cache = (uint8_t*)k_cache;
  a.v_cache = (uint8_t*)v_cache;
  a.table = rope_table;
  a.positions = positions;
  a.slots = slot_mapping;
  a.dev_status = dev_status;
  a.num_tokens = num_tokens;
  a.num_slots = num_blocks * block_size;
  a.max_pos = max_pos;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.H = H;
  a.Hkv = H_kv;
  a.head_dim = head_dim;
  a.rope_dim = rope_dim;
  a.num_axes = num_axes;
  a.block_size = block_size;
  return PKV_OK;
}

}  // namespace

extern "C" {

int pkv_rope_kv_cache_write(void* k_cache, void* v_cache, void* q_out, int64_t q_out_stride,
                            const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, const float* rope_table,
                            int64_t max_pos, int32_t rope_dim, const int32_t* positions,
                            int32_t num_axes, const int32_t* pair_axis, int32_t interleaved,
                            const int32_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
                            int32_t block_size, int32_t H, int32_t H_kv, int32_t head_dim,
                            int* dev_status, void* stream) {
  RopeArgs a;
  const int rc = rope_setup(a, "pkv_rope_kv_cache_write", k_cache, v_cache, q_out, q_out_stride, q,
                            q_stride, k, k_stride, v, v_stride, rope_table, max_pos, rope_dim,
                            positions, num_axes, pair_axis, slot_mapping, num_tokens, num_blocks,
                            block_size, H, H_kv, head_dim, dev_status);
  if (rc != PKV_OK) return rc;
  clear_error();
  return launch_status(launch_rope_write(a, false, interleaved != 0, (cudaStream_t)stream,
                                         current_num_sms()),
                       "pkv_rope_kv_cache_write");
}

int pkv_rope_kv_cache_write_fp8(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                void* q_out, int64_t q_out_stride, const void* q,
                                int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const float* rope_table, int64_t max_pos,
                                int32_t rope_dim, const int32_t* positions, int32_t num_axes,
                                const int32_t* pair_axis, int32_t interleaved,
                                const int32_t* slot_mapping, int64_t num_tokens,
                                int64_t num_blocks, int32_t block_size, int32_t H, int32_t H_kv,
                                int32_t head_dim, int* dev_status, void* stream) {
  PKV_REQUIRE(head_dim == 128, PKV_ERR_UNSUPPORTED,
              "pkv_rope_kv_cache_write_fp8: only head_dim 128 is implemented");
  RopeArgs a;
  const int rc = rope_setup(a, "pkv_rope_kv_cache_write_fp8", k_cache, v_cache, q_out, q_out_stride,
                            q, q_stride, k, k_stride, v, v_stride, rope_table, max_pos, rope_dim,
                            positions, num_axes, pair_axis, slot_mapping, num_tokens, num_blocks,
                            block_size, H, H_kv, head_dim, dev_status);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(k_scale && v_scale && (((uintptr_t)k_scale) & 3) == 0 &&
                  (((uintptr_t)v_scale) & 3) == 0,
              PKV_ERR_INVALID_ARG,
              "pkv_rope_kv_cache_write_fp8: scale arrays must be set and 4-byte aligned");
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  clear_error();
  return launch_status(launch_rope_write(a, true, interleaved != 0, (cudaStream_t)stream,
                                         current_num_sms()),
                       "pkv_rope_kv_cache_write_fp8");
}

int pkv_kv_cache_read_fp8(void* k, void* v, const void* k_cache, const void* v_cache,
                          const float* k_scale, const float* v_scale, const int32_t* slot_mapping,
                          int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                          int32_t num_kv_heads, int32_t head_dim, int* dev_status, void* stream) {
  PKV_REQUIRE(num_tokens >= 0 && num_blocks > 0 && block_size > 0 && num_kv_heads > 0,
              PKV_ERR_INVALID_ARG, "pkv_kv_cache_read_fp8: bad sizes");
  PKV_REQUIRE(head_dim == 128, PKV_ERR_UNSUPPORTED,
              "pkv_kv_cache_read_fp8: only head_dim 128 is implemented");
  PKV_REQUIRE(k_cache && v_cache && k_scale && v_scale && (num_tokens == 0 || (k && v && slot_mapping)),
              PKV_ERR_INVALID_ARG, "pkv_kv_cache_read_fp8: null pointer");
  PKV_REQUIRE(aligned16(k_cache) && aligned16(v_cache) && aligned16(k) && aligned16(v) &&
                  (((uintptr_t)k_scale) & 3) == 0 && (((uintptr_t)v_scale) & 3) == 0,
              PKV_ERR_INVALID_ARG, "pkv_kv_cache_read_fp8: misaligned pointer");
  const int64_t rows = num_tokens * num_kv_heads, cached = num_blocks * block_size * num_kv_heads;
  auto reads = [&](const void* out) {  // whether an output lies in what the call reads
    return overlap(out, rows * 256, k_cache, cached * 128) ||
           overlap(out, rows * 256, v_cache, cached * 128) ||
           overlap(out, rows * 256, k_scale, cached * 4) ||
           overlap(out, rows * 256, v_scale, cached * 4) ||
           overlap(out, rows * 256, slot_mapping, num_tokens * 4);
  };
  PKV_REQUIRE(!overlap(k, rows * 256, v, rows * 256) && !reads(k) && !reads(v), PKV_ERR_INVALID_ARG,
              "pkv_kv_cache_read_fp8: k or v overlaps the other or an input");
  clear_error();
  return launch_status(launch_kv_read_fp8(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping,
                                          num_tokens, num_blocks, block_size, num_kv_heads,
                                          dev_status, (cudaStream_t)stream, current_num_sms()),
                       "pkv_kv_cache_read_fp8");
}

int pkv_paged_attention_decode_fp8(void* out, int32_t out_dtype, float* lse, const void* q,
                                   const void* k_cache, const void* v_cache, const float* k_scale,
                                   const float* v_scale, const int32_t* block_table,
                                   int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t B,
                                   int32_t H, int32_t H_kv, int32_t head_dim, int32_t block_size,
                                   int64_t num_blocks, float scale, int32_t window,
                                   void* workspace, size_t workspace_bytes, int* dev_status,
                                   void* stream) {
  DecodeArgs a;
  bool empty;
  const int rc0 = decode_setup(a, &empty, "pkv_paged_attention_decode_fp8", out, out_dtype, lse, q,
                               k_cache, v_cache, block_table, max_blocks_per_seq, seq_lens, B, H,
                               H_kv, head_dim, block_size, num_blocks, scale, window, workspace,
                               workspace_bytes, dev_status);
  if (rc0 != PKV_OK || empty) return rc0;
  PKV_REQUIRE(k_scale && v_scale && aligned16(k_scale) && aligned16(v_scale), PKV_ERR_INVALID_ARG,
              "pkv_paged_attention_decode_fp8: scale arrays must be set and 16-byte aligned");
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  clear_error();
  cudaStream_t s = (cudaStream_t)stream;
  int rc = launch_status(launch_decode_fp8(a, s), "pkv_paged_attention_decode_fp8 (attention)");
  if (rc != PKV_OK) return rc;
  return launch_status(launch_decode_merge(a, s), "pkv_paged_attention_decode_fp8 (merge)");
}

int pkv_kv_cache_write_fp4(void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                           const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const int32_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
                           int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                           int* dev_status, void* stream) {
  const char* what = "pkv_kv_cache_write_fp4";
  KvFp4Args a;
  const int rc = fp4_setup(a, what, k_cache, v_cache, k_scale, v_scale, k, v, slot_mapping, num_tokens,
                           num_blocks, block_size, num_kv_heads, head_dim, dev_status);
  if (rc != PKV_OK) return rc;
  const int64_t width = (int64_t)num_kv_heads * head_dim;
  PKV_REQUIRE(k_stride >= 0 && v_stride >= 0 && k_stride % 8 == 0 && v_stride % 8 == 0,
              PKV_ERR_INVALID_ARG, "%s: bad token stride", what);
  if (num_tokens > 0)
    PKV_REQUIRE(!fp4_overlaps(a, k, ((num_tokens - 1) * k_stride + width) * 2) &&
                    !fp4_overlaps(a, v, ((num_tokens - 1) * v_stride + width) * 2) &&
                    !fp4_overlaps(a, slot_mapping, num_tokens * 4),
                PKV_ERR_INVALID_ARG, "%s: an input overlaps the caches", what);
  clear_error();
  return launch_status(launch_kv_write_fp4(a, k, k_stride, v, v_stride, (cudaStream_t)stream,
                                           current_num_sms()),
                       what);
}

int pkv_kv_cache_read_fp4(void* k, void* v, const void* k_cache, const void* v_cache,
                          const void* k_scale, const void* v_scale, const int32_t* slot_mapping,
                          int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                          int32_t num_kv_heads, int32_t head_dim, int* dev_status, void* stream) {
  const char* what = "pkv_kv_cache_read_fp4";
  KvFp4Args a;
  const int rc = fp4_setup(a, what, k_cache, v_cache, k_scale, v_scale, k, v, slot_mapping, num_tokens,
                           num_blocks, block_size, num_kv_heads, head_dim, dev_status);
  if (rc != PKV_OK) return rc;
  const int64_t bytes = num_tokens * num_kv_heads * 256;
  PKV_REQUIRE(!overlap(k, bytes, v, bytes) && !fp4_overlaps(a, k, bytes) && !fp4_overlaps(a, v, bytes) &&
                  !overlap(k, bytes, slot_mapping, num_tokens * 4) &&
                  !overlap(v, bytes, slot_mapping, num_tokens * 4),
              PKV_ERR_INVALID_ARG, "%s: k or v overlaps the other or an input", what);
  clear_error();
  return launch_status(launch_kv_read_fp4(a, k, v, (cudaStream_t)stream, current_num_sms()), what);
}

int pkv_paged_attention_decode_fp4(void* out, int32_t out_dtype, float* lse, const void* q,
                                   const void* k_cache, const void* v_cache, const void* k_scale,
                                   const void* v_scale, const int32_t* block_table,
                                   int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t B,
                                   int32_t q_len, int32_t H, int32_t H_kv, int32_t head_dim,
                                   int32_t block_size, int64_t num_blocks, float scale,
                                   int32_t window, void* workspace, size_t workspace_bytes,
                                   int* dev_status, void* stream) {
  const char* what = "pkv_paged_attention_decode_fp4";
  PKV_REQUIRE(max_blocks_per_seq <= INT32_MAX / 128, PKV_ERR_UNSUPPORTED,
              "%s: max_blocks_per_seq * 128 must fit in int32", what);
  PKV_REQUIRE(B < 0 || H_kv < 0 || B <= INT32_MAX / (H_kv > 0 ? H_kv : 1), PKV_ERR_UNSUPPORTED,
              "%s: B * H_kv must fit in int32", what);
  DecodeFp4Args a;
  bool empty;
  const int rc0 = decode_setup(a, &empty, what, out, out_dtype, lse, q, k_cache, v_cache,
                               block_table, max_blocks_per_seq, seq_lens, B, H, H_kv, head_dim,
                               block_size, num_blocks, scale, window, workspace, workspace_bytes,
                               dev_status, q_len);
  if (rc0 != PKV_OK || empty) return rc0;
  PKV_REQUIRE(k_scale && v_scale && aligned16(k_scale) && aligned16(v_scale), PKV_ERR_INVALID_ARG,
              "%s: scale arrays must be set and 16-byte aligned", what);
  a.q_total = q_len;
  a.k_scale4 = (const uint8_t*)k_scale;
  a.v_scale4 = (const uint8_t*)v_scale;
  clear_error();
  return launch_status(launch_decode_fp4(a, (cudaStream_t)stream), what);
}

size_t pkv_decode_sparse_workspace_size(int32_t B, int32_t q_len, int32_t H, int32_t H_kv,
                                        int32_t head_dim) {
  if (B < 0 || q_len < 1 || H <= 0 || H_kv <= 0 || H % H_kv || head_dim <= 0 ||
      (int64_t)B * q_len > INT32_MAX)
    return 0;
  return decode_workspace_bytes(B * q_len, H, H_kv, head_dim, current_num_sms());
}

int pkv_paged_attention_decode_sparse(void* out, int32_t out_dtype, float* lse, const void* q,
                                      const void* k_cache, const void* v_cache,
                                      const int32_t* block_table, int32_t max_blocks_per_seq,
                                      const int32_t* seq_lens, const int32_t* block_indices,
                                      int32_t num_selected, int32_t B, int32_t q_len, int32_t H,
                                      int32_t H_kv, int32_t head_dim, int32_t block_size,
                                      int64_t num_blocks, float scale, void* workspace,
                                      size_t workspace_bytes, int* dev_status, void* stream) {
  const char* what = "pkv_paged_attention_decode_sparse";
  PKV_REQUIRE(q_len >= 1 && num_selected >= 1, PKV_ERR_INVALID_ARG, "%s: bad sizes", what);
  // Rows of all sequences are numbered together, and so are their kv heads.
  PKV_REQUIRE(B < 0 || H_kv < 0 || (int64_t)B * q_len <= INT32_MAX / (H_kv > 0 ? H_kv : 1),
              PKV_ERR_UNSUPPORTED, "%s: B * q_len * H_kv must fit in int32", what);
  PKV_REQUIRE(max_blocks_per_seq <= INT32_MAX / 128, PKV_ERR_UNSUPPORTED,
              "%s: max_blocks_per_seq * 128 must fit in int32", what);
  DecodeArgs a;
  bool empty;
  const int rc0 = decode_setup(a, &empty, what, out, out_dtype, lse, q, k_cache, v_cache,
                               block_table, max_blocks_per_seq, seq_lens, B * q_len, H, H_kv,
                               head_dim, block_size, num_blocks, scale, 0, workspace,
                               workspace_bytes, dev_status);
  if (rc0 != PKV_OK || empty) return rc0;
  PKV_REQUIRE(block_indices, PKV_ERR_INVALID_ARG, "%s: null pointer", what);
  a.block_indices = block_indices;
  a.num_selected = num_selected;
  a.rows_per_seq = q_len;
  clear_error();
  return launch_status(launch_decode_sparse(a, (cudaStream_t)stream), what);
}

int pkv_update_block_summaries(void* summaries, const void* k_cache, const int32_t* block_table,
                               int32_t max_blocks_per_seq, const int32_t* seq_lens,
                               const int32_t* num_new, int32_t max_new, int32_t B, int32_t H_kv,
                               int32_t head_dim, int32_t block_size, int64_t num_blocks,
                               int* dev_status, void* stream) {
  const char* what = "pkv_update_block_summaries";
  PKV_REQUIRE(B >= 0 && H_kv > 0 && max_blocks_per_seq > 0 && num_blocks > 0 && max_new >= 0,
              PKV_ERR_INVALID_ARG, "%s: bad sizes", what);
  PKV_REQUIRE(head_dim == 128 && block_size == 128, PKV_ERR_UNSUPPORTED,
              "%s: only head_dim 128 and block_size 128 are implemented", what);
  PKV_REQUIRE(summaries && k_cache && (B == 0 || (block_table && seq_lens && num_new)),
              PKV_ERR_INVALID_ARG, "%s: null pointer", what);
  PKV_REQUIRE(aligned16(summaries) && aligned16(k_cache), PKV_ERR_INVALID_ARG,
              "%s: pointers must be 16-byte aligned", what);
  if (B == 0 || max_new == 0) return PKV_OK;
  SummaryArgs a = {};
  a.span = (int)(((int64_t)max_new + block_size - 2) / block_size + 1);
  if (a.span > max_blocks_per_seq) a.span = max_blocks_per_seq;
  PKV_REQUIRE((int64_t)B * a.span <= INT32_MAX / H_kv, PKV_ERR_UNSUPPORTED,
              "%s: B * blocks of max_new * H_kv must fit in int32", what);
  const int64_t summary_bytes = num_blocks * H_kv * (4 * (int64_t)head_dim);
  PKV_REQUIRE(!overlap(summaries, summary_bytes, k_cache,
                       num_blocks * block_size * H_kv * (2 * (int64_t)head_dim)) &&
                  !overlap(summaries, summary_bytes, block_table, (int64_t)B * max_blocks_per_seq * 4) &&
                  !overlap(summaries, summary_bytes, seq_lens, (int64_t)B * 4) &&
                  !overlap(summaries, summary_bytes, num_new, (int64_t)B * 4),
              PKV_ERR_INVALID_ARG, "%s: summaries overlaps an input", what);
  a.summaries = (uint8_t*)summaries;
  a.k_cache = (const uint8_t*)k_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.num_new = num_new;
  a.dev_status = dev_status;
  a.num_blocks = num_blocks;
  a.B = B;
  a.Hkv = H_kv;
  a.max_blocks = max_blocks_per_seq;
  a.max_new = max_new;
  clear_error();
  return launch_status(launch_block_summaries(a, (cudaStream_t)stream, current_num_sms()), what);
}

int pkv_accumulate_attention_weights(float* weights, const void* q, const float* lse,
                                     const void* k_cache, const void* k_scale, int32_t key_format,
                                     const int32_t* block_table, int32_t max_blocks_per_seq,
                                     const int32_t* seq_lens, const int32_t* num_fresh, int32_t B,
                                     int32_t q_len, int32_t H, int32_t H_kv, int32_t head_dim,
                                     int32_t block_size, int64_t num_blocks, float scale,
                                     float decay, int* dev_status, void* stream) {
  const char* what = "pkv_accumulate_attention_weights";
  PKV_REQUIRE(B >= 0 && q_len >= 1 && H > 0 && H_kv > 0 && max_blocks_per_seq > 0 && num_blocks > 0,
              PKV_ERR_INVALID_ARG, "%s: bad sizes", what);
  PKV_REQUIRE(H % H_kv == 0, PKV_ERR_INVALID_ARG, "%s: H (%d) not a multiple of H_kv (%d)", what, H, H_kv);
  PKV_REQUIRE(key_format == PKV_KEYS_BF16 || key_format == PKV_KEYS_FP8 || key_format == PKV_KEYS_FP4,
              PKV_ERR_INVALID_ARG, "%s: bad key_format", what);
  PKV_REQUIRE(head_dim == 128 && block_size == 128, PKV_ERR_UNSUPPORTED,
              "%s: only head_dim 128 and block_size 128 are implemented", what);
  PKV_REQUIRE(H / H_kv <= 16, PKV_ERR_UNSUPPORTED, "%s: H / H_kv = %d exceeds 16", what, H / H_kv);
  PKV_REQUIRE(q_len <= (1 << 20), PKV_ERR_UNSUPPORTED, "%s: q_len too large", what);
  PKV_REQUIRE(max_blocks_per_seq <= INT32_MAX / 128 && num_blocks * block_size <= INT32_MAX &&
                  B <= INT32_MAX / H_kv,
              PKV_ERR_UNSUPPORTED,
              "%s: max_blocks_per_seq * 128, num_blocks * 128 and B * H_kv must fit in int32", what);
  PKV_REQUIRE(std::isfinite(scale) && scale > 0.f, PKV_ERR_INVALID_ARG,
              "%s: scale must be a positive finite number", what);
  PKV_REQUIRE(decay >= 0.f && decay <= 1.f, PKV_ERR_INVALID_ARG, "%s: decay outside [0, 1]", what);
  if (B == 0) return PKV_OK;
  const bool scaled = key_format != PKV_KEYS_BF16;
  PKV_REQUIRE(weights && q && lse && k_cache && block_table && seq_lens && num_fresh &&
                  (scaled == (k_scale != nullptr)),
              PKV_ERR_INVALID_ARG, "%s: null pointer, or k_scale where the format has none", what);
  PKV_REQUIRE(aligned16(weights) && aligned16(q) && aligned16(k_cache) && aligned16(k_scale) &&
                  (((uintptr_t)lse) & 3) == 0,
              PKV_ERR_INVALID_ARG, "%s: misaligned pointer", what);
  const int64_t rows = num_blocks * block_size * H_kv, queries = (int64_t)B * q_len * H;
  auto reads = [&](const void* p, int64_t bytes) { return overlap(weights, rows * 4, p, bytes); };
  PKV_REQUIRE(!reads(q, queries * 256) && !reads(lse, queries * 4) &&
                  !reads(k_cache, rows * (key_format == PKV_KEYS_BF16 ? 256 : key_format == PKV_KEYS_FP8 ? 128 : 64)) &&
                  !(scaled && reads(k_scale, rows * (key_format == PKV_KEYS_FP8 ? 4 : 8))) &&
                  !reads(block_table, (int64_t)B * max_blocks_per_seq * 4) && !reads(seq_lens, B * (int64_t)4) &&
                  !reads(num_fresh, B * (int64_t)4),
              PKV_ERR_INVALID_ARG, "%s: weights overlaps an input", what);
  WeightsArgs a = {};
  a.weights = weights;
  a.q = (const uint16_t*)q;
  a.lse = lse;
  a.k_cache = (const uint8_t*)k_cache;
  a.k_scale = (const uint8_t*)k_scale;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.num_fresh = num_fresh;
  a.dev_status = dev_status;
  a.num_blocks = num_blocks;
  a.B = B;
  a.q_len = q_len;
  a.H = H;
  a.Hkv = H_kv;
  a.n_rep = H / H_kv;
  a.max_blocks = max_blocks_per_seq;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.decay = decay;
  clear_error();
  return launch_status(launch_attn_weights(a, key_format, (cudaStream_t)stream, current_num_sms()), what);
}

int pkv_select_rows(int32_t* kept, const float* weights, const int32_t* block_table,
                    int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t B, int32_t H_kv,
                    int32_t block_size, int64_t num_blocks, int32_t num_keep, int32_t num_sink,
                    int32_t num_recent, int* dev_status, void* stream) {
  const char* what = "pkv_select_rows";
  PKV_REQUIRE(B >= 0 && H_kv > 0 && max_blocks_per_seq > 0 && num_blocks > 0 && num_keep >= 1 &&
                  num_sink >= 0 && num_recent >= 0,
              PKV_ERR_INVALID_ARG, "%s: bad sizes", what);
  PKV_REQUIRE(block_size == 128, PKV_ERR_UNSUPPORTED, "%s: only block_size 128 is implemented", what);
  PKV_REQUIRE((int64_t)num_sink + num_recent <= num_keep, PKV_ERR_INVALID_ARG,
              "%s: num_sink + num_recent exceeds num_keep", what);
  PKV_REQUIRE(num_keep <= kMaxKept, PKV_ERR_UNSUPPORTED, "%s: num_keep exceeds %d", what, kMaxKept);
  PKV_REQUIRE(max_blocks_per_seq <= kSelectRowsMaxBlocks, PKV_ERR_UNSUPPORTED,
              "%s: max_blocks_per_seq exceeds %d", what, kSelectRowsMaxBlocks);
  PKV_REQUIRE(num_blocks * block_size <= INT32_MAX && B <= INT32_MAX / 8 / H_kv, PKV_ERR_UNSUPPORTED,
              "%s: num_blocks * 128 and 8 B * H_kv must fit in int32", what);
  if (B == 0) return PKV_OK;
  PKV_REQUIRE(kept && weights && block_table && seq_lens, PKV_ERR_INVALID_ARG, "%s: null pointer", what);
  PKV_REQUIRE(aligned16(weights) && aligned16(kept), PKV_ERR_INVALID_ARG,
              "%s: pointers must be 16-byte aligned", what);
  const int64_t bytes = (int64_t)B * H_kv * num_keep * 4;
  PKV_REQUIRE(!overlap(kept, bytes, weights, num_blocks * H_kv * block_size * 4) &&
                  !overlap(kept, bytes, block_table, (int64_t)B * max_blocks_per_seq * 4) &&
                  !overlap(kept, bytes, seq_lens, (int64_t)B * 4),
              PKV_ERR_INVALID_ARG, "%s: kept overlaps an input", what);
  SelectRowsArgs a = {weights, block_table, seq_lens, kept, dev_status, num_blocks, B, H_kv, block_size,
                      max_blocks_per_seq, num_keep, num_sink, num_recent};
  clear_error();
  return launch_status(launch_select_rows(a, (cudaStream_t)stream, current_num_sms()), what);
}

int pkv_compact_rows(void* const* caches, const int32_t* row_bytes, const int32_t* head_major,
                     int32_t num_caches, const int32_t* kept, int32_t num_keep,
                     const int32_t* block_table, int32_t max_blocks_per_seq,
                     const int32_t* new_block_table, int32_t new_max_blocks_per_seq, int32_t B,
                     int32_t H_kv, int32_t block_size, int64_t num_blocks, int* dev_status,
                     void* stream) {
  const char* what = "pkv_compact_rows";
  PKV_REQUIRE(B >= 0 && H_kv > 0 && max_blocks_per_seq > 0 && num_blocks > 0 && num_keep >= 1 &&
                  block_size > 0 && num_caches >= 1,
              PKV_ERR_INVALID_ARG, "%s: bad sizes", what);
  PKV_REQUIRE(num_caches <= kCompactMaxCaches, PKV_ERR_UNSUPPORTED, "%s: more than %d caches", what,
              kCompactMaxCaches);
  PKV_REQUIRE(num_keep <= kMaxKept, PKV_ERR_UNSUPPORTED, "%s: num_keep exceeds %d", what, kMaxKept);
  PKV_REQUIRE(num_blocks * block_size <= INT32_MAX && B <= INT32_MAX / H_kv, PKV_ERR_UNSUPPORTED,
              "%s: num_blocks * block_size and B * H_kv must fit in int32", what);
  PKV_REQUIRE(!new_block_table || (new_max_blocks_per_seq > 0 &&
                                   num_keep <= (int64_t)new_max_blocks_per_seq * block_size),
              PKV_ERR_INVALID_ARG, "%s: num_keep rows do not fit in the new table", what);
  if (B == 0) return PKV_OK;
  PKV_REQUIRE(caches && row_bytes && head_major && kept && block_table, PKV_ERR_INVALID_ARG,
              "%s: null pointer", what);
  CompactArgs a = {};
  const int64_t rows = num_blocks * block_size * H_kv;
  auto reads = [&](const void* p, int64_t bytes) {
    return overlap(p, bytes, kept, (int64_t)B * H_kv * num_keep * 4) ||
           overlap(p, bytes, block_table, (int64_t)B * max_blocks_per_seq * 4) ||
           (new_block_table &&
            overlap(p, bytes, new_block_table, (int64_t)B * new_max_blocks_per_seq * 4));
  };
  for (int i = 0; i < num_caches; ++i) {
    PKV_REQUIRE(caches[i], PKV_ERR_INVALID_ARG, "%s: null pointer", what);
    PKV_REQUIRE(row_bytes[i] > 0 && row_bytes[i] % 4 == 0 && row_bytes[i] <= (1 << 16), PKV_ERR_UNSUPPORTED,
                "%s: rows of %d bytes (a multiple of 4 up to 2^16 is implemented)", what, row_bytes[i]);
    PKV_REQUIRE(aligned16(caches[i]), PKV_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", what);
    PKV_REQUIRE(!reads(caches[i], rows * row_bytes[i]), PKV_ERR_INVALID_ARG,
                "%s: cache %d overlaps kept or a table", what, i);
    for (int j = 0; j < i; ++j)
      PKV_REQUIRE(!overlap(caches[i], rows * row_bytes[i], caches[j], rows * row_bytes[j]),
                  PKV_ERR_INVALID_ARG, "%s: caches %d and %d overlap", what, j, i);
    CompactCache& c = a.cache[i];
    c.data = (uint8_t*)caches[i];
    c.row_bytes = row_bytes[i];
    c.block_stride = (int64_t)block_size * H_kv * row_bytes[i];
    c.row_stride = head_major[i] ? row_bytes[i] : (int64_t)H_kv * row_bytes[i];
    c.head_stride = head_major[i] ? (int64_t)block_size * row_bytes[i] : row_bytes[i];
  }
  a.kept = kept;
  a.block_table = block_table;
  a.new_table = new_block_table ? new_block_table : block_table;
  a.dev_status = dev_status;
  a.num_blocks = num_blocks;
  a.B = B;
  a.Hkv = H_kv;
  a.block_size = block_size;
  a.max_blocks = max_blocks_per_seq;
  a.new_max_blocks = new_block_table ? new_max_blocks_per_seq : max_blocks_per_seq;
  a.num_keep = num_keep;
  a.num_caches = num_caches;
  clear_error();
  return launch_status(launch_compact_rows(a, (cudaStream_t)stream, current_num_sms()), what);
}

int pkv_select_blocks(int32_t* block_indices, const void* q, const void* summaries,
                      const int32_t* block_table, int32_t max_blocks_per_seq,
                      const int32_t* seq_lens, int32_t B, int32_t q_len, int32_t H, int32_t H_kv,
                      int32_t head_dim, int32_t block_size, int64_t num_blocks,
                      int32_t num_selected, int32_t num_sink, int32_t num_recent, int* dev_status,
                      void* stream) {
  const char* what = "pkv_select_blocks";
  PKV_REQUIRE(B >= 0 && q_len >= 1 && H > 0 && H_kv > 0 && max_blocks_per_seq > 0 && num_blocks > 0,
              PKV_ERR_INVALID_ARG, "%s: bad sizes", what);
  PKV_REQUIRE(H % H_kv == 0, PKV_ERR_INVALID_ARG, "%s: H (%d) not a multiple of H_kv (%d)", what, H,
              H_kv);
  PKV_REQUIRE(num_selected >= 1 && num_sink >= 0 && num_recent >= 0 &&
                  (int64_t)num_sink + num_recent <= num_selected,
              PKV_ERR_INVALID_ARG, "%s: num_sink + num_recent must be at most num_selected", what);
  PKV_REQUIRE(head_dim == 128 && block_size == 128, PKV_ERR_UNSUPPORTED,
              "%s: only head_dim 128 and block_size 128 are implemented", what);
  PKV_REQUIRE(H / H_kv <= 16, PKV_ERR_UNSUPPORTED, "%s: H / H_kv = %d unsupported", what, H / H_kv);
  PKV_REQUIRE(max_blocks_per_seq <= kSelectMaxBlocks, PKV_ERR_UNSUPPORTED,
              "%s: at most %d blocks per sequence", what, kSelectMaxBlocks);
  // A cluster of up to 8 CTAs per row and kv head.
  PKV_REQUIRE((int64_t)B * q_len <= INT32_MAX / 8 / H_kv, PKV_ERR_UNSUPPORTED,
              "%s: B * q_len * H_kv too large", what);
  if (B == 0) return PKV_OK;
  PKV_REQUIRE(block_indices && q && summaries && block_table && seq_lens, PKV_ERR_INVALID_ARG,
              "%s: null pointer", what);
  PKV_REQUIRE(aligned16(q) && aligned16(summaries), PKV_ERR_INVALID_ARG,
              "%s: pointers must be 16-byte aligned", what);
  const int64_t rows = (int64_t)B * q_len, out_bytes = rows * H_kv * num_selected * 4;
  PKV_REQUIRE(!overlap(block_indices, out_bytes, q, rows * H * head_dim * 2) &&
                  !overlap(block_indices, out_bytes, summaries, num_blocks * H_kv * (4 * (int64_t)head_dim)) &&
                  !overlap(block_indices, out_bytes, block_table, (int64_t)B * max_blocks_per_seq * 4) &&
                  !overlap(block_indices, out_bytes, seq_lens, (int64_t)B * 4),
              PKV_ERR_INVALID_ARG, "%s: block_indices overlaps an input", what);
  SelectArgs a = {};
  a.q = (const uint16_t*)q;
  a.summaries = (const uint8_t*)summaries;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = block_indices;
  a.dev_status = dev_status;
  a.num_blocks = num_blocks;
  a.B = B;
  a.q_len = q_len;
  a.H = H;
  a.Hkv = H_kv;
  a.n_rep = H / H_kv;
  a.max_blocks = max_blocks_per_seq;
  a.num_selected = num_selected;
  a.num_sink = num_sink;
  a.num_recent = num_recent;
  clear_error();
  return launch_status(launch_select_blocks(a, (cudaStream_t)stream, current_num_sms()), what);
}

size_t pkv_prefill_workspace_size(void) { return prefill_workspace_bytes(current_num_sms()); }

int pkv_paged_attention_prefill(void* out, int32_t out_dtype, float* lse, const void* q,
                                const int32_t* cu_seqlens_q, int32_t num_tokens,
                                const void* k_cache, const void* v_cache,
                                const int32_t* block_table, int32_t max_blocks_per_seq,
                                const int32_t* seq_lens_kv, int32_t B, int32_t H, int32_t H_kv,
                                int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                float scale, int32_t causal, void* workspace,
                                size_t workspace_bytes, int* dev_status, void* stream) {
  PKV_REQUIRE(B >= 0 && num_tokens >= 0 && H > 0 && H_kv > 0 && max_blocks_per_seq > 0 &&
                  num_blocks > 0,
              PKV_ERR_INVALID_ARG, "pkv_paged_attention_prefill: bad sizes");
  PKV_REQUIRE(H % H_kv == 0, PKV_ERR_INVALID_ARG,
              "pkv_paged_attention_prefill: H (%d) not a multiple of H_kv (%d)", H, H_kv);
  const int n_rep = H / H_kv;
  PKV_REQUIRE(head_dim == 128 && block_size == 128, PKV_ERR_UNSUPPORTED,
              "pkv_paged_attention_prefill: only head_dim 128 and block_size 128 are implemented");
  PKV_REQUIRE(n_rep == 1 || n_rep == 2 || n_rep == 4 || n_rep == 8 || n_rep == 16,
              PKV_ERR_UNSUPPORTED, "pkv_paged_attention_prefill: H / H_kv = %d unsupported", n_rep);
  PKV_REQUIRE(out_dtype == PKV_BF16 || out_dtype == PKV_F32, PKV_ERR_INVALID_ARG,
              "pkv_paged_attention_prefill: bad out_dtype");
  PKV_REQUIRE(std::isfinite(scale) && scale > 0.f, PKV_ERR_INVALID_ARG,
              "pkv_paged_attention_prefill: scale must be a positive finite number");
  PKV_REQUIRE(causal == 0 || causal == 1, PKV_ERR_INVALID_ARG, "pkv_paged_attention_prefill: causal");
  PKV_REQUIRE(num_blocks * block_size <= INT32_MAX, PKV_ERR_UNSUPPORTED,
              "pkv_paged_attention_prefill: num_blocks * block_size must fit in int32");
  if (B == 0 || num_tokens == 0) return PKV_OK;
  PKV_REQUIRE(out && q && cu_seqlens_q && k_cache && v_cache && block_table && seq_lens_kv,
              PKV_ERR_INVALID_ARG, "pkv_paged_attention_prefill: null pointer");
  PKV_REQUIRE(aligned16(out) && aligned16(q) && aligned16(k_cache) && aligned16(v_cache),
              PKV_ERR_INVALID_ARG, "pkv_paged_attention_prefill: pointers must be 16-byte aligned");
  const int G = current_num_sms();
  PKV_REQUIRE(G > 0, PKV_ERR_LAUNCH, "pkv_paged_attention_prefill: no CUDA device");
  const size_t need = prefill_workspace_bytes(G);
  PKV_REQUIRE(workspace && workspace_bytes >= need && (((uintptr_t)workspace) & 255) == 0,
              PKV_ERR_WORKSPACE, "pkv_paged_attention_prefill: workspace needs %zu bytes, 256-aligned",
              need);
  clear_error();
  return launch_status(launch_prefill(q, cu_seqlens_q, k_cache, v_cache, block_table,
                                      max_blocks_per_seq, seq_lens_kv, out, out_dtype == PKV_F32, lse,
                                      num_tokens, B, H, H_kv, num_blocks, scale, causal, workspace,
                                      dev_status, G, (cudaStream_t)stream),
                       "pkv_paged_attention_prefill");
}

// Absorbed MLA decode of q_len query rows per sequence (q_len = 1: plain decode).
static int mla_decode(const char* name, void* out, int32_t out_dtype, float* lse,
                      const void* q_nope, const void* q_rope, const void* cache_nope,
                      const void* cache_rope, const int32_t* block_table, int32_t max_blocks_per_seq,
                      const int32_t* seq_lens, int32_t B, int32_t q_len, int32_t H,
                      int32_t kv_lora_rank, int32_t rope_dim, int32_t block_size, int64_t num_blocks,
                      float scale, void* workspace, size_t workspace_bytes, int* dev_status,
                      void* stream) {
  PKV_REQUIRE(B >= 0 && H > 0 && max_blocks_per_seq > 0 && num_blocks > 0, PKV_ERR_INVALID_ARG,
              "%s: bad sizes", name);
  PKV_REQUIRE(q_len >= 1 && q_len <= 4, PKV_ERR_UNSUPPORTED, "%s: q_len must be 1..4", name);
  PKV_REQUIRE(kv_lora_rank == 512 && rope_dim == 64 && block_size == 128 && H <= 128,
              PKV_ERR_UNSUPPORTED,
              "%s: implemented for kv_lora_rank 512, rope 64, block_size 128, H <= 128", name);
  PKV_REQUIRE(out_dtype == PKV_BF16 || out_dtype == PKV_F32, PKV_ERR_INVALID_ARG,
              "%s: bad out_dtype", name);
  PKV_REQUIRE(std::isfinite(scale) && scale > 0.f, PKV_ERR_INVALID_ARG,
              "%s: scale must be a positive finite number", name);
  PKV_REQUIRE(num_blocks * block_size <= INT32_MAX, PKV_ERR_UNSUPPORTED,
              "%s: num_blocks * block_size must fit in int32", name);
  PKV_REQUIRE((int64_t)B * q_len * H <= INT32_MAX, PKV_ERR_UNSUPPORTED,
              "%s: B * q_len * H must fit in int32", name);
  if (B == 0) return PKV_OK;
  PKV_REQUIRE(out && q_nope && q_rope && cache_nope && cache_rope && block_table && seq_lens,
              PKV_ERR_INVALID_ARG, "%s: null pointer", name);
  PKV_REQUIRE(aligned16(out) && aligned16(q_nope) && aligned16(q_rope) && aligned16(cache_nope) &&
                  aligned16(cache_rope),
              PKV_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", name);
  const int G = current_num_sms();
  PKV_REQUIRE(G >= 2, PKV_ERR_LAUNCH, "%s: no CUDA device", name);
  const size_t need = mla_workspace_bytes(B * q_len, G / 2);
  PKV_REQUIRE(workspace && workspace_bytes >= need && (((uintptr_t)workspace) & 255) == 0,
              PKV_ERR_WORKSPACE, "%s: workspace needs %zu bytes, 256-aligned", name, need);
  clear_error();
  return launch_status(launch_mla_decode(q_nope, q_rope, cache_nope, cache_rope, block_table,
                                         max_blocks_per_seq, seq_lens, out, out_dtype == PKV_F32,
                                         lse, B, q_len, H, num_blocks, scale, workspace, dev_status,
                                         G, (cudaStream_t)stream),
                       name);
}

size_t pkv_mla_decode_workspace_size(int32_t B, int32_t H) {
  if (B < 0 || H <= 0) return 0;
  return mla_workspace_bytes(B, current_num_sms() / 2);
}

int pkv_mla_paged_decode(void* out, int32_t out_dtype, float* lse, const void* q_nope,
                         const void* q_rope, const void* cache_nope, const void* cache_rope,
                         const int32_t* block_table, int32_t max_blocks_per_seq,
                         const int32_t* seq_lens, int32_t B, int32_t H, int32_t kv_lora_rank,
                         int32_t rope_dim, int32_t block_size, int64_t num_blocks, float scale,
                         void* workspace, size_t workspace_bytes, int* dev_status, void* stream) {
  return mla_decode("pkv_mla_paged_decode", out, out_dtype, lse, q_nope, q_rope, cache_nope,
                    cache_rope, block_table, max_blocks_per_seq, seq_lens, B, 1, H, kv_lora_rank,
                    rope_dim, block_size, num_blocks, scale, workspace, workspace_bytes, dev_status,
                    stream);
}

size_t pkv_mla_decode_spec_workspace_size(int32_t B, int32_t q_len, int32_t H) {
  if (B < 0 || q_len < 1 || H <= 0) return 0;
  return mla_workspace_bytes(B * q_len, current_num_sms() / 2);
}

int pkv_mla_paged_decode_spec(void* out, int32_t out_dtype, float* lse, const void* q_nope,
                              const void* q_rope, const void* cache_nope, const void* cache_rope,
                              const int32_t* block_table, int32_t max_blocks_per_seq,
                              const int32_t* seq_lens, int32_t B, int32_t q_len, int32_t H,
                              int32_t kv_lora_rank, int32_t rope_dim, int32_t block_size,
                              int64_t num_blocks, float scale, void* workspace,
                              size_t workspace_bytes, int* dev_status, void* stream) {
  return mla_decode("pkv_mla_paged_decode_spec", out, out_dtype, lse, q_nope, q_rope, cache_nope,
                    cache_rope, block_table, max_blocks_per_seq, seq_lens, B, q_len, H,
                    kv_lora_rank, rope_dim, block_size, num_blocks, scale, workspace,
                    workspace_bytes, dev_status, stream);
}

int pkv_selftest_bounded_wait(int* dev_status, void* stream) {
  PKV_REQUIRE(dev_status != nullptr, PKV_ERR_INVALID_ARG, "pkv_selftest_bounded_wait: null dev_status");
  return launch_status(launch_bounded_wait(dev_status, static_cast<cudaStream_t>(stream)),
                       "pkv_selftest_bounded_wait");
}

int pkv_selftest_bf16_products(float* d, const void* a, const void* b, int32_t n, void* stream) {
  PKV_REQUIRE(n >= 0 && (n == 0 || (d && a && b)) && aligned16(d) && aligned16(a) && aligned16(b),
              PKV_ERR_INVALID_ARG, "pkv_selftest_bf16_products: bad size or pointer");
  clear_error();
  return launch_status(launch_bf16_products(d, a, b, n, static_cast<cudaStream_t>(stream)),
                       "pkv_selftest_bf16_products");
}

}  // extern "C"
