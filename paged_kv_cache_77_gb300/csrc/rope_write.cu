// Rotary embedding of new q and k rows fused with the paged write of k and v, for
// positions with one or several axes (time, height, width), into a bf16 or an FP8 cache.
//
// Pair i of a head (i < rope_dim / 2) turns by the angle of position p = positions[axis(i)][t],
// whose cosine and sine are c = table[p][i], s = table[p][rope_dim / 2 + i]:
//
//   (x1, x2) -> (x1 c - x2 s, x2 c + x1 s)
//
// with x1, x2 the elements i and i + rope_dim / 2 (the rotate_half form the pages print for
// the Llama forward, "KV Cache 笔记") or 2i and 2i + 1. Elements from rope_dim on pass
// through. fp32 arithmetic and one rounding: to bf16, or (FP8 cache) to E4M3 of the fp32
// value over the row's scale, amax / 448. Angles come from the caller's table, so far
// positions cost no accuracy here.
//
// Layout: a lane holds 16 elements of one head, either 8 whole pairs (two 16-byte vectors,
// which are rope_dim / 2 apart or neighbours) or 16 elements that pass through, so a
// head_dim of 128 takes 8 lanes and a warp 4 heads. A warp's item is the q, the k or the v
// heads of a token, up to kUnroll passes of 4 (one pass of heads that are quantised); every
// load of an item is issued before any arithmetic. The cosines and sines of a lane's 8 pairs
// are the same for every head: a q or k item loads them once for its heads, the token's other
// items load them again, mostly from cache. Elements are read and written by the same thread,
// so q may be rotated in place.
//
// Roofline: HBM. Algorithmic bytes per token = 2 (q) + 2 (k, v to bf16; 1.5 to FP8) times
// the rows' bytes, the table row and 4 bytes of slot and of each position.
#include <cuda_fp8.h>

#include "device_common.cuh"
#include "ieee_math.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace pkv {

namespace {

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(u[i]);
    f[2 * i + 1] = bf16hi(u[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// E4M3 codes of a lane's 16 values over their row's scale: the code of the fp32 quotient
// x / scale, correctly rounded (0: an all-zero row, zero codes). With y the correctly rounded
// 1 / scale and q within one unit of the quotient, q + y (x - q scale) rounds to the quotient
// correctly rounded, the remainder being exact (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990). The product x y can be 1.5 units
// off, so it is corrected once before: one division a row and five operations a value in place
// of a division a value (FP8 prefill of 9,001 tokens: 61.4 us with divisions). Scales for which a remainder, y or an
// infinite value would leave the normal numbers divide. (Telling the codes of two enclosing
// products apart and dividing in between gained little, 65.5 to 64.6 us at the time: bf16 rows
// hit exact ties often.)
__device__ __forceinline__ uint4 codes16(const float* f, float scale) {
  uint32_t u[4] = {0, 0, 0, 0};
  if (!__float_as_uint(scale)) return make_uint4(0, 0, 0, 0);  // (a comparison may flush it)
  if (scale > 0x1p-80f && scale < 0x1p120f) {
    const float y = div_ieee(1.f, scale), minus = neg_ieee(scale);
    auto quotient = [&](float x) {
      float q = mul_ieee(x, y);
      q = fma_ieee(fma_ieee(q, minus, x), y, q);
      return fma_ieee(fma_ieee(q, minus, x), y, q);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i >> 1] |= e4m3x2(quotient(f[2 * i]), quotient(f[2 * i + 1])) << (16 * (i & 1));
  } else {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = f[i];
#pragma unroll 1
    for (int n = 0; n < 8; ++n) {  // rolled (rare, and its code is small), the values moving past
      const uint32_t c = e4m3x2(div_ieee(x[0], scale), div_ieee(x[1], scale));
      u[0] = __funnelshift_r(u[0], u[1], 16);
      u[1] = __funnelshift_r(u[1], u[2], 16);
      u[2] = __funnelshift_r(u[2], u[3], 16);
      u[3] = u[3] >> 16 | c << 16;
#pragma unroll
      for (int i = 0; i < 14; ++i) x[i] = x[i + 2];
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Rotates the lane's 8 pairs in place (f: the 16 values of its two vectors).
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate(float* f, const float* c, const float* s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& a = f[INTERLEAVED ? 2 * i : i];
    float& b = f[INTERLEAVED ? 2 * i + 1 : 8 + i];
    const float x = fma_ieee(a, c[i], neg_ieee(mul_ieee(b, s[i])));
    b = fma_ieee(b, c[i], mul_ieee(a, s[i]));
    a = x;
  }
}

}  // namespace

// Measured on GB300 (16,001 tokens of 32 / 8 heads in bf16; 9,001 of 64 / 8 heads in FP8): 4
// passes an item, 3 resident CTAs per SM and a grid of them 64.3 and 56.3 us, 92 % of the copy
// rate each; 2 passes and 4 CTAs 63.4 and 58.4; 8 passes and 2 CTAs 63.8 and 64.0; 4 passes and
// 2 CTAs 74.8 and 70.2; 8 CTAs per SM of grid 66.0 and 59.3.
constexpr int kUnroll = 4;
constexpr int kCtasPerSm = 3;
template <bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(256, kCtasPerSm) rope_write_kernel(const __grid_constant__ RopeArgs a) {
  pdl_wait_then_launch();
  const int lane = threadIdx.x & 31;
  const int lanes = a.head_dim / 16;       // lanes of one head
  const int per_pass = 32 / lanes;         // heads a warp holds at a time
  const int sub = lane / lanes, c = lane - sub * lanes;
  const bool active = sub < per_pass;      // head_dim not a power of two leaves lanes over
  const int nrot = a.rope_dim / 16;
  const bool rot = c < nrot;
  // The lane's two vectors, from the first head of a pass.
  const int lo = sub * a.head_dim + (rot && !INTERLEAVED ? 8 * c : 16 * c);
  const int hi = sub * a.head_dim + (rot && !INTERLEAVED ? a.rope_dim / 2 + 8 * c : 16 * c + 8);
  // An item is up to kUnroll passes over the q, the k or the v heads of a token; one pass where
  // the heads are quantised. All of an item's addresses are offsets from two uniform pointers.
  const int q_share = per_pass * kUnroll, kv_share = FP8 ? per_pass : q_share;
  const int q_parts = (a.H + q_share - 1) / q_share, kv_parts = (a.Hkv + kv_share - 1) / kv_share;
  const int parts = q_parts + 2 * kv_parts;
  const int pass_stride = per_pass * a.head_dim;
  // A warp's items are one stride apart; the division is done once.
  const int stride = (int)gridDim.x * 8, step_t = stride / parts, step_part = stride % parts;
  const int warp0 = (int)blockIdx.x * 8 + __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  int64_t t = warp0 / parts;
  int part = warp0 % parts;
  auto advance = [&]() {
    t += step_t;
    part += step_part;
    if (part >= parts) {
      part -= parts;
      ++t;
    }
  };
  for (; t < a.num_tokens; advance()) {
    const bool is_q = part < q_parts, is_v = part >= q_parts + kv_parts;
    const int head0 = is_q ? part * q_share : (part - q_parts - (is_v ? kv_parts : 0)) * kv_share;
    const int left = (is_q ? a.H : a.Hkv) - head0 - sub;  // heads from the lane's first on
    const uint16_t* src = (is_q    ? a.q + t * a.q_stride
                           : is_v ? a.v + t * a.v_stride
                                  : a.k + t * a.k_stride) +
                          head0 * a.head_dim;
    uint4 w0[kUnroll], w1[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      w0[u] = w1[u] = make_uint4(0, 0, 0, 0);
      if (active && u * per_pass < left && (!FP8 || is_q || u == 0)) {
        w0[u] = *reinterpret_cast<const uint4*>(src + u * pass_stride + lo);
        w1[u] = *reinterpret_cast<const uint4*>(src + u * pass_stride + hi);
      }
    }
    const int32_t slot = __ldg(a.slots + t);
    bool bad_pos = false;
    int pos[kRopeMaxAxes];
#pragma unroll
    for (int x = 0; x < kRopeMaxAxes; ++x) {
      pos[x] = x < a.num_axes ? __ldg(a.positions + x * a.num_tokens + t) : 0;
      bad_pos |= pos[x] < 0 || pos[x] >= a.max_pos;
    }
    if (bad_pos) {  // the same for the whole warp
      if (lane == 0) flag_status(a.dev_status, PKV_DEV_BAD_POSITION);
      continue;
    }
    const bool bad_slot = (int64_t)slot >= a.num_slots;
    if (bad_slot && lane == 0) flag_status(a.dev_status, PKV_DEV_BAD_SLOT);
    const bool store = slot >= 0 && !bad_slot;
    float cs[8], sn[8];
    if (rot && !is_v) {
      const int axis = a.chunk_axis[c];
      if (axis >= 0) {  // the 8 pairs share one axis: whole vectors of its table row
        const int p = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
        const float4* row = reinterpret_cast<const float4*>(a.table + (int64_t)p * a.rope_dim + 8 * c);
        const float4* row_s = reinterpret_cast<const float4*>(
            a.table + (int64_t)p * a.rope_dim + a.rope_dim / 2 + 8 * c);
        const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row_s), s1 = __ldg(row_s + 1);
        cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w;
        cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
        sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
        sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int x = a.pair_axis[8 * c + i];
          const int p = x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3];
          const float* row = a.table + (int64_t)p * a.rope_dim + 8 * c + i;
          cs[i] = __ldg(row);
          sn[i] = __ldg(row + a.rope_dim / 2);
        }
      }
    }
    if (FP8 && !is_q) {
      float f[16];
      unpack8(w0[0], f);
      unpack8(w1[0], f + 8);
      if (rot && !is_v) rotate<INTERLEAVED>(f, cs, sn);
      // Largest magnitude of the row, over its 8 lanes (head_dim is 128); NaN if any value is,
      // so that the row's scale and codes are.
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = max_nan(amax, abs_ieee(f[i]));
#pragma unroll
      for (int o = 4; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (left <= 0 || !store) continue;
      const float scale = div_ieee(amax, 448.f);
      uint8_t* dst = (is_v ? a.v_cache : a.k_cache) + ((int64_t)slot * a.Hkv + head0) * 128;
      const uint4 codes = codes16(f, scale);
      *reinterpret_cast<uint2*>(dst + lo) = make_uint2(codes.x, codes.y);
      *reinterpret_cast<uint2*>(dst + hi) = make_uint2(codes.z, codes.w);
      if (c == 0) {
        const int blk = slot / a.block_size, off = slot - blk * a.block_size;
        (is_v ? a.v_scale : a.k_scale)[((int64_t)blk * a.Hkv + head0 + sub) * a.block_size + off] = scale;
      }
      continue;
    }
    if (!is_q && !store) continue;
    uint16_t* dst = is_q ? a.q_out + t * a.q_out_stride + head0 * a.head_dim
                         : reinterpret_cast<uint16_t*>(is_v ? a.v_cache : a.k_cache) +
                               ((int64_t)slot * a.Hkv + head0) * a.head_dim;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!active || u * per_pass >= left) continue;
      if (rot && !is_v) {
        float f[16];
        unpack8(w0[u], f);
        unpack8(w1[u], f + 8);
        rotate<INTERLEAVED>(f, cs, sn);
        w0[u] = pack8(f);
        w1[u] = pack8(f + 8);
      }
      *reinterpret_cast<uint4*>(dst + u * pass_stride + lo) = w0[u];
      *reinterpret_cast<uint4*>(dst + u * pass_stride + hi) = w1[u];
    }
  }
}

template <bool FP8, bool INTERLEAVED>
static cudaError_t launch_rope_n(const RopeArgs& a, cudaStream_t stream, int num_sms) {
  const int per_pass = 32 / (a.head_dim / 16), q_share = per_pass * kUnroll;
  const int kv_share = FP8 ? per_pass : q_share;
  const int64_t items = a.num_tokens * ((a.H + q_share - 1) / q_share + 2 * ((a.Hkv + kv_share - 1) / kv_share));
  int64_t blocks = (items + 7) / 8;
  const int64_t cap = (int64_t)num_sms * kCtasPerSm;
  if (blocks > cap) blocks = cap;
  return launch_dependent(rope_write_kernel<FP8, INTERLEAVED>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
}

cudaError_t launch_rope_write(const RopeArgs& a, bool fp8, bool interleaved, cudaStream_t stream,
                              int num_sms) {
  if (a.num_tokens == 0) return cudaSuccess;
  if (fp8)
    return interleaved ? launch_rope_n<true, true>(a, stream, num_sms)
                       : launch_rope_n<true, false>(a, stream, num_sms);
  return interleaved ? launch_rope_n<false, true>(a, stream, num_sms)
                     : launch_rope_n<false, false>(a, stream, num_sms);
}

}  // namespace pkv
