// Eviction: the choice of the rows that stay.
//
// For each sequence and kv head the num_keep positions with the largest weights, ascending. The
// first num_sink and the last num_recent are taken without being ranked; of the others, as
// integers in the weights' order, the border is searched, the weight of the last row taken:
//   - a sample of the weights (8 of each block's 128, a sector of memory) gives a bracket that
//     holds the border with near certainty: the digits (11 bits) of the weights that lie three
//     and a half standard deviations of the sample's rank to either side;
//   - one pass over the weights: two bit masks in shared memory, of those above the bracket and
//     of those inside it; the few inside (some 10 %; all of a short row, without a sample) go into
//     a list;
//   - the border is found in the list digit by digit, a histogram and a scan from the top each;
//   - the list's rows above it enter the first mask, those that equal it a mask of their own, of
//     which the lowest positions are taken; every lane writes the positions of words of the masks.
// Where the bracket misses, or the list overflows, all of it is done again with every digit over all
// weights, read from L2 each time. The bracket is a digit wide at least, a quarter of an octave, so the list
// overflows where many weights lie that close together: few different values, but sums of a narrow
// spread too. Measured on GB300, 512 rows of up to 32,768 weights, 4,096 kept: lognormal weights with a
// spread of 2.5 30 us, of 0.3 81, uniform ones 89, sums of 128 steps and 8 heads of independent normal
// scores 89; 16 rows of a million 62, 228, 229, 228; 512 rows of up to 8,192 17, 16, 16, 29.
//
// A row (sequence, kv head) is the work of a cluster of 1 to 8 CTAs, each with its own run of
// blocks, list and histograms; every CTA sums the histograms of the cluster for itself through
// distributed shared memory.
//
// Roofline: HBM by bytes (4 per weight), instructions in practice: some 350 of a warp per block of 128
// weights, issue slots 67 % busy. Measured on GB300: 512 rows of up to 32,768 weights (4,096 kept) 30 us,
// where the bytes take 5.5: a CTA of 256 blocks, one of three on its SM, spends some 45,000 cycles, 2,900
// on the sample, 10,700 on the pass over the weights, 5,400 on the list, 6,000 on scans and digits, 5,500
// on the positions, the rest on lookups and barriers. 16 rows of a million weights (65,536 kept) 61 us
// where the bytes take 10: clusters of 8, one CTA to an SM. More blocks in flight (eight: 84 us),
// prefetches into L2 (68) and the longest sequences first (512 rows 31 us, 1,600 rows 100 and 116) do not help.
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int BS = 128, BINS = 2048, MAX_WARPS = 16;
constexpr int FLIGHT = 2;        // blocks of a warp in flight while as many are worked on
constexpr int SHORT = 1024;      // rows of a CTA that need no bracket
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_PER_CTA = 4096;  // blocks of a CTA, whose masks take 128 KB
static_assert(kSelectRowsMaxBlocks <= MAX_CLUSTER * MAX_PER_CTA, "a row's masks fit its cluster");
constexpr uint32_t ABSENT = 0, BAD = 1;  // keys of positions that are not ranked, and of bad blocks

// Whole numbers in the order of weights given by their bits: -0 equals 0, NaN is above all; the
// least, of -infinity, is 0x7fffff. (The weights are read as integers: as floats, the compiler may
// turn the tests below into comparisons that take subnormals for zero.)
__device__ __forceinline__ uint32_t weight_key(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if ((u & 0x7fffffffu) == 0) return 0x80000000u;
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint4 weight_keys(uint4 w) {
  // Numbers from 0 to infinity, as sums of weights are, need one bit set.
  if (max(max(w.x, w.y), max(w.z, w.w)) <= 0x7f800000u)
    return make_uint4(w.x | 0x80000000u, w.y | 0x80000000u, w.z | 0x80000000u, w.w | 0x80000000u);
  return make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
}

struct Shared {
  int hist[2][BINS];
  int wsum[MAX_WARPS], wabove[MAX_WARPS], wequal[MAX_WARPS];
  int bin[2], rest, all, total;          // what a scan found
  int above, inside;                     // of this CTA: rows above the bracket, rows in the list
  int taken, equal;                      // rows taken without ties, rows of the border's weight
};

// Dynamic shared memory: masks of a CTA's blocks, four words each (bit l of word j: position 4 l + j),
// of rows taken and of rows inside the bracket, later of rows that equal the border; then the list,
// its rows' places as 4 * 32 * block + 32 j + l.
struct Lists {
  uint4 *take, *other;
  uint32_t *key, *place;
  __device__ __forceinline__ Lists(uint4* base, int blocks, int rows)
      : take(base), other(take + blocks), key(reinterpret_cast<uint32_t*>(other + blocks)), place(key + rows) {}
};

// Bits 0 to 7 of x as bits 0, 4, .. 28.
__device__ __forceinline__ uint32_t spread8(uint32_t x) {
  x &= 0xffu;
  x = (x | x << 12) & 0x000f000fu;
  x = (x | x << 6) & 0x03030303u;
  return (x | x << 3) & 0x11111111u;
}
// Positions 32 t .. 32 t + 31 of a block's mask in order.
__device__ __forceinline__ uint32_t in_order(uint4 m, int t) {
  return spread8(m.x >> 8 * t) | spread8(m.y >> 8 * t) << 1 | spread8(m.z >> 8 * t) << 2 | spread8(m.w >> 8 * t) << 3;
}
__device__ __forceinline__ int size(uint4 m) { return __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w); }

// LIST: rows of a CTA inside the bracket; RESIDENT: CTAs that an SM holds.
template <int THREADS, int LIST, int RESIDENT>
__global__ void __launch_bounds__(THREADS, RESIDENT)
    select_rows_kernel(const __grid_constant__ SelectRowsArgs a, int cta_blocks) {
  constexpr int WARPS = THREADS / 32;
  __shared__ __align__(16) Shared sh;
  extern __shared__ __align__(16) uint4 dynamic[];
  pdl_wait_then_launch();
  const int C = (int)cg::this_cluster().num_blocks(), rank = (int)cg::this_cluster().block_rank();
  const int row = blockIdx.x / C, b = row / a.Hkv, g = row % a.Hkv;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int raw = __ldg(a.seq_lens + b), n = clamp_len(raw, a.max_blocks * BS);
  if (n != raw && g == 0 && rank == 0 && tid == 0) flag_status(a.dev_status, PKV_DEV_BAD_LENGTH);
  int32_t* out = a.out + (int64_t)row * a.num_keep;
  if (n <= a.num_keep) {
    for (int i = rank * THREADS + tid; i < a.num_keep; i += C * THREADS) out[i] = i < n ? i : -1;
    return;
  }
  const int lo = a.num_sink, hi = n - a.num_recent;  // ranked: [lo, hi)
  for (int i = rank * THREADS + tid; i < a.num_sink; i += C * THREADS) out[i] = i;
  for (int i = rank * THREADS + tid; i < a.num_recent; i += C * THREADS)
    out[a.num_keep - a.num_recent + i] = hi + i;
  const int want = a.num_keep - a.num_sink - a.num_recent;  // of hi - lo > want
  if (want == 0) return;
  auto sync = [&] {
    if (C == 1)
      __syncthreads();
    else
      cg::this_cluster().sync();
  };
  const Lists list(dynamic, cta_blocks, LIST);

  // This warp's blocks: `count` from `first` on; their masks begin at the own-th of the CTA's.
  const int blocks = (hi + BS - 1) / BS, per = (blocks + C * WARPS - 1) / (C * WARPS);
  const int first = (rank * WARPS + warp) * per, count = max(0, min(per, blocks - first)), own = warp * per;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks + first;
  const uint32_t* weights = reinterpret_cast<const uint32_t*>(a.weights) + (int64_t)g * BS;
  const int64_t stride = (int64_t)a.Hkv * BS;  // from block to block
  // What another CTA of the cluster has where this one has *mine; r is clamped to the cluster.
  auto theirs = [&](auto* mine, int r) { return cg::this_cluster().map_shared_rank(mine, min(r, C - 1)); };
  // The warp's blocks in order: f(block, its four keys of this lane). FLIGHT blocks are loaded while
  // those before them are worked on.
  auto stream = [&](auto&& f) {
    int ids = 0;        // of 32 blocks, lane l's that of block l of them
    unsigned bad = 0;
    auto load = [&](int q, uint4(&w)[FLIGHT]) {
      if (q % 32 == 0) {
        ids = q + lane < count ? __ldg(table + q + lane) : 0;
        const bool wrong = ids < 0 || (int64_t)ids >= a.num_blocks;
        if (wrong) {
          flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
          ids = 0;
        }
        bad = __ballot_sync(0xffffffffu, wrong);
      }
#pragma unroll
      for (int i = 0; i < FLIGHT; ++i) {
        const int blk = __shfl_sync(0xffffffffu, ids, (q + i) % 32);
        if (q + i < count) w[i] = __ldg(reinterpret_cast<const uint4*>(weights + blk * stride) + lane);
      }
      return bad >> (q % 32);
    };
    uint4 now[FLIGHT], then[FLIGHT];
    unsigned bad_now = load(0, now), bad_then = 0;
    for (int q = 0; q < count; q += FLIGHT) {
      if (q + FLIGHT < count) bad_then = load(q + FLIGHT, then);
#pragma unroll
      for (int i = 0; i < FLIGHT; ++i) {
        if (q + i >= count) break;
        uint4 k = bad_now >> i & 1 ? make_uint4(BAD, BAD, BAD, BAD) : weight_keys(now[i]);
        const int start = (first + q + i) * BS, pos = start + 4 * lane;
        if (start < lo || start + BS > hi) {
          if (pos < lo || pos >= hi) k.x = ABSENT;
          if (pos + 1 < lo || pos + 1 >= hi) k.y = ABSENT;
          if (pos + 2 < lo || pos + 2 >= hi) k.z = ABSENT;
          if (pos + 3 < lo || pos + 3 >= hi) k.w = ABSENT;
        }
        f(q + i, k);
      }
#pragma unroll
      for (int i = 0; i < FLIGHT; ++i) now[i] = then[i];
      bad_now = bad_then;
    }
  };
  // The mask of the keys that p holds for.
  auto mask = [&](uint4 k, auto&& p) {
    return make_uint4(__ballot_sync(0xffffffffu, p(k.x)), __ballot_sync(0xffffffffu, p(k.y)),
                      __ballot_sync(0xffffffffu, p(k.z)), __ballot_sync(0xffffffffu, p(k.w)));
  };
  // Sums of x over the lanes before this one, and over all.
  auto before = [&](int x, int& all) {
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    all = __shfl_sync(0xffffffffu, incl, 31);
    return incl - x;
  };
  // Lanes take words of the masks, or bytes of them where a warp has a block or two: lane or item w of a
  // warp's words, 32 >> fine bits each, as bits of the whole word.
  const int fine = per <= 2 ? 2 : 0;
  auto share = [&](uint32_t word, int w) { return fine ? word & 0xffu << 8 * (w & 3) : word; };
  // Behind a sync(): EACH bins of a histogram, from bin BINS - 1 - EACH * tid down, summed over the
  // cluster, and how many rows lie in the bins above them.
  constexpr int EACH = BINS / THREADS;
  int held[EACH], higher;
  auto scan = [&](const int* hist) {
#pragma unroll
    for (int i = 0; i < EACH; ++i) held[i] = 0;
    for (int r = 0; r < C; ++r) {
      const int* from = C == 1 ? hist : theirs(hist, r);
#pragma unroll
      for (int i = 0; i < EACH; i += 4) {
        const int4 x = reinterpret_cast<const int4*>(from + BINS - EACH * (tid + 1))[EACH / 4 - 1 - i / 4];
        held[i] += x.w;
        held[i + 1] += x.z;
        held[i + 2] += x.y;
        held[i + 3] += x.x;
      }
    }
    int sum = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) sum += held[i];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh.wsum[warp] = incl;
    __syncthreads();
    incl += __reduce_add_sync(0xffffffffu, lane < warp ? sh.wsum[lane & (WARPS - 1)] : 0);
    higher = incl - sum;
    if (tid == THREADS - 1) sh.total = incl;
  };
  // The bin with the rank-th row from the top (1 <= rank <= total), in the thread that holds it:
  // f(bin, rows still to take in it, rows in it).
  auto find = [&](int rank_, auto&& f) {
    int rest = rank_ - higher;
    if (rest <= 0) return;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      if (rest > 0 && rest <= held[i]) f(BINS - 1 - EACH * tid - i, rest, held[i]);
      rest -= held[i];
    }
  };

  // Two histograms in turn: one is cleared once every CTA has come to the barrier behind which the
  // other is read.
  auto clear = [&](int* hist) {
    for (int i = tid; i < BINS / 4; i += THREADS) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
  };
  clear(sh.hist[0]);
  clear(sh.hist[1]);
  if (tid == 0) sh.above = sh.inside = 0;
  __syncthreads();

  // ---- bracket [low, top]
  uint32_t low = 1, top = 0xffffffffu;
  if (per * WARPS * BS > SHORT) {
    for (int q = 0; q < count; q += 4 * 4) {
      // Four blocks a load, eight lanes each: a sector of the block, another one for every block.
      uint32_t w[4];
      int pos[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = q + 4 * i + (lane >> 3);
        const int blk = at < count ? __ldg(table + at) : -1;
        const int off = ((first + at) * 5 % 16) * 8 + (lane & 7);
        pos[i] = blk < 0 || (int64_t)blk >= a.num_blocks ? -1 : (first + at) * BS + off;
        w[i] = pos[i] < 0 ? 0u : __ldg(weights + blk * stride + off);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (pos[i] >= lo && pos[i] < hi) atomicAdd(&sh.hist[0][weight_key(w[i]) >> 21], 1);
    }
    sync();
    scan(sh.hist[0]);
    if (tid == 0) {
      sh.bin[0] = BINS - 1;  // (the last bin: no row is above the bracket)
      sh.bin[1] = 0;
    }
    __syncthreads();
    const float m = (float)sh.total, p = (float)want / (float)(hi - lo);
    const float margin = 3.5f * sqrtf(m * p * (1.f - p)) + 2.f;
    const int upper = (int)floorf(m * p - margin), lower = (int)ceilf(m * p + margin);
    if (upper >= 1) find(upper, [&](int bin, int, int) { sh.bin[0] = bin; });
    if (lower <= sh.total) find(lower, [&](int bin, int, int) { sh.bin[1] = bin; });
    __syncthreads();
    top = (uint32_t)sh.bin[0] << 21 | 0x1fffffu;
    low = max(1u, (uint32_t)sh.bin[1] << 21);
  }

  // ---- masks of the rows above the bracket and inside it
  uint32_t border = 0;  // rows above it are taken
  int rest = 0;         // and so many of those that equal it
  {
    int above = 0, inside = 0;
    const uint32_t width = top - low;
    stream([&](int q, uint4 k) {
      const uint4 high = mask(k, [&](uint32_t x) { return x > top; });
      const uint4 in = mask(k, [&](uint32_t x) { return x - low <= width; });
      if (lane == 0) {
        list.take[own + q] = high;
        list.other[own + q] = in;
      }
    });
    __syncwarp();
    for (int q = lane; q < count; q += 32) {
      above += size(list.take[own + q]);
      inside += size(list.other[own + q]);
    }
    above = __reduce_add_sync(0xffffffffu, above);
    inside = __reduce_add_sync(0xffffffffu, inside);
    if (lane == 0) {
      atomicAdd(&sh.above, above);
      sh.wequal[warp] = inside;
    }
  }
  __syncthreads();
  // ---- the list, and the histogram of its first digit; a word of the masks per lane
  int shift = max(0, 32 - __clz(top - low) - 11);
  {
    int at = lane < WARPS ? sh.wequal[lane] : 0;
    const int inside = __reduce_add_sync(0xffffffffu, at);
    at = __reduce_add_sync(0xffffffffu, lane < warp ? at : 0);
    if (tid == 0) sh.inside = inside;
    if (inside <= LIST) {
      uint32_t* words = reinterpret_cast<uint32_t*>(list.other + own);
      for (int w0 = 0; w0 < 4 * count << fine; w0 += 32) {
        const int w = w0 + lane;
        const bool mine = w < 4 * count << fine;
        uint32_t bits = mine ? share(words[w >> fine], w) : 0;
        __syncwarp();
        if (mine) words[w >> fine] = 0;
        int all;
        int to = at + before(__popc(bits), all);
        at += all;
        const int word = w >> fine;
        const int blk = bits ? __ldg(table + word / 4) : 0;
        const bool good = blk >= 0 && (int64_t)blk < a.num_blocks;
        const uint32_t* from = weights + (good ? blk : 0) * stride + word % 4;
        while (bits) {
          uint32_t key[4];
          int bit[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            bit[i] = __ffs((int)bits) - 1;
            bits &= bits - 1;
            key[i] = bit[i] >= 0 && good ? __ldg(from + 4 * bit[i]) : 0u;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (bit[i] >= 0) {
              uint32_t k = key[i] | 0x80000000u;
              if (key[i] > 0x7f800000u || !good) k = good ? weight_key(key[i]) : BAD;
              list.key[to] = k;
              list.place[to] = 32 * (4 * own + word) + bit[i];
              ++to;
              // (At most the last bin, even if somebody else writes the weights meanwhile.)
              atomicAdd(&sh.hist[1][min((k - low) >> shift, BINS - 1u)], 1);
            }
          }
        }
        __syncwarp();
      }
    }
  }
  sync();
  bool found;
  {
    int over = 0, sum_above = 0;
    const Shared* s = C == 1 ? &sh : theirs(&sh, lane);
    if (lane < C) {
      over = s->inside > LIST;
      sum_above = s->above;
    }
    sum_above = __reduce_add_sync(0xffffffffu, sum_above);
    int left = want - sum_above;
    scan(sh.hist[1]);
    __syncthreads();
    // (All CTAs of the cluster come to the same answer.)
    found = !__any_sync(0xffffffffu, over) && left >= 1 && left <= sh.total;
    if (found) {
      // ---- the border among the list
      const int inside = sh.inside;
      uint32_t base = low;
      for (int round = 1;; ++round) {
        find(left, [&](int bin, int r, int size) {
          sh.bin[0] = bin;
          sh.rest = r;
          sh.all = r == size;
        });
        __syncthreads();
        base += (uint32_t)sh.bin[0] << shift;
        left = sh.rest;
        if (sh.all) {  // every row of the bin is taken: the border lies below its least weight
          border = base - 1;
          left = 0;
          break;
        }
        if (shift == 0) {
          border = base;
          break;
        }
        const uint32_t width = (1u << shift) - 1;
        shift = max(0, shift - 11);
        int* hist = sh.hist[(round + 1) & 1];
        clear(hist);
        __syncthreads();
        for (int i = tid; i < inside; i += THREADS) {
          const uint32_t d = list.key[i] - base;
          if (d <= width) atomicAdd(hist + (d >> shift), 1);
        }
        sync();
        scan(hist);
        __syncthreads();
      }
      rest = left;
      for (int i = tid; i < inside; i += THREADS) {
        const uint32_t k = list.key[i], p = list.place[i];
        uint4* to = k > border ? list.take : list.other;
        if (k > border || (k == border && rest > 0))
          atomicOr(reinterpret_cast<uint32_t*>(to) + p / 32, 1u << (p % 32));
      }
      __syncthreads();
    }
  }

  if (!found) {
    // ---- every digit over all weights
    sync();  // nobody reads the histograms any more
    clear(sh.hist[0]);
    __syncthreads();
    rest = want;
    for (int pass = 0; pass < 3; ++pass) {
      const int down = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      int* hist = sh.hist[pass & 1];
      stream([&](int, uint4 k) {
        auto add = [&](uint32_t x) {
          if (x != ABSENT && (pass == 0 || x >> (down + bits) == border))
            atomicAdd(hist + (x >> down & ((1 << bits) - 1)), 1);
        };
        add(k.x);
        add(k.y);
        add(k.z);
        add(k.w);
      });
      sync();
      clear(sh.hist[~pass & 1]);
      scan(hist);
      find(rest, [&](int bin, int r, int) {
        sh.bin[0] = bin;
        sh.rest = r;
      });
      __syncthreads();
      border = border << bits | (uint32_t)sh.bin[0];
      rest = sh.rest;
      __syncthreads();
    }
    stream([&](int q, uint4 k) {
      const uint4 high = mask(k, [&](uint32_t x) { return x > border; });
      const uint4 same = mask(k, [&](uint32_t x) { return x == border; });
      if (lane == 0) {
        list.take[own + q] = high;
        list.other[own + q] = same;
      }
    });
    __syncwarp();
  }

  // ---- positions: a word of the masks per lane, its positions in order; `rest` rows of exactly the
  // border's weight go, lowest first
  int above = 0, equal = 0;
  for (int q = lane; q < count; q += 32) {
    above += size(list.take[own + q]);
    if (rest > 0) equal += size(list.other[own + q]);
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  __syncthreads();  // (the sums below were counts of the list)
  if (lane == 0) {
    sh.wabove[warp] = above;
    sh.wequal[warp] = equal;
  }
  __syncthreads();
  int at = lane < WARPS ? sh.wabove[lane] : 0, eq = lane < WARPS ? sh.wequal[lane] : 0;
  if (C > 1) {
    if (warp == 0) {
      const int x = __reduce_add_sync(0xffffffffu, at), y = __reduce_add_sync(0xffffffffu, eq);
      if (lane == 0) {
        sh.taken = x;
        sh.equal = y;
      }
    }
    sync();
  }
  if (lane >= warp) at = eq = 0;
  if (C > 1) {
    const int *t = theirs(&sh.taken, lane), *e = theirs(&sh.equal, lane);
    if (lane < rank) {
      at += *t;
      eq += *e;
    }
  }
  at = __reduce_add_sync(0xffffffffu, at);  // rows above the border, and at it, before this warp's
  eq = __reduce_add_sync(0xffffffffu, eq);
  at += a.num_sink + min(eq, rest);
  for (int w0 = 0; w0 < 4 * count << fine; w0 += 32) {
    const int w = w0 + lane, word = w >> fine;
    const bool mine = w < 4 * count << fine;
    uint32_t bits = mine ? share(in_order(list.take[own + word / 4], word % 4), w) : 0;
    int all;
    if (eq < rest) {
      uint32_t same = mine ? share(in_order(list.other[own + word / 4], word % 4), w) : 0;
      int places = rest - eq - before(__popc(same), all);
      eq += all;
      for (; same && places > 0; --places) {
        bits |= same & (0u - same);
        same &= same - 1;
      }
      __syncwarp();
    }
    int to = at + before(__popc(bits), all);
    at += all;
    const int pos = first * BS + 32 * word;
    // (The masks hold `want` rows, unless somebody else writes the weights meanwhile.)
    for (; bits; bits &= bits - 1, ++to)
      if ((unsigned)to < (unsigned)(a.num_keep - a.num_recent)) out[to] = pos + __ffs((int)bits) - 1;
    __syncwarp();
  }
  if (C > 1) sync();  // no CTA goes while another may read its shared memory
}

template <int THREADS, int LIST, int RESIDENT>
cudaError_t launch(const SelectRowsArgs& a, int C, cudaStream_t stream) {
  constexpr int WARPS = THREADS / 32;
  static_assert(RESIDENT * (sizeof(Shared) + LIST * 8 + WARPS * 2 * sizeof(uint4) + 1024) <= 228 * 1024,
                "RESIDENT CTAs fit an SM's shared memory, 1 KB of it reserved for each");
  const auto kernel = select_rows_kernel<THREADS, LIST, RESIDENT>;
  const int cta_blocks = (a.max_blocks + C * WARPS - 1) / (C * WARPS) * WARPS;
  const size_t smem = (size_t)cta_blocks * 2 * sizeof(uint4) + LIST * 8;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             MAX_PER_CTA * 2 * (int)sizeof(uint4) + LIST * 8);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.Hkv * C));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, cta_blocks);
}

}  // namespace

cudaError_t launch_select_rows(const SelectRowsArgs& a, cudaStream_t stream, int num_sms) {
  const int64_t rows = (int64_t)a.B * a.Hkv;
  // Cluster width: room for the rows inside the bracket (some 13 % of 256 blocks), and CTAs for every
  // SM where the rows are few, of four blocks a warp or more. Measured on GB300 with wider and narrower
  // clusters (us for 1, 2, 4, 8 CTAs a row): 8 rows of 256 blocks 15.5, 12.9, 12.6, 15.9; 64 of 64 10.2,
  // 12.5, 20, 42; 512 of up to 256 31, 44, 83, 258; 128 of up to 1,024 145 (the lists overflow), 46, 46,
  // 94; 16 of 8,192 535, 535, 285, 68, with 16 CTAs 98. The host knows the table's width, not the lengths: the 512
  // rows of up to 256 blocks take 30 us behind a table of 256, 43 behind 512, 80 behind 1,024, 249 behind 2,048,
  // 270 behind 8,192 and 448 behind 32,768; 512 rows of up to 32 blocks 13, 30, 64, 220, 240 and 389.
  int C = 1;
  while (C < MAX_CLUSTER && (a.max_blocks > 256 * C || (a.max_blocks > 64 * C && rows * 2 * C <= num_sms)))
    C *= 2;
  // Much of a CTA's work does not depend on the row's length, so short rows take fewer warps, and more CTAs to
  // an SM. Measured on GB300 (us with 512 threads, 256, 128): 512 rows of up to 512 weights 11.1, 8.2, 9.2, of
  // 4,096 14.4, 12.7, 14.3, of 16,384 20.2, 20.4, 26.5; 4,096 rows of up to 512 69, 40, 34, of 4,096 105, 80, 67;
  // 2,048 rows of up to 8,192 53, 39, 37, of 16,384 97, 89, 131; 160 rows of 4,096 8.6, 9.0, 10.3.
  if (C == 1 && a.max_blocks <= 32 && rows > 4 * num_sms) return launch<128, 2048, 6>(a, 1, stream);
  if (C == 1 && a.max_blocks <= 128 && rows > 2 * num_sms) return launch<256, 3584, 4>(a, 1, stream);
  return launch<512, 5120, 3>(a, C, stream);
}

}  // namespace pkv
