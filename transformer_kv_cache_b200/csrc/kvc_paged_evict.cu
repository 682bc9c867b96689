// kvc_paged_evict.cu -- eviction from a paged batch by accumulated attention weight.
//
// Per sequence longer than `keep` and per KV head: the kept tokens are the protected ones
// (position < sinks or position >= next position - recent) and then those of highest score,
// ties to the lower slot. Kept tokens in the first `keep` slots stay where they are; the
// others move, in ascending slot, into the slots of the evicted ones, in ascending slot, so
// an eviction moves as few rows as it can and never a row onto one that is still to be read.
//
// Two launches: the selection writes each (sequence, head)'s moves into the workspace, and the
// moves, which then spread over the whole GPU, also set the lengths (every head has read the old
// ones by then).
//
// Selection. A token's key is the order-preserving integer of its score (NaN lowest, protected
// highest). One cluster of 1 to 8 CTAs works on a (sequence, head), its keys read once into
// shared memory, four to a load.
//   Up to kFew evicted (a decode step): they are taken one by one as the lowest (key, then
//   highest slot), a reduction each over the keys.
//   More: the keep-th largest key is found exactly by three passes of 11, 11 and 10 bits: a
//   histogram of the bits below the prefix found so far, summed over distributed shared memory,
//   and the bin that holds the keep-th (11 bits take the sign, the exponent and two bits of the
//   mantissa first, so that the scores spread over the bins). Slot order makes every rank a count
//   over lower slots: warps own consecutive runs of slots, CTAs consecutive runs of warps.
// Moves. Bound by memory (two rows read and written each). The selection looks the pages up, so
// that a move is two dependent loads, its entry in the list and its rows, and a thread has kUnroll
// moves under way.
// The keys' shared memory is laid out for what a sequence has room for, since no length is known on the
// host: room for 32,768 tokens leaves an SM one CTA of the selection, and 64 of 4,160 tokens go in 74 us where
// room for 4,160 takes 22 (64 sequences of 8 heads).
//
// 64 sequences of 8 heads of 4,097 tokens, one of which goes: 14 us a step with the append, most of it
// the three launches' own. 4 sequences of up to 32,768 tokens cut to 4,096: 51 us (120 MB: 2.4 TB/s),
// a third of it the selection, three passes whose barriers a cluster of four waits for.
#include <algorithm>

#include "kvc_paged.cuh"

namespace kvc {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;                 // the portable size
constexpr int kMaxChunk = 49152;               // keys a CTA holds: 192 KB
constexpr int kBins = 2048;
constexpr int kFew = 8;                        // evicted tokens that are taken one by one
constexpr int kMoveThreads = 256;
constexpr int kMoves = 32;                     // moves of a CTA, or the slots of a page where those are more
constexpr int kMoveCtas = 16;                  // of an SM, at most
constexpr int kSlots = 8192;                   // slots from which on a (sequence, head) gets another CTA
constexpr int kUnroll = 2;

// Scores ascending as unsigned integers: -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t caddr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(caddr) : "memory");
  return v;
}
// Barrier of the (sequence, head)'s CTAs.
__device__ __forceinline__ void sync_all(int ranks) {
  if (ranks == 1) {
    __syncthreads();
  } else {
    cluster_arrive_release();
    cluster_wait_acquire();
  }
}

struct Shared {
  uint32_t hist[2][kBins];
  uint32_t counts[4];           // this CTA's: above the threshold from slot `keep` on and below it, ties likewise
  uint32_t warp_counts[kWarps][4];
  uint32_t group[2][kBins / 32];
  uint64_t lowest[2];           // this CTA's lowest (key, slot), two rounds in turn
  uint64_t warp_low[kWarps];
  uint32_t bin, need;
};

__device__ __forceinline__ uint32_t warp_sum(uint32_t x) { return __reduce_add_sync(0xffffffffu, x); }
// A shared variable summed over the cluster's CTAs.
__device__ __forceinline__ uint32_t sum_over(const uint32_t* x, int ranks) {
  if (ranks == 1) return *x;
  uint32_t sum = 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < ranks) sum += ld_cluster_u32(cluster_map(smem_u32(x), r));
  return sum;
}
// The lane in whose `count` the need-th of all lanes' counts falls, lane 0 first; `above` gains
// the counts of the lanes before it.
__device__ __forceinline__ int find_rank(uint32_t count, uint32_t need, uint32_t& above) {
  const int lane = threadIdx.x & 31;
  uint32_t incl = count;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  const uint32_t hit = __ballot_sync(0xffffffffu, incl >= need);
  const int at = hit ? __ffs(hit) - 1 : 31;
  above += __shfl_sync(0xffffffffu, incl - count, at);
  return at;
}

__global__ void __launch_bounds__(kThreads, 4) paged_evict_select_kernel(const EvictParams p, int chunk) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ Shared sh;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rank = blockIdx.x, ranks = gridDim.x;          // the cluster spans x
  const int h = blockIdx.y, b = blockIdx.z;
  const int cap = p.max_pages << p.page_shift;
  int len = p.lengths[b];
  if (len < 0 || len > cap) {
    if (t == 0) latch_error(p.err, DERR_BOUNDS);
    len = min(max(len, 0), cap);
  }
  const long long bh = static_cast<long long>(b) * p.Hkv + h;
  if (len <= p.keep) {                                     // the same for the whole cluster
    if (t == 0 && rank == 0) p.counts[bh] = -1;
    return;
  }
  const float* scores = p.scores + bh * cap;
  const int32_t* positions = p.positions + bh * cap;
  const int recent_from = p.next_positions[b] - p.recent;
  const int c0 = min(len, rank * chunk), c1 = min(len, c0 + chunk), n = c1 - c0;
  const int gone = len - p.keep;
  int2* list_to = p.moves + bh * 2 * p.move_cap;
  int2* list_from = list_to + p.move_cap;
  const int32_t* table = p.page_table + static_cast<long long>(b) * p.max_pages;
  // a slot and its row in the pools (-1: the table names no page)
  auto place = [&](int slot) {
    const int32_t page = __ldg(table + (slot >> p.page_shift));
    if (page >= 0 && page < p.pool_pages)
      return make_int2(slot, ((page * p.Hkv + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1)));
    latch_error(p.err, DERR_BOUNDS);
    return make_int2(slot, -1);
  };
  auto key_of = [&](int pos, float x) { return pos < p.sinks || pos >= recent_from ? 0xffffffffu : score_key(x); };
#pragma unroll 2
  for (int i = 4 * t; i < n; i += 4 * kThreads) {          // rows of cap slots, a multiple of 16; reads past n stay in them
    const int4 pos = *reinterpret_cast<const int4*>(positions + c0 + i);
    const float4 x = *reinterpret_cast<const float4*>(scores + c0 + i);
    *reinterpret_cast<uint4*>(keys + i) =
        make_uint4(key_of(pos.x, x.x), key_of(pos.y, x.y), key_of(pos.z, x.z), key_of(pos.w, x.w));
  }
  uint32_t moves = 0;
  if (gone <= kFew) {
    // the lowest key, the highest slot among equals, `gone` times; its key then counts as highest
    int out[kFew];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kFew; ++r) {
      out[r] = cap;
      if (r >= gone) continue;
      uint64_t low = ~0ull;
      for (int i = t; i < n; i += kThreads) {
        bool taken = false;
#pragma unroll
        for (int q = 0; q < kFew; ++q)
          if (q < r) taken |= c0 + i == out[q];
        // slots descend in the low half, so that the highest comes first
        if (!taken) low = min(low, (static_cast<uint64_t>(keys[i]) << 32) | static_cast<uint32_t>(~(c0 + i)));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, d));
      if (lane == 0) sh.warp_low[warp] = low;
      __syncthreads();
      if (warp == 0) {
        low = lane < kWarps ? sh.warp_low[lane] : ~0ull;
#pragma unroll
        for (int d = 16; d; d >>= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, d));
        if (lane == 0) sh.lowest[r & 1] = low;
      }
      sync_all(ranks);
      low = sh.lowest[r & 1];
      if (ranks > 1)
        for (int k = 0; k < ranks; ++k) low = min(low, ld_cluster_u64(cluster_map(smem_u32(&sh.lowest[r & 1]), k)));
      out[r] = static_cast<int>(~static_cast<uint32_t>(low));
    }
    if (ranks > 1) sync_all(ranks);                        // nobody leaves while its lowest is read
    // at most kFew moves: every thread finds move t of its own
    if (rank == 0 && t < kFew) {
      // the t-th evicted slot below `keep`, and the t-th kept slot from `keep` on
      int to = -1, from = -1, k = 0;
      for (int s = 0; s < p.keep && k <= t; ++k) {         // ascending, by picking the least left
        int best = p.keep;
#pragma unroll
        for (int q = 0; q < kFew; ++q)
          if (out[q] >= s && out[q] < best) best = out[q];
        if (best == p.keep) break;
        to = k == t ? best : -1;
        s = best + 1;
      }
      k = 0;
      for (int s = p.keep; s < len; ++s) {
        bool taken = false;
#pragma unroll
        for (int q = 0; q < kFew; ++q) taken |= out[q] == s;
        if (!taken && k++ == t) from = s;
      }
      if (to >= 0 && from >= 0) {
        list_to[t] = place(to);
        list_from[t] = place(from);
      }
    }
    // how many: evicted slots below `keep`
#pragma unroll
    for (int q = 0; q < kFew; ++q) moves += out[q] < p.keep;
  } else {
    for (int i = t; i < 2 * kBins; i += kThreads) sh.hist[i / kBins][i % kBins] = 0;
    __syncthreads();
    // the keep-th largest key: `prefix` its bits so far, `need` how many of the tokens with that
    // prefix are kept
    uint32_t prefix = 0, mask = 0;
    uint32_t need = p.keep;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bins = 1u << bits;
      uint32_t* hist = sh.hist[pass & 1];
      for (int i = t; i < n; i += kThreads) {
        const uint32_t k = keys[i];
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      // sums of 32 bins each, so that a CTA reads few of its peers' counts
      for (int g = warp; g < static_cast<int>(bins) / 32; g += kWarps) {
        const uint32_t sum = warp_sum(hist[32 * g + lane]);
        if (lane == 0) sh.group[pass & 1][g] = sum;
      }
      sync_all(ranks);
      if (warp == 0) {
        // the group, then the bin, that holds the keep-th from the top
        const int groups = bins / 32;
        uint32_t two[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int g = groups - 1 - (2 * lane + i);
          if (g >= 0) two[i] = sum_over(sh.group[pass & 1] + g, ranks);
        }
        uint32_t above = 0;
        int g = find_rank(two[0] + two[1], need, above);   // the lane
        const uint32_t upper = __shfl_sync(0xffffffffu, two[0], g);
        g *= 2;
        if (above + upper < need) {
          above += upper;
          ++g;
        }
        g = groups - 1 - g;
        need -= above;
        above = 0;
        const uint32_t one = sum_over(hist + 32 * g + 31 - lane, ranks);
        const int bin = 32 * g + 31 - find_rank(one, need, above);
        if (lane == 0) {
          sh.bin = bin;
          sh.need = need - above;
        }
      }
      // the next pass but one counts here again: every CTA has read it, this pass's barrier came after
      if (pass == 1)
        for (int i = t; i < kBins; i += kThreads) sh.hist[0][i] = 0;
      __syncthreads();
      prefix |= sh.bin << shift;
      mask |= (bins - 1) << shift;
      need = sh.need;
    }
    const uint32_t threshold = prefix;                     // kept: key > threshold, or one of the first `need` ties

    // Counts by warp, each over its run of slots, then by CTA: [0] above the threshold from slot
    // `keep` on, [1] above it before that, [2] and [3] ties likewise.
    const int per_warp = (((chunk + kWarps - 1) / kWarps) + 31) & ~31;
    const int w0 = min(n, warp * per_warp), w1 = min(n, w0 + per_warp);
    uint32_t count[4] = {0, 0, 0, 0};
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint32_t k = keys[i];
      const bool high = c0 + i >= p.keep;
      count[0] += k > threshold && high;
      count[1] += k > threshold && !high;
      count[2] += k == threshold && high;
      count[3] += k == threshold && !high;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      count[q] = warp_sum(count[q]);
      if (lane == 0) sh.warp_counts[warp][q] = count[q];
    }
    __syncthreads();
    if (t < 4) {
      uint32_t sum = 0;
      for (int w = 0; w < kWarps; ++w) sum += sh.warp_counts[w][t];
      sh.counts[t] = sum;
    }
    sync_all(ranks);
    // Of a run of slots with `ties` ties behind `seen` earlier ones, the first need - seen are kept,
    // slots below `keep` first. from0, to0: moved tokens and holes in lower slots.
    uint32_t seen = 0, from0 = 0, to0 = 0;
    auto pass_run = [&](uint32_t high, uint32_t low, uint32_t tie_high, uint32_t tie_low, int slots_low) {
      const uint32_t left = need > seen ? need - seen : 0;
      const uint32_t kept_low = min(left, tie_low), kept_high = min(left - kept_low, tie_high);
      from0 += high + kept_high;
      to0 += slots_low - low - kept_low;
      seen += tie_high + tie_low;
    };
    uint32_t my_seen = 0, my_from = 0, my_to = 0;
    for (int r = 0; r < ranks; ++r) {
      if (r == rank) {
        my_seen = seen;
        my_from = from0;
        my_to = to0;
      }
      uint32_t c[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        c[q] = ranks == 1 ? sh.counts[q] : ld_cluster_u32(cluster_map(smem_u32(&sh.counts[q]), r));
      const int a = min(len, r * chunk), z = min(len, a + chunk);
      pass_run(c[0], c[1], c[2], c[3], min(z, p.keep) - min(a, p.keep));
    }
    moves = from0;
    seen = my_seen;
    from0 = my_from;
    to0 = my_to;
    for (int w = 0; w < warp; ++w) {
      const uint32_t* c = sh.warp_counts[w];
      const int a = c0 + min(n, w * per_warp), z = c0 + min(n, (w + 1) * per_warp);
      pass_run(c[0], c[1], c[2], c[3], min(z, p.keep) - min(a, p.keep));
    }
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane, slot = c0 + i;
      const uint32_t k = i < w1 ? keys[i] : 0;
      const uint32_t eq = __ballot_sync(0xffffffffu, i < w1 && k == threshold);
      const uint32_t below = (1u << lane) - 1u;
      const bool kept = i < w1 && (k > threshold || (k == threshold && seen + __popc(eq & below) < need));
      seen += __popc(eq);
      const uint32_t f = __ballot_sync(0xffffffffu, kept && slot >= p.keep);
      const uint32_t g = __ballot_sync(0xffffffffu, i < w1 && !kept && slot < p.keep);
      if (f >> lane & 1u) list_from[from0 + __popc(f & below)] = place(slot);
      if (g >> lane & 1u) list_to[to0 + __popc(g & below)] = place(slot);
      from0 += __popc(f);
      to0 += __popc(g);
    }
    if (ranks > 1) sync_all(ranks);                        // nobody leaves while its counts are read
  }
  if (t == 0 && rank == 0) p.counts[bh] = static_cast<int>(moves);
}

// Moves [per_cta x, + per_cta) of (sequence z, head y), and so on by the grid. The first CTA of a head also
// clears the slots behind the last kept one, to the end of its page: they are the lowest slots that moves
// can come from, so that those moves, if any, are among its first. What comes from the workspace is bounded again: a
// call that wrongly runs beside another with the same workspace moves the wrong tokens, but none elsewhere.
__global__ void __launch_bounds__(kMoveThreads, 4) paged_evict_move_kernel(const EvictParams p, int32_t* lengths, int per_cta) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x, h = blockIdx.y, b = blockIdx.z;
  const long long bh = static_cast<long long>(b) * p.Hkv + h;
  const int moves = min(p.counts[bh], p.move_cap);
  const int stride = static_cast<int>(gridDim.x) * per_cta;
  if (moves < 0) return;
  const int cap = p.max_pages << p.page_shift;
  const int pool_rows = static_cast<int>((p.pool_pages * p.Hkv) << p.page_shift);
  auto sound = [&](int2 at) {
    return static_cast<unsigned>(at.x) < static_cast<unsigned>(cap) && at.y < pool_rows ? at : make_int2(-1, -1);
  };
  float* scores = p.scores + bh * cap;
  int32_t* positions = p.positions + bh * cap;
  const int2* list_to = p.moves + bh * 2 * p.move_cap;
  const int2* list_from = list_to + p.move_cap;
  const int32_t* table = p.page_table + static_cast<long long>(b) * p.max_pages;
  const int page_mask = (1 << p.page_shift) - 1;
  const int lanes = p.row_bytes >> 4;                      // lanes of a row: 8, 16 or 32
  const int per = kMoveThreads / lanes;                    // rows a CTA moves at once
  const int part = (t % lanes) * 16;
  for (int first = blockIdx.x * per_cta; first < moves; first += stride) {
    const int end = min(moves, first + per_cta);
    for (int r = first + t / lanes; r < end; r += kUnroll * per) {
      int2 src[kUnroll], dst[kUnroll];
      uint4 k[kUnroll], v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = r + u * per;
        src[u] = i < end ? sound(list_from[i]) : make_int2(-1, -1);
        dst[u] = i < end ? sound(list_to[i]) : make_int2(-1, -1);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (src[u].y >= 0 && dst[u].y >= 0) {
          const long long a = static_cast<long long>(src[u].y) * p.row_bytes + part;
          k[u] = *reinterpret_cast<const uint4*>(p.k_pool + a);
          v[u] = *reinterpret_cast<const uint4*>(p.v_pool + a);
        }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (src[u].y >= 0 && dst[u].y >= 0) {
          const long long c = static_cast<long long>(dst[u].y) * p.row_bytes + part;
          *reinterpret_cast<uint4*>(p.k_pool + c) = k[u];
          *reinterpret_cast<uint4*>(p.v_pool + c) = v[u];
        }
        if (src[u].x >= 0 && dst[u].x >= 0 && part == 0) {
          scores[dst[u].x] = scores[src[u].x];
          positions[dst[u].x] = positions[src[u].x];
        }
      }
    }
  }
  if (blockIdx.x > 0) return;
  if (t == 0 && h == 0) lengths[b] = p.keep;
  if (p.keep & page_mask) {
    __syncthreads();
    const int tail = (page_mask + 1) - (p.keep & page_mask);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const int32_t page = __ldg(table + (p.keep >> p.page_shift));
    if (page < 0 || page >= p.pool_pages) {
      latch_error(p.err, DERR_BOUNDS);
      return;
    }
    const long long row0 = ((static_cast<long long>(page) * p.Hkv + h) << p.page_shift) + (p.keep & page_mask);
    for (int r = t / lanes; r < tail; r += per) {
      const long long c = (row0 + r) * p.row_bytes;
      *reinterpret_cast<uint4*>(p.k_pool + c + part) = zero;
      *reinterpret_cast<uint4*>(p.v_pool + c + part) = zero;
    }
  }
}

}  // namespace

int paged_evict_max_slots() { return kMaxCluster * kMaxChunk; }

cudaError_t launch_paged_evict(cudaStream_t s, const EvictParams& p, int sms, int32_t* lengths) {
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(paged_evict_select_kernel),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxChunk * 4);
  });
  if (e != cudaSuccess) return e;
  // one CTA for a (sequence, head) unless its slots do not fit, or the CTAs would not fill the
  // GPU and have kSlots each to share: below that the cluster's barriers cost more than it saves
  const int cap = p.max_pages << p.page_shift;
  int ranks = 1;
  while (ranks < kMaxCluster &&
         (cap > ranks * kMaxChunk || (cap > ranks * kSlots && static_cast<long long>(p.B) * p.Hkv * ranks < sms)))
    ranks *= 2;
  const int chunk = (((cap + ranks - 1) / ranks) + 31) & ~31;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ranks, p.Hkv, p.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(chunk) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, paged_evict_select_kernel, p, chunk);
  if (e != cudaSuccess) return e;
  const int per_cta = std::max(kMoves, 1 << p.page_shift);
  // A CTA for per_cta moves where all that the sequences have room for need no more than kMoveCtas an SM;
  // else that many, which then run through the moves. Without the limit a token a step of 64 sequences of
  // 8 heads, kept 4,096 with room for as many, takes 76 us, 73 of them for CTAs that find no move; with it
  // 11.5 (9.9 at 4 an SM, which cut 16 sequences from 12,000 tokens to 6,000 in 135 us, 16 in 107).
  const long long heads = static_cast<long long>(p.B) * p.Hkv;
  const int ctas = static_cast<int>(std::min<long long>((p.move_cap + per_cta - 1) / per_cta,
                                                        (static_cast<long long>(kMoveCtas) * sms + heads - 1) / heads));
  return launch_pdl(paged_evict_move_kernel, dim3(ctas, p.Hkv, p.B), dim3(kMoveThreads), 0, s, p, lengths, per_cta);
}

}  // namespace kvc
