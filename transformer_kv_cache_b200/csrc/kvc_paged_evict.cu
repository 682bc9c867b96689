// kvc_paged_evict.cu -- eviction from a paged batch by accumulated attention weight.
//
// Per sequence longer than `keep` and per KV head: the kept tokens are the protected ones
// (position < sinks or position >= next position - recent) and then those of highest score,
// ties to the lower slot. Kept tokens in the first `keep` slots stay where they are; the
// others move, in ascending slot, into the slots of the evicted ones, in ascending slot, so
// an eviction moves as few rows as it can and never a row onto one that is still to be read.
//
// Selection. A token's key is the order-preserving integer of its score (NaN lowest, protected
// highest), so the keep-th largest key is found exactly by four passes of 8 bits over the
// keys: a histogram of the bits below the prefix found so far, summed over the cluster, and the
// bin that holds the keep-th. One cluster of 1 to 8 CTAs works on a (sequence, head); its
// keys are read from memory once and stay in shared memory; histograms are summed over
// distributed shared memory. Slot order makes every rank a count over lower slots: warps own
// consecutive runs of slots, CTAs consecutive runs of warps.
#include "kvc_paged.cuh"

namespace kvc {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;                 // the portable size
constexpr int kMaxChunk = 49152;               // keys a CTA holds: 192 KB

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
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive_release();
  cluster_wait_acquire();
}

struct Shared {
  uint32_t hist[2][256];
  uint32_t total[256];
  uint32_t counts[3];           // this CTA's ties, moved tokens and holes
  uint32_t warp_a[kWarps], warp_b[kWarps];
  uint32_t bin, above;
};

__device__ __forceinline__ uint32_t warp_sum(uint32_t x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

__global__ void __launch_bounds__(kThreads) paged_evict_kernel(const EvictParams p, int chunk) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ uint32_t keys[];
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
  if (len <= p.keep) return;                               // the same for the whole cluster
  const long long bh = static_cast<long long>(b) * p.Hkv + h;
  float* scores = p.scores + bh * cap;
  int32_t* positions = p.positions + bh * cap;
  const int recent_from = p.next_positions[b] - p.recent;
  const int c0 = min(len, rank * chunk), c1 = min(len, c0 + chunk), n = c1 - c0;
  for (int i = t; i < n; i += kThreads) {
    const int pos = positions[c0 + i];
    const uint32_t k = score_key(scores[c0 + i]);
    keys[i] = pos < p.sinks || pos >= recent_from ? 0xffffffffu : k;
  }
  for (int i = t; i < 512; i += kThreads) sh.hist[i >> 8][i & 255] = 0;
  __syncthreads();

  // the keep-th largest key: `prefix` its bits so far, `need` how many of the tokens with that
  // prefix are kept
  uint32_t prefix = 0, mask = 0;
  uint32_t need = p.keep;
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t* hist = sh.hist[pass & 1];
    for (int i = t; i < ((n + 31) & ~31); i += kThreads) {
      const uint32_t k = i < n ? keys[i] : 0;
      const bool in = i < n && (k & mask) == prefix;
      const uint32_t bin = in ? (k >> shift) & 255u : 256u;
      // lanes of one bin add once: scores crowd into few exponents
      const uint32_t same = __match_any_sync(0xffffffffu, bin);
      if (in && lane == __ffs(same) - 1) atomicAdd(&hist[bin], static_cast<uint32_t>(__popc(same)));
    }
    cluster_sync();
    if (t < 256) {
      uint32_t sum = 0;
      for (int r = 0; r < ranks; ++r) sum += ld_cluster_u32(cluster_map(smem_u32(&hist[t]), r));
      sh.total[t] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      // bins from the top, 8 a lane: lane 0 holds the highest
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += sh.total[255 - (lane * 8 + i)];
      uint32_t incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      const uint32_t before = incl - mine;
      if (before < need && need <= incl) {
        uint32_t above = before;
        int bin = 255 - lane * 8;
        while (above + sh.total[bin] < need) above += sh.total[bin--];
        sh.bin = bin;
        sh.above = above;
      }
    }
    // the buffer of the next pass: every CTA has read it, this pass's barrier came after
    if (pass >= 1 && pass < 3)
      for (int i = t; i < 256; i += kThreads) sh.hist[(pass + 1) & 1][i] = 0;
    __syncthreads();
    prefix |= sh.bin << shift;
    mask |= 255u << shift;
    need -= sh.above;
  }
  const uint32_t threshold = prefix;                       // kept: key > threshold, or one of `need` ties

  // ranks: each warp owns a run of slots
  const int per_warp = (((chunk + kWarps - 1) / kWarps) + 31) & ~31;
  const int w0 = min(n, warp * per_warp), w1 = min(n, w0 + per_warp);
  uint32_t ties = 0;
  for (int i = w0 + lane; i < w1; i += 32) ties += keys[i] == threshold;
  ties = warp_sum(ties);
  if (lane == 0) sh.warp_a[warp] = ties;
  __syncthreads();
  if (t == 0) {
    uint32_t sum = 0;
    for (int w = 0; w < kWarps; ++w) sum += sh.warp_a[w];
    sh.counts[0] = sum;
  }
  cluster_sync();
  uint32_t tie = 0;                                        // ties in lower slots than this warp's
  for (int r = 0; r < rank; ++r) tie += ld_cluster_u32(cluster_map(smem_u32(&sh.counts[0]), r));
  for (int w = 0; w < warp; ++w) tie += sh.warp_a[w];

  // kept tokens from slot `keep` on and evicted ones below it
  const uint32_t tie0 = tie;
  uint32_t from = 0, to = 0;
  auto each = [&](auto&& f) {
    tie = tie0;
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < w1 ? keys[i] : 0;
      const uint32_t eq = __ballot_sync(0xffffffffu, i < w1 && k == threshold);
      const uint32_t below = (1u << lane) - 1u;
      const bool kept = i < w1 && (k > threshold || (k == threshold && tie + __popc(eq & below) < need));
      tie += __popc(eq);
      const int slot = c0 + i;
      const uint32_t f_mask = __ballot_sync(0xffffffffu, kept && slot >= p.keep);
      const uint32_t t_mask = __ballot_sync(0xffffffffu, i < w1 && !kept && slot < p.keep);
      f(slot, f_mask, t_mask, below);
    }
  };
  each([&](int, uint32_t f_mask, uint32_t t_mask, uint32_t) {
    from += __popc(f_mask);
    to += __popc(t_mask);
  });
  __syncthreads();                                         // warp_a is read
  if (lane == 0) {
    sh.warp_a[warp] = from;
    sh.warp_b[warp] = to;
  }
  __syncthreads();
  if (t == 0) {
    uint32_t a = 0, c = 0;
    for (int w = 0; w < kWarps; ++w) {
      a += sh.warp_a[w];
      c += sh.warp_b[w];
    }
    sh.counts[1] = a;
    sh.counts[2] = c;
  }
  cluster_sync();
  uint32_t from0 = 0, to0 = 0, moves = 0;
  for (int r = 0; r < ranks; ++r) {
    const uint32_t a = ld_cluster_u32(cluster_map(smem_u32(&sh.counts[1]), r));
    const uint32_t c = ld_cluster_u32(cluster_map(smem_u32(&sh.counts[2]), r));
    moves += a;
    if (r < rank) {
      from0 += a;
      to0 += c;
    }
  }
  for (int w = 0; w < warp; ++w) {
    from0 += sh.warp_a[w];
    to0 += sh.warp_b[w];
  }
  int32_t* list_to = p.moves + bh * 2 * p.move_cap;
  int32_t* list_from = list_to + p.move_cap;
  each([&](int slot, uint32_t f_mask, uint32_t t_mask, uint32_t below) {
    if (f_mask >> lane & 1u) list_from[from0 + __popc(f_mask & below)] = slot;
    if (t_mask >> lane & 1u) list_to[to0 + __popc(t_mask & below)] = slot;
    from0 += __popc(f_mask);
    to0 += __popc(t_mask);
  });
  __threadfence();
  cluster_sync();                                          // the lists stand; nobody reads scores any more

  const int32_t* table = p.page_table + static_cast<long long>(b) * p.max_pages;
  const int page_mask = (1 << p.page_shift) - 1;
  auto row_of = [&](int slot) -> long long {
    const int32_t page = __ldg(table + (slot >> p.page_shift));
    if (page < 0 || page >= p.pool_pages) {
      latch_error(p.err, DERR_BOUNDS);
      return -1;
    }
    return (((static_cast<long long>(page) * p.Hkv + h) << p.page_shift) + (slot & page_mask)) * p.row_bytes;
  };
  const int lanes = p.row_bytes >> 4;                      // lanes of a row: 8, 16 or 32
  const int per = kThreads / lanes;                        // rows a CTA moves at once
  const int part = (t % lanes) * 16;
  for (uint32_t r = rank * per + t / lanes; r < moves; r += ranks * per) {
    const int src = __ldcg(list_from + r), dst = __ldcg(list_to + r);
    const long long a = row_of(src), c = row_of(dst);
    if (a >= 0 && c >= 0) {
      const uint4 k = *reinterpret_cast<const uint4*>(p.k_pool + a + part);
      const uint4 v = *reinterpret_cast<const uint4*>(p.v_pool + a + part);
      *reinterpret_cast<uint4*>(p.k_pool + c + part) = k;
      *reinterpret_cast<uint4*>(p.v_pool + c + part) = v;
    }
    if (part == 0) {
      scores[dst] = scores[src];
      positions[dst] = positions[src];
    }
  }
  // the last kept page ends in zeros; its slots from `keep` on may be read by a move, so only
  // after all of them
  if (p.keep & page_mask) {
    cluster_sync();
    const int tail = (page_mask + 1) - (p.keep & page_mask);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int r = rank * per + t / lanes; r < tail; r += ranks * per) {
      const long long c = row_of(p.keep + r);
      if (c < 0) continue;
      *reinterpret_cast<uint4*>(p.k_pool + c + part) = zero;
      *reinterpret_cast<uint4*>(p.v_pool + c + part) = zero;
    }
  }
  // nobody reads another CTA's shared memory after the barrier above the moves
}

// lengths = min(lengths, keep), once every head of the sequence is done with the old ones.
__global__ void paged_cut_lengths_kernel(int32_t* lengths, int B, int keep) {
  griddep_wait();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < B) lengths[b] = min(lengths[b], keep);
}

}  // namespace

int paged_evict_max_slots() { return kMaxCluster * kMaxChunk; }

cudaError_t launch_paged_evict(cudaStream_t s, const EvictParams& p, int32_t* lengths) {
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(paged_evict_kernel),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxChunk * 4);
  });
  if (e != cudaSuccess) return e;
  const int cap = p.max_pages << p.page_shift;
  int ranks = 1;
  while (ranks < kMaxCluster &&
         (cap > ranks * kMaxChunk || (cap > ranks * 2048 && static_cast<long long>(p.B) * p.Hkv * ranks < 148)))
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
  e = cudaLaunchKernelEx(&cfg, paged_evict_kernel, p, chunk);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_cut_lengths_kernel, dim3((p.B + 255) / 256), dim3(256), 0, s, lengths, p.B, p.keep);
}

}  // namespace kvc
