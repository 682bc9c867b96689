// kvc_paged_weights_tc.cu -- the attention weight that each cached token of a paged batch
// receives, on sm_100a tensor cores (bf16).
//
// w_j = sum over query rows i and the G query heads of a KV head of 2^(c q_i . k_j - lse2_i). The
// product is taken transposed, S^T = K Q^T (M = 128 keys, N = query rows): a thread owns a key
// (a TMEM lane) and adds up its row of S^T in registers, so the sum over the queries needs no
// exchange between threads, and few query rows cost few columns (N is their number rounded up
// to 16) while the keys fill the tile.
//
// A CTA (one per SM) takes blocks of 256 keys of one KV head, a tile of 128 keys for each of
// two streams, and runs the sequence's query tiles past them (units of kvc_paged.cuh, query tiles
// fastest). A stream has two S^T buffers in TMEM (4 x 128 columns), so that its next product
// runs under this one's exponentials.
//
// Roles (320 threads): warps 0-3 and 4-7 exponentials and sums of stream 0 and 1 (thread = key);
// warp 8 issues the MMAs (both operands in shared memory); warp 9 loads by TMA: key tiles into
// a ring of their own, query tiles into another; the rows' log2-sum-exp and last visible key go
// beside the query tile by plain stores.
#include "kvc_attn_common.cuh"
#include "kvc_paged.cuh"

namespace kvc {
namespace {

constexpr int kThreads = 320;
constexpr int kTile = 128;                     // keys of a stream, query rows of a tile
constexpr int kKeyStages = 4;                  // key tiles (two to a block)
constexpr int kQueryStages = 2;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kSmem = 1024 + (kKeyStages + kQueryStages) * kTileBytes + kQueryStages * kTile * 8 + 512;
};

struct Bars {
  uint64_t k_full[kKeyStages], k_empty[kKeyStages];
  uint64_t q_full[kQueryStages], q_empty[kQueryStages];
  uint64_t s_full[2][2], s_empty[2][2];        // [stream][buffer]
  uint64_t drained;
  uint32_t tmem;
  int abort;
  long long plan[2 + kThreads / 32];
};

// Query rows of tile t of the segment's sequence.
__device__ __forceinline__ int tile_rows(const PagedParams& p, const WeightSegment& g, int t) {
  return min(p.tile_tokens, g.v.n - t * p.tile_tokens) * p.G;
}
// Key tiles of the block: 2, or 1 at the end of a sequence.
__device__ __forceinline__ int block_tiles(const WeightSegment& g) {
  return g.v.len - g.kb * (2 * kTile) > kTile ? 2 : 1;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_weights_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                            const __grid_constant__ PagedParams p) {
  griddep_wait();
  griddep_launch_dependents();
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* k_s = smem;                                     // [stage][8 keys][half][key][128 B]
  uint8_t* q_s = k_s + kKeyStages * C::kTileBytes;         // [stage][half][128 rows][128 B]
  float2* row_s = reinterpret_cast<float2*>(q_s + kQueryStages * C::kTileBytes);   // [stage][128] (-lse2, limit)
  Bars& bar = *reinterpret_cast<Bars*>(row_s + kQueryStages * kTile);
  static_assert(sizeof(Bars) <= 512, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bar.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kKeyStages; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
    }
    for (int i = 0; i < kQueryStages; ++i) {
      mbar_init(&bar.q_full[i], 2);            // the bytes, and the rows' statistics
      mbar_init(&bar.q_empty[i], 9);           // the products, and the 8 warps that read the statistics
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.s_full[i >> 1][i & 1], 1);
      mbar_init(&bar.s_empty[i >> 1][i & 1], 4);
    }
    mbar_init(&bar.drained, 1);
    bar.abort = 0;
    mbar_fence_init();
    p.part_id[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  if (warp == 8) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  Walk walk = plan_walk(p, bar.plan, [&](int, const SeqView& v) { return weight_head_units(p, v); });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;              // S^T buffer x of stream w: columns (2 w + x) * 128
  WeightSegment g;

  if (warp == 9) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmap_q);
      tma_prefetch_desc(&tmap_k);
    }
    const int blk = min(1 << p.page_shift, kTile);
    const int blocks = kTile / blk;
    const int my_blk = lane % blocks;
    const bool loads = lane < blocks;
    const int past = static_cast<int>((p.pool_pages * p.Hkv) << p.page_shift);
    int ek = 0, eq = 0;
    bool ok = true;
    while (ok && next_weight_segment(p, walk, g)) {
      const int key0 = g.kb * 2 * kTile;
      const int nt = block_tiles(g);
      int row[2];
      for (int w = 0; w < nt; ++w) {
        const int key = key0 + w * kTile + my_blk * blk;
        const long long r = loads && key < g.v.len ? pool_row(p, g.b, g.h, key) : -1;
        row[w] = r < 0 ? past : static_cast<int>(r);
      }
      for (int w = 0; w < nt && ok; ++w, ++ek) {
        const int st = ek % kKeyStages;
        ok = ek < kKeyStages || mbar_wait_bounded(&bar.k_empty[st], ((ek / kKeyStages) - 1) & 1, abort, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar.k_full[st], C::kTileBytes);
        __syncwarp();
        if (loads)
          tma_load_4d(k_s + st * C::kTileBytes + my_blk * blk * (D * 2), &tmap_k, &bar.k_full[st], 0, 0, 0, row[w] >> 3);
      }
      for (int t = g.t0; t < g.t1 && ok; ++t, ++eq) {
        const int st = eq % kQueryStages;
        const int tok0 = t * p.tile_tokens, rows = tile_rows(p, g, t);
        ok = eq < kQueryStages || mbar_wait_bounded(&bar.q_empty[st], ((eq / kQueryStages) - 1) & 1, abort, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane < C::kHalves) {
          if (lane == 0) mbar_arrive_expect_tx(&bar.q_full[st], C::kHalves * p.tile_tokens * p.G * 128);
        }
        __syncwarp();
        if (lane < C::kHalves)
          tma_load_3d(q_s + st * C::kTileBytes + lane * (kTile * 128), &tmap_q, &bar.q_full[st], lane * 64, g.h * p.G,
                      g.v.r0 + tok0);
        for (int r = lane; r < kTile; r += 32) {
          float2 x = make_float2(0.f, 0.f);    // no key is below 0: nothing is added
          if (r < rows) {
            const int tok = tok0 + r / p.G;
            x.x = -1.4426950408889634f *
                  __ldg(p.lse + static_cast<long long>(g.v.r0 + tok) * p.Hq + g.h * p.G + r % p.G);
            x.y = __int_as_float(key_limit(p, g.b, g.v, tok));
          }
          row_s[st * kTile + r] = x;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.q_full[st]);
      }
    }
    if (lane == 0) {
      for (int i = max(0, ek - kKeyStages); i < ek; ++i)
        mbar_wait_drain(&bar.k_full[i % kKeyStages], (i / kKeyStages) & 1, p.err);
      for (int i = max(0, eq - kQueryStages); i < eq; ++i)
        mbar_wait_drain(&bar.q_full[i % kQueryStages], (i / kQueryStages) & 1, p.err);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t q_addr = smem_u32(q_s), k_addr = smem_u32(k_s);
    const bool leader = elect_one();
    int ek = 0, eq = 0;
    int steps[2] = {0, 0};
    bool ok = true;
    while (ok && next_weight_segment(p, walk, g)) {
      const int nt = block_tiles(g);
      for (int t = g.t0; t < g.t1 && ok; ++t, ++eq) {
        const int st = eq % kQueryStages;
        const int cols = (tile_rows(p, g, t) + 15) & ~15;
        const uint32_t idesc = idesc_f16kind(1, kTile, 16, 0, 0) + (static_cast<uint32_t>(cols - 16) >> 3 << 17);
        ok = mbar_wait_bounded(&bar.q_full[st], (eq / kQueryStages) & 1, abort, p.err);
        ok = __all_sync(0xffffffffu, ok);
        for (int w = 0; w < nt && ok; ++w) {
          const int ks = (ek + w) % kKeyStages, x = steps[w] & 1;
          if (t == g.t0) ok = mbar_wait_bounded(&bar.k_full[ks], ((ek + w) / kKeyStages) & 1, abort, p.err);
          if (steps[w] >= 2) ok = ok && mbar_wait_bounded(&bar.s_empty[w][x], ((steps[w] >> 1) - 1) & 1, abort, p.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++steps[w];
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              mma_ss(tmem + (2 * w + x) * 128,
                     sw128_desc(k_addr + ks * C::kTileBytes + (c >> 2) * 1024 + (c & 3) * 32, 16, C::kHalves * 1024),
                     sw128_desc(q_addr + st * C::kTileBytes + (c >> 2) * (kTile * 128) + (c & 3) * 32, 16, 1024), idesc,
                     c > 0 ? 1u : 0u);
            }
            mma_commit(&bar.s_full[w][x]);
            if (t + 1 == g.t1) mma_commit(&bar.k_empty[ks]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (leader) mma_commit(&bar.q_empty[st]);
        __syncwarp();
      }
      ek += nt;
    }
    if (leader) mma_commit(&bar.drained);
    __syncwarp();
    mbar_wait_drain(&bar.drained, 0, p.err);
  } else {
    // ------------------------------------------------------------------ sums of stream w
    const int w = warp >> 2, wq = warp & 3;
    const uint32_t s_col = tmem + (static_cast<uint32_t>(wq * 32) << 16) + 2 * w * 128;
    const float c = p.scale_log2;
    int steps = 0, eq = 0;
    bool ok = true;
    while (ok && next_weight_segment(p, walk, g)) {
      const bool mine = w < block_tiles(g);
      const int key = g.kb * 2 * kTile + w * kTile + wq * 32 + lane;
      float total = 0.f;
      for (int t = g.t0; t < g.t1 && ok; ++t, ++eq) {
        const int st = eq % kQueryStages;
        ok = mbar_wait_bounded(&bar.q_full[st], (eq / kQueryStages) & 1, abort, p.err);   // the statistics
        if (mine) {
          const int rows = tile_rows(p, g, t);
          const int x = steps & 1;
          ok = ok && mbar_wait_bounded(&bar.s_full[w][x], (steps >> 1) & 1, abort, p.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++steps;
          tc_fence_after();
          const float2* st_row = row_s + st * kTile;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          for (int q = 0; q < rows; q += 32) {
            uint32_t s[32];
            tmem_ld32(s_col + x * 128 + q, s);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float2 y = st_row[q + k];
              const float e = ex2(fmaf(__uint_as_float(s[k]), c, y.x));
              sum[k & 3] += key < __float_as_int(y.y) ? e : 0.f;
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.s_empty[w][x]);
          total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive(&bar.q_empty[st]);
      }
      if (!ok) break;
      if (g.t0 > 0) {
        p.part_w[static_cast<long long>(blockIdx.x) * p.slot_rows + w * kTile + wq * 32 + lane] = total;
        if (threadIdx.x == 0) p.part_id[blockIdx.x] = make_int4(g.b, g.h, g.kb, 1);
      } else if (key < g.v.len) {
        p.scores[(static_cast<long long>(g.b) * p.Hkv + g.h) * paged_cap(p) + key] += total;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(cudaStream_t s, const PagedParams& p, const CUtensorMap& q, const CUtensorMap& k) {
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(paged_weights_tc_kernel<D>),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  });
  return e != cudaSuccess
             ? e
             : launch_pdl(paged_weights_tc_kernel<D>, dim3(p.grid), dim3(kThreads), Cfg<D>::kSmem, s, q, k, p);
}

}  // namespace

cudaError_t launch_paged_weights_tc(cudaStream_t s, const PagedParams& p) {
  CUtensorMap q, k;
  if (!encode_rows_tmap(&q, p.q, p) || !encode_slots_tmap(&k, p.k_pool, p)) return cudaErrorInvalidValue;
  return p.D == 64 ? launch<64>(s, p, q, k) : launch<128>(s, p, q, k);
}

}  // namespace kvc
