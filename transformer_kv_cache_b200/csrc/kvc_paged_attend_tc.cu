// kvc_paged_attend_tc.cu -- attention of a paged batch on sm_100a tensor cores (bf16).
//
// O_i = sum_j softmax_j(scale q_i . k_j) v_j as a flash-attention pipeline over the units of
// kvc_paged.cuh: one persistent CTA per SM walks its units, an item at a time, and leaves one
// partial (O, maximum, sum) per row and piece, which paged_merge_kernel joins.
//
// An item is up to two tiles of 128 packed query rows (tokens x the G query heads of one KV
// head, whole tokens only) that share the K and V tiles in shared memory. The CTA runs two
// streams, each with a TMEM score tile S (128 x 128 fp32, overwritten by its own weights P as
// bf16), an accumulator O (128 x D fp32) and a softmax warpgroup, so that one stream's
// products run under the other's exponentials. With two tiles a stream is a tile; an item
// of one tile (a decode step's few rows) gives its even key tiles to one stream and its odd ones
// to the other, each with a maximum and sum of its own.
//
// Roles (320 threads): warps 0-3 and 4-7 softmax of stream 0 and 1 (thread = row = TMEM lane);
// warp 8 issues the MMAs (S = Q K^T: both operands in shared memory; O += P V: P in TMEM, V as
// an MN-major operand); warp 9 loads by TMA: queries as a 3-D box (dims, heads, tokens), which
// packs the rows of any group size, and a key tile's pages as boxes of a page's slots. K and V
// tiles share one ring in the order K0 V0 K1 V1 ...
//
// Slots past a sequence's length are never used: blocks past it are loaded from behind the
// pool's end, which TMA fills with zeros, the MMA warp clears the rest of the last block's V
// rows, and their scores are set to -inf whatever K held.
//
// Every barrier wait is bounded; a role that gives up sets the error word, and the CTA drains
// its copies and products, frees its TMEM and returns.
#include "kvc_attn_common.cuh"
#include "kvc_paged.cuh"

namespace kvc {
namespace {

constexpr int kThreads = 320;
constexpr int kTile = 128;                     // query rows of a tile, keys of a unit
constexpr float kGrow = 8.0f;                  // a weight above 2^8 moves the row's reference maximum

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;                       // 128-byte swizzled blocks of a row
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kSmem = 1024 + 2 * kTileBytes + kStages * kTileBytes + 512;
};

struct Bars {
  uint64_t full[10], empty[10];                // K and V tiles
  uint64_t q_full[2], q_empty[2];              // query slots
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t drained;
  uint32_t tmem;
  int abort;
  long long plan[2 + kThreads / 32];
};

// The streams of a segment of n key tiles.
__device__ __forceinline__ int stream_steps(bool two, int w, int n) { return two ? n : (n - w + 1) >> 1; }

__device__ __forceinline__ bool seg_two(const PagedParams& p, const Segment& g) {
  return g.v.n - g.i * p.item_tokens > p.tile_tokens;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attend_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ PagedParams p) {
  griddep_wait();
  griddep_launch_dependents();
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;                                     // [slot][half][128 rows][128 B]
  uint8_t* kv_s = q_s + 2 * C::kTileBytes;                 // [stage][half][128 keys][128 B]
  Bars& bar = *reinterpret_cast<Bars*>(kv_s + C::kStages * C::kTileBytes);
  static_assert(sizeof(Bars) <= 512, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bar.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.o_full[i], 1);
      mbar_init(&bar.o_free[i], 4);
    }
    mbar_init(&bar.drained, 1);
    bar.abort = 0;
    mbar_fence_init();
  }
  if (warp == 8) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  Walk walk = plan_walk(p, bar.plan, [&](int b, const SeqView& v) { return head_units(p, b, v); });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  // TMEM columns: S0, S1 (128 each), O0, O1 (D each)
  Segment g;

  if (warp == 9) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tmap_q);
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_v);
    }
    const int blk = min(1 << p.page_shift, kTile);         // slots of a box
    const int blocks = kTile / blk;
    const int my_blk = lane % blocks, my_half = lane / blocks;   // lanes of a tile's boxes
    const bool loads = lane < blocks * C::kHalves;
    const int past = static_cast<int>((p.pool_pages * p.Hkv) << p.page_shift);
    int e = 0, slot = 0;
    int used[2] = {0, 0};
    bool ok = true;
    while (ok && next_segment(p, walk, g)) {
      const bool two = seg_two(p, g);
      for (int w = 0; w < (two ? 2 : 1) && ok; ++w) {
        ok = used[slot] == 0 || mbar_wait_bounded(&bar.q_empty[slot], (used[slot] - 1) & 1, abort, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&bar.q_full[slot], C::kHalves * p.tile_tokens * p.G * 128);
          for (int c = 0; c < C::kHalves; ++c)
            tma_load_3d(q_s + slot * C::kTileBytes + c * (kTile * 128), &tmap_q, &bar.q_full[slot], c * 64, g.h * p.G,
                        g.v.r0 + g.i * p.item_tokens + w * p.tile_tokens);
        }
        if (ok) ++used[slot];
        slot ^= 1;
      }
      int row_next = past;
      auto row_at = [&](int kt) {
        const int key = kt * kTile + my_blk * blk;
        if (!loads || key >= g.v.len) return past;
        const long long r = pool_row(p, g.b, g.h, key);
        return r < 0 ? past : static_cast<int>(r);
      };
      row_next = row_at(g.k0);
      for (int kt = g.k0; kt < g.k1 && ok; ++kt) {
        const int row = row_next;
        if (kt + 1 < g.k1) row_next = row_at(kt + 1);
        for (int kv = 0; kv < 2 && ok; ++kv, ++e) {
          const int st = e % C::kStages;
          ok = e < C::kStages || mbar_wait_bounded(&bar.empty[st], ((e / C::kStages) - 1) & 1, abort, p.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&bar.full[st], C::kTileBytes);
          __syncwarp();
          if (loads)
            tma_load_2d(kv_s + st * C::kTileBytes + my_half * (kTile * 128) + my_blk * blk * 128,
                        kv ? &tmap_v : &tmap_k, &bar.full[st], my_half * 64, row);
        }
      }
    }
    // every copy that was issued has landed before the CTA's shared memory goes
    if (lane == 0) {
      for (int i = max(0, e - C::kStages); i < e; ++i)
        mbar_wait_drain(&bar.full[i % C::kStages], (i / C::kStages) & 1, p.err);
      for (int i = 0; i < 2; ++i)
        if (used[i]) mbar_wait_drain(&bar.q_full[i], (used[i] - 1) & 1, p.err);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t idesc_s = idesc_f16kind(1, kTile, kTile, 0, 0);
    const uint32_t idesc_o = idesc_f16kind(1, kTile, D, 0, 1);
    const uint32_t q_addr = smem_u32(q_s), kv_addr = smem_u32(kv_s);
    const int blk = min(1 << p.page_shift, kTile);         // slots of a box
    const bool leader = elect_one();
    int e0 = 0, slot = 0;                      // first ring entry of the segment, next query slot
    int used[2] = {0, 0}, steps[2] = {0, 0}, segs[2] = {0, 0};
    bool ok = true;
    while (ok && next_segment(p, walk, g)) {
      const bool two = seg_two(p, g);
      const int n = g.k1 - g.k0;
      int qs[2];
      for (int w = 0; w < (two ? 2 : 1); ++w) {
        qs[w] = slot;
        ok = ok && mbar_wait_bounded(&bar.q_full[slot], used[slot] & 1, abort, p.err);
        ++used[slot];
        slot ^= 1;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!two) qs[1] = qs[0];
      auto wait_stage = [&](int e) {
        return mbar_wait_bounded(&bar.full[e % C::kStages], (e / C::kStages) & 1, abort, p.err);
      };
      auto issue_qk = [&](int w, int t, bool release) {
        const int e = e0 + 2 * t, st = e % C::kStages;
        if (!__all_sync(0xffffffffu, wait_stage(e))) return false;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t off = (c >> 2) * (kTile * 128) + (c & 3) * 32;
            mma_ss(tmem + w * 128, sw128_desc(q_addr + qs[w] * C::kTileBytes + off, 16, 1024),
                   sw128_desc(kv_addr + st * C::kTileBytes + off, 16, 1024), idesc_s, c > 0 ? 1u : 0u);
          }
          mma_commit(&bar.s_full[w]);
          if (release) mma_commit(&bar.empty[st]);
          // the last product that reads these queries
          if (t + 1 == n) mma_commit(&bar.q_empty[qs[w]]);
        }
        __syncwarp();
        return true;
      };
      auto issue_pv = [&](int w, int t, bool first, bool last, bool release) {
        const int e = e0 + 2 * t + 1, st = e % C::kStages;
        bool r = wait_stage(e);
        const int valid = g.v.len - (g.k0 + t) * kTile;
        if (r && valid < kTile && (valid & (blk - 1)) && (w == 0 || !two)) {
          // the rest of the last box: whatever the cache held there
          const int rows = blk - (valid & (blk - 1));
          for (int i = lane; i < rows * 8 * C::kHalves; i += 32) {
            const int c = i / (rows * 8), at = i % (rows * 8);
            *reinterpret_cast<uint4*>(kv_s + st * C::kTileBytes + c * (kTile * 128) + valid * 128 + at * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_shared();
        }
        r = r && mbar_wait_bounded(&bar.p_full[w], steps[w] & 1, abort, p.err);
        if (first && segs[w] > 0) r = r && mbar_wait_bounded(&bar.o_free[w], (segs[w] - 1) & 1, abort, p.err);
        if (!__all_sync(0xffffffffu, r)) return false;
        ++steps[w];
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int c = 0; c < kTile / 16; ++c)
            mma_ts(tmem + 256 + w * D, tmem + w * 128 + c * 8,
                   sw128_desc(kv_addr + st * C::kTileBytes + c * 2048, kTile * 128, 1024), idesc_o,
                   !first || c > 0 ? 1u : 0u);
          if (release) mma_commit(&bar.empty[st]);
          if (last) mma_commit(&bar.o_full[w]);
        }
        __syncwarp();
        return true;
      };
      if (two) {
        ok = ok && issue_qk(0, 0, false) && issue_qk(1, 0, true);
        for (int t = 0; ok && t < n; ++t) {
          const bool more = t + 1 < n;
          ok = issue_pv(0, t, t == 0, !more, false) && (!more || issue_qk(0, t + 1, false)) &&
               issue_pv(1, t, t == 0, !more, true) && (!more || issue_qk(1, t + 1, true));
        }
        if (ok) {
          ++segs[0];
          ++segs[1];
        }
      } else {
        ok = ok && issue_qk(0, 0, true) && (n < 2 || issue_qk(1, 1, true));
        for (int t = 0; ok && t < n; ++t) {
          const int w = t & 1;
          ok = issue_pv(w, t, t < 2, t + 2 >= n, true) && (t + 2 >= n || issue_qk(w, t + 2, true));
        }
        if (ok) {
          ++segs[0];
          if (n > 1) ++segs[1];
        }
      }
      e0 += 2 * n;
    }
    if (leader) mma_commit(&bar.drained);
    __syncwarp();
    mbar_wait_drain(&bar.drained, 0, p.err);
  } else {
    // ------------------------------------------------------------------ softmax of stream w
    const int w = warp >> 2, wq = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_col = tmem + lane_base + w * 128, o_col = tmem + lane_base + 256 + w * D;
    const float c = p.scale_log2;
    int steps = 0, segs = 0;
    bool ok = true;
    while (ok && next_segment(p, walk, g)) {
      const bool two = seg_two(p, g);
      const int n = g.k1 - g.k0;
      const int mine = stream_steps(two, w, n);
      const int t0 = g.i * p.item_tokens + (two ? w * p.tile_tokens : 0);
      const int rows = min(p.tile_tokens, g.v.n - t0) * p.G;
      const int r = wq * 32 + lane;
      const int tok = t0 + r / p.G;
      const int hq = g.h * p.G + r % p.G;
      const bool active = wq * 32 < rows;      // this warp has rows
      const int limit = r < rows ? key_limit(p, g.b, g.v, tok) : 0;
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < mine; ++i, ++steps) {
        ok = mbar_wait_bounded(&bar.s_full[w], steps & 1, abort, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const int kt = g.k0 + (two ? i : 2 * i + w);
          uint32_t s[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(s_col + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]));
          tmem_ld_wait();
          const int valid = limit - kt * kTile;
          if (__any_sync(0xffffffffu, valid < kTile)) {
#pragma unroll
            for (int k = 0; k < 128; ++k)
              if (k >= valid) s[k] = 0xff800000u;
          }
          float a[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) a[k] = __uint_as_float(s[k]);
#pragma unroll
          for (int k = 8; k < 120; k += 16)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              a[j] = max3(a[j], __uint_as_float(s[k + 2 * j]), __uint_as_float(s[k + 2 * j + 1]));
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] = fmaxf(a[j], __uint_as_float(s[120 + j]));
          const float mx = max3(max3(a[0], a[1], a[2]), max3(a[3], a[4], a[5]), fmaxf(a[6], a[7])) * c;
          if (__any_sync(0xffffffffu, mx > m + kGrow)) {
            const float m_new = mx > m + kGrow ? mx : m;
            const float f = m == m_new ? 1.f : ex2(m - m_new);     // 0 from -inf
            l *= f;
            m = m_new;
            if (i > 0) {
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tmem_ld32(o_col + 32 * q, o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st32(o_col + 32 * q, o);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : m;             // nothing seen yet: every weight is 0
          const uint64_t c2 = pk2(c, c), nm2 = pk2(-base, -base);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pb[32];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              float x0, x1;
              up2(fma2_pair(s[64 * q + 2 * k], s[64 * q + 2 * k + 1], c2, nm2), x0, x1);
              x0 = ex2(x0);
              x1 = ex2(x1);
              sum[(2 * k) & 3] += x0;
              sum[(2 * k + 1) & 3] += x1;
              pb[k] = pack_bf16(x0, x1);
            }
            tmem_st32(s_col + 32 * q, pb);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[w]);
      }
      if (!ok) break;
      const long long slot = g.k0 == 0 ? row_slot(p, g.b, two ? 0 : w, g.v.r0 + tok, hq)
                                       : cta_slot(p, blockIdx.x, w * kTile + r);
      if (r < rows) p.part_ml[slot] = make_float2(m, l);
      if (mine > 0) {
        ok = mbar_wait_bounded(&bar.o_full[w], segs & 1, abort, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (active) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(o_col + 32 * q, o);
            tmem_ld_wait();
            if (r < rows) {
              float4* dst = reinterpret_cast<float4*>(p.part_o + slot * D + 32 * q);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                     __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.o_free[w]);
        ++segs;
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
cudaError_t launch(cudaStream_t s, const PagedParams& p, const CUtensorMap& q, const CUtensorMap& k,
                   const CUtensorMap& v) {
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(paged_attend_tc_kernel<D>),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  });
  return e != cudaSuccess ? e
                          : launch_pdl(paged_attend_tc_kernel<D>, dim3(p.grid), dim3(kThreads), Cfg<D>::kSmem, s, q, k,
                                       v, p);
}

}  // namespace

cudaError_t launch_paged_attend_tc(cudaStream_t s, const PagedParams& p) {
  CUtensorMap q, k, v;
  if (!encode_rows_tmap(&q, p.q, p) ||
      !encode_slots_tmap(&k, p.k_pool, p) || !encode_slots_tmap(&v, p.v_pool, p))
    return cudaErrorInvalidValue;
  return p.D == 64 ? launch<64>(s, p, q, k, v) : launch<128>(s, p, q, k, v);
}

}  // namespace kvc
