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
// runs under this one's exponentials. A sequence whose rows fit one tile keeps it in shared memory
// from key block to key block.
//
// Roles: warp 3 walks the schedule and hands out its segments through a ring; warp 0 loads the key
// tiles by TMA (a page to a copy, looked up one block ahead); warp 2 loads the query tiles and puts
// their rows' log2-sum-exp and last visible key beside them; warp 1 and the last one issue the MMAs
// of stream 0 and 1 (both operands in shared memory); the warps between are the exponentials and
// sums (thread = key). A warp whose keys every row of the tile sees, which is all but the last
// tiles of a causal call, adds without looking at the rows' limits (where a row's log2-sum-exp is
// not finite, nothing is skipped: +inf adds exactly nothing, NaN stays NaN).
//
// Two forms. Where the sequences' rows do not fill a query tile, on average (decode steps), the
// keys' bytes are the bound: 4 sum warps a stream. Else the exponentials and their sums are, by their
// instructions (issue slots 61 %, shared memory 38 %, MUFU 37 % of their peaks): 8 sum warps a stream,
// four for a query tile's first 64 rows and four for the others (the halves of a key's sum meet in
// shared memory at the end of a block), so that four warps a scheduler cover one another's waits,
// and as much room for query tiles as for key tiles. The frame of 1,004 rows below takes 134 us with
// four sum warps a stream and one issuer. 32 sequences of 4,096 to 8,192 tokens, a row of 32 heads
// over 8 KV heads of 128 dims each: 70 us, 5.9 TB/s. A frame of 1,004 rows of 16 heads of 64 dims over
// 16,064 keys: 99 us, 2.6 x 10^12 exponentials a second, where the MUFU alone gives 4.5 x 10^12.
#include "kvc_paged.cuh"
#include "kvc_paged_math.cuh"

namespace kvc {
namespace {

using namespace paged;

constexpr int kTile = 128;                     // keys of a stream, query rows of a tile
constexpr int kPoly8 = 3;                      // of 8 pairs, the exponentials on the FMA pipe

template <int D, bool kMany>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kKeyStages = (kMany ? 3 : 4) * (D == 128 ? 1 : 2);    // key tiles (two to a block)
  static constexpr int kQueryStages = kMany ? 3 * (D == 128 ? 1 : 2) : 2;
  static constexpr int kSumWarps = kMany ? 16 : 8;
  static constexpr int kThreads = 32 * (5 + kSumWarps);    // the last warp issues stream 1's products
  static constexpr int kSmem =
      1024 + (kKeyStages + kQueryStages) * kTileBytes + kQueryStages * kTile * 8 + 2 * kTile * 4 + 1408;
};

struct Bars {
  uint64_t k_full[8], k_empty[8];
  uint64_t q_full[6], q_empty[6];
  uint64_t s_full[2][2], s_empty[2][2];        // [stream][buffer]
  uint64_t x_full[2], x_empty[2];              // a stream's second half sums
  uint64_t drained[2];
  SegmentRing ring;
  int finite[6];                               // 1: every row's log-sum-exp is
  uint32_t tmem;
  int abort;
  long long plan[kPlanWords + 24];
};

// Segments in the ring: i = key block, [k0, k1) = query tiles, nk = the sequence's query tiles,
// two = the query tile is not the last segment's (one tile in all, same sequence and head).
__device__ __forceinline__ int tile_rows(const PagedParams& p, const Segment& g, int t) {
  return min(p.tile_tokens, g.v.n - t * p.tile_tokens) * p.G;
}
// Key tiles of the block: 2, or 1 at the end of a sequence.
__device__ __forceinline__ int block_tiles(const Segment& g) { return g.v.len - g.i * (2 * kTile) > kTile ? 2 : 1; }

// The walk of a consumer of query tiles through the ring's segments: a tile that stays (nk == 1)
// is given back when the next one is due, any other after its use.
struct QueryWalk {
  int eq = -1;                                 // tile in use
  bool held = false;                           // it was kept
};

// Sums of 2^(c s + y) over 32 columns that the thread's key is seen by: sum0 and sum1 gain.
__device__ __forceinline__ void add_all(const uint32_t (&s)[32], const float* y, uint64_t c2, uint64_t& sum0,
                                        uint64_t& sum1) {
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    const float4 v = *reinterpret_cast<const float4*>(y + 2 * k);
    const uint64_t x0 = fma2(pk2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), c2, pk2(v.x, v.y));
    const uint64_t x1 = fma2(pk2(__uint_as_float(s[2 * k + 2]), __uint_as_float(s[2 * k + 3])), c2, pk2(v.z, v.w));
    sum0 = add2(sum0, (k & 7) >= 8 - kPoly8 ? exp2_pair(x0) : exp2_pair_mufu(x0));
    sum1 = add2(sum1, ((k + 1) & 7) >= 8 - kPoly8 ? exp2_pair(x1) : exp2_pair_mufu(x1));
  }
}

template <int D, bool kMany>
__global__ void __launch_bounds__(Cfg<D, kMany>::kThreads, 1)
    paged_weights_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                            const __grid_constant__ PagedParams p) {
  using C = Cfg<D, kMany>;
  constexpr int kQueryStages = C::kQueryStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* k_s = smem;                                     // [stage][8 keys][half][key][128 B]
  uint8_t* q_s = k_s + C::kKeyStages * C::kTileBytes;      // [stage][half][128 rows][128 B]
  float* lse_s = reinterpret_cast<float*>(q_s + kQueryStages * C::kTileBytes);   // [stage][128] -lse2
  int* limit_s = reinterpret_cast<int*>(lse_s + kQueryStages * kTile);           // [stage][128] keys that the row sees
  float* half_s = reinterpret_cast<float*>(limit_s + kQueryStages * kTile);      // [stream][128] sums of the second rows
  Bars& bar = *reinterpret_cast<Bars*>(half_s + 2 * kTile);
  static_assert(sizeof(Bars) <= 1408, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bar.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kKeyStages; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 2);           // both issuers, see there
    }
    for (int i = 0; i < kQueryStages; ++i) {
      mbar_init(&bar.q_full[i], 2);            // the bytes, and the rows' statistics
      mbar_init(&bar.q_empty[i], 2 + C::kSumWarps);   // the products, and who reads the statistics
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.s_full[i >> 1][i & 1], 1);
      mbar_init(&bar.s_empty[i >> 1][i & 1], C::kSumWarps / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.x_full[i], 4);
      mbar_init(&bar.x_empty[i], 4);
      mbar_init(&bar.drained[i], 1);
    }
    ring_init(bar.ring, C::kThreads / 32 - 1); // every warp but the one that fills it
    bar.abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();                              // everything above is this CTA's own
  griddep_launch_dependents();
  if (threadIdx.x == 4 * 32) p.part_id[blockIdx.x] = make_int4(0, 0, 0, 0);   // the thread that may write it later
  Walk walk{};
  if (warp == 3 || !plan_by_warp(p))
    walk = plan_walk(p, bar.plan, [&](int, const SeqView& v) { return weight_head_units(p, v); });
  const uint32_t tmem = bar.tmem;              // S^T buffer x of stream w: columns (2 w + x) * 128

  if (warp == 3) {
    // ------------------------------------------------------------------ schedule
    if (lane == 0) {
      bool ok = true, more = true;
      int last_b = -1, last_h = -1;
#pragma unroll 1
      for (int put = 0; ok && more; ++put) {
        WeightSegment w{};
        more = next_weight_segment(p, walk, w);
        Segment g{};                           // the last one handed out has no query tiles
        if (more) {
          const int tiles = (w.v.n + p.tile_tokens - 1) / p.tile_tokens;
          g = {w.b, w.h, w.kb, w.v, w.t0, w.t1, tiles, tiles > 1 || w.b != last_b || w.h != last_h, 0};
          last_b = w.b;
          last_h = w.h;
        }
        ok = ring_put(bar.ring, put, g, abort);
      }
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------------ keys
    if (lane == 0) tma_prefetch_desc(&tmap_k);
    const int blk = min(1 << p.page_shift, kTile);
    const int blocks = kTile / blk;                        // boxes of a tile, two lanes for each of a block's
    const int past = static_cast<int>((p.pool_pages * p.Hkv) << p.page_shift);
    const bool leader = elect_one();
    int ek = 0, sg = 0;
    bool ok = true;
    struct Box {
      int page, key, tiles, h;
    };
    auto box_of = [&](const Segment& g) {
      const int key = g.i * (2 * kTile) + lane * blk;
      Box b{-1, key, block_tiles(g), g.h};
      if (lane < 2 * blocks && key < g.v.len)
        b.page = __ldg(p.page_table + static_cast<long long>(g.b) * p.max_pages + (key >> p.page_shift));
      else
        b.key = -1;
      return b;
    };
    Segment g;
    ok = ring_take(bar.ring, sg++, g, abort);
    bool more = ok && g.nk > 0;
    Box next = more ? box_of(g) : Box{-1, -1, 0, 0};
    while (ok && more) {
      const Box box = next;
      ok = ring_take(bar.ring, sg++, g, abort);
      if (!ok) break;
      more = g.nk > 0;
      if (more) next = box_of(g);
      int row = past;
      if (box.key >= 0) {
        if (box.page < 0 || box.page >= p.pool_pages) latch_error(p.err, DERR_BOUNDS);
        else row = ((box.page * p.Hkv + box.h) << p.page_shift) + (box.key & ((1 << p.page_shift) - 1));
      }
      for (int w = 0; w < box.tiles; ++w, ++ek) {
        const int st = ek % C::kKeyStages;
        ok = ek < C::kKeyStages || wait_segment(&bar.k_empty[st], ((ek / C::kKeyStages) - 1) & 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        int rows[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) rows[i] = __shfl_sync(0xffffffffu, row, w * blocks + i);
        if (leader) {
          mbar_arrive_expect_tx(&bar.k_full[st], C::kTileBytes);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < blocks)
              tma_load_4d(k_s + st * C::kTileBytes + i * blk * (D * 2), &tmap_k, &bar.k_full[st], 0, 0, 0, rows[i] >> 3);
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      for (int i = max(0, ek - C::kKeyStages); i < ek; ++i)
        wait_drain(&bar.k_full[i % C::kKeyStages], (i / C::kKeyStages) & 1, abort);
  } else if (warp == 2) {
    // ------------------------------------------------------------------ queries and their statistics
    if (lane == 0) tma_prefetch_desc(&tmap_q);
    int tok[4], head[4];                       // this lane's rows of any tile
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tok[i] = (32 * i + lane) / p.G;
      head[i] = (32 * i + lane) % p.G;
    }
    int eq = 0, sg = 0, t = 0;
    Segment g{};
    // to the next tile that is to be loaded; its rows' log-sum-exp arrives while a stage is waited for
    float next[4];
    auto advance = [&](bool first) {
      ++t;
      while (first || t >= g.k1) {
        first = false;
        if (!ring_take(bar.ring, sg++, g, abort) || g.nk == 0) return false;
        t = g.two ? g.k0 : g.k1;               // else the tile is there already
      }
      const int rows = tile_rows(p, g, t);
      const float* lse = p.lse + static_cast<long long>(g.v.r0 + t * p.tile_tokens) * p.Hq + g.h * p.G;
#pragma unroll
      for (int i = 0; i < 4; ++i) next[i] = 32 * i + lane < rows ? __ldg(lse + static_cast<long long>(tok[i]) * p.Hq + head[i]) : 0.f;
      return true;
    };
    bool more = advance(true);
    while (more) {
      const int st = eq % kQueryStages;
      const int tok0 = t * p.tile_tokens, rows = tile_rows(p, g, t);
      bool ok = eq < kQueryStages || wait_segment(&bar.q_empty[st], ((eq / kQueryStages) - 1) & 1, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar.q_full[st], C::kHalves * p.tile_tokens * p.G * 128);
        for (int c = 0; c < C::kHalves; ++c)
          tma_load_3d(q_s + st * C::kTileBytes + c * (kTile * 128), &tmap_q, &bar.q_full[st], c * 64, g.h * p.G,
                      g.v.r0 + tok0);
      }
      const bool fin =
          __all_sync(0xffffffffu, isfinite(next[0]) && isfinite(next[1]) && isfinite(next[2]) && isfinite(next[3]));
      if (lane == 0) bar.finite[st] = fin;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 32 * i + lane;
        lse_s[st * kTile + r] = -1.4426950408889634f * next[i];
        limit_s[st * kTile + r] = r < rows ? key_limit(p, g.b, g.v, tok0 + tok[i]) : 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_full[st]);
      ++eq;
      // only now: the next tile may lie many segments on, which wait for this one
      more = advance(false);
    }
    if (lane == 0)
      for (int i = max(0, eq - kQueryStages); i < eq; ++i)
        wait_drain(&bar.q_full[i % kQueryStages], (i / kQueryStages) & 1, abort);
  } else if (warp == 1 || warp == 4 + C::kSumWarps) {
    // ------------------------------------------------------------------ products of stream w
    const int w = warp == 1 ? 0 : 1;
    const uint64_t q_desc = sw128_desc(smem_u32(q_s), 16, 1024);
    const uint64_t k_desc = sw128_desc(smem_u32(k_s), 16, C::kHalves * 1024);
    const bool leader = elect_one();
    int ek = 0, steps = 0;
    QueryWalk q;
    bool ok = true;
    for (int sg = 0; ok; ++sg) {
      Segment g;
      ok = ring_take(bar.ring, sg, g, abort);
      if (!ok || g.nk == 0) break;
      const int nt = block_tiles(g);
      if (g.two && q.held) {
        if (leader) mma_commit(&bar.q_empty[q.eq % kQueryStages]);
        __syncwarp();
        q.held = false;
      }
      for (int t = g.k0; t < g.k1 && ok; ++t) {
        bool r = true;
        if (g.two) {
          ++q.eq;
          r = wait_near(&bar.q_full[q.eq % kQueryStages], (q.eq / kQueryStages) & 1, abort);
        }
        const int st = q.eq % kQueryStages;
        const int cols = (tile_rows(p, g, t) + 15) & ~15;
        const uint32_t idesc = idesc_f16kind(1, kTile, 16, 0, 0) + ((static_cast<uint32_t>(cols - 16) >> 3) << 17);
        // A tile's stage serves either stream from one round of the ring to the next (a block may have
        // one tile), and a wait by parity tells a phase only from the one before. So each issuer sees
        // every tile land, and gives every tile back, the other stream's at once.
        if (t == g.k0)
          for (int i = 0; i < nt; ++i) {
            const int e = ek + i, stage = e % C::kKeyStages;
            r = r && wait_near(&bar.k_full[stage], (e / C::kKeyStages) & 1, abort);
            if (r && i != w && leader) mbar_arrive(&bar.k_empty[stage]);
          }
        if (w < nt) {
          const int ks = (ek + w) % C::kKeyStages, x = steps & 1;
          if (steps >= 2) r = r && wait_near(&bar.s_empty[w][x], ((steps >> 1) - 1) & 1, abort);
          ok = __all_sync(0xffffffffu, r);
          if (!ok) break;
          ++steps;
          tc_fence_after();
          if (leader) {
            // addresses stay below 2^18: an offset adds to the descriptor's address field
            const uint64_t kd = k_desc + (ks * C::kTileBytes >> 4), qd = q_desc + (st * C::kTileBytes >> 4);
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
              mma_ss(tmem + (2 * w + x) * 128, kd + (((c >> 2) * 1024 + (c & 3) * 32) >> 4),
                     qd + (((c >> 2) * (kTile * 128) + (c & 3) * 32) >> 4), idesc, c > 0 ? 1u : 0u);
            mma_commit(&bar.s_full[w][x]);
            if (t + 1 == g.k1) mma_commit(&bar.k_empty[ks]);
          }
          __syncwarp();
        } else {
          ok = __all_sync(0xffffffffu, r);
        }
        if (!ok) break;
        if (g.nk > 1) {
          if (leader) mma_commit(&bar.q_empty[st]);
          __syncwarp();
        } else {
          q.held = true;
        }
      }
      ek += nt;
    }
    if (leader) mma_commit(&bar.drained[w]);
    __syncwarp();
    wait_drain(&bar.drained[w], 0, abort);
  } else {
    // ------------------------------------------------------------------ sums of stream w (rows 64 half ..)
    const int w = kMany ? (warp - 4) >> 3 : (warp - 4) >> 2, half = kMany ? ((warp - 4) >> 2) & 1 : 0, wq = warp & 3;
    const uint32_t s_col = tmem + (static_cast<uint32_t>(wq * 32) << 16) + 2 * w * 128;
    const float c = p.scale_log2;
    const uint64_t c2 = pk2(c, c);
    int steps = 0, met = 0;                    // products, and blocks whose halves met
    QueryWalk q;
    bool ok = true;
    for (int sg = 0; ok; ++sg) {
      Segment g;
      ok = ring_take(bar.ring, sg, g, abort);
      if (!ok || g.nk == 0) break;
      const bool mine = w < block_tiles(g);
      const int key0 = g.i * 2 * kTile + w * kTile + wq * 32, key = key0 + lane;
      if (g.two && q.held) {
        if (lane == 0) mbar_arrive(&bar.q_empty[q.eq % kQueryStages]);
        q.held = false;
      }
      // the score that the sum goes to, asked for now
      float* score = p.scores + (static_cast<long long>(g.b) * p.Hkv + g.h) * paged_cap(p) + key;
      const bool adds = half == 0 && g.k0 == 0 && key < g.v.len;
      const float old = adds ? *score : 0.f;
      float total = 0.f;
      for (int t = g.k0; t < g.k1; ++t) {
        if (g.two) {
          ++q.eq;
          ok = wait_near(&bar.q_full[q.eq % kQueryStages], (q.eq / kQueryStages) & 1, abort);
        }
        const int st = q.eq % kQueryStages;
        if (mine) {
          const int rows = min(tile_rows(p, g, t), kMany ? 64 * half + 64 : kTile);
          const int x = steps & 1;
          ok = ok && wait_near(&bar.s_full[w][x], (steps >> 1) & 1, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++steps;
          tc_fence_after();
          const uint32_t buf = s_col + x * 128;
          const float* y = lse_s + st * kTile;
          const int* limit = limit_s + st * kTile;
          // rows see more keys the later they are: the first one's limit is the tile's least
          const bool all = bar.finite[st] && min(key0 + 31, g.v.len - 1) < limit[0];
          float rest = 0.f;
          uint64_t sum0 = 0, sum1 = 0;
          int done = 64 * half;
          if (all)
            for (; done + 32 <= rows; done += 32) {
              uint32_t s[32];
              tmem_ld32(buf + done, s);
              tmem_ld_wait();
              add_all(s, y + done, c2, sum0, sum1);
            }
          for (; done < rows; done += 16) {
            uint32_t s[16];
            tmem_ld16(buf + done, s);
            tmem_ld_wait();
            if (all) {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                if (done + k >= rows) break;
                rest += ex2(fmaf(__uint_as_float(s[k]), c, y[done + k]));
              }
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (done + k < rows && key < limit[done + k])
                  rest += ex2(fmaf(__uint_as_float(s[k]), c, y[done + k]));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.s_empty[w][x]);
          float e0, e1;
          up2(add2(sum0, sum1), e0, e1);
          total += (e0 + e1) + rest;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (g.nk > 1) {
          if (lane == 0) mbar_arrive(&bar.q_empty[st]);
        } else {
          q.held = true;
        }
      }
      if (!ok) break;
      const int at = w * kTile + wq * 32 + lane;
      if (kMany && (g.nk > 1 || tile_rows(p, g, 0) > 64)) {
        // the second rows' sum to the first ones' warp of the same keys
        if (half == 1) {
          ok = met == 0 || wait_near(&bar.x_empty[w], (met - 1) & 1, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          half_s[at] = total;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.x_full[w]);
        } else {
          ok = wait_near(&bar.x_full[w], met & 1, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          total += half_s[at];
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.x_empty[w]);
        }
        ++met;
      }
      if (half == 1) continue;
      if (g.k0 > 0) {
        p.part_w[static_cast<long long>(blockIdx.x) * p.slot_rows + at] = total;
        if (warp == 4 && lane == 0) p.part_id[blockIdx.x] = make_int4(g.b, g.h, g.i, 1);
      } else if (adds) {
        *score = old + total;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  report_abort(p, abort);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kMany>
cudaError_t launch(cudaStream_t s, const PagedParams& p, const CUtensorMap& q, const CUtensorMap& k) {
  using C = Cfg<D, kMany>;
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(paged_weights_tc_kernel<D, kMany>),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  return e != cudaSuccess
             ? e
             : launch_pdl(paged_weights_tc_kernel<D, kMany>, dim3(p.grid), dim3(C::kThreads), C::kSmem, s, q, k, p);
}

}  // namespace

cudaError_t launch_paged_weights_tc(cudaStream_t s, const PagedParams& p) {
  CUtensorMap q, k;
  if (!encode_rows_tmap(&q, p.q, p) || !encode_slots_tmap(&k, p.k_pool, p)) return cudaErrorInvalidValue;
  // A sequence's rows fill more than one tile, on average. Over 4,096 tokens, 32 heads on 8 of 128 dims: 64
  // sequences of 5 rows 96 us, in the form for many 129, of 40 223 and 221, of 100 445 and 420. No length is
  // known here, so a chunk among single rows may get the slower one: 63 rows of one and one of 900 439, 266.
  const bool many = p.rows > static_cast<long long>(p.B) * p.tile_tokens;
  if (p.D == 64) return many ? launch<64, true>(s, p, q, k) : launch<64, false>(s, p, q, k);
  return many ? launch<128, true>(s, p, q, k) : launch<128, false>(s, p, q, k);
}

}  // namespace kvc
