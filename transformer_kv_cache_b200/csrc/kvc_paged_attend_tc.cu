// kvc_paged_attend_tc.cu -- attention of a paged batch on sm_100a tensor cores (bf16).
//
// O_i = sum_j softmax_j(scale q_i . k_j) v_j as a flash-attention pipeline over the units of
// kvc_paged.cuh: one persistent CTA per SM walks its units, an item at a time. A piece that
// has all of its rows' keys writes O; any other leaves a partial (O, maximum, sum) per row, which
// paged_merge_kernel joins.
//
// An item is up to two tiles of 128 packed query rows (tokens x the G query heads of one KV
// head, whole tokens only) that share the K and V tiles in shared memory. The CTA runs two
// streams, each with score buffers S in TMEM (128 rows x kStep keys fp32, overwritten by their
// own weights P as bf16), an accumulator O (128 x D fp32) and a softmax
// warpgroup, so that one stream's products run under the other's exponentials. With two tiles a
// stream is a tile; an item of one tile (a decode step's few rows) gives its key blocks to the
// streams by turns, each with a maximum and sum of its own.
//
// TMEM decides the step: with D = 64 a stream has two S buffers of 64 keys, and the issuer keeps
// S one step ahead of the softmax; with D = 128 the accumulators leave one S buffer of 128 keys
// (a product of 64 keys would read the query operand from shared memory faster than that can
// give it: 48 cycles for 32 of the tensor core).
//
// Roles (384 threads): warp 3 walks the schedule and hands out its segments through a ring in
// shared memory, some segments ahead (the walk's loads and divisions are off everybody else's
// path), and loads the queries by TMA as a 3-D box (dims, heads, tokens), which packs the rows of
// any group size; warp 0 loads K and V by TMA (a page's slots, all dims, to a box: its rows go by
// eights, the 64-dim halves of eight rows after one another, so that one copy serves a page and
// rows keep one distance; one ring in the order K0 V0 K1 V1 ..., the next tile's pages looked up
// one tile ahead, across segments); warp 1 issues the
// MMAs (S = Q K^T: both operands in shared memory; O += P V: P in TMEM, V as an MN-major
// operand); with D = 128 it takes the streams by turns, which
// keeps one stream's products under the other's softmax; with D = 64, where a product is so short
// that issuing it is what takes the time, warp 2 issues stream 1's; warps 4-7 and 8-11 are the
// softmax of stream 0 and 1 (thread = row = TMEM lane).
//
// Slots past a sequence's length are never used: boxes past it are loaded from behind the
// pool's end, which TMA fills with zeros, the last box of V is copied by the loading warp's threads
// with zeros behind the last token, and those keys' scores are set to -inf whatever K held.
//
// Every barrier wait is bounded; a role that gives up sets the error word, and the CTA drains
// its copies and products, frees its TMEM and returns.
#include "kvc_paged.cuh"
#include "kvc_paged_math.cuh"

namespace kvc {
namespace {

using namespace paged;

constexpr int kThreads = 384;
constexpr int kTile = 128;                     // query rows of a tile, keys of a unit
constexpr float kGrow = 8.0f;                  // a weight above 2^8 moves the row's reference maximum
constexpr int kRegsLow = 88, kRegsHigh = 208;  // 128 x 88 + 256 x 208 = 384 x 168, the registers at launch
constexpr int kAhead = 3;                      // segments handed out before their queries are loaded

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;                       // 128-byte swizzled blocks of a row
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kStep = D == 128 ? 128 : 64;            // keys of a step of a stream
  static constexpr int kBufs = D == 128 ? 1 : 2;               // score buffers of a stream
  static constexpr int kPerTile = kTile / kStep;               // steps of a key tile
  static constexpr int kIssuers = D == 128 ? 1 : 2;            // warps that issue the products
  static constexpr int kPoly8 = D == 128 ? 0 : 2;              // of 8 pairs, the exponentials on the FMA pipe
  static constexpr int kSmem = 1024 + 2 * kTileBytes + kStages * kTileBytes + 1152;
};

struct Bars {
  uint64_t full[10], empty[10];                // K and V tiles
  uint64_t q_full[2], q_empty[2];              // query slots
  uint64_t s_full[2][2], p_full[2][2];         // [stream][buffer]
  uint64_t pv_done[2], o_full[2], o_free[2], drained[2];
  SegmentRing ring;
  uint32_t tmem;
  int abort;
  long long plan[kPlanWords + kThreads / 32];
};

// Steps of stream w in a segment of `blocks` key blocks.
__device__ __forceinline__ int stream_steps(bool two, int w, int blocks) { return two ? blocks : (blocks - w + 1) >> 1; }

// Weights of one row's step: P = 2^(s c - m) as bf16 pairs, returning their sum (before the
// rounding). kPoly of every 8 pairs go to the FMA pipe, the others to the MUFU, spread through the
// row. Masked steps hold -inf and use the MUFU alone, which gives exact zeros.
template <int kPoly>
__device__ __forceinline__ float weigh(const uint32_t* s, uint64_t c2, uint64_t nm2, uint32_t (&pb)[32]) {
  uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const uint64_t x = fma2_pair(s[2 * k], s[2 * k + 1], c2, nm2);
    const uint64_t e = (k & 7) >= 8 - kPoly ? exp2_pair(x) : exp2_pair_mufu(x);
    if (k & 1) sum1 = add2(sum1, e);
    else sum0 = add2(sum0, e);
    float e0, e1;
    up2(e, e0, e1);
    pb[k] = pack_bf16(e0, e1);
  }
  float a, b;
  up2(add2(sum0, sum1), a, b);
  return a + b;
}

template <int N>
__device__ __forceinline__ float row_max(const uint32_t (&s)[N]) {
  float a[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) a[k] = __uint_as_float(s[k]);
#pragma unroll
  for (int k = 8; k + 16 <= N; k += 16)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      a[j] = max3_nan(a[j], __uint_as_float(s[k + 2 * j]), __uint_as_float(s[k + 2 * j + 1]));
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] = max_nan(a[j], __uint_as_float(s[N - 8 + j]));
  return max3_nan(max3_nan(a[0], a[1], a[2]), max3_nan(a[3], a[4], a[5]), max_nan(a[6], a[7]));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attend_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ PagedParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;                                     // [slot][half][128 rows][128 B]
  uint8_t* kv_s = q_s + 2 * C::kTileBytes;                 // [stage][8 keys][half][key][128 B]
  Bars& bar = *reinterpret_cast<Bars*>(kv_s + C::kStages * C::kTileBytes);
  static_assert(sizeof(Bars) <= 1152, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bar.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], C::kIssuers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_empty[i], C::kIssuers);
      for (int x = 0; x < 2; ++x) {
        mbar_init(&bar.s_full[i][x], 1);
        mbar_init(&bar.p_full[i][x], 4);
      }
      mbar_init(&bar.pv_done[i], 1);
      mbar_init(&bar.o_full[i], 1);
      mbar_init(&bar.o_free[i], 4);
      mbar_init(&bar.drained[i], 1);
    }
    ring_init(bar.ring, 9 + C::kIssuers);      // everybody but warp 3 and an idle warp 2
    bar.abort = 0;
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  griddep_wait();                              // everything above is this CTA's own
  griddep_launch_dependents();
  Walk walk = plan_walk(p, bar.plan, [&](int b, const SeqView& v) { return head_units(p, b, v); });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  // TMEM columns: S buffer x of stream w at w * 128 + x * kStep, O of stream w at 256 + w * D
  const int blk = min(1 << p.page_shift, kTile);           // slots of a box

  if (warp == 0) {
    reg_dealloc<kRegsLow>();
    // ------------------------------------------------------------------ K and V
    if (lane == 0) {
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_v);
    }
    const int blocks = kTile / blk;                        // boxes of a tile, a lane for each
    const int past = static_cast<int>((p.pool_pages * p.Hkv) << p.page_shift);
    const bool leader = elect_one();
    // The page of this lane's box of key tile kt (as the table has it, so that nothing waits for
    // the load yet) and how many keys the tile has.
    struct Box {
      int page, key, valid, h;
    };
    Segment g;
    auto box_at = [&](int kt) {
      const KeyTile t = key_tile_at(p, g, kt);
      const int key = t.key0 + lane * blk;
      Box b{-1, key, t.len - t.key0, g.h};
      if (lane < blocks && key < t.len)
        b.page = __ldg((t.b < 0 ? p.prefix_pages : p.page_table + static_cast<long long>(t.b) * p.max_pages) +
                       (key >> p.page_shift));
      return b;
    };
    // The last box of a sequence's V ends inside: what the cache holds behind the length must not
    // meet a weight of 0 (0 x NaN), so its rows are copied here, zeros after the last, as the
    // 128-byte swizzle places them.
    auto copy_last = [&](uint8_t* dst, int row, int first, int rows) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v_pool) +
                                                        static_cast<long long>(row) * D);
      constexpr int kChunks = D / 8;
#pragma unroll 4
      for (int i = lane; i < blk * kChunks; i += 32) {
        const int r = i / kChunks, c = i % kChunks, at = first + r;
        const uint4 x = row < past && r < rows ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(dst + ((at >> 3) * C::kHalves + (c >> 3)) * 1024 + (at & 7) * 128 +
                                  (((c & 7) ^ (at & 7)) << 4)) = x;
      }
      fence_proxy_async_shared();
      __syncwarp();
    };
    int e = 0, sg = 0;
    bool ok = ring_take(bar.ring, sg++, g, abort, p.err), more = ok && g.nk > 0;
    int kt = g.k0;
    Box next = more ? box_at(kt) : Box{-1, 0, 0, 0};
    while (ok && more) {
      const Box box = next;
      if (++kt >= g.k1) {
        ok = ring_take(bar.ring, sg++, g, abort, p.err);
        if (!ok) break;
        more = g.nk > 0;
        kt = g.k0;
      }
      if (more) next = box_at(kt);
      // pool row of this lane's box; behind the pool's end where there is no page (zeros)
      int row = past;
      if (lane < blocks && lane * blk < box.valid) {
        if (box.page < 0 || box.page >= p.pool_pages) latch_error(p.err, DERR_BOUNDS);
        else row = ((box.page * p.Hkv + box.h) << p.page_shift) + (box.key & ((1 << p.page_shift) - 1));
      }
      int rows[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) rows[i] = __shfl_sync(0xffffffffu, row, i);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int st = e % C::kStages;
        ok = e < C::kStages || mbar_wait_bounded(&bar.empty[st], ((e / C::kStages) - 1) & 1, abort, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* dst = kv_s + st * C::kTileBytes;
        int last = 8;                          // the box that is copied by hand
        if (kv == 1 && box.valid < kTile && (box.valid & (blk - 1))) {
          last = box.valid / blk;
          copy_last(dst, __shfl_sync(0xffffffffu, row, last), last * blk, box.valid & (blk - 1));
        }
        if (leader) {
          mbar_arrive_expect_tx(&bar.full[st], C::kTileBytes - (last < 8 ? C::kHalves * blk * 128 : 0));
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < blocks && i != last)
              tma_load_4d(dst + i * blk * (D * 2), kv ? &tmap_v : &tmap_k, &bar.full[st], 0, 0, 0, rows[i] >> 3);
        }
        __syncwarp();
        ++e;
      }
    }
    // every copy that was issued has landed before the CTA's shared memory goes
    if (lane == 0)
      for (int i = max(0, e - C::kStages); i < e; ++i)
        mbar_wait_drain(&bar.full[i % C::kStages], (i / C::kStages) & 1, p.err);
  } else if (warp == 3) {
    reg_dealloc<kRegsLow>();
    // ------------------------------------------------------------------ schedule and queries
    if (lane == 0) {
      tma_prefetch_desc(&tmap_q);
      walk_to_item(p, walk);
      int slot = 0, used[2] = {0, 0}, put = 0;
      bool ok = true, more = true;
      for (int sg = 0; ok; ++sg) {
        while (ok && more && put <= sg + kAhead) {
          Segment g{};
          more = next_segment(p, walk, g);     // the last one handed out has no key tiles
          ok = ring_put(bar.ring, put++, g, abort, p.err);
        }
        if (!ok) break;
        const Segment g = ring_peek(bar.ring, sg);
        if (g.nk == 0) break;
        const int tiles = g.two ? 2 : 1;
        for (int w = 0; w < tiles && ok; ++w) {
          ok = used[slot] == 0 || mbar_wait_bounded(&bar.q_empty[slot], (used[slot] - 1) & 1, abort, p.err);
          if (!ok) break;
          mbar_arrive_expect_tx(&bar.q_full[slot], C::kHalves * p.tile_tokens * p.G * 128);
          for (int c = 0; c < C::kHalves; ++c)
            tma_load_3d(q_s + slot * C::kTileBytes + c * (kTile * 128), &tmap_q, &bar.q_full[slot], c * 64, g.h * p.G,
                        g.v.r0 + g.i * p.item_tokens + w * p.tile_tokens);
          ++used[slot];
          slot ^= 1;
        }
      }
      for (int i = 0; i < 2; ++i)
        if (used[i]) mbar_wait_drain(&bar.q_full[i], (used[i] - 1) & 1, p.err);
    }
  } else if (warp < 3) {
    reg_dealloc<kRegsLow>();
    // ------------------------------------------------------------------ products of streams [w0, w1)
    const int w0 = C::kIssuers == 2 ? warp - 1 : 0, w1 = C::kIssuers == 2 ? w0 + 1 : 2;
    if (warp <= C::kIssuers) {
      const bool leader = elect_one();         // the warp waits, one lane issues
      const uint32_t idesc_s = idesc_f16kind(1, kTile, C::kStep, 0, 0);
      const uint32_t idesc_o = idesc_f16kind(1, kTile, D, 0, 1);
      // addresses stay below 2^18: an offset adds to the descriptor's address field
      const uint64_t q_desc = sw128_desc(smem_u32(q_s), 16, 1024);
      const uint64_t k_desc = sw128_desc(smem_u32(kv_s), 16, C::kHalves * 1024);
      const uint64_t v_desc = sw128_desc(smem_u32(kv_s), 1024, C::kHalves * 1024);
      int e0 = 0, slot = 0, used[2] = {0, 0};  // first ring entry of the segment, next query slot
      int uu[2] = {0, 0}, segs[2] = {0, 0};    // steps and segments of each stream
      bool ok = true;
      for (int sg = 0;; ++sg) {
        Segment g;
        ok = ok && ring_take(bar.ring, sg, g, abort, p.err);
        if (!ok || g.nk == 0) break;
        const bool two = g.two;
        const int blocks = (g.k1 - g.k0) * C::kPerTile;
        const int steps[2] = {stream_steps(two, 0, blocks), stream_steps(two, 1, blocks)};
        const int qs[2] = {slot, two ? slot ^ 1 : slot};
        for (int w = w0; w < w1 && (w == w0 || two); ++w)
          ok = ok && mbar_wait_bounded(&bar.q_full[qs[w]], used[qs[w]] & 1, abort, p.err);
        ok = __all_sync(0xffffffffu, ok);
        ++used[slot];
        if (two) ++used[slot ^ 1];
        else slot ^= 1;
        // Stream w's step u takes key block two ? u : 2 u + w. One issuer takes the streams by turns,
        // so the later one's product frees a tile; of two issuers each has a vote.
        auto issue_s = [&](int w, int u) {
          const int bk = two ? u : 2 * u + w, hb = bk % C::kPerTile;
          const int e = e0 + 2 * (bk / C::kPerTile), st = e % C::kStages;
          if (!two || (hb == 0 && w == w0)) {  // else waited for already
            const bool r = mbar_wait_bounded(&bar.full[st], (e / C::kStages) & 1, abort, p.err);
            if (!__all_sync(0xffffffffu, r)) return false;
          }
          tc_fence_after();
          const int x = (uu[w] + u) % C::kBufs;
          const uint64_t qd = q_desc + (qs[w] * C::kTileBytes >> 4);
          const uint64_t kd = k_desc + (st * C::kTileBytes + hb * (C::kStep * D * 2) >> 4);
          if (leader) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const uint32_t qo = ((c >> 2) * (kTile * 128) + (c & 3) * 32) >> 4;
              const uint32_t ko = ((c >> 2) * 1024 + (c & 3) * 32) >> 4;
              mma_ss(tmem + w * 128 + x * C::kStep, qd + qo, kd + ko, idesc_s, c > 0 ? 1u : 0u);
            }
            mma_commit(&bar.s_full[w][x]);
            const bool last = two ? u + 1 == steps[w] : C::kIssuers == 2 ? u + 1 == steps[w] : bk + 1 == blocks;
            if (C::kIssuers == 2 ? !two || hb == C::kPerTile - 1 : hb == C::kPerTile - 1 && (w == 1 || !two))
              mma_commit(&bar.empty[st]);
            if (last) {                          // the last product that reads these queries
              mma_commit(&bar.q_empty[qs[w]]);
              if (C::kIssuers == 2 && two) mma_commit(&bar.q_empty[qs[w]]);
            }
          }
          __syncwarp();
          return true;
        };
        auto issue_pv = [&](int w, int u) {
          const int bk = two ? u : 2 * u + w, hb = bk % C::kPerTile;
          const int e = e0 + 2 * (bk / C::kPerTile) + 1, st = e % C::kStages;
          const int x = (uu[w] + u) % C::kBufs;
          bool r = true;
          if (!two || (hb == 0 && w == w0)) r = mbar_wait_bounded(&bar.full[st], (e / C::kStages) & 1, abort, p.err);
          if (u == 0 && segs[w] > 0) r = r && mbar_wait_bounded(&bar.o_free[w], (segs[w] - 1) & 1, abort, p.err);
          r = r && mbar_wait_bounded(&bar.p_full[w][x], ((uu[w] + u) / C::kBufs) & 1, abort, p.err);
          if (!__all_sync(0xffffffffu, r)) return false;
          tc_fence_after();
          const uint64_t vd = v_desc + (st * C::kTileBytes + hb * (C::kStep * D * 2) >> 4);
          if (leader) {
#pragma unroll
            for (int c = 0; c < C::kStep / 16; ++c)
              mma_ts(tmem + 256 + w * D, tmem + w * 128 + x * C::kStep + c * 8, vd + c * (D * 32 >> 4), idesc_o,
                     u > 0 || c > 0 ? 1u : 0u);
            if (C::kBufs > 1) mma_commit(&bar.pv_done[w]);
            if (u + 1 == steps[w]) mma_commit(&bar.o_full[w]);
          }
          __syncwarp();
          return true;
        };
        auto release_v = [&](int w, int u) {
          const int bk = two ? u : 2 * u + w, hb = bk % C::kPerTile;
          if (leader && (C::kIssuers == 2 ? !two || hb == C::kPerTile - 1 : hb == C::kPerTile - 1 && (w == 1 || !two)))
            mma_commit(&bar.empty[(e0 + 2 * (bk / C::kPerTile) + 1) % C::kStages]);
          __syncwarp();
        };
        for (int u = 0; u < C::kBufs && ok; ++u)
          for (int w = w0; w < w1 && ok; ++w)
            if (u < steps[w]) ok = issue_s(w, u);
        for (int u = 0; u < steps[w0] && ok; ++u)
          for (int w = w0; w < w1 && ok; ++w) {
            if (u >= steps[w]) continue;
            ok = issue_pv(w, u);
            if (ok && u + C::kBufs < steps[w]) ok = issue_s(w, u + C::kBufs);
            if (ok) release_v(w, u);
          }
        for (int w = w0; w < w1; ++w) {
          uu[w] += steps[w];
          segs[w] += steps[w] > 0;
        }
        e0 += 2 * (g.k1 - g.k0);
      }
      if (leader) mma_commit(&bar.drained[w0]);
      __syncwarp();
      mbar_wait_drain(&bar.drained[w0], 0, p.err);
    }
  } else {
    reg_alloc<kRegsHigh>();
    // ------------------------------------------------------------------ softmax of stream w
    const int w = (warp - 4) >> 2, wq = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_base = tmem + lane_base + w * 128, o_col = tmem + lane_base + 256 + w * D;
    const float c = p.scale_log2;
    int uu = 0, segs = 0;
    bool ok = true;
    for (int sg = 0;; ++sg) {
      Segment g;
      ok = ok && ring_take(bar.ring, sg, g, abort, p.err);
      if (!ok || g.nk == 0) break;
      const bool two = g.two;
      const int steps = stream_steps(two, w, (g.k1 - g.k0) * C::kPerTile);
      const int t0 = g.i * p.item_tokens + (two ? w * p.tile_tokens : 0);
      const int rows = min(p.tile_tokens, g.v.n - t0) * p.G;
      const int r = wq * 32 + lane;
      const int tok = t0 + r / p.G;
      const int hq = g.h * p.G + r % p.G;
      const bool active = wq * 32 < rows;      // this warp has rows
      // rows of nobody compute what nobody reads: they mask nothing and move nothing
      const int limit = r < rows ? key_limit(p, g.b, g.v, tok) : 1 << 30;
      float m = -INFINITY, l = 0.f;
      for (int u = 0; u < steps; ++u) {
        const int x = (uu + u) % C::kBufs;
        const uint32_t s_col = s_base + x * C::kStep;
        ok = mbar_wait_bounded(&bar.s_full[w][x], ((uu + u) / C::kBufs) & 1, abort, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const int bk = two ? u : 2 * u + w;
          uint32_t s[C::kStep];
#pragma unroll
          for (int q = 0; q < C::kStep / 32; ++q)
            tmem_ld32(s_col + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]));
          const KeyTile kt = key_tile_at(p, g, g.k0 + bk / C::kPerTile);
          const int valid = (kt.b == g.b ? limit : kt.len) - kt.key0 - (bk % C::kPerTile) * C::kStep;
          const bool masked = __any_sync(0xffffffffu, valid < C::kStep);
          tmem_ld_wait();
          if (masked) {
#pragma unroll
            for (int k = 0; k < C::kStep; ++k)
              if (k >= valid) s[k] = 0xff800000u;
          }
          // the row's reference maximum moves when a weight would pass 2^8, or on a NaN
          const float mx = row_max(s) * c;
          const bool move = r < rows && !(mx <= m + kGrow);
          if (__any_sync(0xffffffffu, move)) {
            const float m_new = move ? mx : m;
            const float f = move ? ex2(m - m_new) : 1.f;           // 0 from -inf
            l *= f;
            m = m_new;
            if (u > 0) {
              if (C::kBufs > 1) {
                // S is ahead of O here: the product of the step before must be done
                ok = mbar_wait_bounded(&bar.pv_done[w], (uu + u - 1) & 1, abort, p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
              }
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
          uint32_t pb[32];
#pragma unroll
          for (int q = 0; q < C::kStep / 64; ++q) {
            l += masked ? weigh<0>(&s[64 * q], c2, nm2, pb) : weigh<C::kPoly8>(&s[64 * q], c2, nm2, pb);
            tmem_st32(s_col + 32 * q, pb);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[w][x]);
      }
      if (!ok) break;
      uu += steps;
      const bool whole = g.k0 == 0 && g.k1 == g.nk && two && writes_rows(p, g.v, g.i);
      const long long out = static_cast<long long>(g.v.r0 + tok) * p.Hq + hq;
      const long long slot = g.k0 == 0 ? row_slot(p, g.b, two ? 0 : w, g.v.r0 + tok, hq)
                                       : cta_slot(p, blockIdx.x, w * kTile + r);
      if (r < rows) {
        if (!whole) p.part_ml[slot] = make_float2(m, l);
        else if (p.lse) p.lse[out] = (m + log2f(l)) * 0.6931471805599453f;
      }
      if (steps == 0) continue;
      ok = mbar_wait_bounded(&bar.o_full[w], segs & 1, abort, p.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (active) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(o_col + 32 * q, o);
          tmem_ld_wait();
          if (r >= rows) {
          } else if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + out * D + 32 * q);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t y[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                y[j] = pack_bf16(__uint_as_float(o[8 * k + 2 * j]) * inv, __uint_as_float(o[8 * k + 2 * j + 1]) * inv);
              dst[k] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(p.part_o + slot * D + 32 * q);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                   __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.o_free[w]);
      ++segs;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
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
  if (!encode_rows_tmap(&q, p.q, p) || !encode_slots_tmap(&k, p.k_pool, p) || !encode_slots_tmap(&v, p.v_pool, p))
    return cudaErrorInvalidValue;
  return p.D == 64 ? launch<64>(s, p, q, k, v) : launch<128>(s, p, q, k, v);
}

}  // namespace kvc
