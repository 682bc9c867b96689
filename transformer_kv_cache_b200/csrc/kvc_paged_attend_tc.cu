// kvc_paged_attend_tc.cu -- attention of a paged batch on sm_100a tensor cores (bf16).
//
// O_i = sum_j softmax_j(scale q_i . k_j) v_j as a flash-attention pipeline over the units of
// kvc_paged.cuh: one persistent CTA per SM walks its units, an item at a time. A piece that
// has all of its rows' keys writes O; any other leaves a partial (O, maximum, sum) per row, which
// paged_merge_kernel joins.
//
// An item is up to two tiles of 128 packed query rows (tokens x the G query heads of one KV
// head, whole tokens only) that share the K and V tiles in shared memory. The CTA runs two
// streams, each with a score tile S in TMEM (128 rows x 128 keys fp32, overwritten by its own
// weights P as bf16), so that one stream's products run under the other's exponentials. With
// two tiles a stream is a tile; an item of one tile (a decode step's few rows) gives its key tiles
// to the streams by turns, each with a maximum and sum of its own.
//
// A stream's softmax is one warpgroup, a row to a thread, for 64 dims as for 128. (With 64 dims TMEM has
// room for two accumulators a stream, each with half of the keys: four warps a scheduler, a quarter of the
// exponentials on the FMA pipe, but 96 registers a thread, 7 stages for 10 and a join at a segment's end.
// Slower throughout: 1,004 rows over 73,292 keys 457 us for 442, 64 sequences of 130 rows 291 for 258.)
//
// Roles: warp 3 walks the schedule and hands out its segments through a ring in shared memory,
// some segments ahead (the walk's loads and divisions are off everybody else's path), and loads the
// queries by TMA as a 3-D box (dims, heads, tokens), which packs the rows of any group size; warp 0
// loads K and V by TMA (a page's slots, all dims, to a box: its rows go by eights, the 64-dim
// halves of eight rows after one another, so that one copy serves a page and rows keep one
// distance; one ring, a tile's V behind the next one's K, the next tile's pages looked up one tile ahead,
// across segments); warp 1 issues the MMAs (S = Q K^T: both operands in shared memory; O += P V:
// P in TMEM, V as an MN-major operand), the streams by turns, which keeps one stream's products
// under the other's softmax (a warp for each let them run in step: 771 for 952 TFLOP/s at D =
// 128); the warps from 4 on are the softmax (thread = row = TMEM lane).
//
// Slots past a sequence's length are never used: boxes past it are loaded from behind the
// pool's end, which TMA fills with zeros, warp 2 clears the last box of V behind the last token
// (the loading warp copying that box instead held up all loads: 90 for 55 us at 64 sequences of 512
// to 1,024 tokens in pages of 128 slots), and those keys' scores are set to -inf whatever K held.
//
// What bounds it. Few rows: the bytes of K and V (32 sequences of 4,096 to 8,192 tokens, 8 KV heads
// of 128 dims: 133 us, 6.1 TB/s), and where sequences are short a segment's end and start, some 1 us,
// and the call's own, some 12 us (64 of 512 to 1,024: 51 us). Both come from beyond the instruction cache, so
// the code is kept small (121 KB of it took 64 us there, 90 KB 50). Many rows, 128 dims: S = Q K^T
// reads both operands from shared memory, 8 KB for 64 cycles of the tensor core, all that it gives
// (4,096 rows of 8 heads over 16,384 keys: 245 us, 1,122 TFLOP/s); 64 dims: no pipe, but a stream's chain of
// product, score load, maximum, exponentials and weight store, which two warps a scheduler cover in part
// (MUFU 57 % of its peak, issue slots 34 %, tensor core 29 %; 2 sequences' 1,004 rows of 16 heads over 8,032
// shared keys and 4,016 and 8,032 of their own: 191 us, 606 TFLOP/s).
//
// Every barrier wait is bounded; a role that gives up sets the error word, and the CTA drains
// its copies and products, frees its TMEM and returns.
#include "kvc_paged.cuh"
#include "kvc_paged_math.cuh"

namespace kvc {
namespace {

using namespace paged;

constexpr int kTile = 128;                     // query rows of a tile, keys of a unit
constexpr float kGrow = 8.0f;                  // a weight above 2^8 moves the row's reference maximum
constexpr int kAhead = 3;                      // segments handed out before their queries are loaded
constexpr int kSoftWarps = 8;                  // four to a stream
constexpr int kThreads = 128 + 32 * kSoftWarps;
constexpr int kRegsLow = 88, kRegsHigh = 208;  // of warps 0 to 3 and of the softmax: in all 168 a thread, as at launch

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;                       // 128-byte swizzled blocks of a row
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + 1216;
};

struct Bars {
  uint64_t full[10], empty[10];                // K and V tiles
  uint64_t q_full[2], q_empty[2];              // query slots
  uint64_t s_full[2], p_full[2];
  uint64_t o_full[2], o_free[2];
  uint64_t tail_full[10];                      // tiles of V that end inside a box, before full
  uint64_t drained;
  SegmentRing ring;
  uint32_t tmem;
  int abort;
  long long plan[kPlanWords + 20];
};

// The key tiles of stream w in a segment of n: all of them where the item has two tiles of rows,
// else every other one (a segment of an odd number hands the next one's first
// tile to the other stream, so that segments of a single tile keep both busy).
__device__ __forceinline__ int stream_steps(const Segment& g, int w) {
  return g.two ? g.k1 - g.k0 : (g.k1 - g.k0 - (w ^ g.phase) + 1) >> 1;
}
__device__ __forceinline__ int stream_tile(const Segment& g, int w, int u) {
  return g.two ? u : 2 * u + (w ^ g.phase);
}
// The ring holds the tiles of a segment of n in the order in which the streams use them: K0, K1 V0,
// K2 V1, ..., V(n-1). The entry of V(t):
__device__ __forceinline__ int v_entry(int t, int n) { return t + 1 == n ? 2 * n - 1 : 2 * t + 2; }
// Weights of one row's step: P = 2^(s c - m) as bf16 pairs, returning their sum before the rounding, which
// the log-sum-exp keeps in full. The tensor core takes 16-bit weights, and bf16 ones need no scaling; a
// rounding is half a step (2^-8) at most, of each weight apart, so that over a row they mostly cancel: the
// outputs, rounded to bf16 themselves, are 1.7e-3 from the exact ones where fp32 weights give 1.66e-3.
__device__ __forceinline__ float weigh(const uint32_t* s, uint64_t c2, uint64_t nm2, uint32_t (&pb)[32]) {
  uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const uint64_t x = fma2_pair(s[2 * k], s[2 * k + 1], c2, nm2);
    const uint64_t e = exp2_pair_mufu(x);
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

// Whether a tile with `valid` keys before the sequence's end has its last inside a box of blk slots.
__device__ __forceinline__ bool ends_inside(int valid, int blk) { return valid < kTile && (valid & (blk - 1)); }

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
  static_assert(sizeof(Bars) <= 1216, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bar.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
      mbar_init(&bar.tail_full[i], 1);
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
    ring_init(bar.ring, 3 + kSoftWarps);       // warps 0, 1, 2 and the softmax
    bar.abort = 0;
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();                              // everything above is this CTA's own
  griddep_launch_dependents();
  Walk walk{};
  if (warp == 3 || !plan_by_warp(p))
    walk = plan_walk(p, bar.plan, [&](int b, const SeqView& v) { return head_units(p, b, v); });
  const uint32_t tmem = bar.tmem;
  // TMEM columns: S of stream w at 128 w, overwritten by its weights, O at 256 + w D
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
    int e = 0, sg = 0;
    bool ok = ring_take(bar.ring, sg++, g, abort), more = ok && g.nk > 0;
    int kt = g.k0;
    Box next = more ? box_at(kt) : Box{-1, 0, 0, 0};
    int row = past, valid = 0;                 // of the tile before: its V comes behind the next K
    int st = 0;                                // the next ring entry's stage
    auto load = [&](const CUtensorMap& map, uint64_t* landed, int from) {
      ok = ok && (e < C::kStages || wait_near(&bar.empty[st], ((e / C::kStages) - 1) & 1, abort));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      int rows[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) rows[i] = __shfl_sync(0xffffffffu, from, i) >> 3;
      if (leader) {
        uint8_t* dst = kv_s + st * C::kTileBytes;
        mbar_arrive_expect_tx(landed, C::kTileBytes);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < blocks) tma_load_4d(dst + i * blk * (D * 2), &map, landed, 0, 0, 0, rows[i]);
      }
      __syncwarp();
      ++e;
      st = st + 1 == C::kStages ? 0 : st + 1;
    };
    bool first = true;                         // of its segment
#pragma unroll 1
    while (ok && more) {
      const Box box = next;
      bool last = false;
      if (++kt >= g.k1) {
        last = true;
        ok = ring_take(bar.ring, sg++, g, abort);
        if (!ok) break;
        more = g.nk > 0;
        kt = g.k0;
      }
      if (more) next = box_at(kt);
      // pool row of this lane's box; behind the pool's end where there is no page (zeros)
      int here = past;
      if (lane < blocks && lane * blk < box.valid) {
        if (box.page < 0 || box.page >= p.pool_pages) latch_error(p.err, DERR_BOUNDS);
        else here = ((box.page * p.Hkv + box.h) << p.page_shift) + (box.key & ((1 << p.page_shift) - 1));
      }
      load(tmap_k, &bar.full[st], here);
      // the V of the tile before, and this one's where no other comes
#pragma unroll 1
      for (int j = first ? 1 : 0; j < (last ? 2 : 1); ++j)
        // a tile of V that ends inside a box goes through warp 2
        load(tmap_v, ends_inside(j ? box.valid : valid, blk) ? &bar.tail_full[st] : &bar.full[st], j ? here : row);
      row = here;
      valid = box.valid;
      first = last;
    }
    // every copy that was issued has landed before the CTA's shared memory goes
    if (lane == 0)
      for (int i = max(0, e - C::kStages); i < e; ++i)
        wait_drain(&bar.full[i % C::kStages], (i / C::kStages) & 1, abort);
  } else if (warp == 3) {
    reg_dealloc<kRegsLow>();
    // ------------------------------------------------------------------ schedule and queries
    if (lane == 0) {
      tma_prefetch_desc(&tmap_q);
      walk_to_item(p, walk);
      int slot = 0, used[2] = {0, 0}, put = 0, phase = 0;
      bool ok = true, more = true;
#pragma unroll 1
      for (int sg = 0; ok; ++sg) {
        // the first queries go out before the segments behind theirs
        const int ahead = used[slot] == 0 ? 0 : kAhead;
#pragma unroll 1
        while (ok && more && put <= sg + ahead) {
          Segment g{};
          more = next_segment(p, walk, g);     // the last one handed out has no key tiles
          g.phase = phase;
          if (!g.two) phase ^= (g.k1 - g.k0) & 1;
          ok = ring_put(bar.ring, put++, g, abort);
        }
        if (!ok) break;
        const Segment g = ring_peek(bar.ring, sg);
        if (g.nk == 0) break;
        const int tiles = g.two ? 2 : 1;
#pragma unroll 1
        for (int w = 0; w < tiles && ok; ++w) {
          ok = used[slot] == 0 || wait_segment(&bar.q_empty[slot], (used[slot] - 1) & 1, abort);
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
        if (used[i]) wait_drain(&bar.q_full[i], (used[i] - 1) & 1, abort);
    }
  } else if (warp == 1) {
    reg_dealloc<kRegsLow>();
    // ------------------------------------------------------------------ products
    const uint32_t idesc_s = idesc_f16kind(1, kTile, kTile, 0, 0);
    const uint32_t idesc_o = idesc_f16kind(1, kTile, D, 0, 1);
    // addresses stay below 2^18: an offset adds to the descriptor's address field
    const uint64_t q_desc = sw128_desc(smem_u32(q_s), 16, 1024);
    const uint64_t k_desc = sw128_desc(smem_u32(kv_s), 16, C::kHalves * 1024);
    const uint64_t v_desc = sw128_desc(smem_u32(kv_s), 1024, C::kHalves * 1024);
    const bool leader = elect_one();           // the warp waits, one lane issues
    int st = 0, slot = 0;                      // the next ring entry's stage, the next query slot
    uint32_t phase = 0;                        // of that stage
    auto advance = [&] {
      if (++st == C::kStages) {
        st = 0;
        phase ^= 1;
      }
    };
    // bit w: the phases of the query slots, of the streams' P and of their O
    uint32_t q_phase = 0, p_phase = 0, o_phase = 0;
    bool ok = true;
    // P of step u of the segment stands, and O may be written
    auto weighed = [&](int w, int u) {
      if (u == 0 && !wait_near(&bar.o_free[w], (o_phase >> w & 1) ^ 1, abort)) return false;   // at once the first time
      return wait_near(&bar.p_full[w], ((p_phase >> w) + u) & 1, abort);
    };
    auto score = [&](int w, int q, int stage) {            // S = Q K^T
      const uint64_t qd = q_desc + (q * C::kTileBytes >> 4), kd = k_desc + (stage * C::kTileBytes >> 4);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        mma_ss(tmem + w * 128, qd + (((c >> 2) * (kTile * 128) + (c & 3) * 32) >> 4),
               kd + (((c >> 2) * 1024 + (c & 3) * 32) >> 4), idesc_s, c > 0 ? 1u : 0u);
      mma_commit(&bar.s_full[w]);
    };
    auto add_v = [&](int w, int u, int stage) {            // O += P V
      const uint64_t vd = v_desc + (stage * C::kTileBytes >> 4);
#pragma unroll
      for (int c = 0; c < kTile / 16; ++c)
        mma_ts(tmem + 256 + w * D, tmem + w * 128 + c * 8, vd + (c * 16 * (D * 2) >> 4), idesc_o,
               u > 0 || c > 0 ? 1u : 0u);
    };
#pragma unroll 1
    for (int sg = 0;; ++sg) {
      Segment g;
      ok = ok && ring_take(bar.ring, sg, g, abort);
      if (!ok || g.nk == 0) break;
      const bool two = g.two;
      const int n = g.k1 - g.k0;
      const int q0 = slot;
      ok = wait_near(&bar.q_full[q0], q_phase >> q0 & 1, abort);
      if (two) ok = ok && wait_near(&bar.q_full[q0 ^ 1], q_phase >> (q0 ^ 1) & 1, abort);
      ok = __all_sync(0xffffffffu, ok);
      q_phase ^= two ? 3u : 1u << q0;
      if (!two) slot ^= 1;
      if (two) {
        // Step u of both streams: O += P V(u), S of K(u + 1); K comes first in the ring. Both products of
        // a stream go out back to back behind all of their waits (with 64 columns they take no longer
        // than their issue: a wait between them 627 for 676 TFLOP/s).
        ok = ok && __all_sync(0xffffffffu, wait_near(&bar.full[st], phase, abort));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll 1
          for (int w = 0; w < 2; ++w) {
            score(w, q0 ^ w, st);
            if (n == 1) mma_commit(&bar.q_empty[q0 ^ w]);
          }
          mma_commit(&bar.empty[st]);
        }
        __syncwarp();
        advance();
#pragma unroll 1
        for (int u = 0; u < n && ok; ++u) {
          const bool more = u + 1 < n;
          const int sk = st;
          const uint32_t pk = phase;
          if (more) advance();
          const int sv = st;
          const uint32_t pv = phase;
          advance();
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            bool r = ok;
            if (w == 0)
              r = r && wait_near(&bar.full[sv], pv, abort) && (!more || wait_near(&bar.full[sk], pk, abort));
            r = r && weighed(w, u);
            ok = __all_sync(0xffffffffu, r);
            if (!ok) break;
            tc_fence_after();
            if (leader) {
              add_v(w, u, sv);
              if (more) {
                score(w, q0 ^ w, sk);
                if (w == 1) mma_commit(&bar.empty[sk]);
                if (u + 2 == n) mma_commit(&bar.q_empty[q0 ^ w]);
              } else {
                mma_commit(&bar.o_full[w]);
              }
              if (w == 1) mma_commit(&bar.empty[sv]);
            }
            __syncwarp();
          }
        }
      } else {
        // The streams take the tiles by turns: V(t), then S of K(t + 2) as soon as it is there.
#pragma unroll 1
        for (int t = -2; t < n && ok; ++t) {
          const int w = (t & 1) ^ g.phase, u = t >> 1, sv = st;
          if (t >= 0) {
            ok = __all_sync(0xffffffffu, wait_near(&bar.full[st], phase, abort) && weighed(w, u));
            if (!ok) break;
            advance();
            tc_fence_after();
            if (leader) {
              add_v(w, u, sv);
              if (t + 2 >= n) mma_commit(&bar.o_full[w]);
            }
            __syncwarp();
          }
          if (t + 2 < n) {
            ok = __all_sync(0xffffffffu, wait_near(&bar.full[st], phase, abort));
            if (!ok) break;
            tc_fence_after();
            if (leader) {
              score(w, q0, st);
              mma_commit(&bar.empty[st]);
              if (t + 3 == n) mma_commit(&bar.q_empty[q0]);
            }
            __syncwarp();
            advance();
          }
          if (t >= 0 && leader) mma_commit(&bar.empty[sv]);
          __syncwarp();
        }
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int steps = stream_steps(g, w);
        p_phase ^= static_cast<uint32_t>(steps & 1) << w;
        o_phase ^= static_cast<uint32_t>(steps > 0) << w;
      }
    }
    if (leader) mma_commit(&bar.drained);
    __syncwarp();
    wait_drain(&bar.drained, 0, abort);
  } else if (warp == 2) {
    reg_dealloc<kRegsLow>();
    // ------------------------------------------------------------------ the last values of a sequence
    // What the cache holds behind a length must not meet a weight of 0 (0 x NaN): zeros to V's rows
    // behind the last token, up to the end of its box, then the tile is handed on.
    int e0 = 0;
    uint32_t phases = 0;                       // of the stages' tail_full
    bool ok = true;
    for (int sg = 0; ok; ++sg) {
      Segment g;
      ok = ring_take(bar.ring, sg, g, abort);
      if (!ok || g.nk == 0) break;
      // the prefix's last tile, where the item has it before its own, and the segment's last
#pragma unroll 1
      for (int i = 0; i < 2 && ok; ++i) {
        const int kt = i ? g.k1 - 1 : prefix_tiles(p) - 1;
        if (!i && (kt < g.k0 || kt >= g.k1 - 1)) continue;
        const KeyTile tile = key_tile_at(p, g, kt);
        const int valid = tile.len - tile.key0;
        if (!ends_inside(valid, blk)) continue;
        const int st = (e0 + v_entry(kt - g.k0, g.k1 - g.k0)) % C::kStages;
        ok = __all_sync(0xffffffffu, wait_segment(&bar.tail_full[st], phases >> st & 1, abort));
        if (!ok) break;
        phases ^= 1u << st;
        uint8_t* v = kv_s + st * C::kTileBytes;
        const int end = (valid | (blk - 1)) + 1;
#pragma unroll 1
        for (int k = valid * C::kHalves + (lane >> 3); k < end * C::kHalves; k += 4) {
          const int at = k / C::kHalves;       // eight lanes for 128 bytes of a row
          *reinterpret_cast<uint4*>(v + ((at >> 3) * C::kHalves + k % C::kHalves) * 1024 + (at & 7) * 128 +
                                    (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.full[st]);
      }
      e0 += 2 * (g.k1 - g.k0);
    }
  } else {
    reg_alloc<kRegsHigh>();
    // ------------------------------------------------------------------ softmax of stream w
    const int w = (warp - 4) >> 2, wq = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_col = tmem + lane_base + w * 128;
    const uint32_t o_col = tmem + lane_base + 256 + w * D;
    const float c = p.scale_log2;
    const int r = wq * 32 + lane, r_tok = r / p.G, r_head = r - r_tok * p.G;   // row, its token and head
    int done = 0, segs = 0;
    bool ok = true;
    for (int sg = 0;; ++sg) {
      // the segment stays in the ring until its end, where it is read again: its fields are not
      // held in registers through the steps
      ok = ok && wait_near(&bar.ring.full[sg % kRing], (sg / kRing) & 1, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      int steps, first, stride, limit;         // of the steps' key tiles: the first and their distance; keys seen
      bool mine, active;                       // this row, this warp has rows
      {
        const Segment g = ring_peek(bar.ring, sg);
        if (g.nk == 0) break;
        steps = stream_steps(g, w);
        first = g.k0 + stream_tile(g, w, 0);
        stride = g.two ? 1 : 2;
        const int t0 = g.i * p.item_tokens + (g.two ? w * p.tile_tokens : 0);
        const int rows = min(p.tile_tokens, g.v.n - t0) * p.G;
        mine = r < rows;
        active = wq * 32 < rows;
        // rows of nobody compute what nobody reads: they mask nothing and move nothing. The keys that
        // the row sees, counted from the segment's tile 0 of its own (a joined prefix comes before).
        limit = mine ? key_limit(p, g.b, g.v, t0 + r_tok) + prefix_tiles(p) * kTile : 1 << 30;
      }
      float m = -INFINITY, l = 0.f;
      for (int u = 0; u < steps; ++u) {
        ok = wait_near(&bar.s_full[w], (done + u) & 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (active) {
          uint32_t s[kTile];
#pragma unroll
          for (int q = 0; q < kTile / 32; ++q)
            tmem_ld32(s_col + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]));
          const int tile = first + u * stride;
          const int valid = (tile < prefix_tiles(p) ? p.prefix_tokens : limit) - tile * kTile;
          const bool masked = __any_sync(0xffffffffu, valid < kTile);
          tmem_ld_wait();
          if (masked) {
#pragma unroll
            for (int k = 0; k < kTile; ++k)
              if (k >= valid) s[k] = 0xff800000u;
          }
          // the row's reference maximum moves when a weight would pass 2^8, or on a NaN
          const float mx = row_max(s) * c;
          const bool move = mine && !(mx <= m + kGrow);
          if (__any_sync(0xffffffffu, move)) {
            const float m_new = move ? mx : m;
            const float f = move ? ex2(m - m_new) : 1.f;           // 0 from -inf
            l *= f;
            m = m_new;
            if (u > 0) {                       // S of this step is complete, and so the product of the last
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tmem_ld16(o_col + 16 * q, o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st16(o_col + 16 * q, o);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : m;             // nothing seen yet: every weight is 0
          const uint64_t c2 = pk2(c, c), nm2 = pk2(-base, -base);
          uint32_t pb[32];
#pragma unroll
          for (int q = 0; q < kTile / 64; ++q) {
            l += weigh(&s[64 * q], c2, nm2, pb);
            tmem_st32(s_col + 32 * q, pb);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[w]);
      }
      if (!ok) break;
      done += steps;
      bool whole;
      long long out, slot;                     // the row and head of O, the partial's slot
      {
        const Segment g = ring_peek(bar.ring, sg);
        const int row = g.v.r0 + g.i * p.item_tokens + (g.two ? w * p.tile_tokens : 0) + r_tok;
        const int hq = g.h * p.G + r_head;
        whole = g.k0 == 0 && g.k1 == g.nk && g.two && writes_rows(p, g.v, g.i);
        out = static_cast<long long>(row) * p.Hq + hq;
        slot = g.k0 == 0 ? row_slot(p, g.b, g.two ? 0 : w, row, hq) : cta_slot(p, blockIdx.x, w * kTile + r);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ring.empty[sg % kRing]);
      if (steps == 0) {
        if (mine) p.part_ml[slot] = make_float2(m, l);
        continue;
      }
      ok = wait_near(&bar.o_full[w], segs & 1, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (mine) {
        if (!whole) p.part_ml[slot] = make_float2(m, l);
        else if (p.lse) p.lse[out] = (m + log2f(l)) * 0.6931471805599453f;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      // 32 columns of the row: O or a partial
      auto store = [&](const uint32_t* o, int q) {
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + out * D + 32 * q);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              y[i] = pack_bf16(__uint_as_float(o[8 * k + 2 * i]) * inv, __uint_as_float(o[8 * k + 2 * i + 1]) * inv);
            dst[k] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_o + slot * D + 32 * q);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                 __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
        }
      };
      if (active) {
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(o_col + 32 * q, o);
          tmem_ld_wait();
          if (mine) store(o, q);
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
  report_abort(p, abort);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(cudaStream_t s, const PagedParams& p, const CUtensorMap& q, const CUtensorMap& k,
                   const CUtensorMap& v) {
  using C = Cfg<D>;
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    const void* kernel = reinterpret_cast<const void*>(paged_attend_tc_kernel<D>);
    // the warps' shares come out of what the block is launched with; a larger sum would wait forever
    cudaFuncAttributes at;
    if (const cudaError_t got = cudaFuncGetAttributes(&at, kernel); got != cudaSuccess) return got;
    if (at.numRegs * kThreads < 32 * (4 * kRegsLow + kSoftWarps * kRegsHigh))
      return cudaErrorLaunchOutOfResources;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  return e != cudaSuccess ? e
                          : launch_pdl(paged_attend_tc_kernel<D>, dim3(p.grid), dim3(kThreads), C::kSmem, s, q,
                                       k, v, p);
}

}  // namespace

cudaError_t launch_paged_attend_tc(cudaStream_t s, const PagedParams& p) {
  CUtensorMap q, k, v;
  if (!encode_rows_tmap(&q, p.q, p) || !encode_slots_tmap(&k, p.k_pool, p) || !encode_slots_tmap(&v, p.v_pool, p))
    return cudaErrorInvalidValue;
  return p.D == 64 ? launch<64>(s, p, q, k, v) : launch<128>(s, p, q, k, v);
}

}  // namespace kvc
