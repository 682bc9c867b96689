// kvc_paged.cuh -- what the paged-batch operators share: the batch as the kernels see it, the
// schedule of the attention and weight kernels, and the layout of their workspace.
//
// Schedule. The work of a call is a sequence of units; CTA c of the grid takes the units
// [c * U, (c + 1) * U) with U = ceil(units / CTAs), whatever the lengths on the device are, so
// a long sequence is split over CTAs and short ones share one, and no host copy of a length is
// needed (a captured graph follows the lengths of its replay). A key tile of an attention item is
// cost_one or cost_two units (and U no less), and belongs to the CTA that has its first one; an
// item is one KV head with up to item_tokens query tokens of one
// sequence (its G query heads each), or, for the shared prefix, of the whole batch: there the
// queries of all sequences are packed, so the prefix is read once for the batch and not once
// per sequence. The prefix is sequence -1 of the schedule. An item whose units fall into several
// CTAs leaves several partial results; the CTA that has its first unit puts its partial into
// the row's own slot, every other CTA into the CTA's slot (a CTA continues at most one item,
// the one it begins with).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvc_internal.h"
#include "sm100_ptx.cuh"

namespace kvc {

struct PagedParams {
  int B, Hq, Hkv, G, D;
  int page_shift;               // page size = 1 << page_shift
  int max_pages;                // pages of a sequence's page-table row
  int prefix_tokens;
  int rows;                     // rows of Q (the tensors' size; row_start tells which are in use)
  int causal;
  int join;                     // 1: an item reads the prefix's key tiles before its own
  long long pool_pages;
  const int32_t* page_table;
  const int32_t* lengths;
  const int32_t* prefix_pages;
  const int32_t* row_start;
  const void* q;
  long long q_stride;           // elements between Q rows
  const void* k_pool;
  const void* v_pool;
  void* o;
  float* lse;                   // attention: out (may be null); weights: in
  float* scores;
  float scale_log2;             // softmax scale * log2(e)
  int* err;
  // schedule
  int item_tokens;              // query tokens of an item
  int prefix_item_tokens;       // the same for the prefix's items
  int tile_tokens;              // query tokens of a tile (the item's, or half of them)
  int key_tile, key_shift;      // keys of a unit, 1 << key_shift
  int prefix_units;             // key tiles of the prefix
  int streams;                  // tiles of an item: 1, or 2 (an item of one tile splits its keys in two streams)
  int cost_one, cost_two;       // units of a key tile with one tile of queries, and with two
  int slot_rows;                // rows of a CTA's partial slot
  int grid;                     // CTAs of the schedule
  // workspace
  long long* plan;              // [0] U, [1 + b] first unit of sequence b (b = -1 starts at 0)
  float* part_o;                // attention: [row slots | CTA slots][D]
  float2* part_ml;              // their running maximum (base-2 logit) and sum
  float* part_w;                // weights: [CTA][slot_rows] sums of continued items
  int4* part_id;                // weights: [CTA] (b, h, key block, 1 when it continues an item)
};

struct SeqView {
  int r0, n, len;               // first row, rows, keys
};

__device__ __forceinline__ int paged_cap(const PagedParams& p) { return p.max_pages << p.page_shift; }

// x / y (neither negative) in 32 bits where they hold both.
__device__ __forceinline__ long long quotient(long long x, long long y) {
  if ((x | y) >> 32 == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}
// Sequence b (-1: the prefix and the whole batch's rows), clamped into the tensors.
__device__ __forceinline__ SeqView seq_view(const PagedParams& p, int b) {
  SeqView v;
  const int lo = __ldcg(p.row_start + (b < 0 ? 0 : b));
  const int hi = __ldcg(p.row_start + (b < 0 ? p.B : b + 1));
  v.r0 = min(max(lo, 0), p.rows);
  v.n = min(max(hi, v.r0), p.rows) - v.r0;
  v.len = b < 0 ? p.prefix_tokens : min(max(__ldcg(p.lengths + b), 0), paged_cap(p));
  return v;
}
// Latch an error when sequence b's length or rows are outside its tensors.
__device__ __forceinline__ void seq_check(const PagedParams& p, int b) {
  const int lo = p.row_start[b], hi = p.row_start[b + 1], len = p.lengths[b];
  if (lo < 0 || hi < lo || hi > p.rows || len < 0 || len > paged_cap(p)) latch_error(p.err, DERR_BOUNDS);
}

__device__ __forceinline__ int item_tokens(const PagedParams& p, int b) {
  return b < 0 ? p.prefix_item_tokens : p.item_tokens;
}
__device__ __forceinline__ int seq_items(const PagedParams& p, int b, const SeqView& v) {
  const int it = item_tokens(p, b);
  return (v.n + it - 1) / it;
}
// Key tiles of the prefix that each item reads before its own (p.join).
__device__ __forceinline__ int prefix_tiles(const PagedParams& p) { return p.join ? p.prefix_units : 0; }
// Own keys that some row among the first t tokens of the sequence sees.
__device__ __forceinline__ int keys_before(const PagedParams& p, int b, const SeqView& v, int t) {
  return b >= 0 && p.causal ? min(v.len, max(0, v.len - v.n + t)) : v.len;
}
// Key tiles of item i, and the units of each.
__device__ __forceinline__ int item_tiles(const PagedParams& p, int b, const SeqView& v, int i) {
  const int t = min(v.n, (i + 1) * item_tokens(p, b));
  return prefix_tiles(p) + ((keys_before(p, b, v, t) + p.key_tile - 1) >> p.key_shift);
}
__device__ __forceinline__ bool two_tiles(const PagedParams& p, const SeqView& v, int i) {
  return p.streams == 2 && v.n - i * p.item_tokens > p.tile_tokens;
}
__device__ __forceinline__ int tile_cost(const PagedParams& p, const SeqView& v, int i) {
  return two_tiles(p, v, i) ? p.cost_two : p.cost_one;
}
// sum over j < n of floor((a j + b) / m), for a, b >= 0, by the known Euclid-like floor sum: whole
// multiples of m come out in closed
// form, and the rest counts lattice points under a line, which is the same sum with a and m
// exchanged and fewer terms (the steps of Euclid's algorithm on a and m).
// Every value stays below 2^32: rows and keys of a sequence do.
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  long long s = 0;
#pragma unroll 1
  for (;;) {
    s += static_cast<long long>(a / m) * (static_cast<long long>(n) * (n - 1) / 2) +
         static_cast<long long>(b / m) * n;
    a %= m;
    b %= m;
    const uint32_t top = a * n + b;
    if (top < m) return s;
    n = top / m;
    b = top % m;
    const uint32_t x = a;
    a = m;
    m = x;
  }
}
// Units of a sequence's items [0, i) for one head.
__device__ __forceinline__ long long units_before(const PagedParams& p, int b, const SeqView& v, int i) {
  if (i <= 0) return 0;
  // items before the last are full
  const int last = seq_items(p, b, v) - 1, whole = min(i, last);
  const int full = p.streams == 2 ? p.cost_two : p.cost_one;
  long long s;
  if (b < 0 || !p.causal) {
    s = static_cast<long long>(whole) * item_tiles(p, b, v, 0) * full;
  } else {
    // they see len - n + (j + 1) item_tokens keys, none while that is negative
    const int it = p.item_tokens, first = v.len - v.n;
    const int skip = first < 0 ? min(whole, -first / it) : 0;
    s = static_cast<long long>(whole) * prefix_tiles(p);
    if (whole > skip) s += floor_sum(whole - skip, p.key_tile, it, first + (skip + 1) * it + p.key_tile - 1);
    s *= full;
  }
  if (i > whole) s += static_cast<long long>(item_tiles(p, b, v, last)) * tile_cost(p, v, last);
  return s;
}
__device__ __forceinline__ long long head_units(const PagedParams& p, int b, const SeqView& v) {
  return units_before(p, b, v, seq_items(p, b, v));
}

// The schedule's walk through a CTA's units.
struct Segment {
  int b, h, i;                  // sequence, KV head, item
  SeqView v;
  int k0, k1, nk;               // key tiles [k0, k1) of the item's nk
  bool two;                     // the item has two tiles of query tokens
  int phase;                    // which stream takes the first tile of an item that has one
};
// Key tile kt of an item: the sequence whose pages hold it (-1: the prefix), its first key there
// and that sequence's keys.
struct KeyTile {
  int b, key0, len;
};
__device__ __forceinline__ KeyTile key_tile_at(const PagedParams& p, const Segment& g, int kt) {
  const int before = prefix_tiles(p);
  if (kt < before) return {-1, kt * p.key_tile, p.prefix_tokens};
  return {g.b, (kt - before) * p.key_tile, g.v.len};
}
struct Walk {
  long long u, u1;              // units left
  long long item_first;         // first unit of the item (b, h, i)
  int b, h, i;
  SeqView v, next;              // sequence b, and b + 1 loaded ahead
  int items;
};
__device__ __forceinline__ void walk_to(const PagedParams& p, Walk& w, int b) {
  w.b = b;
  w.items = seq_items(p, b, w.v);
  if (b + 1 < p.B) w.next = seq_view(p, b + 1);
}

// The first unit of every sequence, and this CTA's place in them. units_of_head(b, view) gives the
// units of one head of sequence b. Of 32 sequences any warp finds out by itself (plan_by_warp), and
// only a warp that needs the walk calls this (a decode step of 4: 15.6 us block-wide, 14.7 so; of 64
// with two or three to a lane: 70 and 74); else every thread of the block does. s must hold
// kPlanWords + blockDim.x / 32 long longs. CTA 0 writes the plan. (The schedule is written for
// little code, one place for each computation and no unrolling: it runs once, from a cold cache.)
constexpr int kPlanWords = 5;
__device__ __forceinline__ int first_sequence(const PagedParams& p) { return p.prefix_tokens > 0 && !p.join ? -1 : 0; }
__device__ __forceinline__ bool plan_by_warp(const PagedParams& p) { return p.B - first_sequence(p) <= 32; }
template <typename HeadUnits>
__device__ __forceinline__ Walk plan_walk(const PagedParams& p, long long* s, HeadUnits&& units_of_head) {
  const bool alone = plan_by_warp(p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int nt = alone ? 32 : blockDim.x, t = alone ? lane : threadIdx.x;
  const int b_first = first_sequence(p);
  const int n_seq = p.B - b_first;
  const int per = alone ? 1 : (n_seq + nt - 1) / nt;
  const int b0 = b_first + min(n_seq, t * per), b1 = b_first + min(n_seq, (t + 1) * per);
  long long at = 0, units = 0, U = 0, u0 = 0, u1 = 0;      // at: units before sequence b
  SeqView view{};
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      if (pass == 0 || per > 1) {              // else they are at hand
        view = seq_view(p, b);
        units = units_of_head(b, view);
      }
      const long long x = p.Hkv * units;
      if (pass == 1) {
        if (blockIdx.x == 0 && b >= 0) {
          seq_check(p, b);
          p.plan[1 + b] = at;
        }
        if (u0 < u1 && u0 >= at && u0 < at + x) {          // this CTA begins here
          s[0] = at;
          s[1] = b;
          s[2] = (static_cast<long long>(view.n) << 32) | static_cast<uint32_t>(view.r0);
          s[3] = view.len;
          s[4] = units;
        }
      }
      at += x;
    }
    if (pass == 0) {
      const long long mine = at;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, at, d);
        if (lane >= d) at += o;
      }
      long long total = __shfl_sync(0xffffffffu, at, 31);
      at -= mine;
      if (!alone) {                            // the warps' sums, a lane for each
        if (lane == 0) s[kPlanWords + warp] = total;
        __syncthreads();
        long long x = lane < warps ? s[kPlanWords + lane] : 0, y = lane < warp ? x : 0;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
          x += __shfl_xor_sync(0xffffffffu, x, d);
          y += __shfl_xor_sync(0xffffffffu, y, d);
        }
        total = x;
        at += y;
      }
      U = max(quotient(total + p.grid - 1, p.grid), static_cast<long long>(p.cost_two));
      u0 = min(total, U * blockIdx.x);
      u1 = min(total, u0 + U);
    }
  }
  if (blockIdx.x == 0 && t == 0) p.plan[0] = U;
  // (several warps that are alone write the same)
  if (alone) __syncwarp();
  else __syncthreads();
  Walk w{};
  w.u = u0;
  w.u1 = u1;
  if (u0 < u1) {
    const int b = static_cast<int>(s[1]);
    w.v = {static_cast<int>(s[2]), static_cast<int>(s[2] >> 32), static_cast<int>(s[3])};
    walk_to(p, w, b);
    w.h = static_cast<int>(quotient(u0 - s[0], s[4]));
    w.item_first = s[0] + w.h * s[4];
    w.i = 0;
  }
  return w;
}
// To the item that holds the walk's first unit (attention; a search over the items' first units).
__device__ __forceinline__ void walk_to_item(const PagedParams& p, Walk& w) {
  if (w.u >= w.u1) return;
  const long long rel = w.u - w.item_first;
  long long before = 0;
  int lo = 0, hi = w.items;                    // units_before(lo) <= rel < units_before(hi)
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const long long x = units_before(p, w.b, w.v, mid);
    if (x <= rel) {
      lo = mid;
      before = x;
    } else {
      hi = mid;
    }
  }
  w.item_first += before;
  w.i = lo;
}

// Tiles of an item whose first unit lies in its first n.
__device__ __forceinline__ int tiles_before(int n, int cost) {
  return cost == 1 ? n : static_cast<int>(static_cast<uint32_t>(n + cost - 1) / static_cast<uint32_t>(cost));
}
// The next piece of one item in the CTA's units (attention).
__device__ __forceinline__ bool next_segment(const PagedParams& p, Walk& w, Segment& g) {
#pragma unroll 1
  while (w.u < w.u1) {
    if (w.i >= w.items) {
      w.i = 0;
      if (++w.h >= p.Hkv) {
        w.h = 0;
        w.v = w.next;
        walk_to(p, w, w.b + 1);
      }
      continue;
    }
    const int nk = item_tiles(p, w.b, w.v, w.i), cost = tile_cost(p, w.v, w.i);
    // the tiles whose first unit lies in [u, u1)
    const long long end = w.item_first + nk * cost;
    if (w.u > end - cost) {
      w.u = max(w.u, end);
      w.item_first = end;
      ++w.i;
      continue;
    }
    const int k0 = tiles_before(static_cast<int>(w.u - w.item_first), cost);
    const int k1 = tiles_before(static_cast<int>(min(end, w.u1) - w.item_first), cost);
    if (k1 <= k0) return false;
    g.b = w.b;
    g.h = w.h;
    g.i = w.i;
    g.v = w.v;
    g.k0 = k0;
    g.k1 = k1;
    g.nk = nk;
    g.two = two_tiles(p, w.v, w.i);
    w.u = w.item_first + k1 * cost;
    return true;
  }
  return false;
}

// Waits for phase `parity` of `bar`, giving up after a limit or as soon as another role of the CTA
// has: then *abort is set (the kernel's end latches the error, report_abort) and false returned, and the
// caller leaves its loop. A kernel has some forty of these, so they are kept short: its code is to
// fit the instruction cache.
template <bool kDrain>
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (!kDrain && *abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_near(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return wait_on<false>(bar, parity, abort, KVC_WAIT_LIMIT_NS);
}
// For something a whole segment away, which may pass the usual limit: a sequence's 2^22 key tiles
// take some 10 s.
__device__ __forceinline__ bool wait_segment(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return wait_on<false>(bar, parity, abort, 30 * KVC_WAIT_LIMIT_NS);
}
// For a CTA's own work in flight, whoever gave up.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity, volatile int* abort) {
  wait_on<true>(bar, parity, abort, KVC_WAIT_LIMIT_NS);
}
// Behind the block's last barrier.
__device__ __forceinline__ void report_abort(const PagedParams& p, const volatile int* abort) {
  if (threadIdx.x == 0 && *abort) latch_error(p.err, DERR_TIMEOUT);
}

// Segments handed from the warp that walks the schedule to the others of its CTA.
constexpr int kRing = 8;
struct SegmentRing {
  uint64_t full[kRing], empty[kRing];
  int4 a[kRing], b[kRing], c[kRing];
};
__device__ __forceinline__ void ring_init(SegmentRing& r, int readers) {
  for (int i = 0; i < kRing; ++i) {
    mbar_init(&r.full[i], 1);
    mbar_init(&r.empty[i], readers);
  }
}
// The k-th segment into the ring (one thread).
__device__ __forceinline__ bool ring_put(SegmentRing& r, int k, const Segment& g, volatile int* abort) {
  const int i = k % kRing;
  if (k >= kRing && !wait_segment(&r.empty[i], ((k / kRing) - 1) & 1, abort)) return false;
  r.a[i] = make_int4(g.b, g.h, g.i, g.two);
  r.b[i] = make_int4(g.v.r0, g.v.n, g.v.len, g.nk);
  r.c[i] = make_int4(g.k0, g.k1, g.phase, 0);
  mbar_arrive(&r.full[i]);
  return true;
}
__device__ __forceinline__ Segment ring_peek(const SegmentRing& r, int k) {
  const int i = k % kRing;
  const int4 a = r.a[i], b = r.b[i], c = r.c[i];
  return {a.x, a.y, a.z, {b.x, b.y, b.z}, c.x, c.y, b.w, a.w != 0, c.z};
}
// The k-th segment out of it (a warp; the same answer in every lane).
__device__ __forceinline__ bool ring_take(SegmentRing& r, int k, Segment& g, volatile int* abort) {
  const int i = k % kRing;
  const bool ok = wait_segment(&r.full[i], (k / kRing) & 1, abort);
  if (!__all_sync(0xffffffffu, ok)) return false;
  g = ring_peek(r, k);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&r.empty[i]);
  return true;
}

// Physical page of key `slot` of sequence b; -1 (and an error) when the table names none.
__device__ __forceinline__ long long page_of(const PagedParams& p, int b, int slot) {
  const int k = slot >> p.page_shift;
  const int32_t page = b < 0 ? __ldg(p.prefix_pages + k)
                             : __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + k);
  if (page < 0 || page >= p.pool_pages) {
    latch_error(p.err, DERR_BOUNDS);
    return -1;
  }
  return page;
}
// Row of the pool (rows of D elements) that holds key `slot` of sequence b for KV head h, or -1.
__device__ __forceinline__ long long pool_row(const PagedParams& p, int b, int h, int slot) {
  const long long page = page_of(p, b, slot);
  return page < 0 ? -1 : (((page * p.Hkv + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1)));
}
// Keys that token t of the sequence sees.
__device__ __forceinline__ int key_limit(const PagedParams& p, int b, const SeqView& v, int t) {
  return b >= 0 && p.causal ? min(v.len, max(0, v.len - v.n + t + 1)) : v.len;
}

// Parts of a row's keys: the prefix and its own, or both in one.
__host__ __device__ __forceinline__ int parts_of(const PagedParams& p) { return p.prefix_tokens > 0 && !p.join ? 2 : 1; }
// Partial slots. Row slots: [part][stream][row][query head]; CTA slots after them.
__host__ __device__ __forceinline__ long long row_slots(const PagedParams& p) {
  return static_cast<long long>(parts_of(p)) * p.streams * p.rows * p.Hq;
}
__device__ __forceinline__ long long row_slot(const PagedParams& p, int b, int stream, int row, int hq) {
  const int part = parts_of(p) == 2 && b >= 0 ? 1 : 0;
  return ((static_cast<long long>(part) * p.streams + stream) * p.rows + row) * p.Hq + hq;
}
__device__ __forceinline__ long long cta_slot(const PagedParams& p, int cta, int r) {
  return row_slots(p) + static_cast<long long>(cta) * p.slot_rows + r;
}
// Whether an item's rows are written to O by the CTA that has all of its keys: two tiles (a
// stream each) or one stream, and no other part.
__device__ __forceinline__ bool writes_rows(const PagedParams& p, const SeqView& v, int item) {
  return parts_of(p) == 1 && (p.streams == 1 || two_tiles(p, v, item));
}

// Sequence whose rows hold `row` (row_start[b] <= row < row_start[b + 1]), or -1; warp-wide.
__device__ __forceinline__ int find_sequence(const int32_t* row_start, int B, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B + 1;                                 // row_start entries [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool le = at < n && __ldcg(row_start + lo + at) <= row;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0) return -1;
    const int k = 31 - __clz(m);
    lo += k * step;
    n = min(step, n - k * step);
  }
  if (lo >= B) return -1;
  return __ldcg(row_start + lo) <= row && row < __ldcg(row_start + lo + 1) ? lo : -1;
}

// Weights: a unit is one key block (key_tile keys of a sequence, one KV head) with one tile of
// query tokens, tiles running fastest, so that a key block's sums stay in a CTA.
__device__ __forceinline__ long long weight_head_units(const PagedParams& p, const SeqView& v) {
  return static_cast<long long>((v.len + p.key_tile - 1) >> p.key_shift) *
         ((v.n + p.tile_tokens - 1) / p.tile_tokens);
}
struct WeightSegment {
  int b, h, kb;                 // sequence, KV head, key block
  SeqView v;
  int t0, t1;                   // query tiles [t0, t1)
};
__device__ __forceinline__ bool next_weight_segment(const PagedParams& p, Walk& w, WeightSegment& g) {
#pragma unroll 1
  while (w.u < w.u1) {
    const long long uph = weight_head_units(p, w.v);
    if (w.u >= w.item_first + uph) {
      w.item_first += uph;
      if (++w.h >= p.Hkv) {
        w.h = 0;
        w.v = w.next;
        walk_to(p, w, w.b + 1);
      }
      continue;
    }
    const int tiles = (w.v.n + p.tile_tokens - 1) / p.tile_tokens;
    const long long rel = w.u - w.item_first;
    g.b = w.b;
    g.h = w.h;
    g.v = w.v;
    g.kb = static_cast<int>(quotient(rel, tiles));
    g.t0 = static_cast<int>(rel - static_cast<long long>(g.kb) * tiles);
    g.t1 = static_cast<int>(min(static_cast<long long>(tiles), g.t0 + (w.u1 - w.u)));
    w.u += g.t1 - g.t0;
    return true;
  }
  return false;
}

// ------------------------------------------------------------------ launchers
// Tensor maps of the bf16 kernels. Query rows as (dims, heads, rows), one box a 64-dim half of
// the G heads of tile_tokens rows; pool slots as (64 dims, 8 rows, halves, eights of rows), one
// box a page's slots (128 of them at most).
bool encode_rows_tmap(CUtensorMap* map, const void* rows_dev, const PagedParams& p);
bool encode_slots_tmap(CUtensorMap* map, const void* pool, const PagedParams& p);

cudaError_t launch_paged_attend_tc(cudaStream_t s, const PagedParams& p);
cudaError_t launch_paged_attend_simt(cudaStream_t s, const PagedParams& p);
cudaError_t launch_paged_weights_tc(cudaStream_t s, const PagedParams& p);
cudaError_t launch_paged_weights_simt(cudaStream_t s, const PagedParams& p);
struct EvictParams {
  int B, Hkv, page_shift, max_pages, row_bytes;
  int keep, sinks, recent;
  long long pool_pages;
  const int32_t* page_table;
  const int32_t* lengths;
  const int32_t* next_positions;
  uint8_t* k_pool;
  uint8_t* v_pool;
  float* scores;
  int32_t* positions;
  int32_t* counts;              // workspace: [B * Hkv] moves, -1 where nothing is evicted
  int2* moves;                  // workspace: [B * Hkv][2][move_cap] (slot, pool row) moved to and from
  int move_cap;
  int* err;
};
int paged_evict_max_slots();
cudaError_t launch_paged_evict(cudaStream_t s, const EvictParams& p, int sms, int32_t* lengths);

}  // namespace kvc
