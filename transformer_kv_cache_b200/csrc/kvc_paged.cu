// kvc_paged.cu -- the paged-batch entry points (kvc_paged_*): argument checks, workspace,
// the append and the merge of partial attention results.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "kvc_paged.cuh"

namespace kvc {
namespace {

constexpr int kMaxGroup = 64;                  // query heads per KV head
// A CTA appends a sequence's rows in one launch up to kFewRows a sequence, on average, and kFewBytes of K
// and V in all, since one sequence may have nearly all of them, which one SM then copies at some 40 GB/s. Against
// the form of two launches (rows of 4 KB; 2.5 us of each are copies that reset the lengths): 64 sequences'
// single rows 4.7 for 6.5 us, their 8 rows 5.8 for 7.5; one of 193 rows beside 63 single ones 25 for 7.4, and
// above the limit one of 449 49 for 7.2, 1,024 single rows 11.5 for 8.7 (though 256 sequences' 8 rows 6.7 for 10.1).
constexpr int kFewRows = 8;
constexpr long long kFewBytes = 1 << 20;
constexpr int kManyHeads = 8192;               // rows x heads from which on the merge packs four into a warp
constexpr long long kMaxSlots = 1LL << 29;     // slots of a sequence, tokens of the prefix: their sum is an int

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; }

bool valid_batch(const kvc_paged_batch* b) {
  if (!b) return false;
  if (b->dtype != KVC_F32 && b->dtype != KVC_BF16) return false;
  if (b->head_dim != 64 && b->head_dim != 128) return false;
  const int P = b->page_size;
  if (P < 16 || P > 256 || (P & (P - 1))) return false;
  if (b->num_seqs < 1 || b->num_seqs > 65535 || b->num_kv_heads < 1 || b->num_q_heads < 1 ||
      b->num_q_heads > 65535 || b->num_q_heads % b->num_kv_heads || b->num_q_heads / b->num_kv_heads > kMaxGroup)
    return false;
  if (b->max_pages < 1 || b->max_pages > kMaxSlots / P || b->pool_pages < 1) return false;
  // pool rows (pages x heads x slots) index the tensor maps as int
  if (b->pool_pages > INT_MAX / (static_cast<long long>(b->num_kv_heads) * P)) return false;
  if (b->prefix_tokens < 0 || b->prefix_tokens > kMaxSlots || (b->prefix_tokens > 0 && !b->prefix_pages)) return false;
  if (!(b->softmax_scale > 0.f) || !std::isfinite(b->softmax_scale) || b->reserved != 0) return false;
  if (!b->k_pool || !b->v_pool || !b->page_table || !b->lengths) return false;
  if (b->next_positions == b->lengths) return false;        // both grow by an append's rows
  return aligned16(b->k_pool) && aligned16(b->v_pool) && aligned16(b->scores) && aligned16(b->positions);
}

int page_shift(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

bool valid_rows(const kvc_paged_batch* b, const void* x, long long stride, int heads, int32_t rows) {
  if (rows < 0 || !aligned16(x) || (rows > 0 && !x)) return false;
  const int per16 = b->dtype == KVC_F32 ? 4 : 8;
  return stride >= static_cast<long long>(heads) * b->head_dim && stride % per16 == 0 && stride <= (1LL << 36);
}

// ------------------------------------------------------------------ the schedule and its workspace
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
  size_t plan, part_o, part_ml, part_w, part_id, bytes;
};

PagedParams base_params(const kvc_paged_batch* b, int32_t rows, const int32_t* row_start, int sms) {
  PagedParams p{};
  p.B = b->num_seqs;
  p.Hq = b->num_q_heads;
  p.Hkv = b->num_kv_heads;
  p.G = p.Hq / p.Hkv;
  p.D = b->head_dim;
  p.page_shift = page_shift(b->page_size);
  p.max_pages = b->max_pages;
  p.rows = rows;
  p.pool_pages = b->pool_pages;
  p.page_table = b->page_table;
  p.lengths = b->lengths;
  p.prefix_pages = b->prefix_pages;
  p.row_start = row_start;
  p.k_pool = b->k_pool;
  p.v_pool = b->v_pool;
  p.scale_log2 = b->softmax_scale * 1.4426950408889634f;
  p.err = b->error;
  p.grid = sms;
  p.cost_one = p.cost_two = 1;
  return p;
}

void attend_schedule(PagedParams* p, const kvc_paged_batch* b) {
  p->prefix_tokens = b->prefix_tokens;
  p->prefix_units = (b->prefix_tokens + (b->dtype == KVC_BF16 ? 128 : 64) - 1) / (b->dtype == KVC_BF16 ? 128 : 64);
  // Where the sequences' rows fill their items (on average), packing the batch's rows saves no
  // pass over the prefix: each item then reads the prefix before its own keys, and its rows'
  // partials need no joining with those of a second item. No sequence's rows are known here, so that in a
  // mixed batch the others read the prefix for themselves too; B of them at most, beside a chunk of
  // about B items that read it anyway. 32 heads on 8 of 128 dims behind 16,384 tokens, joined and not: 64
  // sequences of 64 rows 1,040 us and 1,366, 15 single rows and one of 1,100 480 and 504, 63 and one of
  // 4,100 1,668 and 1,356.
  if (b->dtype == KVC_BF16) {
    // two tiles of 128 packed rows share a CTA's key tiles
    p->tile_tokens = 128 / p->G;
    p->item_tokens = p->prefix_item_tokens = 2 * p->tile_tokens;
    p->key_tile = 128;
    p->key_shift = 7;
    p->streams = 2;
    p->slot_rows = 256;
    // a key tile's time with two tiles of queries to its time with one (2.4 to 1.46 us with 128
    // dims); with one alone where no item has more
    p->cost_one = p->rows > p->tile_tokens ? 3 : 1;
    p->cost_two = p->rows > p->tile_tokens ? 5 : 1;
    p->join = p->prefix_tokens > 0 && p->rows >= static_cast<long long>(p->B) * p->item_tokens;
    return;
  }
  // Tiles of 16 query rows where a sequence has no more (a 64-row tile of them would spend its
  // products on padding), else of 64. The prefix's of 16 up to two of them (8 sequences' row of 4 heads
  // each behind 1,500 tokens: 22.5 us, in one tile of 64 26), of 64 from there on (at 31 tokens 29 us, in
  // tiles of 16 33). A chunk among single rows is faster in the small tiles as well (63 rows of one and one of 900:
  // 237 us, in tiles of 64 309).
  const long long all = static_cast<long long>(p->rows) * p->G;
  const int few = p->G <= 16 && (all + p->B - 1) / p->B <= 16 ? 16 : 64;
  const int prefix = few == 16 && all <= 32 ? 16 : 64;
  p->tile_tokens = p->item_tokens = few / p->G;
  p->prefix_item_tokens = prefix / p->G;
  p->slot_rows = std::max(few, p->prefix_tokens > 0 ? prefix : 16);
  p->key_tile = 64;
  p->key_shift = 6;
  p->streams = 1;
  p->join = p->prefix_tokens > 0 && p->rows >= static_cast<long long>(p->B) * p->item_tokens && few == 64;
  if (p->D == 64) p->grid *= 2;                // CTAs that fit an SM
}

void weights_schedule(PagedParams* p, const kvc_paged_batch* b) {
  p->prefix_tokens = 0;                        // the prefix keeps no scores
  if (b->dtype == KVC_BF16) {
    p->tile_tokens = p->item_tokens = 128 / p->G;
    p->key_tile = p->slot_rows = 256;
    p->key_shift = 8;
    p->streams = 1;
    return;
  }
  // tiles of 32 rows, of which only fours that there are cost anything, where a sequence has no more
  // (16 sequences of 4 rows of 6 heads: 82 us, in tiles of 64 120; of 4 heads' one row: 75, in 16 72)
  const long long per_seq = (static_cast<long long>(p->rows) + p->B - 1) / p->B * p->G;
  p->tile_tokens = p->item_tokens = (per_seq <= 32 ? 32 : 64) / p->G;
  p->key_tile = 64;
  p->key_shift = 6;
  p->streams = 1;
  p->slot_rows = p->key_tile;
  p->grid *= 2;                                // CTAs that fit an SM
}

Layout attend_layout(const PagedParams& p) {
  Layout l{};
  const size_t slots = static_cast<size_t>(row_slots(p)) +
                       static_cast<size_t>(p.grid) * p.slot_rows;
  l.plan = 0;
  l.part_ml = align256(8 * (static_cast<size_t>(p.B) + 1));
  l.part_o = l.part_ml + align256(slots * sizeof(float2));
  l.bytes = l.part_o + align256(slots * p.D * sizeof(float));
  return l;
}

Layout weights_layout(const PagedParams& p) {
  Layout l{};
  l.plan = 0;
  l.part_id = align256(8 * (static_cast<size_t>(p.B) + 1));
  l.part_w = l.part_id + align256(static_cast<size_t>(p.grid) * sizeof(int4));
  l.bytes = l.part_w + align256(static_cast<size_t>(p.grid) * p.slot_rows * sizeof(float));
  return l;
}

int move_cap(const kvc_paged_batch* b, int32_t keep) {
  const long long cap = static_cast<long long>(b->max_pages) * b->page_size;
  return static_cast<int>(std::min<long long>(keep, std::max<long long>(cap - keep, 0)));
}
size_t evict_counts_bytes(const kvc_paged_batch* b) {
  return align256(sizeof(int32_t) * static_cast<size_t>(b->num_seqs) * b->num_kv_heads);
}
size_t evict_bytes(const kvc_paged_batch* b, int32_t keep) {
  return evict_counts_bytes(b) +
         align256(sizeof(int2) * 2 * static_cast<size_t>(b->num_seqs) * b->num_kv_heads * move_cap(b, keep));
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr)
               : nullptr;
  }();
  return fn;
}

// ------------------------------------------------------------------ append
struct AppendParams {
  int B, H, page_shift, max_pages, rows, row_bytes;   // row_bytes: one head's
  long long pool_pages, k_stride, v_stride;           // bytes between source rows
  const int32_t* page_table;
  int32_t* lengths;
  int32_t* next_positions;
  const int32_t* row_start;
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* k_pool;
  uint8_t* v_pool;
  float* scores;
  int32_t* positions;
  int* err;
  int behind_warps;                                   // of a sequence, for the slots behind its last token
};

// Slots to clear behind a sequence's last token, where the call begins that page (every page of the
// cache ends in zeros).
__device__ __forceinline__ int append_behind(const AppendParams& p, int n, int len) {
  const int page_size = 1 << p.page_shift, end = len + n, first = end & ~(page_size - 1);
  return n == 0 || end == first || first < len ? 0 : first + page_size - end;
}
// One task of a sequence (a warp): task i < n copies its i-th row, the tasks behind those clear a
// slot behind its last token each. 16 bytes a lane.
__device__ __forceinline__ void append_task(const AppendParams& p, int b, int lo, int n, int len, int task) {
  const int lane = threadIdx.x & 31, page_size = 1 << p.page_shift;
  const bool copy = task < n;
  const int slot = len + task;
  const int32_t page = __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + (slot >> p.page_shift));
  if (page < 0 || page >= p.pool_pages) {
    if (lane == 0) latch_error(p.err, DERR_BOUNDS);
    return;
  }
  const int per_head = p.row_bytes >> 4, chunks = p.H * per_head;
  const long long head_bytes = static_cast<long long>(p.row_bytes) << p.page_shift;
  const long long base = page * p.H * head_bytes + (slot & (page_size - 1)) * static_cast<long long>(p.row_bytes);
  const long long row = lo + task;
  const uint4* k = reinterpret_cast<const uint4*>(p.k + (copy ? row * p.k_stride : 0));
  const uint4* v = reinterpret_cast<const uint4*>(p.v + (copy ? row * p.v_stride : 0));
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 4
  for (int c = lane; c < chunks; c += 32) {
    const long long to = base + (c / per_head) * head_bytes + (c % per_head) * 16;
    *reinterpret_cast<uint4*>(p.k_pool + to) = copy ? __ldg(k + c) : zero;
    *reinterpret_cast<uint4*>(p.v_pool + to) = copy ? __ldg(v + c) : zero;
  }
  if (!copy) return;
  const int cap = p.max_pages << p.page_shift;
  const int position = p.positions ? p.next_positions[b] + task : 0;
  for (int h = lane; h < p.H; h += 32) {
    const long long at = (static_cast<long long>(b) * p.H + h) * cap + slot;
    if (p.scores) p.scores[at] = 0.f;
    if (p.positions) p.positions[at] = position;
  }
}
// A sequence's rows and length; false (and an error) where they are out of range, would take the next
// position out of it (2^31 is passed by a day of frames), or do not fit.
__device__ __forceinline__ bool append_view(const AppendParams& p, int b, int& lo, int& n, int& len) {
  lo = p.row_start[b];
  const int hi = p.row_start[b + 1], cap = p.max_pages << p.page_shift;
  len = p.lengths[b];
  n = hi - lo;
  const int next = p.next_positions ? p.next_positions[b] : 0;
  const bool in = lo >= 0 && hi >= lo && hi <= p.rows && len >= 0 && len <= cap && next <= INT_MAX - n;
  if (in && n <= cap - len) return true;
  latch_error(p.err, in ? DERR_POOL : DERR_BOUNDS);
  return false;
}
__device__ __forceinline__ void grow(const AppendParams& p, int b, int n, int len) {
  p.lengths[b] = len + n;
  if (p.next_positions) p.next_positions[b] += n;
}

// A CTA per sequence, which then grows by its rows. Bound by its chain of loads (rows, lengths, table,
// rows): 64 sequences, 3 to 5 rows of 8 heads of 128 dims each (3 MB): 4 us.
__global__ void __launch_bounds__(512) paged_append_few_kernel(const AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x, warps = blockDim.x >> 5;
  int lo, n, len;
  if (!append_view(p, b, lo, n, len)) return;
  const int tasks = n + append_behind(p, n, len);
  for (int task = threadIdx.x >> 5; task < tasks; task += warps) append_task(p, b, lo, n, len, task);
  __syncthreads();
  if (threadIdx.x == 0) grow(p, b, n, len);
}

// A warp per row of the batch, and `behind_warps` a sequence for the slots behind its last token; the
// lengths grow in a kernel of their own, once nobody reads the old ones. 2 x 1,004 rows of 16 heads of 64 dims (16 MB): 6 us, half
// of them the two launches.
__global__ void __launch_bounds__(256) paged_append_kernel(const AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int z = warp - p.rows;
  const int b = z < 0 ? find_sequence(p.row_start, p.B, warp) : z / p.behind_warps;
  if (b < 0 || b >= p.B) return;                       // behind the last sequence
  int lo, n, len;
  if (!append_view(p, b, lo, n, len)) return;
  if (z < 0) {
    append_task(p, b, lo, n, len, warp - lo);
    return;
  }
  const int behind = append_behind(p, n, len);
  for (int i = z % p.behind_warps; i < behind; i += p.behind_warps) append_task(p, b, lo, n, len, n + i);
}
__global__ void paged_grow_kernel(const AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  int lo, n, len;
  if (b < p.B && append_view(p, b, lo, n, len)) grow(p, b, n, len);
}

// ------------------------------------------------------------------ merging partial results
// LANES lanes per (row, query head): O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i over the row's
// partials in the order of their keys, LSE = ln 2 (M + log2 of that sum). A row that sees no key
// gets O = 0 and LSE = -inf. Rows that their CTA wrote itself are left alone. What the row needs
// of the batch is read before the wait for the attention kernel (which had waited for whatever
// wrote it), the partials after it.
// Bound by its chain of loads: some 4 us behind a step of 4 sequences, 7 behind one of 64 with a prefix.
template <typename T, int D, int LANES>
__global__ void __launch_bounds__(128) paged_merge_kernel(const PagedParams p) {
  constexpr int kPer = D / LANES;                      // dims of a lane, as vectors of kVec
  constexpr int kVec = kPer < 4 ? kPer : 4;
  const int lane = threadIdx.x % LANES;
  const int row = blockIdx.x, hq = (blockIdx.y * 128 + threadIdx.x) / LANES;
  const int b = find_sequence(p.row_start, p.B, row);
  const int h = hq / p.G, g = hq % p.G;
  const int parts = parts_of(p);
  // Half of the lanes look up the row's part of the prefix, the others its own (one place in the code
  // for both): the item's units up to its last key tile's first, its first unit (without the
  // sequence's), and the row's place.
  const bool second = lane >= LANES / 2;
  int nk = 0, place = 0;                               // row of the tile << 2 | tile << 1 | the keys are split
  long long first = 0;
  bool whole = false, mine = hq < p.Hq;
  if (b >= 0 && (second || parts == 2)) {
    const int s = second ? b : -1;
    const SeqView v = seq_view(p, s);
    const int t = row - v.r0;
    if (t >= 0 && t < v.n) {
      const int it = item_tokens(p, s), item = t / it, in = t - item * it;
      const int tiles = item_tiles(p, s, v, item);
      if (tiles > 0) nk = (tiles - 1) * tile_cost(p, v, item) + 1;
      // the heads before, then the items before
#pragma unroll 1
      for (int k = 0; k < 2; ++k)
        first += (k == 0 ? h : 1) * units_before(p, s, v, k == 0 ? seq_items(p, s, v) : item);
      const int tile = p.streams == 2 ? in / p.tile_tokens : 0;
      place = ((in - tile * p.tile_tokens) * p.G + g) << 2 | tile << 1 | (p.streams == 2 && !two_tiles(p, v, item));
      whole = second && writes_rows(p, v, item);
    }
  }
  griddep_wait();
  griddep_launch_dependents();
  if (b < 0) return;                                   // behind the last sequence: left as it was
  // (a call that wrongly runs beside another with the same workspace merges other partials, but reads
  // none outside of it: the CTAs are bounded)
  const long long U = max(__ldcg(p.plan), 1LL), own = __ldcg(p.plan + 1 + b);
  // the partials in the order of their keys: per part its CTAs' pieces, per piece its streams
  int c = 0, n = 0;
  if (nk > 0) {
    const long long u0 = first + (second ? own : 0);
    int end = 0;                                       // its CTA, then that of the first unit
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      end = c;
      c = static_cast<int>(min(quotient(max(k == 0 ? u0 + nk - 1 : u0, 0LL), U), p.grid - 1LL));
    }
    const int pieces = max(end - c, 0) + 1;
    n = pieces == 1 && whole ? -1 : pieces << (place & 1);
  }
  const int c0 = __shfl_sync(0xffffffffu, c, 0, LANES), c1 = __shfl_sync(0xffffffffu, c, LANES / 2, LANES);
  const int n0 = __shfl_sync(0xffffffffu, n, 0, LANES), n1 = __shfl_sync(0xffffffffu, n, LANES / 2, LANES);
  const int place0 = __shfl_sync(0xffffffffu, place, 0, LANES),
            place1 = __shfl_sync(0xffffffffu, place, LANES / 2, LANES);
  if (n1 < 0) mine = false;                            // written by its CTA
  const int total = mine ? n0 + n1 : 0;
  auto slot_of = [&](int i) {
    const bool k = i >= n0;
    const int at = k ? place1 : place0, j = k ? i - n0 : i;
    const int piece = at & 1 ? j >> 1 : j, stream = at & 1 ? j & 1 : 0;
    if (piece == 0) return row_slot(p, k ? b : -1, stream, row, hq);
    return cta_slot(p, (k ? c1 : c0) + piece, (at & 1 ? stream : at >> 1 & 1) * (p.slot_rows / p.streams) + (at >> 2));
  };
  float M = -INFINITY, L = 0.f, acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  for (int i0 = 0; __any_sync(0xffffffffu, i0 < total); i0 += LANES) {
    // a lane for each of LANES partials: their common maximum, their weights
    const bool there = i0 + lane < total;
    const long long slot = there ? slot_of(i0 + lane) : 0;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (there) ml = __ldcg(p.part_ml + slot);
    if (ml.y == 0.f) ml.x = -INFINITY;                 // saw none of its keys
    float top = fmaxf(M, ml.x);
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float f = M == -INFINITY ? 0.f : exp2f(M - top);
    const float w = ml.y == 0.f ? 0.f : exp2f(ml.x - top);
    M = top;
    float l = w * ml.y;
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    L = L * f + l;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] *= f;
#pragma unroll 4
    for (int j = 0; j < LANES; ++j) {
      if (!__any_sync(0xffffffffu, i0 + j < total)) break;
      const float wj = __shfl_sync(0xffffffffu, w, j, LANES);
      const float* src = p.part_o + __shfl_sync(0xffffffffu, slot, j, LANES) * D + lane * kVec;
      if (wj != 0.f) {                                 // a partial that saw no key holds no numbers
#pragma unroll
        for (int i = 0; i < kPer; i += kVec) {
          if constexpr (kVec == 2) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(src + i * LANES));
            acc[i] = fmaf(wj, x.x, acc[i]);
            acc[i + 1] = fmaf(wj, x.y, acc[i + 1]);
          } else {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src + i * LANES));
            acc[i] = fmaf(wj, x.x, acc[i]);
            acc[i + 1] = fmaf(wj, x.y, acc[i + 1]);
            acc[i + 2] = fmaf(wj, x.z, acc[i + 2]);
            acc[i + 3] = fmaf(wj, x.w, acc[i + 3]);
          }
        }
      }
    }
  }
  if (!mine) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  T* out = static_cast<T*>(p.o) + (static_cast<long long>(row) * p.Hq + hq) * D + lane * kVec;
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    T* at = out + (i / kVec) * kVec * LANES + i % kVec;
    if constexpr (sizeof(T) == 2) *reinterpret_cast<__nv_bfloat162*>(at) = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
    else *reinterpret_cast<float2*>(at) = make_float2(acc[i] * inv, acc[i + 1] * inv);
  }
  if (p.lse && lane == 0)
    p.lse[static_cast<long long>(row) * p.Hq + hq] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <typename T, int D>
cudaError_t launch_merge(cudaStream_t s, const PagedParams& p) {
  // A warp for a row's head takes up to 32 partials at once (a long sequence's few rows); eight
  // lanes for one where there are many rows, whose partials are few: four times fewer warps to
  // look everything up.
  if (static_cast<long long>(p.rows) * p.Hq < kManyHeads)
    return launch_pdl(paged_merge_kernel<T, D, 32>, dim3(p.rows, (p.Hq + 3) / 4), dim3(128), 0, s, p);
  return launch_pdl(paged_merge_kernel<T, D, 8>, dim3(p.rows, (p.Hq + 15) / 16), dim3(128), 0, s, p);
}
template <typename T>
cudaError_t launch_merge(cudaStream_t s, const PagedParams& p) {
  return p.D == 64 ? launch_merge<T, 64>(s, p) : launch_merge<T, 128>(s, p);
}

// Weights of key blocks whose query tiles were split over CTAs: the run of continuing CTAs of a
// key block is summed in order by the CTA that stands first in it.
__global__ void __launch_bounds__(256) paged_weights_merge_kernel(const PagedParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x;
  const int4 id = p.part_id[c];
  // what a concurrent call may have left in a workspace that it wrongly shares is no place outside the scores
  auto within = [](int x, int n) { return static_cast<unsigned>(x) < static_cast<unsigned>(n); };
  if (!id.w || !within(id.x, p.B) || !within(id.y, p.Hkv) ||
      !within(id.z, (paged_cap(p) + p.key_tile - 1) >> p.key_shift))
    return;
  auto same = [&](int k) {
    if (k < 0 || k >= p.grid) return false;
    const int4 o = p.part_id[k];
    return o.w && o.x == id.x && o.y == id.y && o.z == id.z;
  };
  if (same(c - 1)) return;
  int end = c + 1;
  while (same(end)) ++end;
  const SeqView v = seq_view(p, id.x);
  for (int i = threadIdx.x; i < p.key_tile; i += blockDim.x) {
    const int key = id.z * p.key_tile + i;
    if (key >= v.len) continue;
    float sum = 0.f;
    for (int k = c; k < end; ++k) sum += p.part_w[static_cast<long long>(k) * p.slot_rows + i];
    p.scores[(static_cast<long long>(id.x) * p.Hkv + id.y) * paged_cap(p) + key] += sum;
  }
}

kvc_status status_of(cudaError_t e) { return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA; }

}  // namespace

bool encode_rows_tmap(CUtensorMap* map, const void* rows_dev, const PagedParams& p) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.D), static_cast<cuuint64_t>(p.Hq),
                              static_cast<cuuint64_t>(p.rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.D) * 2, static_cast<cuuint64_t>(p.q_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(p.tile_tokens)};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(rows_dev), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_slots_tmap(CUtensorMap* map, const void* pool, const PagedParams& p) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(p.D) * 2;
  const cuuint32_t halves = static_cast<cuuint32_t>(p.D / 64);
  const cuuint64_t dims[4] = {64, 8, halves, static_cast<cuuint64_t>((p.pool_pages * p.Hkv) << p.page_shift) / 8};
  const cuuint64_t strides[3] = {row, 128, row * 8};
  const cuuint32_t box[4] = {64, 8, halves, static_cast<cuuint32_t>(std::min(1 << p.page_shift, 128)) / 8};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kvc

extern "C" kvc_status kvc_paged_workspace(const kvc_paged_batch* batch, int32_t rows, int32_t keep,
                                          int64_t* bytes_out) {
  using namespace kvc;
  if (!bytes_out || !valid_batch(batch) || rows < 0 || keep < 0) return KVC_ERR_ARG;
  const int sms = sm_count();
  if (sms < 1) return KVC_ERR_CUDA;
  size_t most = 256;
  PagedParams p = base_params(batch, rows, nullptr, sms);
  attend_schedule(&p, batch);
  p.join = 0;                                  // fewer rows may not join: this layout holds either
  most = std::max(most, attend_layout(p).bytes);
  p = base_params(batch, rows, nullptr, sms);
  weights_schedule(&p, batch);
  most = std::max(most, weights_layout(p).bytes);
  most = std::max(most, evict_bytes(batch, keep));
  *bytes_out = static_cast<int64_t>(most);
  return KVC_OK;
}

extern "C" kvc_status kvc_paged_append(const kvc_paged_batch* batch, const void* k_dev, const void* v_dev,
                                       int64_t k_row_stride, int64_t v_row_stride, int32_t rows,
                                       const int32_t* row_start_dev, void* stream) {
  using namespace kvc;
  if (!valid_batch(batch) || !row_start_dev || !valid_rows(batch, k_dev, k_row_stride, batch->num_kv_heads, rows) ||
      !valid_rows(batch, v_dev, v_row_stride, batch->num_kv_heads, rows) ||
      (batch->positions && !batch->next_positions))
    return KVC_ERR_ARG;
  if (rows == 0) return KVC_OK;
  const int elem = batch->dtype == KVC_F32 ? 4 : 2;
  AppendParams p{};
  p.B = batch->num_seqs;
  p.H = batch->num_kv_heads;
  p.page_shift = page_shift(batch->page_size);
  p.max_pages = batch->max_pages;
  p.rows = rows;
  p.row_bytes = batch->head_dim * elem;
  p.pool_pages = batch->pool_pages;
  p.k_stride = k_row_stride * elem;
  p.v_stride = v_row_stride * elem;
  p.page_table = batch->page_table;
  p.lengths = batch->lengths;
  p.next_positions = batch->next_positions;
  p.row_start = row_start_dev;
  p.k = static_cast<const uint8_t*>(k_dev);
  p.v = static_cast<const uint8_t*>(v_dev);
  p.k_pool = static_cast<uint8_t*>(batch->k_pool);
  p.v_pool = static_cast<uint8_t*>(batch->v_pool);
  p.scores = batch->scores;
  p.positions = batch->positions;
  p.err = batch->error;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows <= kFewRows * p.B && 2LL * rows * p.H * p.row_bytes <= kFewBytes)
    return status_of(launch_pdl(paged_append_few_kernel, dim3(p.B), dim3(512), 0, s, p));
  // One for each slot that a page may need cleared, in all up to 4,096 and never fewer than a page of 16
  // needs: 1,024 sequences' single rows in pages of 256 take 8.8 us, with a warp for every slot 41; 8
  // sequences' 512 rows 11.8, with 15 warps a sequence 15.5.
  p.behind_warps = std::min(batch->page_size - 1, std::max(15, 4096 / p.B));
  const long long warps = rows + static_cast<long long>(p.B) * p.behind_warps;
  if (warps > INT_MAX - 8) return KVC_ERR_ARG;
  cudaError_t e = launch_pdl(paged_append_kernel, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(256), 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(paged_grow_kernel, dim3((p.B + 255) / 256), dim3(256), 0, s, p);
  return status_of(e);
}

extern "C" kvc_status kvc_paged_attend(const kvc_paged_batch* batch, const void* q_dev, int64_t q_row_stride,
                                       void* o_dev, float* lse_dev, int32_t rows, const int32_t* row_start_dev,
                                       int32_t causal, void* workspace_dev, int64_t workspace_bytes, void* stream) {
  using namespace kvc;
  if (!valid_batch(batch) || !row_start_dev || !valid_rows(batch, q_dev, q_row_stride, batch->num_q_heads, rows) ||
      !aligned16(o_dev) || (rows > 0 && !o_dev) || !workspace_dev || !aligned16(workspace_dev) ||
      (causal != 0 && causal != 1) || static_cast<long long>(rows) * batch->num_q_heads > (1LL << 32))
    return KVC_ERR_ARG;
  if (rows == 0) return KVC_OK;
  const int sms = sm_count();
  if (sms < 1) return KVC_ERR_CUDA;
  PagedParams p = base_params(batch, rows, row_start_dev, sms);
  attend_schedule(&p, batch);
  const Layout l = attend_layout(p);
  if (workspace_bytes < static_cast<int64_t>(l.bytes)) return KVC_ERR_ARG;
  uint8_t* w = static_cast<uint8_t*>(workspace_dev);
  p.plan = reinterpret_cast<long long*>(w + l.plan);
  p.part_ml = reinterpret_cast<float2*>(w + l.part_ml);
  p.part_o = reinterpret_cast<float*>(w + l.part_o);
  p.q = q_dev;
  p.q_stride = q_row_stride;
  p.o = o_dev;
  p.lse = lse_dev;
  p.causal = causal;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = batch->dtype == KVC_BF16 ? launch_paged_attend_tc(s, p) : launch_paged_attend_simt(s, p);
  if (e == cudaSuccess) e = batch->dtype == KVC_F32 ? launch_merge<float>(s, p) : launch_merge<__nv_bfloat16>(s, p);
  return status_of(e);
}

extern "C" kvc_status kvc_paged_weights(const kvc_paged_batch* batch, const void* q_dev, int64_t q_row_stride,
                                        const float* lse_dev, int32_t rows, const int32_t* row_start_dev,
                                        int32_t causal, void* workspace_dev, int64_t workspace_bytes, void* stream) {
  using namespace kvc;
  if (!valid_batch(batch) || !batch->scores || !row_start_dev ||
      !valid_rows(batch, q_dev, q_row_stride, batch->num_q_heads, rows) || (rows > 0 && !lse_dev) || !workspace_dev ||
      !aligned16(workspace_dev) || (causal != 0 && causal != 1))
    return KVC_ERR_ARG;
  if (rows == 0) return KVC_OK;
  const int sms = sm_count();
  if (sms < 1) return KVC_ERR_CUDA;
  PagedParams p = base_params(batch, rows, row_start_dev, sms);
  weights_schedule(&p, batch);
  const Layout l = weights_layout(p);
  if (workspace_bytes < static_cast<int64_t>(l.bytes)) return KVC_ERR_ARG;
  uint8_t* w = static_cast<uint8_t*>(workspace_dev);
  p.plan = reinterpret_cast<long long*>(w + l.plan);
  p.part_id = reinterpret_cast<int4*>(w + l.part_id);
  p.part_w = reinterpret_cast<float*>(w + l.part_w);
  p.q = q_dev;
  p.q_stride = q_row_stride;
  p.lse = const_cast<float*>(lse_dev);
  p.scores = batch->scores;
  p.causal = causal;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = batch->dtype == KVC_BF16 ? launch_paged_weights_tc(s, p) : launch_paged_weights_simt(s, p);
  // one tile of rows holds every sequence's: no key block is split
  if (e == cudaSuccess && rows > p.tile_tokens)
    e = launch_pdl(paged_weights_merge_kernel, dim3(p.grid), dim3(256), 0, s, p);
  return status_of(e);
}

extern "C" kvc_status kvc_paged_evict(const kvc_paged_batch* batch, int32_t keep, int32_t sinks, int32_t recent,
                                      void* workspace_dev, int64_t workspace_bytes, void* stream) {
  using namespace kvc;
  if (!valid_batch(batch) || !batch->scores || !batch->positions || !batch->next_positions || keep < 1 || sinks < 0 ||
      recent < 0 || static_cast<long long>(sinks) + recent > keep || !workspace_dev || !aligned16(workspace_dev) ||
      workspace_bytes < static_cast<int64_t>(evict_bytes(batch, keep)))
    return KVC_ERR_ARG;
  const long long cap = static_cast<long long>(batch->max_pages) * batch->page_size;
  if (cap <= keep) return KVC_OK;              // no sequence can be longer
  if (cap > paged_evict_max_slots()) return KVC_ERR_UNSUPPORTED;
  const int sms = sm_count();
  if (sms < 1) return KVC_ERR_CUDA;
  EvictParams p{};
  p.B = batch->num_seqs;
  p.Hkv = batch->num_kv_heads;
  p.page_shift = page_shift(batch->page_size);
  p.max_pages = batch->max_pages;
  p.row_bytes = batch->head_dim * (batch->dtype == KVC_F32 ? 4 : 2);
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  p.pool_pages = batch->pool_pages;
  p.page_table = batch->page_table;
  p.lengths = batch->lengths;
  p.next_positions = batch->next_positions;
  p.k_pool = static_cast<uint8_t*>(batch->k_pool);
  p.v_pool = static_cast<uint8_t*>(batch->v_pool);
  p.scores = batch->scores;
  p.positions = batch->positions;
  p.counts = static_cast<int32_t*>(workspace_dev);
  p.moves = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace_dev) + evict_counts_bytes(batch));
  p.move_cap = move_cap(batch, keep);
  p.err = batch->error;
  return status_of(launch_paged_evict(static_cast<cudaStream_t>(stream), p, sms, batch->lengths));
}
