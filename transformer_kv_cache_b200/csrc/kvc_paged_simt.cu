// kvc_paged_simt.cu -- attention of a paged batch and the weights of its cached tokens in fp32
// storage and arithmetic (FFMA), with the schedule of kvc_paged.cuh.
//
// Attention: one pass over an item's keys with the running maximum and sum of the softmax, the
// next tile's keys and values arriving by cp.async under this one's products. A tile is 16 rows
// where sequences have no more, else 64, the prefix's chosen by the batch's rows. Weights: a block
// of keys with a tile of 32 or 64 rows, a key's sum over the rows in one thread or half-warp.
//
// What shared memory gives back (512 bytes in four cycles for a load of 16 bytes a lane) bounds the
// products: 64 rows are 4 x 4 of them to a thread, 16 x 16 threads, eight loads for 64 FFMA, twice the
// FFMAs' own time (300 rows over 4,000 tokens: attention 26 TFLOP/s with 64 dims, 29 with 128, weights 21
// and 25). Few rows are dealt out so that no thread computes rows that there are not: 16 sequences of 2,048
// to 4,096 tokens, 8 heads of 64 dims: attention 59 us, 3.4 TB/s (128 as 16 x 16 threads), the weights
// with 128 dims 74 us, 2.8 TB/s (247).
#include <math_constants.h>

#include "kvc_paged.cuh"

namespace kvc {
namespace {

constexpr int kKT = 64;                        // keys of a tile
constexpr int kThreads = 256;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// The tile's query rows [token t0 .., G heads each]; rows past `tokens` are zeros.
template <int D, int LD, int ROWS>
__device__ __forceinline__ void load_queries(const PagedParams& p, const SeqView& v, int h, int t0, int rows,
                                             float* dst) {
  constexpr int kChunks = D / 4;
  for (int i = threadIdx.x; i < ROWS * kChunks; i += kThreads) {
    const int r = i / kChunks, c = i % kChunks;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      const long long row = v.r0 + t0 + r / p.G;
      x = load4(static_cast<const float*>(p.q) + row * p.q_stride + (h * p.G + r % p.G) * D + c * 4);
    }
    *reinterpret_cast<float4*>(dst + r * LD + c * 4) = x;
  }
}

// Scores of RA rows of `a` by RB rows of `b`, rows ra + i * sa and rb + j * sb.
template <int D, int RA, int RB>
__device__ __forceinline__ void dots(const float* a, int lda, int sa, const float* b, int ldb, int sb,
                                     float (&s)[RA][RB]) {
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int j = 0; j < RB; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 x[RA], y[RB];
#pragma unroll
    for (int i = 0; i < RA; ++i) x[i] = load4(a + i * sa * lda + d);
#pragma unroll
    for (int j = 0; j < RB; ++j) y[j] = load4(b + j * sb * ldb + d);
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
      for (int j = 0; j < RB; ++j)
        s[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, s[i][j]))));
  }
}

// Scores of 4 keys by 4 rows in 16 lanes, a sixteenth of the dims in each (64 products for eight loads,
// which bound these kernels); summed over the lanes, that of key `part / 4` and row `part % 4` ends
// in lane `part`. k4 and q4 are the lane's first 16 bytes of the first key and row.
template <int D, int LD>
__device__ __forceinline__ float dots_by_lanes(const float* k4, const float* q4, int part) {
  float a[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) a[i] = 0.f;
#pragma unroll
  for (int x = 0; x < D; x += 64) {
    float4 k[4], q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k[i] = load4(k4 + i * LD + x);
      q[i] = load4(q4 + i * LD + x);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float4 u = k[i >> 2], v = q[i & 3];
      a[i] = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, a[i]))));
    }
  }
#pragma unroll
  for (int n = 8; n; n >>= 1) {
    const bool upper = part & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, upper ? a[i] : a[i + n], n);
      a[i] = (upper ? a[i + n] : a[i]) + other;
    }
  }
  return a[0];
}

// 16 bytes to shared memory behind the registers' back, or zeros where `there` is false.
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}

// A CTA's loads of key tiles: a thread copies the same 16 bytes of kKeys of a tile's keys, whose
// pages it asks for one tile ahead. Keys that no page holds are zeros.
template <int D>
struct KeyLoader {
  static constexpr int kChunks = D / 4, kKeys = kKT * kChunks / kThreads, kStep = kThreads / kChunks;
  int page[kKeys];
  KeyTile tile;

  __device__ __forceinline__ void look(const PagedParams& p, const KeyTile& t) {
    tile = t;
    const int32_t* table =
        tile.b < 0 ? p.prefix_pages : p.page_table + static_cast<long long>(tile.b) * p.max_pages;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int key = tile.key0 + static_cast<int>(threadIdx.x) / kChunks + i * kStep;
      page[i] = key < tile.len ? __ldg(table + (key >> p.page_shift)) : -1;
    }
  }
  template <bool kValues>
  __device__ __forceinline__ void load(const PagedParams& p, int h, float* ks, float* vs, int ld) const {
    const int c = static_cast<int>(threadIdx.x) % kChunks;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int at = static_cast<int>(threadIdx.x) / kChunks + i * kStep, key = tile.key0 + at;
      const bool in = key < tile.len, there = in && page[i] >= 0 && page[i] < p.pool_pages;
      if (in && !there) latch_error(p.err, DERR_BOUNDS);
      const long long row = there ? ((static_cast<long long>(page[i]) * p.Hkv + h) << p.page_shift) +
                                        (key & ((1 << p.page_shift) - 1))
                                  : 0;
      cp_async16_or_zero(ks + at * ld + c * 4, static_cast<const float*>(p.k_pool) + row * D + c * 4, there);
      if (kValues) cp_async16_or_zero(vs + at * ld + c * 4, static_cast<const float*>(p.v_pool) + row * D + c * 4, there);
    }
  }
};
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One segment in tiles of 64 query rows; sm holds [rows][LD] queries, two stages of [kKT][LD] keys
// and values, [rows][LP] weights.
template <int D>
__device__ __forceinline__ void attend_segment(const PagedParams& p, const Segment& g, float* sm) {
  constexpr int LD = D + 4, ROWS = 64, RPT = ROWS / 16, LP = kKT + 4;
  float* qs = sm;
  float* kv = qs + ROWS * LD;                  // [stage][K, V][kKT][LD]
  float* ps = kv + 4 * kKT * LD;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int t0 = g.i * item_tokens(p, g.b);
  const int tokens = min(item_tokens(p, g.b), g.v.n - t0), rows = tokens * p.G;
  KeyLoader<D> loader;
  loader.look(p, key_tile_at(p, g, g.k0));
  __syncthreads();                             // the segment before is read
  loader.template load<true>(p, g.h, kv, kv + kKT * LD, LD);
  cp_async_commit();
  load_queries<D, LD, ROWS>(p, g.v, g.h, t0, rows, qs);
  float m[RPT], l[RPT], acc[RPT][D / 16];
  int limit[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    m[r] = -CUDART_INF_F;
    l[r] = 0.f;
    const int at = ty * RPT + r;
    limit[r] = at < rows ? key_limit(p, g.b, g.v, t0 + at / p.G) : 0;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[r][c] = 0.f;
  }
  if (g.k0 + 1 < g.k1) loader.look(p, key_tile_at(p, g, g.k0 + 1));
  for (int kt = g.k0; kt < g.k1; ++kt) {
    const int st = (kt - g.k0) & 1;
    const float* ks = kv + st * 2 * kKT * LD;
    const float* vs = ks + kKT * LD;
    if (kt + 1 < g.k1) {
      float* next = kv + (st ^ 1) * 2 * kKT * LD;
      loader.template load<true>(p, g.h, next, next + kKT * LD, LD);
      cp_async_commit();
      if (kt + 2 < g.k1) loader.look(p, key_tile_at(p, g, kt + 2));
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();
    const KeyTile tile = key_tile_at(p, g, kt);
    float s[RPT][4];
    dots<D, RPT, 4>(qs + ty * RPT * LD, LD, 1, ks + tx * LD, LD, 16, s);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      float mx = -CUDART_INF_F;
      const int end = (tile.b == g.b ? limit[r] : tile.len) - tile.key0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[r][j] = tx + 16 * j < end ? s[r][j] * p.scale_log2 : -CUDART_INF_F;
        mx = fmaxf(mx, s[r][j]);
      }
#pragma unroll
      for (int d = 8; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float m_new = fmaxf(m[r], mx);
      const float base = m_new == -CUDART_INF_F ? 0.f : m_new;     // nothing visible yet: every weight is 0
      const float f = exp2f(m[r] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[r][j] - base);
        sum += e;
        ps[(ty * RPT + r) * LP + tx + 16 * j] = e;
      }
#pragma unroll
      for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      l[r] = l[r] * f + sum;
      m[r] = m_new;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) acc[r][c] *= f;
    }
    __syncwarp();                              // a row's weights are written and read by one half-warp
#pragma unroll 2
    for (int k = 0; k < kKT; k += 4) {
      float4 pr[RPT];
#pragma unroll
      for (int r = 0; r < RPT; ++r) pr[r] = load4(ps + (ty * RPT + r) * LP + k);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const float4 v4 = load4(vs + (k + kk) * LD + c * 64 + tx * 4);
#pragma unroll
          for (int r = 0; r < RPT; ++r) {
            const float e = kk == 0 ? pr[r].x : kk == 1 ? pr[r].y : kk == 2 ? pr[r].z : pr[r].w;
            acc[r][4 * c + 0] = fmaf(e, v4.x, acc[r][4 * c + 0]);
            acc[r][4 * c + 1] = fmaf(e, v4.y, acc[r][4 * c + 1]);
            acc[r][4 * c + 2] = fmaf(e, v4.z, acc[r][4 * c + 2]);
            acc[r][4 * c + 3] = fmaf(e, v4.w, acc[r][4 * c + 3]);
          }
        }
      }
    }
    __syncthreads();                           // the stage is read
  }
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int at = ty * RPT + r;
    if (at >= rows) continue;
    if (g.k0 == 0 && g.k1 == g.nk && writes_rows(p, g.v, g.i)) {
      const long long out = static_cast<long long>(g.v.r0 + t0 + at / p.G) * p.Hq + g.h * p.G + at % p.G;
      const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
      if (p.lse && tx == 0) p.lse[out] = (m[r] + log2f(l[r])) * 0.6931471805599453f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        *reinterpret_cast<float4*>(static_cast<float*>(p.o) + out * D + c * 64 + tx * 4) =
            make_float4(acc[r][4 * c] * inv, acc[r][4 * c + 1] * inv, acc[r][4 * c + 2] * inv, acc[r][4 * c + 3] * inv);
      continue;
    }
    const long long slot = g.k0 == 0 ? row_slot(p, g.b, 0, g.v.r0 + t0 + at / p.G, g.h * p.G + at % p.G)
                                     : cta_slot(p, blockIdx.x, at);
    if (tx == 0) p.part_ml[slot] = make_float2(m[r], l[r]);
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      *reinterpret_cast<float4*>(p.part_o + slot * D + c * 64 + tx * 4) =
          make_float4(acc[r][4 * c], acc[r][4 * c + 1], acc[r][4 * c + 2], acc[r][4 * c + 3]);
  }
}

// One segment in tiles of 16 query rows, in three phases of a key tile: scores (a warp has 8 keys),
// softmax (a warp has two rows), sums (16 bytes of the dims, 4 rows and some of the keys to a thread:
// all threads have keys however few the rows are, and are joined at the end of the segment).
// MAXROWS: query rows that the kernel's shared memory is laid out for.
template <int D, int MAXROWS>
__device__ __forceinline__ void attend_few(const PagedParams& p, const Segment& g, float* sm) {
  constexpr int LD = D + 4, LP = kKT + 4, kChunks = D / 4, kGroups = kThreads / kChunks;
  float* qs = sm;
  float* kv = qs + MAXROWS * LD;               // [stage][K, V][kKT][LD]
  float* ss = kv + 4 * kKT * LD;               // [row][LP] scores
  float* pt = ss + 16 * LP;                    // [key][16 rows] weights
  float* fs = pt + kKT * 16;                   // [row] factors of what was summed before; at the end 1 / sum
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane & 15;
  const int t0 = g.i * item_tokens(p, g.b);
  const int tokens = min(item_tokens(p, g.b), g.v.n - t0), rows = tokens * p.G;
  const int quads = rows <= 4 ? 1 : rows <= 8 ? 2 : 4;
  const int c = threadIdx.x % kChunks, quad = threadIdx.x / kChunks % quads, k_first = threadIdx.x / kChunks / quads,
            k_step = kGroups / quads;
  KeyLoader<D> loader;
  loader.look(p, key_tile_at(p, g, g.k0));
  __syncthreads();                             // the segment before is read
  loader.template load<true>(p, g.h, kv, kv + kKT * LD, LD);
  cp_async_commit();
  load_queries<D, LD, 16>(p, g.v, g.h, t0, rows, qs);
  float m[2], l[2];                            // of rows 2 warp, + 1
  int limit[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int at = 2 * warp + r;
    m[r] = -CUDART_INF_F;
    l[r] = 0.f;
    limit[r] = at < rows ? key_limit(p, g.b, g.v, t0 + at / p.G) : 0;
  }
  float acc[4][4] = {};                        // [row][dim]
  if (g.k0 + 1 < g.k1) loader.look(p, key_tile_at(p, g, g.k0 + 1));
#pragma unroll 1
  for (int kt = g.k0; kt < g.k1; ++kt) {
    const int st = (kt - g.k0) & 1;
    const float* ks = kv + st * 2 * kKT * LD;
    const float* vs = ks + kKT * LD;
    if (kt + 1 < g.k1) {
      float* next = kv + (st ^ 1) * 2 * kKT * LD;
      loader.template load<true>(p, g.h, next, next + kKT * LD, LD);
      cp_async_commit();
      if (kt + 2 < g.k1) loader.look(p, key_tile_at(p, g, kt + 2));
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();
    const int key4 = warp * 8 + (lane >> 4) * 4;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 4)
      ss[(r0 + (part & 3)) * LP + key4 + (part >> 2)] =
          dots_by_lanes<D, LD>(ks + key4 * LD + part * 4, qs + r0 * LD + part * 4, part);
    __syncthreads();
    const KeyTile tile = key_tile_at(p, g, kt);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int at = 2 * warp + r;
      if (at >= rows) break;
      const int end = (tile.b == g.b ? limit[r] : tile.len) - tile.key0;
      const float s0 = lane < end ? ss[at * LP + lane] * p.scale_log2 : -CUDART_INF_F;
      const float s1 = lane + 32 < end ? ss[at * LP + lane + 32] * p.scale_log2 : -CUDART_INF_F;
      float mx = fmaxf(s0, s1);
#pragma unroll
      for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float m_new = fmaxf(m[r], mx);
      const float base = m_new == -CUDART_INF_F ? 0.f : m_new;       // nothing visible yet: every weight is 0
      const float f = exp2f(m[r] - base), e0 = exp2f(s0 - base), e1 = exp2f(s1 - base);
      pt[lane * 16 + at] = e0;
      pt[(lane + 32) * 16 + at] = e1;
      float sum = e0 + e1;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      l[r] = l[r] * f + sum;
      m[r] = m_new;
      if (lane == 0) fs[at] = f;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float f = fs[4 * quad + r];        // of rows that there are not: nothing that is kept
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][i] *= f;
    }
#pragma unroll 4
    for (int k = k_first; k < kKT; k += k_step) {
      const float4 v = load4(vs + k * LD + c * 4), e = load4(pt + k * 16 + 4 * quad);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = r == 0 ? e.x : r == 1 ? e.y : r == 2 ? e.z : e.w;
        acc[r][0] = fmaf(x, v.x, acc[r][0]);
        acc[r][1] = fmaf(x, v.y, acc[r][1]);
        acc[r][2] = fmaf(x, v.z, acc[r][2]);
        acc[r][3] = fmaf(x, v.w, acc[r][3]);
      }
    }
    __syncthreads();                           // the stage, the weights and the factors are read
  }
  // the groups' sums to shared memory ([group of keys][row][D], in the first K), then joined in order
  const bool whole = g.k0 == 0 && g.k1 == g.nk && writes_rows(p, g.v, g.i);
  auto place = [&](int at, long long& out, long long& slot) {
    const int row = g.v.r0 + t0 + at / p.G, hq = g.h * p.G + at % p.G;
    out = static_cast<long long>(row) * p.Hq + hq;
    slot = g.k0 == 0 ? row_slot(p, g.b, 0, row, hq) : cta_slot(p, blockIdx.x, at);
  };
#pragma unroll
  for (int r = 0; r < 4; ++r)
    *reinterpret_cast<float4*>(kv + ((k_first * quads + quad) * 4 + r) * D + c * 4) =
        make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int at = 2 * warp + r;
    if (at >= rows || lane > 0) break;
    long long out, slot;
    place(at, out, slot);
    fs[at] = whole ? (l[r] == 0.f ? 0.f : 1.f / l[r]) : 1.f;
    if (!whole) p.part_ml[slot] = make_float2(m[r], l[r]);
    else if (p.lse) p.lse[out] = (m[r] + log2f(l[r])) * 0.6931471805599453f;
  }
  __syncthreads();
  const int at = threadIdx.x / kChunks;        // a thread for 16 bytes of a row, kGroups rows at once
#pragma unroll 1
  for (int r = at; r < rows; r += kGroups) {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < k_step; ++k) {
      const float4 x = load4(kv + (k * quads * 4 + r) * D + c * 4);
      sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
    }
    const float f = fs[r];
    long long out, slot;
    place(r, out, slot);
    float* dst = whole ? static_cast<float*>(p.o) + out * D : p.part_o + slot * D;
    *reinterpret_cast<float4*>(dst + c * 4) = make_float4(sum.x * f, sum.y * f, sum.z * f, sum.w * f);
  }
}

// OWN and PREFIX: query rows of a tile of a sequence's own keys and of the prefix's.
template <int D, int OWN, int PREFIX>
__global__ void __launch_bounds__(kThreads) paged_attend_simt_kernel(const PagedParams p) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ __align__(16) float sm[];
  __shared__ long long plan_s[kPlanWords + kThreads / 32];
  constexpr int kMax = OWN > PREFIX ? OWN : PREFIX;
  Walk w = plan_walk(p, plan_s, [&](int b, const SeqView& v) { return head_units(p, b, v); });
  walk_to_item(p, w);
  Segment g;
  while (next_segment(p, w, g)) {
    const bool few = OWN == PREFIX || g.b >= 0 ? OWN == 16 : PREFIX == 16;
    if (few) attend_few<D, kMax>(p, g, sm);
    else attend_segment<D>(p, g, sm);
  }
}

// Weights: a step of a CTA is a block of kKT keys with one tile of ROWS query rows; keys, rows and
// their log-sum-exp arrive by cp.async kStages - 1 steps ahead, the steps' descriptions beside them.
template <int D, int ROWS>
struct WeightsCfg {
  static constexpr int kLD = D + 4;
  // as many as leave room for two CTAs of an SM. Where a step takes 68 KB the CTAs of an SM cover one
  // another's loads instead (2 x 300 rows over 4,000 tokens, 128 dims: 142 us, and with three stages of
  // one CTA 173)
  static constexpr int kStages = D == 64 ? (ROWS == 32 ? 3 : 2) : (ROWS == 32 ? 2 : 1);
  static constexpr int kFloats = (kKT + ROWS) * kLD + ROWS;
  static constexpr size_t kSmem = sizeof(float) * kStages * kFloats;
};
struct WeightStep {
  int b, h, kb, t;                             // sequence, KV head, key block, query tile
  int last, first;                             // 1: the CTA's last of the block; the CTA has the block's first
  SeqView v;
};

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads) paged_weights_simt_kernel(const PagedParams p) {
  griddep_wait();
  griddep_launch_dependents();
  using C = WeightsCfg<D, ROWS>;
  constexpr int LD = C::kLD, RPT = ROWS / 16, kStages = C::kStages, kChunks = D / 4;
  extern __shared__ __align__(16) float sm[];  // [stage][keys | rows][LD], [rows] log-sum-exp
  __shared__ long long plan_s[kPlanWords + kThreads / 32];
  __shared__ WeightStep steps_s[kStages];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;            // of ROWS = 64
  Walk w = plan_walk(p, plan_s, [&](int, const SeqView& v) { return weight_head_units(p, v); });
  if (threadIdx.x == 0) p.part_id[blockIdx.x] = make_int4(0, 0, 0, 0);
  // the step that is looked up; its head's key blocks and query tiles
  int kb = 0, t = 0, blocks = 0, tiles = 0;
  bool more = w.u < w.u1, first = false;
  auto head_size = [&] {
    blocks = (w.v.len + kKT - 1) / kKT;
    tiles = (w.v.n + p.tile_tokens - 1) / p.tile_tokens;
  };
  KeyLoader<D> loader;
  if (more) {
    head_size();
    kb = static_cast<int>(quotient(w.u - w.item_first, tiles));
    t = static_cast<int>(w.u - w.item_first - static_cast<long long>(kb) * tiles);
    first = t == 0;
    loader.look(p, {w.b, kb * kKT, w.v.len});
  }
  // this thread's 16 bytes of a tile's rows: their token and head
  constexpr int kRows = ROWS * kChunks / kThreads, kStep = kThreads / kChunks;
  const int c = static_cast<int>(threadIdx.x) % kChunks, r0 = static_cast<int>(threadIdx.x) / kChunks;
  int tok[kRows], head[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    tok[i] = (r0 + i * kStep) / p.G;
    head[i] = (r0 + i * kStep) % p.G;
  }
  int put = 0;                                 // steps whose loads are out
  auto issue = [&] {                           // the step's loads, and the look-up of the next one's
    if (more) {
      float* ks = sm + put % kStages * C::kFloats;
      float* qs = ks + kKT * LD + r0 * LD + c * 4;
      float* ls = ks + (kKT + ROWS) * LD + r0;
      loader.template load<false>(p, w.h, ks, nullptr, LD);
      const int tok0 = t * p.tile_tokens, rows = min(p.tile_tokens, w.v.n - tok0) * p.G;
      const float* q = static_cast<const float*>(p.q) + (w.v.r0 + tok0) * p.q_stride + w.h * p.G * D + c * 4;
      const float* lse = p.lse + static_cast<long long>(w.v.r0 + tok0) * p.Hq + w.h * p.G;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const bool in = r0 + i * kStep < rows;
        cp_async16_or_zero(qs + i * kStep * LD, in ? q + tok[i] * p.q_stride + head[i] * D : q, in);
        if (c == 0 && in)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(ls + i * kStep)),
                       "l"(lse + tok[i] * p.Hq + head[i])
                       : "memory");
      }
      more = ++w.u < w.u1;
      if (threadIdx.x == 0) steps_s[put % kStages] = {w.b, w.h, kb, t, t + 1 == tiles || !more, first, w.v};
      ++put;
      if (++t == tiles) {
        t = 0;
        first = true;
        if (++kb == blocks) {
          kb = 0;
          while (more) {                       // the next head that has any
            if (++w.h == p.Hkv) {
              w.h = 0;
              w.v = w.next;
              walk_to(p, w, w.b + 1);
              head_size();
            }
            if (blocks > 0 && tiles > 0) break;
          }
        }
      }
      if (more) loader.look(p, {w.b, kb * kKT, w.v.len});
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) issue();
  // The keys whose sums this thread holds, kKeys from `mine` on; `writes`: the whole of them in the end.
  const int lane = threadIdx.x & 31, part = lane & 15;
  constexpr int kKeys = ROWS == 32 ? 1 : 4;
  const int mine = ROWS == 32 ? (static_cast<int>(threadIdx.x) >> 5) * 8 + (lane >> 4) * 4 + (part >> 2) : ty * 4;
  const bool writes = ROWS == 32 ? (part & 3) == 0 : tx == 0;
  float sum[kKeys] = {};
#pragma unroll 1
  for (int at = 0;; ++at) {
    if (kStages == 1) {
      __syncthreads();                         // the step before is read
      issue();
    }
    if (at == put) break;
    cp_async_wait<kStages == 1 ? 0 : kStages - 2>();
    __syncthreads();                           // step `at` is there, and the step before is read
    if (kStages > 1) issue();
    const WeightStep& d = steps_s[at % kStages];
    const float* ks = sm + at % kStages * C::kFloats;
    const float* qs = ks + kKT * LD;
    const float* ls = qs + ROWS * LD;
    const int key0 = d.kb * kKT + mine, tok0 = d.t * p.tile_tokens;
    const int rows = min(p.tile_tokens, d.v.n - tok0) * p.G;
    // the scores that the sums go to, asked for now
    float* scores = p.scores + (static_cast<long long>(d.b) * p.Hkv + d.h) * paged_cap(p) + key0;
    const bool adds = writes && d.last && d.first;
    float old[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) old[i] = adds && key0 + i < d.v.len ? scores[i] : 0.f;
    auto gain = [&](float s, int key, int r) {
      const float e = exp2f(fmaf(s, p.scale_log2, -1.4426950408889634f * ls[r]));
      return key < key_limit(p, d.b, d.v, tok0 + r / p.G) ? e : 0.f;
    };
    if constexpr (ROWS == 32) {
      const float* k4 = ks + (mine & ~3) * LD + part * 4;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 4) {
        const float x = dots_by_lanes<D, LD>(k4, qs + r0 * LD + part * 4, part);
        const int r = r0 + (part & 3);
        if (r < rows) sum[0] += gain(x, key0, r);
      }
    } else {
      float s[4][RPT];
      dots<D, 4, RPT>(ks + ty * 4 * LD, LD, 1, qs + tx * LD, LD, 16, s);
#pragma unroll
      for (int j = 0; j < RPT; ++j)
        if (tx + 16 * j < rows)
#pragma unroll
          for (int i = 0; i < kKeys; ++i) sum[i] += gain(s[i][j], key0 + i, tx + 16 * j);
    }
    if (!d.last) continue;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
#pragma unroll
      for (int k = ROWS == 32 ? 2 : 8; k; k >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], k);
      if (adds) {
        if (key0 + i < d.v.len) scores[i] = old[i] + sum[i];
      } else if (writes) {
        p.part_w[static_cast<long long>(blockIdx.x) * p.slot_rows + mine + i] = sum[i];
      }
      sum[i] = 0.f;
    }
    if (!d.first && threadIdx.x == 0) p.part_id[blockIdx.x] = make_int4(d.b, d.h, d.kb, 1);
  }
}

template <int D, int OWN, int PREFIX>
cudaError_t attend(cudaStream_t s, const PagedParams& p) {
  constexpr int kMax = OWN > PREFIX ? OWN : PREFIX;
  // scores, weights and factors of the few-row form, or weights
  constexpr int kLast = kMax == 16 ? 16 * (kKT + 4) + kKT * 16 + 16 : kMax * (kKT + 4);
  constexpr size_t smem = sizeof(float) * (kMax * (D + 4) + 4 * kKT * (D + 4) + kLast);
  static PerDeviceOnce once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(paged_attend_simt_kernel<D, OWN, PREFIX>),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  });
  return e != cudaSuccess
             ? e
             : launch_pdl(paged_attend_simt_kernel<D, OWN, PREFIX>, dim3(p.grid), dim3(kThreads), smem, s, p);
}
template <int D>
cudaError_t attend(cudaStream_t s, const PagedParams& p) {
  const bool own16 = p.item_tokens * p.G <= 16, prefix16 = p.prefix_item_tokens * p.G <= 16;
  if (!own16) return attend<D, 64, 64>(s, p);
  return prefix16 ? attend<D, 16, 16>(s, p) : attend<D, 16, 64>(s, p);
}
template <int D, int ROWS>
cudaError_t weights(cudaStream_t s, const PagedParams& p) {
  constexpr size_t smem = WeightsCfg<D, ROWS>::kSmem;
  static PerDeviceOnce once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(paged_weights_simt_kernel<D, ROWS>),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  });
  return e != cudaSuccess ? e
                          : launch_pdl(paged_weights_simt_kernel<D, ROWS>, dim3(p.grid), dim3(kThreads), smem, s, p);
}

}  // namespace

cudaError_t launch_paged_attend_simt(cudaStream_t s, const PagedParams& p) {
  return p.D == 64 ? attend<64>(s, p) : attend<128>(s, p);
}

cudaError_t launch_paged_weights_simt(cudaStream_t s, const PagedParams& p) {
  const bool few = p.tile_tokens * p.G <= 32;
  if (p.D == 64) return few ? weights<64, 32>(s, p) : weights<64, 64>(s, p);
  return few ? weights<128, 32>(s, p) : weights<128, 64>(s, p);
}

}  // namespace kvc
