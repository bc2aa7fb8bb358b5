// The tree attention's partition of a batch into equal shares, and the kernel that joins
// row tiles cut by it (used by the CUDA-core and the tensor-core kernels).
#pragma once

#include <climits>
#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace fm {
namespace {

constexpr int kTreeMaxWidth = kTreeMaxNodes + 1;

// ------------------------------------------------------------------ the partition

struct Request {
  int ctx, n;  // positions before the root, nodes (0: nothing to do)
};

__device__ __forceinline__ Request request_of(const TreeAttnArgs& a, int b, unsigned& err) {
  Request r;
  r.ctx = LDCG(a.ctx_lens + b);
  r.n = a.num_nodes ? LDCG(a.num_nodes + b) : a.width;
  if (r.n < 0 || r.n > a.width) err |= FLASHMAP_DEVERR_TREE, r.n = min(max(r.n, 0), a.width);
  if (r.ctx < 0 || r.ctx > INT_MAX - kTreeMaxWidth - 256) err |= FLASHMAP_DEVERR_POSITION, r.n = 0, r.ctx = 0;
  const int row = LDCG(a.req_pool_idx + b);
  if (row < 0 || row >= a.table_rows) err |= FLASHMAP_DEVERR_REQUEST, r.n = 0;
  return r;
}

template <int TM, int TN>
struct Cut {
  __device__ static int row_tiles(const TreeAttnArgs& a, Request r) { return (r.n * a.group + TM - 1) / TM; }
  __device__ static int pos_tiles(Request r) { return (r.ctx + r.n + TN - 1) / TN; }
  __device__ static int64_t units(const TreeAttnArgs& a, Request r) {
    return r.n > 0 ? static_cast<int64_t>(a.nkv) * row_tiles(a, r) * pos_tiles(r) : 0;
  }
};

struct Spot {
  int b;         // the request that holds the unit
  int64_t base;  // its first unit
};

// Inclusive sum over the block in thread order; `total` over all threads.
template <int THREADS>
__device__ __forceinline__ int64_t unit_scan(int64_t v, int64_t* red, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) red[warp] = v;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int64_t s = red[w];
    if (w < warp) before += s;
    total += s;
  }
  return v + before;
}

// The batch's units T, and the request of unit T c / G (b = bs when there is none, T = 0).
// Called by the whole block; every thread gets the answer.
template <int THREADS, int TM, int TN>
__device__ __forceinline__ int64_t locate(const TreeAttnArgs& a, int c, int G, Spot& spot, unsigned& err,
                                          int64_t* red, Spot* shared_spot) {
  const int t = threadIdx.x;
  int64_t T = 0, mine = 0, incl = 0;
  for (int b0 = 0; b0 < a.bs; b0 += THREADS) {
    const int b = b0 + t;
    const int64_t v = b < a.bs ? Cut<TM, TN>::units(a, request_of(a, b, err)) : 0;
    int64_t chunk;
    const int64_t i = unit_scan<THREADS>(v, red, chunk);
    if (b0 == 0) mine = v, incl = i;
    T += chunk;
  }
  if (t == 0) *shared_spot = Spot{a.bs, 0};
  __syncthreads();
  const int64_t u = T * c / G;
  if (t < a.bs && incl - mine <= u && u < incl) *shared_spot = Spot{t, incl - mine};
  int64_t before = 0;
  if (a.bs > THREADS) {  // the unit may lie past the first chunk
    unsigned none = 0;
    for (int b0 = 0; b0 < a.bs; b0 += THREADS) {
      const int b = b0 + t;
      const int64_t v = b < a.bs ? Cut<TM, TN>::units(a, request_of(a, b, none)) : 0;
      int64_t chunk;
      const int64_t i = before + unit_scan<THREADS>(v, red, chunk);
      if (b0 > 0 && b < a.bs && i - v <= u && u < i) *shared_spot = Spot{b, i - v};
      before += chunk;
    }
  }
  __syncthreads();
  spot = *shared_spot;
  return T;
}

// One CTA's walk over its units, row tile by row tile.
template <int TM, int TN>
struct Walk {
  int64_t u, u1, base;  // next unit, the range's end, the request's first unit
  int b;
  Request r;
  int nt, mt;              // position tiles and row tiles of the request
  int head, tile_m, t0, t1;  // the item: key/value head, row tile, its position tiles
  bool first_item, whole;  // the range's first item; it holds all of the row tile's positions
  bool started;

  __device__ void enter(const TreeAttnArgs& a) {
    unsigned none = 0;
    r = request_of(a, b, none);
    nt = Cut<TM, TN>::pos_tiles(r);
    mt = Cut<TM, TN>::row_tiles(a, r);
  }
  __device__ Walk(const TreeAttnArgs& a, Spot s, int64_t begin, int64_t end)
      : u(begin), u1(end), base(s.base), b(s.b), first_item(false), started(false) {
    if (u < u1) enter(a);
  }
  // The next item; false when the range is done.
  __device__ bool next(const TreeAttnArgs& a) {
    if (u >= u1) return false;
    while (r.n <= 0 || u - base >= static_cast<int64_t>(a.nkv) * mt * nt) {
      base += r.n > 0 ? static_cast<int64_t>(a.nkv) * mt * nt : 0;
      ++b;
      enter(a);
    }
    const int64_t local = u - base;
    const int g = static_cast<int>(local / nt);
    t0 = static_cast<int>(local - static_cast<int64_t>(g) * nt);
    head = g / mt;
    tile_m = g - head * mt;
    t1 = static_cast<int>(min(static_cast<int64_t>(nt), t0 + (u1 - u)));
    first_item = !started;
    started = true;
    whole = t0 == 0 && t1 == nt;
    u += t1 - t0;
    return true;
  }
};

// The parent of node i >= 1: the previous node of a chain, else the node its id names.
__device__ __forceinline__ int parent_of(const TreeAttnArgs& a, int b, int i, unsigned& err) {
  if (!a.tree_ids) return i - 1;
  const int64_t id = LDCG(a.tree_ids + static_cast<int64_t>(b) * (a.width - 1) + (i - 1));
  const int64_t p = id >= 0 ? id / a.width : -1;
  if (p < 0 || p >= i || id - p * a.width != i) {
    err |= FLASHMAP_DEVERR_TREE;
    return -1;  // no ancestors
  }
  return static_cast<int>(p);
}

// ------------------------------------------------------------------ joining split row tiles

// Block c + 1 (x) looks at the border between CTAs c and c + 1 of the kernel before: if it
// is the first border inside a row tile, the block joins that row tile's parts in CTA
// order. Rows are spread over the blocks along y, a warp per row.
constexpr int kJoinThreads = 256, kJoinY = 4;

template <typename T, int HD, int TM, int TN>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeAttnArgs a) {
  __shared__ int64_t red[kJoinThreads / 32];
  __shared__ Spot s_spot;
  pdl_trigger();
  pdl_wait();
  const int G = gridDim.x + 1, c = blockIdx.x + 1;
  unsigned none = 0;
  Spot spot;
  const int64_t units = locate<kJoinThreads, TM, TN>(a, c, G, spot, none, red, &s_spot);
  const int64_t u = units * c / G;
  if (u >= units) return;
  const Request r = request_of(a, spot.b, none);
  const int nt = Cut<TM, TN>::pos_tiles(r), mt = Cut<TM, TN>::row_tiles(a, r);
  const int64_t g = (u - spot.base) / nt;
  const int64_t g0 = spot.base + g * nt, g1 = g0 + nt;  // the row tile's units
  if (u <= g0 || units * (c - 1) / G > g0) return;      // no border inside it, or not its first
  const int head = static_cast<int>(g / mt), tile_m = static_cast<int>(g - static_cast<int64_t>(head) * mt);
  const int rows = min(TM, r.n * a.group - tile_m * TM);
  const int first = 2 * (c - 1) + (units * (c - 1) / G == g0 ? 0 : 1);  // CTA c - 1 may have begun elsewhere
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int E = HD / 32;
  for (int row = blockIdx.y * (kJoinThreads / 32) + warp; row < rows; row += kJoinY * (kJoinThreads / 32)) {
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int p = c - 1; p < G && units * p / G < g1; ++p) {
      if (units * p / G == units * (p + 1) / G) continue;
      const int64_t at = static_cast<int64_t>(p == c - 1 ? first : 2 * p) * TM + row;
      const float2 ml = __ldcg(a.part_ml + at);
      const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.f : mn;
      const float f0 = exp2f(m - base), f1 = exp2f(ml.x - base);
      l = l * f0 + ml.y * f1;
      m = mn;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f0 + LDCG(a.part_o + at * HD + lane + 32 * e) * f1;
    }
    const int rr = tile_m * TM + row, i = rr / a.group, h = rr - i * a.group;
    T* dst = static_cast<T*>(a.out) + ((static_cast<int64_t>(spot.b) * a.width + i) * a.nq + head * a.group + h) * HD;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[lane + 32 * e] = from_f32<T>(o[e] * inv);
  }
}

}  // namespace
}  // namespace fm
