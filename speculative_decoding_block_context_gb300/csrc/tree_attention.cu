// Attention of a tree of drafted tokens over a paged cache. Node i of request b sits at
// cache position ctx[b] + i; it sees positions below ctx[b], itself and its ancestors:
//   out = sum_j softmax_j(scale q k_j) v_j
// with grouped heads: query heads h * group .. h * group + group - 1 read key/value head h.
//
// A request's nodes and a key/value head's group of query heads make n * group query rows
// that read the same keys, so they share one pass over them. The work is cut into units
// (request, key/value head, row tile, position tile), in that order, and CTA c of G takes
// units [T c / G, T (c + 1) / G): every CTA streams the same number of tiles whatever the
// requests' lengths. T hangs on lengths that only the device knows, so each CTA sums the
// batch's units itself. A row tile that spans several CTAs leaves partial sums (running
// maximum, sum and unnormalised output, float32) which a second kernel joins in CTA order.

#include <algorithm>
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

  __device__ void enter(const TreeAttnArgs& a) {
    unsigned none = 0;
    r = request_of(a, b, none);
    nt = Cut<TM, TN>::pos_tiles(r);
    mt = Cut<TM, TN>::row_tiles(a, r);
  }
  __device__ Walk(const TreeAttnArgs& a, Spot s, int64_t begin, int64_t end)
      : u(begin), u1(end), base(s.base), b(s.b), first_item(true) {
    if (u < u1) enter(a);
    t1 = 0;
    first_item = false;
    started = false;
  }
  bool started;
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

// ------------------------------------------------------------------ on the CUDA cores

// float32 (whose products the tensor cores would round) and heads of 32 in bf16: 32 rows
// by 64 positions a tile, each thread 2 rows x 4 positions of the scores and 2 rows x
// HD / 16 channels of the output, operands in shared memory as float32.
template <int HD>
struct Simt {
  static constexpr int TM = 32, TN = 64, THREADS = 256;
  static constexpr int LQ = HD + 4, LP = TN + 4;
  static constexpr int SMEM = static_cast<int>(sizeof(float)) * (TM * LQ + TN * LQ + TN * HD + TM * LP);
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&v)[4]);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x.x));
  const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x.y));
  v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
}

template <typename T, int HD>
__global__ void __launch_bounds__(256) tree_simt_kernel(const TreeAttnArgs a) {
  using C = Simt<HD>;
  constexpr int TM = C::TM, TN = C::TN, LQ = C::LQ, LP = C::LP, EC = HD / 16;
  extern __shared__ float smem_f[];
  float* sq = smem_f;
  float* sk = sq + TM * LQ;
  float* sv = sk + TN * LQ;
  float* sp = sv + TN * HD;
  __shared__ int64_t red[C::THREADS / 32];
  __shared__ Spot s_spot;
  __shared__ short parent[kTreeMaxWidth];
  __shared__ uint32_t vis[TM][TN / 32];  // this tile's visible tree positions per row
  __shared__ uint32_t okbits[TN / 32];   // positions that could be read
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  unsigned err = 0;
  Spot spot;
  const int G = gridDim.x, c = blockIdx.x;
  const int64_t units = locate<C::THREADS, TM, TN>(a, c, G, spot, err, red, &s_spot);
  const int64_t u0 = units * c / G, u1 = units * (c + 1) / G;
  Walk<TM, TN> w(a, spot, u0, u1);
  const float k2 = a.scale * 1.4426950408889634f;
  int tree_b = -1;
  while (w.next(a)) {
    const int rows = min(TM, w.r.n * a.group - w.tile_m * TM);
    const int64_t table = static_cast<int64_t>(LDCG(a.req_pool_idx + w.b)) * a.stride;
    const int end = w.r.ctx + w.r.n;
    __syncthreads();
    if (w.t1 * TN > w.r.ctx && tree_b != w.b) {  // the item reaches the tree
      for (int i = tid; i < w.r.n; i += C::THREADS) parent[i] = static_cast<short>(i ? parent_of(a, w.b, i, err) : -1);
      tree_b = w.b;
    }
    for (int x = tid; x < TM * (HD / 4); x += C::THREADS) {
      const int row = x / (HD / 4), d = (x - row * (HD / 4)) * 4;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (row < rows) {
        const int rr = w.tile_m * TM + row, i = rr / a.group, h = rr - i * a.group;
        load4(static_cast<const T*>(a.q) + (static_cast<int64_t>(w.b) * a.width + i) * a.q_stride +
                  static_cast<int64_t>(w.head * a.group + h) * HD + d, v);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sq[row * LQ + d + e] = v[e];
    }
    float o[2][EC], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int e = 0; e < EC; ++e) o[r][e] = 0.f;
    for (int tile = w.t0; tile < w.t1; ++tile) {
      const int p0 = tile * TN;
      __syncthreads();  // the previous tile's readers are done
      if (tid < TN / 32) okbits[tid] = 0;
      __syncthreads();
      for (int x = tid; x < TN * (HD / 4); x += C::THREADS) {
        const int col = x / (HD / 4), d = (x - col * (HD / 4)) * 4, pos = p0 + col;
        float kv[4] = {0.f, 0.f, 0.f, 0.f}, vv[4] = {0.f, 0.f, 0.f, 0.f};
        if (pos < end) {
          const int pc = pos / a.P;
          const int page = pc < a.stride ? LDCG(a.req_to_page + table + pc) : -1;
          if (page < 0 || page >= a.num_pages) {
            err |= pc < a.stride ? FLASHMAP_DEVERR_PAGE : FLASHMAP_DEVERR_POSITION;
          } else {
            const int64_t at = ((static_cast<int64_t>(page) * a.nkv + w.head) * a.P + (pos - pc * a.P)) * HD + d;
            load4(static_cast<const T*>(a.keys) + at, kv);
            load4(static_cast<const T*>(a.values) + at, vv);
            if (d == 0) atomicOr(&okbits[col >> 5], 1u << (col & 31));
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sk[col * LQ + d + e] = kv[e];
          sv[col * HD + d + e] = vv[e];
        }
      }
      if (p0 + TN > w.r.ctx && tid < rows) {  // what each row sees of a tile that reaches the tree
        uint32_t bits[TN / 32];
#pragma unroll
        for (int x = 0; x < TN / 32; ++x) {
          const int before = w.r.ctx - (p0 + 32 * x);  // context positions of this word
          bits[x] = before >= 32 ? 0xffffffffu : before <= 0 ? 0u : (1u << before) - 1;
        }
        for (int i = (w.tile_m * TM + tid) / a.group; i >= 0; i = parent[i]) {
          const int at = w.r.ctx + i - p0;
          if (at < 0) break;  // ancestors only come earlier
#pragma unroll
          for (int x = 0; x < TN / 32; ++x)
            if ((at >> 5) == x) bits[x] |= 1u << (at & 31);
        }
#pragma unroll
        for (int x = 0; x < TN / 32; ++x) vis[tid][x] = bits[x];
      }
      __syncthreads();
      float s[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[r][j] = 0.f;
      for (int d = 0; d < HD; d += 4) {
        float4 q4[2], k4[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) q4[r] = *reinterpret_cast<const float4*>(sq + (ty + 16 * r) * LQ + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * LQ + d);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[r][j] = fmaf(q4[r].x, k4[j].x, fmaf(q4[r].y, k4[j].y, fmaf(q4[r].z, k4[j].z, fmaf(q4[r].w, k4[j].w, s[r][j]))));
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = ty + 16 * r;
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = tx + 16 * j;
          bool see = row < rows && (okbits[col >> 5] >> (col & 31) & 1u);
          if (see && p0 + TN > w.r.ctx) see = vis[row][col >> 5] >> (col & 31) & 1u;
          s[r][j] = see ? s[r][j] * k2 : -INFINITY;
          mx = fmaxf(mx, s[r][j]);
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float mn = fmaxf(m[r], mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m[r] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(s[r][j] - base);
          sum += e;
          sp[row * LP + tx + 16 * j] = e;
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l[r] = l[r] * f + sum;
        m[r] = mn;
#pragma unroll
        for (int e = 0; e < EC; ++e) o[r][e] *= f;
      }
      __syncwarp();  // a row's probabilities are written and read by one half warp
      for (int j = 0; j < TN; j += 4) {
        float4 p4[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) p4[r] = *reinterpret_cast<const float4*>(sp + (ty + 16 * r) * LP + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          float v[EC];
          if constexpr (EC >= 4) {
#pragma unroll
            for (int x = 0; x < EC / 4; ++x) {
              const float4 v4 = *reinterpret_cast<const float4*>(sv + (j + jj) * HD + x * 64 + tx * 4);
              v[4 * x] = v4.x, v[4 * x + 1] = v4.y, v[4 * x + 2] = v4.z, v[4 * x + 3] = v4.w;
            }
          } else {
            const float2 v2 = *reinterpret_cast<const float2*>(sv + (j + jj) * HD + tx * 2);
            v[0] = v2.x, v[1] = v2.y;
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p = jj == 0 ? p4[r].x : jj == 1 ? p4[r].y : jj == 2 ? p4[r].z : p4[r].w;
#pragma unroll
            for (int e = 0; e < EC; ++e) o[r][e] = fmaf(p, v[e], o[r][e]);
          }
        }
      }
    }
    const int slot = 2 * c + (w.first_item ? 0 : 1);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = ty + 16 * r;
      if (row >= rows) continue;
      if (w.whole) {
        const int rr = w.tile_m * TM + row, i = rr / a.group, h = rr - i * a.group;
        T* dst = static_cast<T*>(a.out) + ((static_cast<int64_t>(w.b) * a.width + i) * a.nq + w.head * a.group + h) * HD;
        const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
#pragma unroll
        for (int e = 0; e < EC; ++e) {
          const int ch = EC >= 4 ? (e >> 2) * 64 + tx * 4 + (e & 3) : tx * 2 + e;
          dst[ch] = from_f32<T>(o[r][e] * inv);
        }
      } else {
        float* dst = a.part_o + (static_cast<int64_t>(slot) * TM + row) * HD;
#pragma unroll
        for (int e = 0; e < EC; ++e) dst[EC >= 4 ? (e >> 2) * 64 + tx * 4 + (e & 3) : tx * 2 + e] = o[r][e];
        if (tx == 0) a.part_ml[static_cast<int64_t>(slot) * TM + row] = make_float2(m[r], l[r]);
      }
    }
  }
  if (err) set_dev_error(a.dev_err, err);
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

template <typename T, int HD>
cudaError_t launch_simt(const Launch& L, const TreeAttnArgs& a, int G) {
  using C = Simt<HD>;
  cudaError_t e = cudaFuncSetAttribute(tree_simt_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e == cudaSuccess) e = launch_k(L, tree_simt_kernel<T, HD>, dim3(G), dim3(C::THREADS), C::SMEM, a);
  if (e == cudaSuccess && G > 1)
    e = launch_k(L, tree_join_kernel<T, HD, C::TM, C::TN>, dim3(G - 1, kJoinY), dim3(kJoinThreads), 0, a);
  return e;
}

template <typename T>
cudaError_t launch_simt_hd(const Launch& L, const TreeAttnArgs& a, int G) {
  switch (a.hd) {
    case 32: return launch_simt<T, 32>(L, a, G);
    case 64: return launch_simt<T, 64>(L, a, G);
    case 128: return launch_simt<T, 128>(L, a, G);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

namespace {
int simt_ctas(int num_sms) { return 2 * num_sms; }
}  // namespace

size_t tree_attention_bytes(int dtype, int hd, int width, int group, int num_sms) {
  const int G = simt_ctas(num_sms);
  return static_cast<size_t>(2 * G) * 32 * (static_cast<size_t>(hd) * 4 + 8);
}

cudaError_t tree_attention(const Launch& L, TreeAttnArgs a, void* workspace) {
  const int G = simt_ctas(L.num_sms);
  a.part_ml = static_cast<float2*>(workspace);
  a.part_o = reinterpret_cast<float*>(a.part_ml + static_cast<size_t>(2 * G) * 32);
  return a.dtype == FLASHMAP_F32 ? launch_simt_hd<float>(L, a, G) : launch_simt_hd<__nv_bfloat16>(L, a, G);
}

}  // namespace fm
