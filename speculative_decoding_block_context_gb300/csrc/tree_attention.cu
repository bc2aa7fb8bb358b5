// Attention of a tree of drafted tokens over a paged cache. Node i of request b sits at
// cache position ctx[b] + i; it sees positions below ctx[b], itself and its ancestors:
//   out = sum_j softmax_j(scale q k_j) v_j
// with grouped heads: query heads h * group .. h * group + group - 1 read key/value head h.
//
// A request's nodes and a key/value head's group of query heads make n * group query rows
// that read the same keys, so they share one pass over them. The work is cut into units
// (request, key/value head, row tile, position tile), in that order, and CTA c of G takes
// units [T c / G, T (c + 1) / G): every CTA streams about the same number of tiles whatever
// the requests' lengths. T hangs on lengths that only the device knows, so each CTA sums the
// batch's units itself. A row tile that spans several CTAs leaves partial sums (running
// maximum, sum and unnormalised output, float32) which a second kernel joins in CTA order.

#include <algorithm>
#include <climits>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "tree_common.cuh"

namespace fm {
namespace {

// ------------------------------------------------------------------ on the CUDA cores

// float32 (whose products the tensor cores would round) and heads of 32 in bf16: 32 rows
// by 64 positions a tile, each thread 2 rows x 4 positions of the scores and 2 rows x
// HD / 16 channels of the output, operands in shared memory as float32. Bound by the float32
// pipe and shared memory: 64 requests of 4 nodes, 8 heads of 64 over up to 3000 positions take
// 453 us; two CTAs an SM, so that one's loads run under the other's sums.
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
  const Share share = locate<C::THREADS, TM, TN, 1, 1>(a, spot, err, red, &s_spot);
  Walk<TM, TN> w(a, share, spot);
  const float k2 = a.scale * 1.4426950408889634f;
  int tree_b = -1;
  while (w.next(a)) {
    const int rows = min(TM, w.r.n * a.group - w.tile_m * TM);
    const int64_t table = static_cast<int64_t>(w.r.row) * a.stride;
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
    const int slot = 2 * static_cast<int>(blockIdx.x) + (w.first_item ? 0 : 1);
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
  if (tid == 0) write_join_task(a, share, w);
  if (err) set_dev_error(a.dev_err, err);
}

template <typename T, int HD>
cudaError_t launch_simt(const Launch& L, const TreeAttnArgs& a, int G) {
  using C = Simt<HD>;
  cudaError_t e = cudaFuncSetAttribute(tree_simt_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e == cudaSuccess) e = launch_k(L, tree_simt_kernel<T, HD>, dim3(G), dim3(C::THREADS), C::SMEM, a);
  if (e == cudaSuccess && G > 1)
    e = launch_k(L, tree_join_kernel<T, HD, C::TM>, dim3(G - 1, kJoinY), dim3(kJoinThreads), 0, a);
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
size_t simt_bytes(int hd, int num_sms) {
  return join_tasks_bytes(simt_ctas(num_sms)) +
         static_cast<size_t>(2 * simt_ctas(num_sms)) * 32 * (static_cast<size_t>(hd) * 4 + 8);
}
}  // namespace

size_t tree_attention_bytes(int dtype, int hd, int width, int group, int num_sms) {
  return tree_mma_fits(dtype, hd) ? tree_mma_bytes(hd, width, group, num_sms) : simt_bytes(hd, num_sms);
}

cudaError_t tree_attention(const Launch& L, TreeAttnArgs a, void* workspace) {
  if (tree_mma_fits(a.dtype, a.hd)) return tree_mma(L, a, workspace);
  const int G = simt_ctas(L.num_sms);
  a.tasks = workspace;
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + join_tasks_bytes(G));
  a.part_o = reinterpret_cast<float*>(a.part_ml + static_cast<size_t>(2 * G) * 32);
  return a.dtype == FLASHMAP_F32 ? launch_simt_hd<float>(L, a, G) : launch_simt<__nv_bfloat16, 32>(L, a, G);
}

}  // namespace fm
