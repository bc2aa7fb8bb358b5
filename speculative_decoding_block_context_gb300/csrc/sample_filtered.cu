// Tokens drawn under temperature, top-k, top-p and min-p from one uniform per row.
//
// With m the row's largest logit, w_j = exp((l_j - m) / T). In the order (l descending,
// j ascending) each filter keeps a prefix: top-k the first k entries; top-p the entries
// whose predecessors among those k hold less than p of their mass; min-p the entries with
// w >= min_p. The drawn entry is the lowest j with sum_{kept i <= j} w_i > u W, W the kept
// mass.
//
// Which entry a border or a draw falls on must not hang on rounding, so weights are
// integers: w 2^44 rounded, from an exponential good to about 1e-9, summed exactly in
// 64 bits in whatever order.
//
// One CTA per row; the row is read from L2 in every pass. Borders are found by radix
// selection on the logits' order-preserving bits, eight bits a pass, by count (top-k) or
// by mass (top-p).

#include <algorithm>
#include <climits>
#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace fm {
namespace {

constexpr int kSfThreads = 1024;
constexpr int kSfWarps = kSfThreads / 32;
constexpr int kFixBits = 44;  // 393216 weights of at most 1 sum below 2^63

__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// log2(e) / T in two float32 parts.
struct Slope {
  float hi, lo;
};
__device__ __forceinline__ Slope slope_of(float T) {
  const double c = 1.4426950408889634074 / static_cast<double>(T);
  Slope s;
  s.hi = static_cast<float>(c);
  s.lo = isinf(s.hi) ? 0.f : static_cast<float>(c - static_cast<double>(s.hi));
  return s;
}

// exp((l - m) / T) 2^44, rounded. With x = (l - m) log2(e) / T carried in two parts,
// x = n / 32 + r, |r| <= 1/64: 2^x = 2^(n / 32) (1 + (2^r - 1)), the first factor from a
// table of 32 values in two parts and the second's excess from four terms of its series
// (the fifth is below 4e-13).
__device__ __forceinline__ unsigned long long weight_fix(float l, float m, Slope c, const float2* tab) {
  if (l == m) return 1ull << kFixBits;
  const float d = __fsub_rn(l, m);  // l - m = d + e exactly
  const float bb = __fsub_rn(d, l);
  const float e = __fadd_rn(__fsub_rn(l, __fsub_rn(d, bb)), __fsub_rn(-m, bb));
  const float x = __fmul_rn(d, c.hi);
  if (!(x > -46.f)) return 0;  // below half a unit (or l not finite)
  const float lo = __fmaf_rn(d, c.hi, -x) + __fmaf_rn(d, c.lo, e * c.hi);
  const float nf = rintf(x * 32.f);
  const int n = static_cast<int>(nf);
  const float r = __fmaf_rn(nf, -0.03125f, x) + lo;
  const float q = r * (0.693147182f + r * (0.240226507f + r * (0.0555041087f + r * 0.00961812911f)));
  const float2 h = tab[n & 31];
  const float scale = __uint_as_float(static_cast<uint32_t>((n >> 5) + kFixBits + 127) << 23);
  return __float2ull_rn(h.x * scale) + __float2ll_rn(__fmaf_rn(h.x, q, h.y) * scale);
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p, int j) {
  return to_f32<T>(p[j]) + 0.f;  // -0 counts as 0
}
__device__ __forceinline__ bool usable(float l) { return l > -INFINITY; }  // neither -inf nor NaN

template <typename V>
__device__ __forceinline__ V warp_incl(V v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ unsigned long long block_sum_u64(unsigned long long v, unsigned long long* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  unsigned long long t = 0;
  for (int w = 0; w < kSfWarps; ++w) t += red[w];
  return t;
}

// A border in the order (l descending, j ascending): entries with a larger key, and the
// first `ties` (by index) of those with this key.
struct Border {
  uint32_t key;
  int ties;
};

template <typename T>
__global__ void __launch_bounds__(kSfThreads) sample_filtered_kernel(const SampleFilteredArgs a) {
  __shared__ float2 tab[32];
  __shared__ unsigned long long red[kSfWarps];
  __shared__ unsigned long long hist[256];
  __shared__ uint32_t s_digit;
  __shared__ unsigned long long s_above;
  __shared__ int s_pick;
  __shared__ unsigned long long s_pickw;
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t < 32) {
    const double h = exp2(t / 32.0);
    tab[t].x = static_cast<float>(h);
    tab[t].y = static_cast<float>(h - static_cast<double>(tab[t].x));
  }
  const int row = blockIdx.x, b = row / a.per, V = a.V;
  const T* lr = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.ld;
  const float temp = a.temperature[b];
  const bool greedy = !(temp > 0.f);
  int k = a.top_k ? a.top_k[b] : 0;
  if (k <= 0 || k > V) k = V;
  const float p = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
  float u = a.uniforms ? a.uniforms[row] : 0.f;
  u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;

  // the largest logit and its lowest index
  unsigned long long best = 0;
  for (int j = t; j < V; j += kSfThreads) {
    const float l = load_logit(lr, j);
    if (usable(l))
      best = max(best, (static_cast<unsigned long long>(order_key(l)) << 32) | (0xffffffffu - static_cast<uint32_t>(j)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) red[warp] = best;
  __syncthreads();
  for (int w = 0; w < kSfWarps; ++w) best = max(best, red[w]);
  const int top = best ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(best)) : 0;
  if (greedy || best == 0) {
    if (t == 0) {
      a.tokens[row] = a.ids ? a.ids[top] : top;
      if (a.probs) a.probs[row] = best ? 1.f : 0.f;
    }
    return;
  }
  const uint32_t top_key = static_cast<uint32_t>(best >> 32);
  const float m = key_value(top_key);
  const Slope c = slope_of(temp);
  __syncthreads();

  Border border{0, INT_MAX};  // everything
  if (k < V) {
    // radix selection by count: digits from the top; `left` entries still to take
    uint32_t prefix = 0;
    int left = k;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (t < 256) hist[t] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int j = t; j < V; j += kSfThreads) {
        const float l = load_logit(lr, j);
        const uint32_t key = order_key(l);
        if (usable(l) && (key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1ull);
      }
      __syncthreads();
      if (t == 0) {
        int d = 255;
        unsigned long long above = 0;
        while (d > 0 && above + hist[d] < static_cast<unsigned long long>(left)) above += hist[d--];
        s_digit = d;
        s_above = above;
      }
      __syncthreads();
      prefix |= s_digit << shift;
      left -= static_cast<int>(s_above);
      __syncthreads();
    }
    border = Border{prefix, left};  // fewer than k usable entries: prefix 0, everything kept
  }
  // the mass of what top-k keeps
  auto mass_of = [&](Border bd) {
    unsigned long long s = 0;
    for (int j = t; j < V; j += kSfThreads) {
      const float l = load_logit(lr, j);
      if (usable(l) && order_key(l) > bd.key) s += weight_fix(l, m, c, tab);
    }
    s = block_sum_u64(s, red);
    if (bd.ties != INT_MAX && bd.key != 0) s += static_cast<unsigned long long>(bd.ties) * weight_fix(key_value(bd.key), m, c, tab);
    return s;
  };
  if (p < 1.f) {
    const unsigned long long all = mass_of(border);
    const double want = p > 0.f ? ceil(static_cast<double>(p) * static_cast<double>(all)) : 1.0;
    unsigned long long left = min(all, max(1ull, static_cast<unsigned long long>(want)));
    uint32_t prefix = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (t < 256) hist[t] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int j = t; j < V; j += kSfThreads) {
        const float l = load_logit(lr, j);
        const uint32_t key = order_key(l);
        if (usable(l) && (key & mask) == prefix) {
          const unsigned long long w = weight_fix(l, m, c, tab);
          if (w) atomicAdd(&hist[(key >> shift) & 255], w);
        }
      }
      __syncthreads();
      if (t == 0) {
        int d = 255;
        unsigned long long above = 0;
        while (d > 0 && above + hist[d] < left) above += hist[d--];
        s_digit = d;
        s_above = above;
      }
      __syncthreads();
      prefix |= s_digit << shift;
      left -= s_above;
      __syncthreads();
    }
    const unsigned long long w = weight_fix(key_value(prefix), m, c, tab);
    const unsigned long long n = w ? (left + w - 1) / w : 1;
    int ties = static_cast<int>(min(n, static_cast<unsigned long long>(INT_MAX - 1)));
    if (prefix == border.key) ties = min(ties, border.ties);
    border = Border{prefix, ties};
  }
  const unsigned long long least =
      mp > 0.f ? static_cast<unsigned long long>(ceil(static_cast<double>(fminf(mp, 1.f)) * (1ull << kFixBits))) : 0;

  // Index order: each warp takes a contiguous share of the row; first the shares' ties
  // (those at the border's key are kept lowest index first), then their kept mass, then
  // the share that holds the draw is walked.
  const int share = ((V + kSfWarps - 1) / kSfWarps + 31) / 32 * 32;
  const int j0 = warp * share, j1 = min(V, j0 + share);
  __shared__ int s_ties[kSfWarps];
  int ties_before = 0;
  if (border.ties != INT_MAX) {
    int n = 0;
    for (int j = j0 + lane; j < j1; j += 32) {
      const float l = load_logit(lr, j);
      n += usable(l) && order_key(l) == border.key;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) s_ties[warp] = n;
    __syncthreads();
    for (int w = 0; w < warp; ++w) ties_before += s_ties[w];
  }
  // kept weight of entry j for a lane, the warp's running tie count in `seen`
  auto kept_weight = [&](int j, int& seen) -> unsigned long long {
    const float l = j < j1 ? load_logit(lr, j) : -INFINITY;
    const uint32_t key = order_key(l);
    bool keep = usable(l) && key > border.key;
    if (border.ties != INT_MAX) {
      const bool tie = usable(l) && key == border.key;
      const unsigned votes = __ballot_sync(0xffffffffu, tie);
      if (tie) keep = seen + __popc(votes & ((1u << lane) - 1)) < border.ties;
      seen += __popc(votes);
    } else {
      keep = usable(l);
    }
    if (!keep) return 0;
    const unsigned long long w = weight_fix(l, m, c, tab);
    return w >= least ? w : 0;
  };
  unsigned long long mine = 0;
  int seen = ties_before;
  for (int j = j0; j < j1; j += 32) mine += kept_weight(j + lane, seen);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  __syncthreads();
  if (lane == 0) red[warp] = mine;
  if (t == 0) s_pick = -1;
  __syncthreads();
  unsigned long long before = 0, total = 0;
  for (int w = 0; w < kSfWarps; ++w) {
    if (w < warp) before += red[w];
    total += red[w];
  }
  const unsigned long long draw = static_cast<unsigned long long>(static_cast<double>(u) * static_cast<double>(total));
  if (before <= draw && draw < before + mine) {
    unsigned long long at = before;
    int s2 = ties_before;
    for (int j = j0; j < j1; j += 32) {
      const unsigned long long w = kept_weight(j + lane, s2);
      const unsigned long long incl = at + warp_incl(w);
      const unsigned hit = __ballot_sync(0xffffffffu, incl > draw);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          s_pick = j + lane;
          s_pickw = w;
        }
        break;
      }
      at = __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  __syncthreads();
  if (t == 0) {
    const int j = s_pick >= 0 ? s_pick : top;
    a.tokens[row] = a.ids ? a.ids[j] : j;
    if (a.probs) a.probs[row] = static_cast<float>(static_cast<double>(s_pickw) / static_cast<double>(total));
  }
}

}  // namespace

cudaError_t sample_filtered(const Launch& L, const SampleFilteredArgs& a) {
  return launch_k(L, a.dtype == FLASHMAP_F32 ? sample_filtered_kernel<float> : sample_filtered_kernel<__nv_bfloat16>,
                  dim3(a.rows), dim3(kSfThreads), 0, a);
}

}  // namespace fm
