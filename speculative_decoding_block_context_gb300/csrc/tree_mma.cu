// Tree attention on the tensor cores, for bf16 caches with heads of 64 or 128 channels.
//
// An item is (request, key/value head, row tile) over a run of position tiles: TM query
// rows (MT tiles of 128: node-major, the group's heads of a node side by side) against 128
// positions at a time. Per position tile and row tile
//   S = Q K^T   tcgen05.mma, both operands in shared memory, S in TMEM (float32)
//   P = exp2(S scale log2 e - m), bf16, written back over S in TMEM
//   O += P V    tcgen05.mma, P from TMEM, V from shared memory as it was loaded
// The running maximum m of a row moves only when a score passes it by more than 2^8, so O
// is seldom rescaled; the row's sum is kept in float32 from the unrounded exponentials.
//
// Warp 0 loads 16-position blocks (a page holds whole ones) by TMA into a ring of K and V
// tiles in the order the products take them; warp 1 issues the products; four warps per
// row tile, one thread per row, do the softmax and the epilogue.

#include <algorithm>
#include <climits>
#include <cstdint>
#include <string>

#include "common.cuh"
#include "internal.h"
#include "tree_common.cuh"

namespace fm {
namespace {

constexpr int TN = 128;  // positions per tile

template <int HD, int MT>
struct MmaCfg {
  static constexpr int TM = 128 * MT;
  static constexpr int THREADS = 64 + 128 * MT;
  static constexpr int NB = MT == 1 ? 2 : 1;  // S buffers per row tile
  static constexpr int TILE = TN * HD * 2;    // bytes of a K, V or Q tile (128 rows)
  static constexpr int SLOTS = HD == 64 ? 8 : MT == 1 ? 5 : 4;
  static constexpr int SMEM = MT * TILE + SLOTS * TILE + 1024;
  static constexpr int O_COL = MT * NB * 128;  // TMEM column of the first row tile's output
};
constexpr int kTmemCols = 512;

__device__ __forceinline__ void tmem_ld32w(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld128w(uint32_t taddr, uint32_t (&r)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]), "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]), "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]), "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]), "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]), "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]), "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]), "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}

// D (TMEM) = A (TMEM, bf16 pairs) x B (shared memory) (+ D).
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// A wait by a whole warp: every lane gets the same answer, so none is left behind at a
// later warp-wide instruction when the wait gives up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Descriptor of an operand tile whose rows run along the product's k (a V tile: rows are
// positions, 64 channels = 128 swizzled bytes a row): 8-row groups 1024 bytes apart (stride
// byte offset), the next 64 channels half a tile further (leading byte offset).
__device__ __forceinline__ uint64_t sdesc_sw128_rows_k(uint32_t saddr, uint32_t half_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(half_bytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

template <int HD, int MT>
__global__ void __launch_bounds__(MmaCfg<HD, MT>::THREADS, 1)
    tree_mma_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const TreeAttnArgs a) {
  using C = MmaCfg<HD, MT>;
  constexpr int TM = C::TM, NB = C::NB, SLOTS = C::SLOTS, HALF = TN * 128;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[SLOTS], empty[SLOTS], q_ready[MT], s_full[MT][NB], p_ready[MT][NB], pv_done[MT][NB],
      o_free[MT], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ int64_t red[C::THREADS / 32];
  __shared__ Spot s_spot;
  __shared__ int s_issued;
  __shared__ volatile uint8_t blocks_ok[16];  // per position tile (mod 16): its readable 16-position blocks
  __shared__ short s_parent[4 * MT][kTreeMaxWidth];  // a copy per warp

  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sq = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* ring = sq + MT * C::TILE;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int m = 0; m < MT; ++m) {
      mbar_init(&q_ready[m], 4);
      mbar_init(&o_free[m], 4);
      for (int i = 0; i < NB; ++i) {
        mbar_init(&s_full[m][i], 1);
        mbar_init(&p_ready[m][i], 4);
        mbar_init(&pv_done[m][i], 1);
      }
    }
    mbar_init(&drain, 1);
    abort_flag = 0;
    s_issued = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_trigger();
  pdl_wait();

  unsigned err = 0;
  Spot spot;
  const int G = gridDim.x, c = blockIdx.x;
  const int64_t units = locate<C::THREADS, TM, TN>(a, c, G, spot, err, red, &s_spot);
  const int64_t u0 = units * c / G, u1 = units * (c + 1) / G;
  Walk<TM, TN> w(a, spot, u0, u1);
  volatile int* ab = &abort_flag;

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    const int total_rows = static_cast<int>(a.num_pages) * a.nkv * a.P;  // a box from here on reads zeros
    const uint64_t pol = a.width * a.group <= TM ? l2_policy_evict_first() : l2_policy_evict_last();
    int slot = 0, issued = 0, seq = 0;
    uint32_t phase = 0;
    bool ok = true;
    // A tile of K (or V): lane j < 8 requests the tile's j-th block.
    auto load_tile = [&](const CUtensorMap* map, int row) {
      if (!warp_wait(&empty[slot], phase ^ 1u, ab)) return false;
      if (lane == 0) mbar_arrive_expect_tx(&full[slot], C::TILE);
      __syncwarp();
      if (lane < 8) {
        uint8_t* dst = ring + slot * C::TILE + lane * 2048;
#pragma unroll
        for (int h = 0; h < HD / 64; ++h) tma_load_2d(dst + h * HALF, map, &full[slot], h * 64, row, pol);
      }
      ++issued;
      if (++slot == SLOTS) slot = 0, phase ^= 1u;
      return true;
    };
    while (ok && w.next(a)) {
      const int end = w.r.ctx + w.r.n;
      const int64_t table = static_cast<int64_t>(LDCG(a.req_pool_idx + w.b)) * a.stride;
      // the page of this lane's block in a tile (INT_MIN: nothing there)
      auto page_of = [&](int t) {
        const int pos = t * TN + lane * 16;
        if (lane >= 8 || t >= w.t1 || pos >= end) return INT_MIN;
        const int pc = pos / a.P;
        if (pc >= a.stride) {
          err |= FLASHMAP_DEVERR_POSITION;
          return INT_MIN;
        }
        return LDCG(a.req_to_page + table + pc);
      };
      auto row_of = [&](int t, int page) {
        if (page < 0 || page >= a.num_pages) {
          if (page != INT_MIN) err |= FLASHMAP_DEVERR_PAGE;
          return total_rows;
        }
        const int pos = t * TN + lane * 16;
        return (page * a.nkv + w.head) * a.P + pos % a.P;
      };
      int page = page_of(w.t0), row_prev = total_rows;
      for (int t = w.t0; t < w.t1; ++t) {
        const int row = row_of(t, page);
        page = page_of(t + 1);  // asked for while the ring is waited for
        const unsigned bits = __ballot_sync(0xffffffffu, row != total_rows) & 0xffu;
        if (lane == 0) blocks_ok[seq & 15] = static_cast<uint8_t>(bits);
        ++seq;
        if (!(ok = load_tile(&kmap, row))) break;
        if (NB == 1) {
          if (!(ok = load_tile(&vmap, row))) break;
        } else if (t > w.t0 && !(ok = load_tile(&vmap, row_prev))) {
          break;
        }
        row_prev = row;
      }
      if (ok && NB == 2) ok = load_tile(&vmap, row_prev);
    }
    if (lane == 0) s_issued = issued;
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, TN);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, HD) | (1u << 16);  // B rows run along k
    const uint32_t q0 = smem_u32(sq), r0 = smem_u32(ring);
    int slot = 0;
    uint32_t phase = 0;
    int items[MT] = {}, ns[MT] = {}, np[MT] = {};  // items, score and value products issued per row tile
    bool ok = true;
    while (ok && w.next(a)) {
      const int rows = min(TM, w.r.n * a.group - w.tile_m * TM);
      const int nm = (rows + 127) >> 7;
      const int end = w.r.ctx + w.r.n;
      auto scores = [&](int m, uint32_t kaddr) {
        const int buf = ns[m] % NB;
        // P of the tile that last used this buffer has been taken by its product
        if (ns[m] >= NB && !warp_wait(&pv_done[m][buf], ((ns[m] / NB) + 1) & 1, ab)) return false;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t d = tmem + static_cast<uint32_t>((m * NB + buf) * 128);
#pragma unroll
          for (int s = 0; s < HD / 16; ++s) {
            const uint32_t off = (s >> 2) * HALF + (s & 3) * 32;
            umma_bf16(d, sdesc_sw128(q0 + m * C::TILE + off), sdesc_sw128(kaddr + off), idesc_s, s > 0);
          }
          umma_commit(&s_full[m][buf]);
        }
        ++ns[m];
        return true;
      };
      auto release_slot = [&]() {
        if (lane == 0) umma_commit(&empty[slot]);  // free once the products issued so far are done
        if (++slot == SLOTS) slot = 0, phase ^= 1u;
      };
      // the values of tile t are in the slot: nothing past the request's end may reach a sum
      auto clear_tail = [&](int t, int at) {
        const int left = end - t * TN;  // positions of the tile that exist
        if (left >= TN || !(left & 15)) return;
        // the last block's rows past the end hold whatever the page held: their weights
        // are 0, but 0 times a NaN is not
        const int r1 = (left + 15) & ~15;
        uint8_t* base = ring + at * C::TILE;
        for (int x = lane; x < (r1 - left) * 8 * (HD / 64); x += 32) {
          const int h = x / ((r1 - left) * 8), y = x - h * (r1 - left) * 8;
          *reinterpret_cast<uint4*>(base + h * HALF + left * 128 + y * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        __syncwarp();
      };
      auto weighted_sum = [&](int t, int m, uint32_t vaddr) {
        const int buf = np[m] % NB;
        if (!warp_wait(&p_ready[m][buf], (np[m] / NB) & 1, ab)) return false;
        // the item before has read its output
        if (t == w.t0 && items[m] > 0 && !warp_wait(&o_free[m], (items[m] - 1) & 1, ab)) return false;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t d = tmem + C::O_COL + static_cast<uint32_t>(m * 128);
          const uint32_t p = tmem + static_cast<uint32_t>((m * NB + buf) * 128);
#pragma unroll
          for (int s = 0; s < TN / 16; ++s)
            umma_bf16_ts(d, p + 8 * s, sdesc_sw128_rows_k(vaddr + s * 2048, HALF), idesc_o, t > w.t0 || s > 0);
          umma_commit(&pv_done[m][buf]);
        }
        ++np[m];
        if (t == w.t1 - 1) ++items[m];
        return true;
      };
      // Step t: the scores of tile t and the values of tile t - 1. With two S buffers the
      // scores go first (they run while the softmax of tile t - 1 does); with one they
      // follow the product that takes P out of it.
      for (int t = w.t0; ok && t <= w.t1; ++t) {
        const bool has_s = t < w.t1, has_v = t > w.t0;
        if constexpr (NB == 2) {
          if (has_s) {
            if (!(ok = warp_wait(&full[slot], phase, ab))) break;
            if (t == w.t0 && !(ok = warp_wait(&q_ready[0], items[0] & 1, ab))) break;
            if (!(ok = scores(0, r0 + slot * C::TILE))) break;
            __syncwarp();
            release_slot();
          }
          if (has_v) {
            if (!(ok = warp_wait(&full[slot], phase, ab))) break;
            clear_tail(t - 1, slot);
            if (!(ok = weighted_sum(t - 1, 0, r0 + slot * C::TILE))) break;
            __syncwarp();
            release_slot();
          }
        } else {
          const int vs = slot, ks = !has_v ? slot : slot + 1 == SLOTS ? 0 : slot + 1;
          const uint32_t k_phase = ks < vs ? phase ^ 1u : phase;
          if (has_v) {
            if (!(ok = warp_wait(&full[vs], phase, ab))) break;
            clear_tail(t - 1, vs);
          }
          for (int m = 0; ok && m < nm; ++m) {
            if (has_v && !(ok = weighted_sum(t - 1, m, r0 + vs * C::TILE))) break;
            if (!has_s) continue;
            if (m == 0 && !(ok = warp_wait(&full[ks], k_phase, ab))) break;
            if (t == w.t0 && !(ok = warp_wait(&q_ready[m], items[m] & 1, ab))) break;
            ok = scores(m, r0 + ks * C::TILE);
          }
          if (!ok) break;
          __syncwarp();
          if (has_v) release_slot();
          if (has_s) release_slot();
        }
      }
    }
    // nothing of this CTA may be in flight when its TMEM is freed
    if (lane == 0) {
      umma_commit(&drain);
      int own = 0;
      mbar_wait(&drain, 0, &own);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax and epilogue
    const int m = (warp - 2) >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t o_addr = tmem + lanes + C::O_COL + static_cast<uint32_t>(m * 128);
    // a negative scale's sign goes into Q; a scale of 0 stays apart from a hidden score's -inf
    const float k2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
    short* parent = s_parent[warp - 2];
    int n = 0, seq = 0, tree_b = -1;
    bool ok = true;
    while (ok && w.next(a)) {
      const int rows = min(128, w.r.n * a.group - w.tile_m * TM - m * 128);
      if (rows <= 0) {
        seq += w.t1 - w.t0;
        continue;
      }
      const bool live = row < rows, warp_live = quad * 32 < rows;
      const int rr = w.tile_m * TM + m * 128 + row, node = rr / a.group;
      const int64_t q_row = static_cast<int64_t>(w.b) * a.width + node;
      const int q_head = w.head * a.group + (rr - node * a.group);
      if (live) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + q_row * a.q_stride +
                                                          static_cast<int64_t>(q_head) * HD);
        uint8_t* dst = sq + m * C::TILE + row * 128;
        uint4 v[HD / 8];
#pragma unroll
        for (int x = 0; x < HD / 8; ++x) v[x] = __ldcg(src + x);
#pragma unroll
        for (int x = 0; x < HD / 8; ++x) {
          v[x].x ^= flip, v[x].y ^= flip, v[x].z ^= flip, v[x].w ^= flip;
          *reinterpret_cast<uint4*>(dst + (x >> 3) * HALF + (((x & 7) ^ (row & 7)) * 16)) = v[x];
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_ready[m]);
      if (a.tree_ids && w.t1 * TN > w.r.ctx && tree_b != w.b) {  // the item reaches the tree
        for (int i = lane; i < w.r.n; i += 32) parent[i] = static_cast<short>(i ? parent_of(a, w.b, i, err) : -1);
        __syncwarp();
        tree_b = w.b;
      }
      float mx = -INFINITY, l = 0.f;  // the maximum the weights are taken against, and their sum
      for (int t = w.t0; t < w.t1; ++t) {
        const int buf = n % NB, p0 = t * TN;
        if (!(ok = warp_wait(&s_full[m][buf], (n / NB) & 1, ab))) break;
        tc_fence_after();
        if (warp_live) {
          const uint32_t s_addr = tmem + lanes + static_cast<uint32_t>((m * NB + buf) * 128);
          uint32_t s[128];
          tmem_ld128w(s_addr, s);
          const uint32_t blocks = blocks_ok[seq & 15];
          if (p0 + TN > w.r.ctx || blocks != 0xffu) {
            uint32_t see[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int before = w.r.ctx + (a.tree_ids ? 0 : node + 1) - (p0 + 32 * x);
              see[x] = before >= 32 ? 0xffffffffu : before <= 0 ? 0u : (1u << before) - 1;
            }
            if (a.tree_ids && live && p0 + TN > w.r.ctx) {
              for (int i = node; i >= 0; i = parent[i]) {
                const int at = w.r.ctx + i - p0;
                if (at < 0) break;  // ancestors only come earlier
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  if ((at >> 5) == x) see[x] |= 1u << (at & 31);
              }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
              see[x] &= (blocks >> (2 * x) & 1u ? 0x0000ffffu : 0u) | (blocks >> (2 * x + 1) & 1u ? 0xffff0000u : 0u);
#pragma unroll
            for (int x = 0; x < 128; ++x)
              if (!(see[x >> 5] >> (x & 31) & 1u)) s[x] = 0xff800000u;
          }
          float top = -INFINITY;
#pragma unroll
          for (int x = 0; x < 128; ++x) top = fmaxf(top, __uint_as_float(s[x]));
          top *= k2;
          if (t == w.t0) {
            mx = top;
          } else if (__any_sync(0xffffffffu, top > mx + 8.f)) {
            const float to = fmaxf(mx, top), f = mx == -INFINITY ? 0.f : ex2(mx - to);
            // the output holds every tile before this one
            if (!(ok = warp_wait(&pv_done[m][(n - 1) % NB], ((n - 1) / NB) & 1, ab))) break;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < HD; x += 32) {
              uint32_t o[32];
              tmem_ld32w(o_addr + x, o);
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st32(o_addr + x, o);
            }
            l *= f;
            mx = to;
          }
          const float base = mx == -INFINITY ? 0.f : mx;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int x = 0; x < 128; x += 32) {
            uint32_t p[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              const float e0 = ex2(fmaf(__uint_as_float(s[x + 2 * y]), k2, -base));
              const float e1 = ex2(fmaf(__uint_as_float(s[x + 2 * y + 1]), k2, -base));
              sum[y & 1] += e0;
              sum[2 + (y & 1)] += e1;
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(e0, e1);
              p[y] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            tmem_st16(s_addr + x / 2, p);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        ++n;
        ++seq;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[m][buf]);
      }
      if (!ok) break;
      if (!(ok = warp_wait(&pv_done[m][(n - 1) % NB], ((n - 1) / NB) & 1, ab))) break;
      tc_fence_after();
      if (warp_live) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int64_t part = (static_cast<int64_t>(2 * c + (w.first_item ? 0 : 1)) * TM + m * 128 + row);
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (q_row * a.nq + q_head) * HD;
#pragma unroll
        for (int x = 0; x < HD; x += 32) {
          uint32_t o[32];
          tmem_ld32w(o_addr + x, o);
          if (!live) continue;
          if (w.whole) {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {
              uint32_t b[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[y + 2 * z]) * inv,
                                                                __uint_as_float(o[y + 2 * z + 1]) * inv);
                b[z] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              *reinterpret_cast<uint4*>(dst + x + y) = make_uint4(b[0], b[1], b[2], b[3]);
            }
          } else {
#pragma unroll
            for (int y = 0; y < 32; y += 4)
              *reinterpret_cast<uint4*>(a.part_o + part * HD + x + y) = make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
          }
        }
        if (live && !w.whole) a.part_ml[part] = make_float2(mx, l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[m]);
    }
  }
  if (err) set_dev_error(a.dev_err, err);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (threadIdx.x == 0 && abort_flag) {
    // copies still in flight land before the CTA's shared memory goes
    set_dev_error(a.dev_err, FLASHMAP_DEVERR_TIMEOUT);
    for (int i = max(0, s_issued - SLOTS); i < s_issued; ++i) {
      int own = 0;
      mbar_wait(&full[i % SLOTS], (i / SLOTS) & 1, &own);
    }
  }
}

template <int HD, int MT>
cudaError_t launch_mma(const Launch& L, const TreeAttnArgs& a, int G, const CUtensorMap& kmap, const CUtensorMap& vmap) {
  using C = MmaCfg<HD, MT>;
  cudaError_t e =
      cudaFuncSetAttribute(tree_mma_kernel<HD, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e == cudaSuccess)
    e = launch_k(L, tree_mma_kernel<HD, MT>, dim3(G), dim3(C::THREADS), C::SMEM, kmap, vmap, a);
  if (e == cudaSuccess && G > 1)
    e = launch_k(L, tree_join_kernel<__nv_bfloat16, HD, C::TM, TN>, dim3(G - 1, kJoinY), dim3(kJoinThreads), 0, a);
  return e;
}

// Two row tiles a CTA once a request's nodes and a group's heads fill more than one.
int row_tiles_per_cta(int width, int group) { return width * group > 128 ? 2 : 1; }

}  // namespace

size_t tree_mma_bytes(int hd, int width, int group, int num_sms) {
  return static_cast<size_t>(2 * num_sms) * 128 * row_tiles_per_cta(width, group) * (static_cast<size_t>(hd) * 4 + 8);
}

cudaError_t tree_mma(const Launch& L, TreeAttnArgs a, void* workspace) {
  const int mt = row_tiles_per_cta(a.width, a.group), G = L.num_sms;
  a.part_ml = static_cast<float2*>(workspace);
  a.part_o = reinterpret_cast<float*>(a.part_ml + static_cast<size_t>(2 * G) * 128 * mt);
  CUtensorMap kmap, vmap;
  std::string err;
  const int64_t rows = a.num_pages * a.nkv * a.P;
  if (!make_tmap_bf16(&kmap, a.keys, rows, a.hd, a.hd, 16, &err) ||
      !make_tmap_bf16(&vmap, a.values, rows, a.hd, a.hd, 16, &err))
    return cudaErrorInvalidValue;
  if (a.hd == 64) return mt == 1 ? launch_mma<64, 1>(L, a, G, kmap, vmap) : launch_mma<64, 2>(L, a, G, kmap, vmap);
  return mt == 1 ? launch_mma<128, 1>(L, a, G, kmap, vmap) : launch_mma<128, 2>(L, a, G, kmap, vmap);
}

}  // namespace fm
