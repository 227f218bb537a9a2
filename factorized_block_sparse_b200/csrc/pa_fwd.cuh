// Forward kernel of packed causal attention on tcgen05.
//
// Persistent: each CTA walks a zig-zag share of the items, longest first.  An
// item is two units of 128 query rows that share their K/V tiles: two query
// heads of one K/V head (same rows), or two neighbouring row tiles of one
// head.  Per key tile of 128 and unit u
//   S_u = Q_u K^T     both operands in shared memory, fp32 in TMEM
//   P = 2^(S c - m)   running maximum and sum of the online softmax in
//                     registers; P back into TMEM, rounded
//   O_u += P V        P read from TMEM, fp32 accumulator in TMEM
// and o = O / sum at the end.  While one unit's softmax runs, the tensor core
// works on the other unit.  The running maximum moves only when it grows by
// more than 2^8, so O is rescaled rarely; numerator and denominator use the
// same maximum, so the quotient is exact up to rounding.
//
// TMEM columns: S_u at 128 u.  D <= 64: P_u at 256 + 64 u and O_u at 384 + D u,
// so the next S is computed while the softmax works on this one (which is in
// registers by then), and each unit has an issuing warp of its own.  D = 128
// has no room for that: P_u over S_u, O_u at 256 + 128 u.  There order makes
// waits unnecessary: one thread's MMAs execute in order, so S_u(j+1) behind
// PV_u(j) cannot overwrite a P_u(j) still being read, and the commit behind
// S_u(j+1) also says that O_u holds PV_u(j), which is what a rescale needs.
//
// What bounds it.  D = 128: per unit the chain S -> softmax -> PV, 3.3k cycles
// for 2.1k of products with two units in turn; one sequence of 32768, 16 / 2
// heads, 3.3 to 3.9 ms (1.1 to 1.3 PFLOP/s; the clock falls with the power).
// D <= 64: the softmax (1024 cycles of exponentials a tile pair of 1430 in
// all); 2 x 12288 rows, 8 heads of 64, 0.38 ms (820 TFLOP/s); 2 x 8192 rows,
// 8 / 4 heads of 32, 0.18 ms.  These times and those below are of runs of
// milliseconds; in runs of seconds, under the power limit, the same calls take
// 0.41 ms (text), 0.49 (ten ragged sequences) and 3.6 (32768).  An eighth or more of
// the exponentials on the FMA pipe did not help either and costs the row sums
// their last bits.
//
// Roles: the softmax and epilogue of a unit in 4 NH warps, NH threads a query
// row (TMEM lane 32 (w mod 4) + lane) with 128 / NH keys and D / NH output
// columns each; one warp whose lane 0 is the TMA producer; two for the MMAs.
// D <= 64 takes NH = 2 (the two threads agree on the row's maximum through
// shared memory): it is bound by the softmax, and two warps a scheduler do not
// hide its latencies (2 x 12288 rows, 8 heads of 64: 389 us, 417 with NH = 1).
// D = 128 takes NH = 1: there the exchange only lengthens the chain S ->
// softmax -> PV (ten ragged sequences, 32 / 8 heads: 426 us, 466 with NH = 2;
// 415 since PV begins with the first quarter of P).
#pragma once

#include "pa_device.cuh"

namespace pa {

// D = 128: k-steps of PV that are issued as soon as the first 32 keys' P is there, while the softmax goes on with the
// others: the product's end, which the unit's next step waits for, comes earlier (one sequence of 8192, 16 / 2 heads:
// 217 us; all at once 223, in halves 218 to 222, three quarters first 226).
constexpr int kEarly = 2;

enum Pairing : int { kSingle = 0, kHeads = 1, kTiles = 2 };

struct FwdArgs {
  const Slot* slots;
  int n_items, heads;  // items = slots x heads (head pairs where two heads make an item)
  int pairing;
  int G;               // query heads of a K/V head
  View o;
  float* lse;
  long long ls;
  float scale_log2;
};

template <int D>
struct FwdCfg {
  using G = TileGeo<D>;
  static constexpr int STAGES = D >= 128 ? 4 : 8;  // K and V tiles in turn
  static constexpr int NH = D <= 64 ? 2 : 1;       // threads a query row
  static constexpr int SOFT_WARPS = 8 * NH;
  static constexpr int STG_COLS = D >= 64 ? 32 : 16;  // staging: 32 rows of so many columns per warp
  static constexpr int STG_ROWB = 2 * STG_COLS;
  static constexpr int STG_BYTES = 32 * STG_ROWB;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * G::BYTES;
  static constexpr int OFF_STG = OFF_KV + STAGES * G::BYTES;
  static constexpr int OFF_RED = OFF_STG + SOFT_WARPS * STG_BYTES;  // [2 tiles in turn][2 units][2 halves][128 rows]
  static constexpr int OFF_BAR = OFF_RED + (NH - 1) * 8 * kTile * 4;
  static constexpr int N_BARS = 2 + 2 + 2 * STAGES + 2 * 6 + 2;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BARS;
  static constexpr int SMEM = OFF_MISC + 16;
  static constexpr bool SEP = D <= 64;  // P in columns of its own
  static constexpr int COL_P = SEP ? 256 : 0, P_STRIDE = SEP ? 64 : 128;
  static constexpr int COL_O = SEP ? 384 : 256;
  static constexpr int THREADS = 32 * (SOFT_WARPS + 3);
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// What an item is: its units' query tiles and heads.
struct FwdItem {
  Slot s;
  int hk;
  int n[2];   // key tiles of each unit (0: no such unit)
  int qt[2];  // query tile in the sequence
  int h[2];   // query head
};

// An item of one unit alone takes the units in turn (k counts the CTA's
// items), so that one's epilogue runs beside the next one's softmax.
__device__ __forceinline__ FwdItem fwd_item(const FwdArgs& a, const Slot& s, int item, int k) {
  FwdItem it;
  const int hi = item % a.heads;
  it.s = s;
  if (a.pairing == kTiles) {
    it.h[0] = it.h[1] = hi;
    it.qt[0] = 2 * it.s.tile;
    it.qt[1] = it.qt[0] + 1;
    it.n[0] = it.qt[0] + 1;
    it.n[1] = it.qt[1] * kTile < it.s.len ? it.qt[1] + 1 : 0;
  } else {
    it.h[0] = a.pairing == kHeads ? 2 * hi : hi;
    it.h[1] = it.h[0] + 1;
    it.qt[0] = it.qt[1] = it.s.tile;
    it.n[0] = it.s.tile + 1;
    it.n[1] = a.pairing == kHeads ? it.n[0] : 0;
  }
  it.hk = it.h[0] / a.G;
  if (it.n[1] == 0 && (k & 1)) {
    it.n[1] = it.n[0];
    it.n[0] = 0;
    it.qt[1] = it.qt[0];
    it.h[1] = it.h[0];
  }
  return it;
}

template <typename T, int D>
__global__ void __launch_bounds__(FwdCfg<D>::THREADS, 1)
    pa_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const FwdArgs a) {
  using C = FwdCfg<D>;
  using G = TileGeo<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sKV = smem + C::OFF_KV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* bar_q_full = bars;                        // [2]
  uint64_t* bar_q_free = bars + 2;                    // [2]
  uint64_t* bar_kv_full = bars + 4;                   // [STAGES]
  uint64_t* bar_kv_free = bar_kv_full + C::STAGES;    // [STAGES]
  uint64_t* bar_s_full = bar_kv_free + C::STAGES;     // [2] S of a tile
  uint64_t* bar_s_free = bar_s_full + 2;              // [2] S has been read (SEP)
  uint64_t* bar_p_full = bar_s_free + 2;              // [2] P of a tile
  uint64_t* bar_pv_done = bar_p_full + 2;             // [2] PV of a tile
  uint64_t* bar_o_free = bar_pv_done + 2;             // [2] the epilogue has read O
  uint64_t* bar_p_early = bar_o_free + 2;             // [2] the first 32 keys' P (not SEP)
  uint64_t* bar_drain = bar_p_early + 2;              // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(smem + C::OFF_MISC + 4);

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int cta = blockIdx.x, n_ctas = gridDim.x;
  if (threadIdx.x == 0) {
    for (int u = 0; u < 2; ++u) {
      mbar_init(bar_q_full + u, 1);
      mbar_init(bar_q_free + u, 1);
      mbar_init(bar_s_full + u, 1);
      mbar_init(bar_s_free + u, 4 * C::NH);
      mbar_init(bar_p_full + u, 4 * C::NH);
      mbar_init(bar_p_early + u, 4 * C::NH);
      mbar_init(bar_pv_done + u, 1);
      mbar_init(bar_o_free + u, 4 * C::NH);
      mbar_init(bar_drain + u, 1);
    }
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar_kv_full + s, 1);
      mbar_init(bar_kv_free + s, C::SEP ? 2 : 1);  // commits of each issuing warp
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::SOFT_WARPS + 1) tmem_alloc<512>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const SlotWalk walk(a.slots, a.n_items, a.heads);

  if (warp == C::SOFT_WARPS) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      bool ok = true;
      int ring = 0, nq[2] = {0, 0};
      for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
        const FwdItem it = fwd_item(a, walk.take(item, k), item, k);
        for (int u = 0; ok && u < 2; ++u) {
          if (it.n[u] == 0) continue;
          if (nq[u] > 0) ok = mbar_wait(bar_q_free + u, (nq[u] - 1) & 1, abort_flag);
          if (!ok) break;
          if (!PA_WITHHELD(kHoldQ, nq[u])) {
            mbar_arrive_expect_tx(bar_q_full + u, G::BYTES);
            load_tile<D>(sQ + u * G::BYTES, &mq, bar_q_full + u, it.h[u], it.s.start + it.qt[u] * kTile);
          }
          ++nq[u];
        }
        const int n = max(it.n[0], it.n[1]);
        for (int j = 0; ok && j < 2 * n; ++j, ++ring) {  // K_0 V_0 K_1 V_1 ...
          const int st = ring % C::STAGES;
          if (ring >= C::STAGES && !mbar_wait(bar_kv_free + st, (ring / C::STAGES - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          if (PA_WITHHELD(kHoldV, ring - 1)) continue;
          mbar_arrive_expect_tx(bar_kv_full + st, G::BYTES);
          load_tile<D>(sKV + st * G::BYTES, (j & 1) ? &mv : &mk, bar_kv_full + st, it.hk, it.s.start + (j >> 1) * kTile);
        }
      }
      // no copy may land after the CTA has gone, whichever role gives up, and when
      for (int u = 0; u < 2; ++u)
        if (nq[u] > 0) mbar_wait_drain(bar_q_full + u, (nq[u] - 1) & 1);
      for (int h = ring > C::STAGES ? ring - C::STAGES : 0; h < ring; ++h)
        mbar_wait_drain(bar_kv_full + h % C::STAGES, (h / C::STAGES) & 1);
    }
  } else if (warp > C::SOFT_WARPS) {
    // ------------------------------------------------------------------ MMAs
    constexpr uint32_t id_s = make_idesc<T>(128, 128, false, false);
    constexpr uint32_t id_o = make_idesc<T>(128, D, false, true);
    bool ok = true;
    int ring = 0;  // K/V tiles so far
    auto full = [&](int r) { return mbar_wait_warp(bar_kv_full + r % C::STAGES, (r / C::STAGES) & 1, abort_flag); };
    auto q_desc = [&](int u) { return G::kmajor(smem_u32(sQ) + u * G::BYTES); };
    // S of unit u's next tile from the K tile at ring position r
    auto issue_s = [&](int u, int r) {
      const Desc q_k = q_desc(u), k_k = G::kmajor(smem_u32(sKV) + r % C::STAGES * G::BYTES);
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16_ss(tmem + u * 128, q_k.at(G::kstep(kk)), k_k.at(G::kstep(kk)), id_s, kk > 0);
        mma_commit(bar_s_full + u);
      }
      __syncwarp();
    };
    // k-steps k0 .. k1 - 1 of O of unit u, from the V tile at ring position r; keys behind the sequence's last are zeroed in it
    auto issue_pv = [&](int u, int r, bool first, int k0, int k1) {
      const Desc v_mn = G::mnmajor(smem_u32(sKV) + r % C::STAGES * G::BYTES);
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          if (kk >= k0 && kk < k1)
            mma_bf16_ts(tmem + C::COL_O + u * D, tmem + C::COL_P + u * C::P_STRIDE + kk * 8, v_mn.at(G::mnstep(kk)), id_o,
                        (!first || kk > 0));
        if (k1 == kTile / 16) mma_commit(bar_pv_done + u);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) mma_commit(bar);
      __syncwarp();
    };
    if constexpr (C::SEP) {
      const int u = warp - C::SOFT_WARPS - 1;
      int ni = 0, ns = 0, np = 0;  // items, S and PV products of this unit so far
      // a tile that only the other unit needs
      auto skip = [&](int r) -> bool {
        if (!full(r)) return false;
        if (lane == 0) mbar_arrive(bar_kv_free + r % C::STAGES);
        __syncwarp();
        return true;
      };
      for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
        const FwdItem it = fwd_item(a, walk.take(item, k), item, k);
        const int n = uniform(u ? it.n[1] : it.n[0]), n_all = uniform(max(it.n[0], it.n[1])), len = uniform(it.s.len);
        if (n > 0) {
          ok = full(ring) && mbar_wait_warp(bar_q_full + u, ni & 1, abort_flag) &&
               (ns == 0 || mbar_wait_warp(bar_s_free + u, (ns - 1) & 1, abort_flag));
          if (!ok) break;
          issue_s(u, ring);
          ++ns;
          commit(bar_kv_free + ring % C::STAGES);
          if (n == 1) commit(bar_q_free + u);
        } else {
          ok = skip(ring);
        }
        for (int j = 0; ok && j < n_all; ++j, ring += 2) {
          const int sv = (ring + 1) % C::STAGES;
          if (j < n) {
            if (j + 1 < n) {
              ok = full(ring + 2) && mbar_wait_warp(bar_s_free + u, (ns - 1) & 1, abort_flag);
              if (!ok) break;
              issue_s(u, ring + 2);
              ++ns;
              commit(bar_kv_free + (ring + 2) % C::STAGES);
              if (j + 2 == n) commit(bar_q_free + u);
            }
            if (!(ok = full(ring + 1))) break;
            if (len - j * kTile < kTile) zero_rows<D>(sKV + sv * G::BYTES, len - j * kTile, lane);
            ok = mbar_wait_warp(bar_p_full + u, np & 1, abort_flag) &&
                 (j > 0 || ni == 0 || mbar_wait_warp(bar_o_free + u, (ni - 1) & 1, abort_flag));
            if (!ok) break;
            ++np;
            issue_pv(u, ring + 1, j == 0, 0, kTile / 16);
            commit(bar_kv_free + sv);
          } else {
            ok = skip(ring + 1);
          }
          if (ok && j + 1 < n_all && j + 1 >= n) ok = skip(ring + 2);
        }
        if (n > 0) ++ni;
      }
    } else if (warp == C::SOFT_WARPS + 1) {
      // One warp for both units, in strict turn: with a warp each (measured: 0.43 -> 0.52 ms for ten ragged sequences,
      // 32 / 8 heads of 128) their products mix, both finish late and both softmaxes then run at the same time.
      int ni[2] = {0, 0}, np[2] = {0, 0};  // items and PV products of each unit so far
      for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
        const FwdItem it = fwd_item(a, walk.take(item, k), item, k);
        const int n0 = uniform(it.n[0]), n1 = uniform(it.n[1]), n = max(n0, n1), len = uniform(it.s.len);
        ok = full(ring);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int nu = u ? n1 : n0;
          if (!ok || nu == 0) continue;
          ok = mbar_wait_warp(bar_q_full + u, ni[u] & 1, abort_flag);
          if (!ok) break;
          issue_s(u, ring);
          if (nu == 1) commit(bar_q_free + u);
        }
        if (!ok) break;
        commit(bar_kv_free + ring % C::STAGES);
        for (int j = 0; ok && j < n; ++j, ring += 2) {
          const int sv = (ring + 1) % C::STAGES, sk = (ring + 2) % C::STAGES;
          ok = full(ring + 1) && (j + 1 == n || full(ring + 2));
          if (!ok) break;
          if (len - j * kTile < kTile) zero_rows<D>(sKV + sv * G::BYTES, len - j * kTile, lane);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int nu = u ? n1 : n0;
            if (!ok || j >= nu) continue;
            ok = mbar_wait_warp(bar_p_early + u, np[u] & 1, abort_flag) &&
                 (j > 0 || ni[u] == 0 || mbar_wait_warp(bar_o_free + u, (ni[u] - 1) & 1, abort_flag));
            if (!ok) break;
            issue_pv(u, ring + 1, j == 0, 0, kEarly);
            if (!(ok = mbar_wait_warp(bar_p_full + u, np[u] & 1, abort_flag))) break;
            ++np[u];
            issue_pv(u, ring + 1, j == 0, kEarly, kTile / 16);
            if (j + 1 < nu) {
              issue_s(u, ring + 2);
              if (j + 2 == nu) commit(bar_q_free + u);
            }
          }
          if (!ok) break;
          commit(bar_kv_free + sv);
          if (j + 1 < n) commit(bar_kv_free + sk);
        }
        ni[0] += n0 > 0;
        ni[1] += n1 > 0;
      }
    }
    if (elect_one()) {  // every MMA has completed before TMEM is released
      mma_commit(bar_drain + (warp - C::SOFT_WARPS - 1));
      mbar_wait_drain(bar_drain + (warp - C::SOFT_WARPS - 1), 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------- softmax, epilogue
    constexpr int NH = C::NH, KPT = kTile / NH;  // threads a row, keys a thread
    const int u = warp / (4 * NH), half = (warp >> 2) & (NH - 1), quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_base + u * 128 + half * KPT;
    const uint32_t t_p = tmem + lane_base + C::COL_P + u * C::P_STRIDE + half * (KPT / 2);
    const uint32_t t_o = tmem + lane_base + C::COL_O + u * D + half * (D / NH);
    uint8_t* stg = smem + C::OFF_STG + warp * C::STG_BYTES;
    // what the two threads of a row tell one another: [turn][unit][half][row]
    float* mine = reinterpret_cast<float*>(smem + C::OFF_RED) + (u * 2 + half) * kTile + row;
    const float* other = reinterpret_cast<float*>(smem + C::OFF_RED) + (u * 2 + (half ^ 1)) * kTile + row;
    int turn = 0;
    auto exchange = [&](float v) -> float {  // the other thread's value: one barrier of the two warps, buffers in turn
      mine[turn * 4 * kTile] = v;
      asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + u * 4 + quarter) : "memory");
      const float r = other[turn * 4 * kTile];
      turn ^= 1;
      return r;
    };
    bool ok = true;
    int ns = 0;
    for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
      const FwdItem it = fwd_item(a, walk.take(item, k), item, k);
      // (selected, not indexed: an index that is not a constant puts the arrays into memory)
      const int n = u ? it.n[1] : it.n[0], qt = u ? it.qt[1] : it.qt[0], head = u ? it.h[1] : it.h[0];
      if (n == 0) continue;
      float m_used = -INFINITY, l_sum = 0.f;
      for (int j = 0; j < n; ++j, ++ns) {
        ok = ok && mbar_wait(bar_s_full + u, ns & 1, abort_flag);
        tc_fence_after();
        float s[KPT];
#pragma unroll
        for (int c = 0; c < KPT / 32; ++c) tmem_ld32(t_s + c * 32, s + c * 32);
        tmem_wait_ld();
        if (C::SEP) {
          tc_fence_before();
          warp_arrive(bar_s_free + u, lane);
        }
        if (j + 1 == n) {  // the diagonal tile: keys up to the row itself
#pragma unroll
          for (int c = 0; c < KPT / 32; ++c) mask_after32(s + c * 32, row - half * KPT - c * 32, -INFINITY);
        }
        float mx[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) mx[x] = max3(s[x], s[8 + x], s[16 + x]);
#pragma unroll
        for (int i = 24; i + 16 < KPT; i += 16)
#pragma unroll
          for (int x = 0; x < 8; ++x) mx[x] = max3(mx[x], s[i + x], s[i + 8 + x]);
#pragma unroll
        for (int x = 0; x < 8; ++x) mx[x] = fmaxf(mx[x], s[KPT - 8 + x]);
        float m_tile = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
        if constexpr (NH == 2) m_tile = fmaxf(m_tile, exchange(m_tile));
        m_tile *= a.scale_log2;
        float factor = 1.f;
        if (m_tile > m_used + 8.f) {
          factor = ex2(m_used - m_tile);  // 0 for the first tile
          m_used = m_tile;
        }
        if (C::SEP && j > 0) {  // P's columns are free, and O holds every tile before this one
          ok = ok && mbar_wait(bar_pv_done + u, (ns - 1) & 1, abort_flag);
          tc_fence_after();
        }
        if (j > 0 && __any_sync(0xffffffffu, factor != 1.f)) {  // each thread its columns of O
#pragma unroll
          for (int i = 0; i < D / NH / 16; ++i) {
            float ov[16];
            tmem_ld16(t_o + i * 16, ov);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) ov[x] *= factor;
            tmem_st16(t_o + i * 16, ov);
          }
        }
        // a row whose keys so far all score -inf: weights of 0, not 2^(-inf + inf)
        const float neg = m_used == -INFINITY ? Elem<T>::kBias : Elem<T>::kBias - m_used;
        const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2), ng2 = f2_pack(neg, neg);
        uint64_t rs[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < KPT / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = f2_unpack(f2_fma(f2_pack(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]), sc2, ng2));
            const float p0 = ex2(e.x), p1 = ex2(e.y);
            rs[i & 3] = f2_add(rs[i & 3], f2_pack(p0, p1));
            pk[i] = Elem<T>::pack(p0, p1);
          }
          tmem_st8(t_p + c * 16, pk);
          tmem_st8(t_p + c * 16 + 8, pk + 8);
          if (!C::SEP && c == 0) {  // the product with the first 32 keys can begin
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(bar_p_early + u, lane);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar_p_full + u, lane);
        const float2 r0 = f2_unpack(f2_add(f2_add(rs[0], rs[1]), f2_add(rs[2], rs[3])));
        l_sum = l_sum * factor + (r0.x + r0.y);
      }
      // ------------------------------------------------------------ epilogue
      ok = warp_ok(ok && mbar_wait(bar_pv_done + u, (ns - 1) & 1, abort_flag));
      tc_fence_after();
      if constexpr (NH == 2) {  // (a negative sum: gave up after a timeout, and so does its partner at the barrier)
        const float theirs = exchange(ok ? l_sum : -1.f);
        ok = ok && !(theirs < 0.f);
        l_sum += theirs;
      }
      const float inv = 1.f / l_sum;
      const int r0 = qt * kTile + quarter * 32;  // the warp's first row in the sequence
      const long long row0 = static_cast<long long>(it.s.start) + r0;
      const int rows = min(32, it.s.len - r0);
      T* out = static_cast<T*>(const_cast<void*>(a.o.p)) + row0 * a.o.rs + static_cast<long long>(head) * a.o.hs +
               half * (D / NH);
      constexpr int CHUNKS = C::STG_ROWB / 16;  // 16-byte chunks of a staged row
      constexpr int PASSES = D / NH / C::STG_COLS;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
#pragma unroll
        for (int i = 0; i < C::STG_COLS / 16; ++i) {
          float ov[16];
          tmem_ld16(t_o + p * C::STG_COLS + i * 16, ov);
          tmem_wait_ld();
          if (p == PASSES - 1 && i == C::STG_COLS / 16 - 1) {
            tc_fence_before();
            warp_arrive(bar_o_free + u, lane);
          }
          uint32_t w[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) w[x] = Elem<T>::pack(ov[2 * x] * inv, ov[2 * x + 1] * inv);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            *reinterpret_cast<uint4*>(stg + lane * C::STG_ROWB + (((2 * i + x) ^ ((lane >> 1) & (CHUNKS - 1))) << 4)) =
                make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
        }
        __syncwarp();
        // whole runs of a row leave together: CHUNKS lanes a row
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
          const int r = i * (32 / CHUNKS) + lane / CHUNKS, c = lane % CHUNKS;
          if (r < rows)
            *reinterpret_cast<uint4*>(out + r * a.o.rs + p * C::STG_COLS + c * 8) =
                *reinterpret_cast<const uint4*>(stg + r * C::STG_ROWB + ((c ^ ((r >> 1) & (CHUNKS - 1))) << 4));
        }
        __syncwarp();
      }
      if (half == 0 && lane < rows)
        a.lse[static_cast<long long>(head) * a.ls + row0 + lane] =
            (m_used + log2f(l_sum) - Elem<T>::kBias) * 0.6931471805599453f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::SOFT_WARPS + 1) {
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

}  // namespace pa
