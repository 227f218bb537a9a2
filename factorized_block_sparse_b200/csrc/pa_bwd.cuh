// Backward kernels of packed causal attention on tcgen05.
//
// pa_bwd_pre_kernel   per (query tile, head): delta_i = <dO_i, o_i>, packed
//                     with -lse log2 e for the main kernel, and zeros for the
//                     tile's dq sum.
// pa_bwd_kernel       persistent; an item is a tile of 128 keys of one K/V
//                     head and all query tiles of all query heads that see it
//                     (diagonal first, head by head).  Per step of 128 queries,
//                     keys on TMEM lanes:
//   S^T = K Q^T                       P^T = 2^(S^T c - lse log2 e), over S^T
//   dP^T = V dO^T                     dS^T = P^T (dP^T - delta), to shared memory
//   dV += P^T dO                      A from TMEM
//   dK += dS^T Q,  dQ = dS K          A from shared memory, dS^T read K-major
//                                     and MN-major
//                     dV and dK stay in TMEM for the whole item, so their sums
//                     run in a fixed order over the group's heads; dQ is
//                     added to a float32 sum per tile in global memory.
// pa_bwd_dq_kernel    dq = scale * sum, rounded once.
//
// The S^T product of the next step is issued behind dV (which frees its
// columns) and so runs under this step's dS; the next step's dP^T runs under
// the products of dS.  With D = 128 TMEM is full (S^T, dP^T, dV, dK of 128
// columns each), so dQ lands in the dP^T columns and the next dP^T waits for
// its read-out, which dK covers.
//
// Roles (704 threads): warps 0..15 four compute groups (thread = key row, 32 of
// the step's queries each), warps 16..19 read-out of dQ and of the item's dK,
// dV, warp 20 lane 0 the TMA producer, warp 21 TMEM and the MMAs.
#pragma once

#include "pa_device.cuh"

namespace pa {

struct BwdArgs {
  const Slot* slots;
  int n_items, Hkv, G;
  int n_tiles;          // 128-row tiles of all sequences
  const float* ld;      // [Hq][n_tiles][2][128]: -lse log2 e (padding -inf), delta (padding 0)
  float* dq_sum;        // [Hq][n_tiles][4 row quarters][D / 32][8][32 rows][4 columns]
  View dk, dv;
  float scale, scale_log2;
};

template <int D>
struct BwdCfg {
  using G = TileGeo<D>;
  static constexpr int KVB = D >= 128 ? 1 : 2;   // K/V buffers
  static constexpr int QST = 2;                  // Q stages (with lse and delta)
  static constexpr int OST = D >= 128 ? 1 : 2;   // dO stages
  static constexpr int NDS = D >= 128 ? 1 : 2;   // dS^T buffers
  static constexpr int NDQ = D >= 128 ? 1 : 2;   // dQ buffers in TMEM
  static constexpr int DS_BYTES = 2 * kTile * 128;
  static constexpr int LD_BYTES = 2 * kTile * 4;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + KVB * G::BYTES;
  static constexpr int OFF_Q = OFF_V + KVB * G::BYTES;
  static constexpr int OFF_DO = OFF_Q + QST * G::BYTES;
  static constexpr int OFF_DS = OFF_DO + OST * G::BYTES;
  static constexpr int OFF_STG = OFF_DS + NDS * DS_BYTES;  // dQ on its way out: two pieces a read-out warp
  static constexpr int STG_BYTES = 32 * 32 * 4;
  static constexpr int OFF_LD = OFF_STG + 8 * STG_BYTES;
  static constexpr int OFF_BAR = OFF_LD + QST * LD_BYTES;
  static constexpr int N_BARS = 2 * KVB + 2 * QST + 2 * OST + 4 + NDS + 2 * NDQ + 2 + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BARS;
  static constexpr int SMEM = OFF_MISC + 16;
  static constexpr int COL_S = 0, COL_DP = 128, COL_DV = 256, COL_DK = 256 + D;
  static constexpr int COL_DQ = D >= 128 ? COL_DP : 256 + 2 * D;  // + b * D
  static constexpr int COMPUTE = 512, THREADS = COMPUTE + 192;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct BwdItem {
  Slot s;
  int hk, n, per;  // K/V head, steps, steps of one query head
};

__device__ __forceinline__ BwdItem bwd_item(const BwdArgs& a, int item) {
  BwdItem it;
  const int slot = item / a.Hkv;
  it.hk = item - slot * a.Hkv;
  it.s = a.slots[slot];
  it.per = (it.s.len + kTile - 1) / kTile - it.s.tile;
  it.n = it.per * a.G;
  return it;
}

// 32 rows of two threads' worth: D / 8 threads a row, 8 columns each.
template <typename T, int D>
__global__ void __launch_bounds__(256)
    pa_bwd_pre_kernel(const Slot* slots, View o, View dO, const float* lse, long long ls, float* ld, float* dq_sum,
                      int n_tiles) {
  constexpr int TPR = D / 8, RPI = 256 / TPR;  // threads a row, rows a turn
  const Slot s = slots[blockIdx.x];
  const int h = blockIdx.y, tid = threadIdx.x;
  const long long tile = static_cast<long long>(h) * n_tiles + s.base + s.tile;
  float* out = ld + tile * 2 * kTile;
  for (int r = tid / TPR; r < kTile; r += RPI) {
    const int i = s.tile * kTile + r;
    const bool in = i < s.len;
    float d = 0.f;
    if (in) {
      const long long row = static_cast<long long>(s.start) + i;
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const T*>(o.p) + row * o.rs + h * o.hs + (tid % TPR) * 8);
      const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const T*>(dO.p) + row * dO.rs + h * dO.hs + (tid % TPR) * 8);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 x = Elem<T>::unpack(aw[u]), y = Elem<T>::unpack(bw[u]);
        d += x.x * y.x + x.y * y.y;
      }
    }
#pragma unroll
    for (int w = TPR / 2; w >= 1; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
    if (tid % TPR == 0) {
      out[r] = in ? -1.4426950408889634f * lse[static_cast<long long>(h) * ls + s.start + i] : -INFINITY;
      out[kTile + r] = d;
    }
  }
  float4* z = reinterpret_cast<float4*>(dq_sum + tile * kTile * D);
  for (int i = tid; i < kTile * D / 4; i += 256) z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
    pa_bwd_dq_kernel(const Slot* slots, const float* dq_sum, View dq, int n_tiles, float scale) {
  const Slot s = slots[blockIdx.x];
  const int h = blockIdx.y;
  const long long tile = static_cast<long long>(h) * n_tiles + s.base + s.tile;
  const float4* in = reinterpret_cast<const float4*>(dq_sum + tile * kTile * D);
  const int rows = min(kTile, s.len - s.tile * kTile);
  T* out = static_cast<T*>(const_cast<void*>(dq.p)) + (static_cast<long long>(s.start) + s.tile * kTile) * dq.rs + h * dq.hs;
#pragma unroll 4
  for (int i = threadIdx.x; i < kTile * D / 8; i += 256) {
    const int r = i % kTile, c = i / kTile;  // 8 columns from 8 c
    if (r >= rows) continue;
    const float4* p = in + (r / 32) * (8 * D) + (c / 4) * 256 + (c % 4) * 64 + r % 32;
    const float4 a = p[0], b = p[32];
    *reinterpret_cast<uint4*>(out + r * dq.rs + c * 8) =
        make_uint4(Elem<T>::pack(a.x * scale, a.y * scale), Elem<T>::pack(a.z * scale, a.w * scale),
                   Elem<T>::pack(b.x * scale, b.y * scale), Elem<T>::pack(b.z * scale, b.w * scale));
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(704, 1)
    pa_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo, const BwdArgs a) {
  using C = BwdCfg<D>;
  using G = TileGeo<D>;
  // fp16's P (at most 1) is scaled up for its product, away from the type's subnormals; dV is scaled back
  constexpr float kP = std::is_same<T, __half>::value ? 4096.f : 1.f;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* bar_kv_full = bars;                        // [KVB]
  uint64_t* bar_kv_free = bar_kv_full + C::KVB;        // [KVB]
  uint64_t* bar_q_full = bar_kv_free + C::KVB;         // [QST] Q, lse and delta of a step
  uint64_t* bar_q_free = bar_q_full + C::QST;          // [QST]
  uint64_t* bar_do_full = bar_q_free + C::QST;         // [OST]
  uint64_t* bar_do_free = bar_do_full + C::OST;        // [OST]
  uint64_t* bar_s_full = bar_do_free + C::OST;         // S^T of a step
  uint64_t* bar_p_full = bar_s_full + 1;               // P^T of a step written
  uint64_t* bar_dp_full = bar_p_full + 1;              // dP^T of a step
  uint64_t* bar_ds_full = bar_dp_full + 1;             // dS^T of a step written
  uint64_t* bar_ds_free = bar_ds_full + 1;             // [NDS]
  uint64_t* bar_dq_full = bar_ds_free + C::NDS;        // [NDQ]
  uint64_t* bar_dq_free = bar_dq_full + C::NDQ;        // [NDQ]
  uint64_t* bar_dkv_full = bar_dq_free + C::NDQ;       // the item's dK, dV
  uint64_t* bar_dkv_free = bar_dkv_full + 1;
  uint64_t* bar_drain = bar_dkv_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(smem + C::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, n_ctas = gridDim.x;
  if (threadIdx.x == 0) {
    for (int b = 0; b < C::KVB; ++b) {
      mbar_init(bar_kv_full + b, 1);
      mbar_init(bar_kv_free + b, 1);
    }
    for (int b = 0; b < C::QST; ++b) {
      mbar_init(bar_q_full + b, 1);
      mbar_init(bar_q_free + b, 1);
    }
    for (int b = 0; b < C::OST; ++b) {
      mbar_init(bar_do_full + b, 1);
      mbar_init(bar_do_free + b, 1);
    }
    mbar_init(bar_s_full, 1);
    mbar_init(bar_p_full, C::COMPUTE);
    mbar_init(bar_dp_full, 1);
    mbar_init(bar_ds_full, C::COMPUTE);
    for (int b = 0; b < C::NDS; ++b) mbar_init(bar_ds_free + b, 1);
    for (int b = 0; b < C::NDQ; ++b) {
      mbar_init(bar_dq_full + b, 1);
      mbar_init(bar_dq_free + b, 128);
    }
    mbar_init(bar_dkv_full, 1);
    mbar_init(bar_dkv_free, 128);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 21) tmem_alloc<512>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 20) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      bool ok = true;
      int g = 0, ni = 0, n_do = 0;
      for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
        const BwdItem it = bwd_item(a, item);
        const int kb = ni % C::KVB;
        if (ni >= C::KVB && !mbar_wait(bar_kv_free + kb, (ni / C::KVB - 1) & 1, abort_flag)) break;
        const int key0 = it.s.start + it.s.tile * kTile;
        mbar_arrive_expect_tx(bar_kv_full + kb, 2 * G::BYTES);
        load_tile<D>(smem + C::OFF_K + kb * G::BYTES, &mk, bar_kv_full + kb, it.hk, key0);
        load_tile<D>(smem + C::OFF_V + kb * G::BYTES, &mv, bar_kv_full + kb, it.hk, key0);
        ++ni;
        for (int j = 0; ok && j < it.n; ++j) {
          const int st = g % C::QST, h = it.hk * a.G + j / it.per, qt = it.s.tile + j % it.per;
          if (g >= C::QST && !mbar_wait(bar_q_free + st, (g / C::QST - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const int row = it.s.start + qt * kTile;
          mbar_arrive_expect_tx(bar_q_full + st, G::BYTES + C::LD_BYTES);
          load_tile<D>(smem + C::OFF_Q + st * G::BYTES, &mq, bar_q_full + st, h, row);
          bulk_load(smem + C::OFF_LD + st * C::LD_BYTES,
                    a.ld + (static_cast<long long>(h) * a.n_tiles + it.s.base + qt) * 2 * kTile, C::LD_BYTES, bar_q_full + st);
          ++g;
          const int so = n_do % C::OST;
          if (n_do >= C::OST && !mbar_wait(bar_do_free + so, (n_do / C::OST - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar_do_full + so, G::BYTES);
          load_tile<D>(smem + C::OFF_DO + so * G::BYTES, &mdo, bar_do_full + so, h, row);
          ++n_do;
        }
      }
      if (*(volatile int*)abort_flag) {  // no copy may land after the CTA has gone
        for (int i = ni > C::KVB ? ni - C::KVB : 0; i < ni; ++i) mbar_wait_drain(bar_kv_full + i % C::KVB, (i / C::KVB) & 1);
        for (int i = g > C::QST ? g - C::QST : 0; i < g; ++i) mbar_wait_drain(bar_q_full + i % C::QST, (i / C::QST) & 1);
        for (int i = n_do > C::OST ? n_do - C::OST : 0; i < n_do; ++i)
          mbar_wait_drain(bar_do_full + i % C::OST, (i / C::OST) & 1);
      }
    }
  } else if (warp == 21) {
    // ------------------------------------------------------------------ MMAs
    constexpr uint32_t id_s = make_idesc<T>(128, 128, false, false);
    constexpr uint32_t id_kv = make_idesc<T>(128, D, false, true);
    constexpr uint32_t id_q = make_idesc<T>(128, D, true, true);
    bool ok = true;
    int g = 0, ni = 0;
    for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas), ++ni) {
      const BwdItem it = bwd_item(a, item);
      const int kb = ni % C::KVB;
      uint8_t* sK = smem + C::OFF_K + kb * G::BYTES;
      uint8_t* sV = smem + C::OFF_V + kb * G::BYTES;
      const Desc k_k = G::kmajor(smem_u32(sK)), k_mn = G::mnmajor(smem_u32(sK)), v_k = G::kmajor(smem_u32(sV));
      ok = mbar_wait(bar_kv_full + kb, (ni / C::KVB) & 1, abort_flag);
      if (!ok) break;
      const int keys = it.s.len - it.s.tile * kTile;
      if (keys < kTile) {
        zero_rows<D>(sK, keys, lane);
        zero_rows<D>(sV, keys, lane);
      }
      // S^T and dP^T of step j (global step gg); a last, partial query tile is zeroed behind its rows first
      auto issue_s = [&](int j, int gg) -> bool {
        const int st = gg % C::QST;
        if (!mbar_wait(bar_q_full + st, (gg / C::QST) & 1, abort_flag)) return false;
        uint8_t* sQ = smem + C::OFF_Q + st * G::BYTES;
        const int rows = it.s.len - (it.s.tile + j % it.per) * kTile;
        if (rows < kTile) zero_rows<D>(sQ, rows, lane);
        tc_fence_after();
        const Desc q_k = G::kmajor(smem_u32(sQ));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(tmem + C::COL_S, k_k.at(G::kstep(kk)), q_k.at(G::kstep(kk)), id_s, kk > 0);
          mma_commit(bar_s_full);
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](int j, int gg) -> bool {
        const int so = gg % C::OST;
        if (!mbar_wait(bar_do_full + so, (gg / C::OST) & 1, abort_flag)) return false;
        // D = 128: the columns are free once the last dQ in them has been read
        if (D >= 128 && gg > 0 && !mbar_wait(bar_dq_free, (gg - 1) & 1, abort_flag)) return false;
        uint8_t* sDO = smem + C::OFF_DO + so * G::BYTES;
        const int rows = it.s.len - (it.s.tile + j % it.per) * kTile;
        if (rows < kTile) zero_rows<D>(sDO, rows, lane);
        tc_fence_after();
        const Desc do_k = G::kmajor(smem_u32(sDO));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(tmem + C::COL_DP, v_k.at(G::kstep(kk)), do_k.at(G::kstep(kk)), id_s, kk > 0);
          mma_commit(bar_dp_full);
        }
        __syncwarp();
        return true;
      };
      ok = issue_s(0, g) && issue_dp(0, g);
      for (int j = 0; ok && j < it.n; ++j, ++g) {
        const int st = g % C::QST;
        ok = mbar_wait(bar_p_full, g & 1, abort_flag);
        if (ok && j == 0 && ni > 0) ok = mbar_wait(bar_dkv_free, (ni - 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const Desc do_mn = G::mnmajor(smem_u32(smem + C::OFF_DO) + (g % C::OST) * G::BYTES);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)  // 16 queries of P^T = 8 TMEM columns; each group's half begins at its S^T columns
            mma_bf16_ts(tmem + C::COL_DV, tmem + C::COL_S + (kk / 2) * 32 + (kk % 2) * 8, do_mn.at(G::mnstep(kk)), id_kv,
                        j > 0 || kk > 0);
          mma_commit(bar_do_free + g % C::OST);
        }
        __syncwarp();
        if (j + 1 < it.n && !(ok = issue_s(j + 1, g + 1))) break;
        if (!(ok = mbar_wait(bar_ds_full, g & 1, abort_flag))) break;
        if (D < 128 && j + 1 < it.n && !(ok = issue_dp(j + 1, g + 1))) break;
        const int qb = g % C::NDQ;
        if (D < 128 && g >= C::NDQ && !(ok = mbar_wait(bar_dq_free + qb, (g / C::NDQ - 1) & 1, abort_flag))) break;
        tc_fence_after();
        // dS as queries x keys (M over two panels, 16 keys a k-step) and dS^T as keys x queries
        const uint32_t ds_base = smem_u32(smem + C::OFF_DS) + (g % C::NDS) * C::DS_BYTES;
        const Desc ds_mn(ds_base, kTile * 128, 1024, kSwizzle128), ds_k(ds_base, 16, 1024, kSwizzle128);
        const Desc q_mn = G::mnmajor(smem_u32(smem + C::OFF_Q) + st * G::BYTES);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_bf16_ss(tmem + C::COL_DQ + qb * D, ds_mn.at(kk * 2048), k_mn.at(G::mnstep(kk)), id_q, kk > 0);
          mma_commit(bar_dq_full + qb);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_bf16_ss(tmem + C::COL_DK, ds_k.at((kk / 4) * kTile * 128 + (kk % 4) * 32), q_mn.at(G::mnstep(kk)), id_kv,
                        j > 0 || kk > 0);
          mma_commit(bar_q_free + st);
          mma_commit(bar_ds_free + g % C::NDS);
        }
        __syncwarp();
        if (D >= 128 && j + 1 < it.n) ok = issue_dp(j + 1, g + 1);
      }
      if (ok && elect_one()) {
        mma_commit(bar_kv_free + kb);
        mma_commit(bar_dkv_full);
      }
    }
    if (elect_one()) {  // every MMA has completed before TMEM is released
      mma_commit(bar_drain);
      mbar_wait_drain(bar_drain, 0);
    }
    __syncwarp();
  } else if (warp >= 16) {
    // ------------------------------------------- read-out of dQ, dK and dV
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    bool ok = true;
    int g = 0, ni = 0, pieces = 0;
    for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas), ++ni) {
      const BwdItem it = bwd_item(a, item);
      for (int j = 0; ok && j < it.n; ++j, ++g) {
        const int qb = g % C::NDQ, h = it.hk * a.G + j / it.per, qt = it.s.tile + j % it.per;
        float* dst = a.dq_sum + (static_cast<long long>(h) * a.n_tiles + it.s.base + qt) * kTile * D + quarter * 32 * D;
        ok = mbar_wait(bar_dq_full + qb, (g / C::NDQ) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          tmem_ld32(tmem + lane_base + C::COL_DQ + qb * D + c * 32, v);
          tmem_wait_ld();
          if (c == D / 32 - 1) {
            tc_fence_before();
            mbar_arrive(bar_dq_free + qb);
          }
          // 32 rows x 32 columns go out as one bulk reduction of 4 KiB
          float4* stg = reinterpret_cast<float4*>(smem + C::OFF_STG + (quarter * 2 + (pieces & 1)) * C::STG_BYTES);
          if (lane == 0 && pieces >= 2) bulk_wait_read<1>();  // the piece two before has been read
          ++pieces;
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) stg[i * 32 + lane] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            bulk_reduce_add(dst + c * 32 * 32, stg, C::STG_BYTES);
            bulk_commit_group();
          }
        }
      }
      ok = ok && mbar_wait(bar_dkv_full, ni & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const int key = it.s.tile * kTile + row;
      const bool in = key < it.s.len;
      const long long krow = static_cast<long long>(it.s.start) + key;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const View& v = half ? a.dk : a.dv;
        const float f = half ? a.scale : 1.f / kP;
        T* out = static_cast<T*>(const_cast<void*>(v.p)) + krow * v.rs + it.hk * v.hs;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float x[32];
          tmem_ld32(tmem + lane_base + (half ? C::COL_DK : C::COL_DV) + c * 32, x);
          tmem_wait_ld();
          if (half == 1 && c == D / 32 - 1) {
            tc_fence_before();
            mbar_arrive(bar_dkv_free);
          }
          if (in)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(out + c * 32 + i * 8) =
                  make_uint4(Elem<T>::pack(x[8 * i] * f, x[8 * i + 1] * f), Elem<T>::pack(x[8 * i + 2] * f, x[8 * i + 3] * f),
                             Elem<T>::pack(x[8 * i + 4] * f, x[8 * i + 5] * f), Elem<T>::pack(x[8 * i + 6] * f, x[8 * i + 7] * f));
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // no reduction may read shared memory after the CTA has gone
  } else {
    // ------------------------------------------------------ P^T and dS^T
    const int w = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;  // w: which 32 queries
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_base + C::COL_S + w * 32, t_dp = tmem + lane_base + C::COL_DP + w * 32;
    const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2);
    const int first = row - w * 32;  // on the diagonal: the first query at or behind the key
    const uint32_t behind = first <= 0 ? 0xffffffffu : (first >= 32 ? 0u : 0xffffffffu << first);
    bool ok = true;
    int g = 0;
    for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
      const BwdItem it = bwd_item(a, item);
      for (int j = 0, in_head = 0; ok && j < it.n; ++j, ++g) {
        const int st = g % C::QST;
        const bool diag = in_head == 0;
        if (++in_head == it.per) in_head = 0;
        const float* ld = reinterpret_cast<const float*>(smem + C::OFF_LD + st * C::LD_BYTES) + w * 32;
        ok = mbar_wait(bar_q_full + st, (g / C::QST) & 1, abort_flag) && mbar_wait(bar_s_full, g & 1, abort_flag);
        tc_fence_after();
        float p[32];
        tmem_ld32(t_s, p);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 l = *reinterpret_cast<const float4*>(ld + 4 * c);
          const float2 e0 = f2_unpack(f2_fma(f2_pack(p[4 * c], p[4 * c + 1]), sc2, f2_pack(l.x, l.y)));
          const float2 e1 = f2_unpack(f2_fma(f2_pack(p[4 * c + 2], p[4 * c + 3]), sc2, f2_pack(l.z, l.w)));
          p[4 * c] = ex2(e0.x);
          p[4 * c + 1] = ex2(e0.y);
          p[4 * c + 2] = ex2(e1.x);
          p[4 * c + 3] = ex2(e1.y);
        }
        if (diag) {
#pragma unroll
          for (int i = 0; i < 32; ++i) p[i] = ((behind >> i) & 1u) ? p[i] : 0.f;
        }
        {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = Elem<T>::pack(p[2 * i] * kP, p[2 * i + 1] * kP);
          tmem_st8(t_s, pk);
          tmem_st8(t_s + 8, pk + 8);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar_p_full);

        ok = ok && mbar_wait(bar_dp_full, g & 1, abort_flag);
        tc_fence_after();
        float dp[32];
        tmem_ld32(t_dp, dp);
        tmem_wait_ld();
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 dl = *reinterpret_cast<const float4*>(ld + kTile + 4 * c);
          float s0 = p[4 * c] * (dp[4 * c] - dl.x), s1 = p[4 * c + 1] * (dp[4 * c + 1] - dl.y);
          float s2 = p[4 * c + 2] * (dp[4 * c + 2] - dl.z), s3 = p[4 * c + 3] * (dp[4 * c + 3] - dl.w);
          if (diag) {  // a masked place stays 0 whatever dP holds there
            const uint32_t m = behind >> (4 * c);
            s0 = (m & 1u) ? s0 : 0.f;
            s1 = (m & 2u) ? s1 : 0.f;
            s2 = (m & 4u) ? s2 : 0.f;
            s3 = (m & 8u) ? s3 : 0.f;
          }
          pk[2 * c] = Elem<T>::pack(s0, s1);
          pk[2 * c + 1] = Elem<T>::pack(s2, s3);
        }
        if (g >= C::NDS) ok = ok && mbar_wait(bar_ds_free + g % C::NDS, (g / C::NDS - 1) & 1, abort_flag);
        uint8_t* ds = smem + C::OFF_DS + (g % C::NDS) * C::DS_BYTES + (w >> 1) * kTile * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(ds + sw128_offset(row, (w & 1) * 4 + c)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar_ds_full);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 21) {
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

}  // namespace pa
