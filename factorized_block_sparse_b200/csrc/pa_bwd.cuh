// Backward kernels of packed causal attention on tcgen05.
//
// pa_bwd_pre_kernel   per (query tile, head): delta_i = <dO_i, o_i> and
//                     -lse_i log2 e, padded to whole tiles (fp16: also largest norms).
// pa_bwd_kernel, dkv_part
//                     an item is a tile of 128 keys of one K/V head and all
//                     query tiles of all query heads that see it (head by
//                     head, diagonal first).  Per step of 128 queries, keys on
//                     TMEM lanes:
//                       S^T = K Q^T,    P^T = 2^(S^T c - lse log2 e)
//                       dP^T = V dO^T,  dS^T = P^T (dP^T - delta)
//                       dV += P^T dO,   dK += dS^T Q
// pa_bwd_kernel, dq_part
//                     an item is a tile of 128 queries of one head and the key
//                     tiles before it; per step S, dP and dS with queries on
//                     TMEM lanes, and dQ += dS K.
//
// The scores are computed twice (7 products of 128 x 128 x D a tile pair in
// place of 5).  The other way, dQ of every tile pair added to a float32 sum in
// global memory by the kernel that holds the keys, was built and measured: it
// moves 512 D bytes of float32 reductions a tile pair, ran into them (12.9 ms
// against 9.8 ms without, one sequence of 32768, 16 heads of 128), needs the
// sums zeroed and converted, and leaves dq's last bits to their order.  Here
// every sum has a fixed order: a call gives the same bits every time.
//
// P^T, dS^T and dS go back into TMEM, rounded to the tensors' type (the one
// rounding before their products), over columns that have been read, and are
// the A operand of their products from there; shared memory only holds what
// TMA brings.  One thread issues all MMAs of a part; they execute in order, so
// a product behind another that reads its destination columns needs no wait.
//
// What bounds it.  D = 128: the products and the power they draw (executed
// rate 1.3 PFLOP/s on one sequence of 32768, at about 1.5 GHz).  D <= 64: the
// exponentials (16 a clock and SM, twice a score) and the arithmetic and waits
// around them, 2.0 us a tile pair against 0.7 us of products (tensor pipe 46 %,
// exponential unit 47 %, issue slots 52 % busy).  Measured there and not kept:
// the step in two halves of 64 columns with barriers of their
// own (text shape 1.02 -> 1.50 ms: twice the waits of the issuing thread), a
// second issuing warp (no change), 64 columns a compute thread (dK/dV part 597
// -> 679 us), dQ's steps in turn by two halves of the warps (1.04 -> 1.07 ms),
// the exponentials of two groups after those of the other two (1.04 -> 1.07
// ms).  Times of runs of milliseconds: 2 x 12288 rows, 8 heads of 64, 1.02 ms;
// ten ragged sequences of 16384 rows, 32 / 8 heads of 128, 1.43 ms; one of
// 32768, 16 / 2 heads of 128, 12.0 ms; 2 x 8192 rows, 8 / 4 heads of 32, 0.44.
// In runs of seconds, under the power limit: 1.19, 1.66 and 12.7 ms.
//
// Roles of both parts: compute groups of four warps (thread = row of the tile,
// kCols columns of the step each), four warps for the read-out of an item's
// result, one whose lane 0 is the TMA producer, one for TMEM and the MMAs.
#pragma once

#include <type_traits>

#include "pa_device.cuh"

namespace pa {

// Of every 8 pairs of exponentials, those on the FMA pipe (P is rounded to
// half the bits right after, and nothing is summed before).  Measured at none
// and here: dK/dV part 687 and 658 us (D = 64, text shape), 839 and 813 (D =
// 128, ragged); dQ part 477 and 466 (D = 64); at D = 128 any share costs.
template <int D>
constexpr int kDkvPoly = D <= 64 ? 1 : 3;
template <int D>
constexpr int kDqPoly = D <= 64 ? 1 : 0;
// Whether the issuing warp waits for the next tiles before it waits for a
// step's weights, so that no other wait stands between them and their products
// (D = 64, text shape: 1013 us, 1033 without; D = 128, ragged: 1434 and 1409 us).
template <int D>
constexpr bool kTilesAhead = D <= 64;
// Columns of the step that a compute thread takes.
constexpr int kCols = 32;
constexpr int kBwdComputeWarps = 4 * 128 / kCols, kBwdThreads = 32 * (kBwdComputeWarps + 6);

// TMEM column, inside its 128, of k-step kk of a weight tile: each group's
// packed pairs begin at the first of its kCols score columns.
__device__ constexpr uint32_t weight_col(int kk) { return (kk / (kCols / 16)) * kCols + (kk % (kCols / 16)) * 8; }

__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float* v) {
#pragma unroll
  for (int c = 0; c < kCols / 32; ++c) tmem_ld32(taddr + c * 32, v + c * 32);
  tmem_wait_ld();
}
__device__ __forceinline__ void tmem_st_weights(uint32_t taddr, const uint32_t* pk) {
#pragma unroll
  for (int c = 0; c < kCols / 16; ++c) tmem_st8(taddr + c * 8, pk + c * 8);
  tmem_wait_st();
}
// Zeroes the pairs' values whose bit is not set (a bit a column, kCols / 32 words).
__device__ __forceinline__ void keep_bits(float* v, const uint32_t* m) {
#pragma unroll
  for (int i = 0; i < kCols; ++i) v[i] = ((m[i / 32] >> (i % 32)) & 1u) ? v[i] : 0.f;
}

// fp16's P (at most 1) is scaled up for its product, away from the type's subnormals, by an addition to the stored
// -lse log2 e; dV is scaled back.
template <typename T>
constexpr int kWeightBits = std::is_same<T, __half>::value ? 12 : 0;

// fp16's dS is scaled, bf16's is not: dO of size 2^-10 over some thousands of keys makes it 2^-20, deep in fp16's
// subnormals, and dO and v of size 2^8 take it out of fp16's range.  |dS| <= P |dP - delta| <= 2 max|dO_i| max|v_j|
// (delta is a mean of dP), so the power of two that takes this bound to [2^14, 2^15) can neither overflow nor cost
// anything, and every sum is divided by it at the end.  The norms are those of the rows that an item's dS is made of
// (finite rows: the others make NaN of theirs whatever the factor).
template <typename T>
constexpr bool kScaleDs = std::is_same<T, __half>::value;

// The exponent of that factor from the largest squared norms.
__device__ __forceinline__ int ds_exponent(float do2, float v2) {
  const float m = do2 * v2;  // within 2^-96 .. 2^78
  if (!(m > 0.f)) return 0;
  const int k = static_cast<int>(__float_as_uint(m) >> 23) - 127;  // the bound is below 2^((k + 3) / 2)
  return 15 - ((k + 4) >> 1);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The exponent from the largest of `rows` runs of n values of p, `step` apart, and the largest of nv values of v, by a whole
// warp: an item starts with it, so eight loads are under way at a time, and its code is there once (2 x 12288 rows, 8
// heads of 64, fp16: 1300 us; copies at its four places 1340, a constant in its place 1275, dS unscaled, mostly
// subnormals that cost less power, 1260).
__device__ __noinline__ int ds_exponent(const float* p, int rows, int n, long long step, const float* v, int nv, int lane) {
  float m[2] = {0.f, 0.f};
  const int all = rows * n;
  for (int i = lane; i - lane < max(all, nv); i += 128) {
    float x[4], y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = i + 32 * u, r = j / n;
      x[u] = j < all ? p[r * step + (j - r * n)] : 0.f;
      y[u] = j < nv ? v[j] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) m[0] = fmaxf(m[0], x[u]), m[1] = fmaxf(m[1], y[u]);
  }
  return ds_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m[0]))),  // (no value is negative)
                     __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m[1]))));
}

// TPR threads a row, 8 columns each.  kScaleDs: peak [Hq + Hkv][n_tiles] takes the largest squared norm of a (head, tile)'s
// rows of dO, and of v behind them.
template <typename T, int D>
__global__ void __launch_bounds__(256)
    pa_bwd_pre_kernel(const Slot* slots, View o, View dO, View v, const float* lse, long long ls, float* ld, float* peak,
                      int n_tiles, int Hkv) {
  constexpr int TPR = D / 8, RPI = 256 / TPR;
  pdl_trigger();
  const Slot s = slots[blockIdx.x];
  const int h = blockIdx.y, tid = threadIdx.x;
  float* out = ld + (static_cast<long long>(h) * n_tiles + s.base + s.tile) * 2 * kTile;
  float most[2] = {0.f, 0.f};  // of dO and v
  auto row_norm = [&](float ss, float& m) {  // ss: the sum of a thread's 8 squares
#pragma unroll
    for (int w = TPR / 2; w >= 1; w >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, w);
    if (ss < INFINITY) m = fmaxf(m, ss);  // (neither NaN)
  };
  for (int r = tid / TPR; r < kTile; r += RPI) {
    const int i = s.tile * kTile + r;
    const bool in = i < s.len;
    float d = 0.f, ss = 0.f, sv = 0.f;
    if (in) {
      const long long row = static_cast<long long>(s.start) + i;
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const T*>(o.p) + row * o.rs + h * o.hs + (tid % TPR) * 8);
      const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const T*>(dO.p) + row * dO.rs + h * dO.hs + (tid % TPR) * 8);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 x = Elem<T>::unpack(aw[u]), y = Elem<T>::unpack(bw[u]);
        d += x.x * y.x + x.y * y.y;
        if constexpr (kScaleDs<T>) ss += y.x * y.x + y.y * y.y;
      }
      if constexpr (kScaleDs<T>)
        if (h < Hkv) {
          const uint4 e = *reinterpret_cast<const uint4*>(static_cast<const T*>(v.p) + row * v.rs + h * v.hs + (tid % TPR) * 8);
          const uint32_t ew[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 x = Elem<T>::unpack(ew[u]);
            sv += x.x * x.x + x.y * x.y;
          }
        }
    }
    if constexpr (kScaleDs<T>) {
      row_norm(ss, most[0]);
      if (h < Hkv) row_norm(sv, most[1]);
    }
#pragma unroll
    for (int w = TPR / 2; w >= 1; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
    if (tid % TPR == 0) {
      out[r] = in ? kWeightBits<T> - 1.4426950408889634f * lse[static_cast<long long>(h) * ls + s.start + i] : -INFINITY;
      out[kTile + r] = -d;
    }
  }
  if constexpr (kScaleDs<T>) {
    __shared__ float warps[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(most[k]));
      if ((tid & 31) == 0) warps[k][tid >> 5] = __uint_as_float(m);
    }
    __syncthreads();
    if (tid < 2 && (tid == 0 || h < Hkv)) {
      float m = warps[tid][0];
#pragma unroll
      for (int w = 1; w < 8; ++w) m = fmaxf(m, warps[tid][w]);
      peak[static_cast<long long>(tid == 0 ? h : static_cast<int>(gridDim.y) + h) * n_tiles + s.base + s.tile] = m;
    }
  }
}

// Steps of part sp of an item of `all` steps.
__host__ __device__ __forceinline__ int part_first(int all, int sp, int split) {
  return static_cast<int>(static_cast<long long>(all) * sp / split);
}

// dV and dK of items in parts: the parts' sums in order, rounded once.  A block
// takes kSumRows rows of a (key tile, K/V head), a thread 8 columns of one.
constexpr int kSumRows = 16;
template <typename T, int D>
__global__ void __launch_bounds__(256)
    pa_bwd_sum_kernel(const Slot* slots, const float* part, int split, int Hkv, int G, long long rows, View dk, View dv,
                      float scale) {
  pdl_wait();
  const Slot s = slots[blockIdx.x];
  const int hk = blockIdx.y, r0 = blockIdx.z * kSumRows, n_rows = min(kSumRows, s.len - s.tile * kTile - r0);
  const int all = ((s.len + kTile - 1) / kTile - s.tile) * G;
  const long long row0 = static_cast<long long>(s.start) + s.tile * kTile + r0, plane = Hkv * rows * D;
  for (int i = threadIdx.x; i < 2 * n_rows * (D / 8); i += 256) {
    const int c = i % (D / 8), which = i / (D / 8) / n_rows, r = i / (D / 8) % n_rows;
    const float* p = part + which * plane + (hk * rows + row0 + r) * D + c * 8;
    float x[8] = {};
    for (int sp = 0; sp < split; ++sp) {
      if (part_first(all, sp, split) == part_first(all, sp + 1, split)) continue;  // (never written)
      const float4 u = *reinterpret_cast<const float4*>(p + sp * 2 * plane);
      const float4 v = *reinterpret_cast<const float4*>(p + sp * 2 * plane + 4);
      x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w, x[4] += v.x, x[5] += v.y, x[6] += v.z, x[7] += v.w;
    }
    const View& o = which ? dk : dv;
    const float f = which ? scale : 1.f / (1 << kWeightBits<T>);
    *reinterpret_cast<uint4*>(static_cast<T*>(const_cast<void*>(o.p)) + (row0 + r) * o.rs + hk * o.hs + c * 8) =
        make_uint4(Elem<T>::pack(x[0] * f, x[1] * f), Elem<T>::pack(x[2] * f, x[3] * f),
                   Elem<T>::pack(x[4] * f, x[5] * f), Elem<T>::pack(x[6] * f, x[7] * f));
  }
}

// Writes one row's D float32 values from TMEM, times f.
template <int D>
__device__ __forceinline__ void row_out_f32(float* out, uint32_t taddr, bool in, float f) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float x[32];
    tmem_ld32(taddr + c * 32, x);
    tmem_wait_ld();
    if (in)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float4*>(out + c * 32 + 4 * i) = make_float4(x[4 * i] * f, x[4 * i + 1] * f, x[4 * i + 2] * f, x[4 * i + 3] * f);
  }
}

// Writes one row's D float32 values from TMEM, times f, as T.
template <typename T, int D>
__device__ __forceinline__ void row_out(T* out, uint32_t taddr, bool in, float f) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float x[32];
    tmem_ld32(taddr + c * 32, x);
    tmem_wait_ld();
    if (in)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(out + c * 32 + i * 8) =
            make_uint4(Elem<T>::pack(x[8 * i] * f, x[8 * i + 1] * f), Elem<T>::pack(x[8 * i + 2] * f, x[8 * i + 3] * f),
                       Elem<T>::pack(x[8 * i + 4] * f, x[8 * i + 5] * f), Elem<T>::pack(x[8 * i + 6] * f, x[8 * i + 7] * f));
  }
}

// Shared memory of the two parts: their tiles from 0 on, then the barriers of each.
template <int D>
struct BwdSmem {
  static constexpr int BARS = D >= 128 ? 19 : 32;
  static constexpr int OFF_BARS = 227 * 1024 - 16 - 16 * BARS;
};
template <int D>
struct BwdCfg {
  static constexpr int OFF_MISC = 227 * 1024 - 16, SMEM = 227 * 1024;
};

// ------------------------------------------------------------------ dK, dV
struct DkvArgs {
  const Slot* slots;
  int n_items, Hkv, G;
  int n_tiles;      // 128-row tiles of all sequences
  const float* ld;  // [Hq][n_tiles][2][128]: kWeightBits - lse log2 e (padding -inf), -delta (padding 0)
  const float *peak_do, *peak_v;  // [Hq][n_tiles], [Hkv][n_tiles]: largest squared norms of the rows (kScaleDs)
  View dk, dv;
  float scale, scale_log2;
  // Few key tiles and many steps each: the steps of an item in `split` parts,
  // whose float32 sums pa_bwd_sum_kernel adds up in order.
  int split;
  float* part;     // [split][dv, dk][Hkv][rows][D], or null
  long long rows;
};

template <int D>
struct DkvCfg {
  using G = TileGeo<D>;
  static constexpr int KVB = D >= 128 ? 1 : 2;  // K/V buffers
  static constexpr int QST = D >= 128 ? 3 : 5;  // Q stages, with delta
  static constexpr int OST = D >= 128 ? 2 : 4;  // dO stages, with lse
  static constexpr int NS = D >= 128 ? 1 : 2;   // S^T buffers in TMEM
  static constexpr int VEC = kTile * 4;         // a tile's lse or delta
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + KVB * G::BYTES;
  static constexpr int OFF_Q = OFF_V + KVB * G::BYTES;
  static constexpr int OFF_DO = OFF_Q + QST * G::BYTES;
  static constexpr int OFF_DELTA = OFF_DO + OST * G::BYTES;
  static constexpr int OFF_LSE = OFF_DELTA + QST * VEC;
  static constexpr int END = OFF_LSE + OST * VEC;  // of the tiles
  static constexpr int N_BARS = 2 * KVB + 2 * QST + 2 * OST + 2 * NS + 2 + 2 + 1;
  static constexpr int OFF_BAR = BwdSmem<D>::OFF_BARS;
  static constexpr int COL_DP = NS * 128, COL_DV = COL_DP + 128, COL_DK = COL_DV + D;
  // P^T takes the first 16 of each group's 32 columns of its S^T buffer.  With
  // two buffers dS^T takes the other 16, so dP^T is free once it has been read
  // and the next one is under way before dK; with one buffer dS^T goes over
  // dP^T, so that the next S^T only waits for dV.
  static constexpr bool DS_IN_S = NS == 2;
  static_assert(END <= OFF_BAR && N_BARS <= BwdSmem<D>::BARS && COL_DK + D <= 512, "shared memory and TMEM");
};

struct DkvItem {
  Slot s;
  int hk, per;       // K/V head, steps of one query head
  int sp, first, n;  // which part of the steps, its first step and how many (0: nothing to do)
};

__device__ __forceinline__ DkvItem dkv_item(const DkvArgs& a, const Slot& s, int item) {
  DkvItem it;
  const int r = item % (a.Hkv * a.split);
  it.hk = r / a.split;
  it.sp = r % a.split;
  it.s = s;
  it.per = (it.s.len + kTile - 1) / kTile - it.s.tile;
  it.first = part_first(it.per * a.G, it.sp, a.split);
  it.n = part_first(it.per * a.G, it.sp + 1, a.split) - it.first;
  return it;
}

// Exponent of an item's factor of dS: dO of the group's heads from the key tile on, v of the whole sequence (delta).
template <typename T>
__device__ __forceinline__ int ds_exponent(const DkvArgs& a, const DkvItem& it, int lane) {
  if constexpr (!kScaleDs<T>) return 0;
  return ds_exponent(a.peak_do + static_cast<long long>(it.hk) * a.G * a.n_tiles + it.s.base + it.s.tile, a.G, it.per, a.n_tiles,
                     a.peak_v + static_cast<long long>(it.hk) * a.n_tiles + it.s.base, it.s.tile + it.per, lane);
}

// One part of the kernel: its barriers (their place in shared memory), initialised by one thread.
// p_full has one for each S^T buffer: with two buffers S^T of step j + 1 is there before the issuing warp has seen the
// weights of step j, so a compute warp may write P^T of both before then.  On one barrier its second arrival could stand
// for a slower warp's first, or two phases could pass unseen; S^T of step j + 2, which the buffer's next arrivals wait
// for, is issued behind dS^T of step j, that is behind all arrivals of step j and the wait for them.
template <int D>
struct DkvBars {
  using C = DkvCfg<D>;
  uint64_t *kv_full, *kv_free, *q_full, *q_free, *do_full, *do_free, *s_full, *p_full, *dp_full, *ds_full, *out_full,
      *out_free, *drain;
  __device__ __forceinline__ explicit DkvBars(uint8_t* smem) {
    kv_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [KVB]
    kv_free = kv_full + C::KVB;                                // [KVB]
    q_full = kv_free + C::KVB;                                 // [QST]
    q_free = q_full + C::QST;                                  // [QST]
    do_full = q_free + C::QST;                                 // [OST]
    do_free = do_full + C::OST;                                // [OST]
    s_full = do_free + C::OST;                                 // [NS] S^T of a step
    p_full = s_full + C::NS;                                   // [NS] P^T of a step written
    dp_full = p_full + C::NS;                                  // dP^T of a step
    ds_full = dp_full + 1;                                     // dS^T of a step written
    out_full = ds_full + 1;                                    // the item's dK, dV
    out_free = out_full + 1;
    drain = out_free + 1;
  }
  __device__ __forceinline__ void init() const {
    for (uint64_t* b = kv_full; b < p_full; ++b) mbar_init(b, 1);
    for (int b = 0; b < C::NS; ++b) mbar_init(p_full + b, kBwdComputeWarps);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, kBwdComputeWarps);
    mbar_init(out_full, 1);
    mbar_init(out_free, 4);
    mbar_init(drain, 1);
  }
};

template <typename T, int D>
__device__ __forceinline__ void dkv_part(uint8_t* smem, const uint32_t tmem, int* abort_flag, const CUtensorMap& mq,
                                         const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo,
                                         const DkvArgs& a) {
  using C = DkvCfg<D>;
  using G = TileGeo<D>;
  const DkvBars<D> bar(smem);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int cta = blockIdx.x, n_ctas = gridDim.x;
  const SlotWalk walk(a.slots, a.n_items, a.Hkv * a.split);

  if (warp == kBwdComputeWarps + 4) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      bool ok = true;
      int g = 0, ni = 0, n_do = 0;
      for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
        const DkvItem it = dkv_item(a, walk.take(item, k), item);
        if (it.n == 0) continue;
        const int kb = ni % C::KVB;
        if (ni >= C::KVB && !mbar_wait(bar.kv_free + kb, (ni / C::KVB - 1) & 1, abort_flag)) break;
        const int key0 = it.s.start + it.s.tile * kTile;
        if (!PA_WITHHELD(kHoldDkvK, ni)) {
          mbar_arrive_expect_tx(bar.kv_full + kb, 2 * G::BYTES);
          load_tile<D>(smem + C::OFF_K + kb * G::BYTES, &mk, bar.kv_full + kb, it.hk, key0);
          load_tile<D>(smem + C::OFF_V + kb * G::BYTES, &mv, bar.kv_full + kb, it.hk, key0);
        }
        ++ni;
        for (int j = it.first; ok && j < it.first + it.n; ++j) {
          const int h = it.hk * a.G + j / it.per, qt = it.s.tile + j % it.per, row = it.s.start + qt * kTile;
          const float* ld = a.ld + (static_cast<long long>(h) * a.n_tiles + it.s.base + qt) * 2 * kTile;
          const int sq = g % C::QST;
          if (g >= C::QST && !mbar_wait(bar.q_free + sq, (g / C::QST - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar.q_full + sq, G::BYTES + C::VEC);
          load_tile<D>(smem + C::OFF_Q + sq * G::BYTES, &mq, bar.q_full + sq, h, row);
          bulk_load(smem + C::OFF_DELTA + sq * C::VEC, ld + kTile, C::VEC, bar.q_full + sq);
          ++g;
          const int so = n_do % C::OST;
          if (n_do >= C::OST && !mbar_wait(bar.do_free + so, (n_do / C::OST - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          if (!PA_WITHHELD(kHoldDkvDO, n_do)) {
            mbar_arrive_expect_tx(bar.do_full + so, G::BYTES + C::VEC);
            load_tile<D>(smem + C::OFF_DO + so * G::BYTES, &mdo, bar.do_full + so, h, row);
            bulk_load(smem + C::OFF_LSE + so * C::VEC, ld, C::VEC, bar.do_full + so);
          }
          ++n_do;
        }
      }
      // no copy may land after the CTA has gone or the other part has begun, whichever role gives up, and when
      for (int i = ni > C::KVB ? ni - C::KVB : 0; i < ni; ++i) mbar_wait_drain(bar.kv_full + i % C::KVB, (i / C::KVB) & 1);
      for (int i = g > C::QST ? g - C::QST : 0; i < g; ++i) mbar_wait_drain(bar.q_full + i % C::QST, (i / C::QST) & 1);
      for (int i = n_do > C::OST ? n_do - C::OST : 0; i < n_do; ++i)
        mbar_wait_drain(bar.do_full + i % C::OST, (i / C::OST) & 1);
    }
  } else if (warp == kBwdComputeWarps + 5) {
    // ------------------------------------------------------------------ MMAs
    constexpr uint32_t id_s = make_idesc<T>(128, 128, false, false);
    constexpr uint32_t id_o = make_idesc<T>(128, D, false, true);
    bool ok = true;
    int ni = 0;
    // next S^T and dP^T to issue; the step whose weights are awaited
    Ring<C::QST> iq, rq;
    Ring<C::OST> io, ro;
    Ring<C::NS> is, rs;
    Ring<C::KVB> rk;
    uint32_t ph = 0;
    for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
      DkvItem it = dkv_item(a, walk.take(item, k), item);
      it.s = uniform(it.s);
      it.per = uniform(it.per);
      it.n = uniform(it.n);
      if (it.n == 0) continue;
      const int skip = uniform(it.first) % it.per;  // query tiles before the first step's
      const int kb = rk.st;
      uint8_t* sK = smem + C::OFF_K + kb * G::BYTES;
      uint8_t* sV = smem + C::OFF_V + kb * G::BYTES;
      const Desc k_k = G::kmajor(smem_u32(sK)), v_k = G::kmajor(smem_u32(sV));
      ok = mbar_wait_warp(bar.kv_full + kb, rk.ph, abort_flag);
      rk.next();
      if (!ok) break;
      const int keys = it.s.len - it.s.tile * kTile;
      if (keys < kTile) {
        zero_rows<D>(sK, keys, lane);
        zero_rows<D>(sV, keys, lane);
      }
      int rows_s = keys - skip * kTile, left_s = it.per - skip, rows_p = rows_s, left_p = left_s;  // of the next query tile
      // S^T (dP^T) of the item's next step; a last, partial query tile is zeroed behind its rows first
      auto has_q = [&]() { return mbar_wait_warp(bar.q_full + iq.st, iq.ph, abort_flag); };
      auto has_do = [&]() { return mbar_wait_warp(bar.do_full + io.st, io.ph, abort_flag); };
      auto issue_s = [&]() {
        uint8_t* sQ = smem + C::OFF_Q + iq.st * G::BYTES;
        if (rows_s < kTile) zero_rows<D>(sQ, rows_s, lane);
        rows_s -= kTile;
        if (--left_s == 0) rows_s = keys, left_s = it.per;
        tc_fence_after();
        const Desc q_k = G::kmajor(smem_u32(sQ));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(tmem + is.st * 128, k_k.at(G::kstep(kk)), q_k.at(G::kstep(kk)), id_s, kk > 0);
          mma_commit(bar.s_full + is.st);
        }
        __syncwarp();
        iq.next();
        is.next();
      };
      auto issue_dp = [&]() {
        uint8_t* sDO = smem + C::OFF_DO + io.st * G::BYTES;
        if (rows_p < kTile) zero_rows<D>(sDO, rows_p, lane);
        rows_p -= kTile;
        if (--left_p == 0) rows_p = keys, left_p = it.per;
        tc_fence_after();
        const Desc do_k = G::kmajor(smem_u32(sDO));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(tmem + C::COL_DP, v_k.at(G::kstep(kk)), do_k.at(G::kstep(kk)), id_s, kk > 0);
          mma_commit(bar.dp_full);
        }
        __syncwarp();
        io.next();
      };
      if (!(ok = has_q())) break;
      issue_s();
      if (!(ok = has_do())) break;
      issue_dp();
      if (C::NS > 1 && it.n > 1) {
        if (!(ok = has_q())) break;
        issue_s();
      }
      for (int j = 0; ok && j < it.n; ++j) {
        if (kTilesAhead<D>) ok = (j + C::NS >= it.n || has_q()) && (j + 1 >= it.n || has_do());
        ok = ok && mbar_wait_warp(bar.p_full + rs.st, rs.ph, abort_flag);
        if (ok && j == 0 && ni > 0) ok = mbar_wait_warp(bar.out_free, (ni - 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const Desc do_mn = G::mnmajor(smem_u32(smem + C::OFF_DO) + ro.st * G::BYTES);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)  // 16 queries = 8 TMEM columns of P^T, each group's from its first column on
            mma_bf16_ts(tmem + C::COL_DV, tmem + rs.st * 128 + weight_col(kk), do_mn.at(G::mnstep(kk)),
                        id_o, j > 0 || kk > 0);
          mma_commit(bar.do_free + ro.st);
        }
        __syncwarp();
        if (!C::DS_IN_S && j + 1 < it.n) {  // over P^T, behind its product
          if (!kTilesAhead<D> && !(ok = has_q())) break;
          issue_s();
        }
        if (!(ok = mbar_wait_warp(bar.ds_full, ph, abort_flag))) break;
        if (C::DS_IN_S && j + 1 < it.n) {
          if (!kTilesAhead<D> && !(ok = has_do())) break;
          issue_dp();
        }
        tc_fence_after();
        const Desc q_mn = G::mnmajor(smem_u32(smem + C::OFF_Q) + rq.st * G::BYTES);
        const uint32_t t_ds = tmem + (C::DS_IN_S ? rs.st * 128 + kCols / 2 : C::COL_DP);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_bf16_ts(tmem + C::COL_DK, t_ds + weight_col(kk), q_mn.at(G::mnstep(kk)), id_o,
                        j > 0 || kk > 0);
          mma_commit(bar.q_free + rq.st);
        }
        __syncwarp();
        rq.next();
        ro.next();
        rs.next();
        ph ^= 1;
        if (C::DS_IN_S && j + 2 < it.n) {  // over P^T and dS^T, behind their products
          if (!kTilesAhead<D> && !(ok = has_q())) break;
          issue_s();
        }
        if (!C::DS_IN_S && j + 1 < it.n) {  // over dS^T, behind its product
          if (!kTilesAhead<D> && !(ok = has_do())) break;
          issue_dp();
        }
      }
      if (ok && elect_one()) {
        mma_commit(bar.kv_free + kb);
        mma_commit(bar.out_full);
      }
      ++ni;
    }
    if (elect_one()) {  // every MMA has completed before TMEM is released
      mma_commit(bar.drain);
      mbar_wait_drain(bar.drain, 0);
    }
    __syncwarp();
  } else if (warp >= kBwdComputeWarps) {
    // --------------------------------------------------- read-out of dK, dV
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    bool ok = true;
    int ni = 0;
    for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
      const DkvItem it = dkv_item(a, walk.take(item, k), item);
      if (it.n == 0) continue;
      const float unscale = pow2(-ds_exponent<T>(a, it, lane));
      ok = warp_ok(mbar_wait_steps(bar.out_full, ni & 1, abort_flag, it.n));
      if (!ok) break;
      ++ni;
      tc_fence_after();
      const int key = it.s.tile * kTile + row;
      const long long krow = static_cast<long long>(it.s.start) + key;
      const bool in = key < it.s.len;
      if (a.part) {
        float* dst = a.part + ((static_cast<long long>(it.sp) * 2 * a.Hkv + it.hk) * a.rows + krow) * D;
        row_out_f32<D>(dst, tmem + lane_base + C::COL_DV, in, 1.f);
        row_out_f32<D>(dst + a.Hkv * a.rows * D, tmem + lane_base + C::COL_DK, in, unscale);
      } else {
        row_out<T, D>(static_cast<T*>(const_cast<void*>(a.dv.p)) + krow * a.dv.rs + it.hk * a.dv.hs,
                      tmem + lane_base + C::COL_DV, in, 1.f / (1 << kWeightBits<T>));
        row_out<T, D>(static_cast<T*>(const_cast<void*>(a.dk.p)) + krow * a.dk.rs + it.hk * a.dk.hs,
                      tmem + lane_base + C::COL_DK, in, a.scale * unscale);
      }
      tc_fence_before();
      warp_arrive(bar.out_free, lane);
    }
  } else {
    // ------------------------------------------------------ P^T and dS^T
    const int w = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;  // w: which kCols queries
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + w * kCols;
    const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2);
    uint32_t behind[kCols / 32];  // on the diagonal: the queries at or behind the key
#pragma unroll
    for (int c = 0; c < kCols / 32; ++c) {
      const int first = row - w * kCols - c * 32;
      behind[c] = first <= 0 ? 0xffffffffu : (first >= 32 ? 0u : 0xffffffffu << first);
    }
    const float* lse0 = reinterpret_cast<const float*>(smem + C::OFF_LSE) + w * kCols;
    const float* delta0 = reinterpret_cast<const float*>(smem + C::OFF_DELTA) + w * kCols;
    bool ok = true;
    Ring<C::QST> rq;
    Ring<C::OST> ro;
    Ring<C::NS> rs;
    uint32_t ph = 0;
    for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
      const DkvItem it = dkv_item(a, walk.take(item, k), item);
      const float up = it.n > 0 ? pow2(ds_exponent<T>(a, it, lane) - kWeightBits<T>) : 1.f;  // of dS
      for (int j = 0, in_head = it.first % it.per; ok && j < it.n; ++j) {
        const bool diag = in_head == 0;
        if (++in_head == it.per) in_head = 0;
        const uint32_t t_s = t_row + rs.st * 128, t_dp = t_row + C::COL_DP;
        const float* lse = lse0 + ro.st * kTile;
        const float* delta = delta0 + rq.st * kTile;
        ok = mbar_wait(bar.do_full + ro.st, ro.ph, abort_flag) && mbar_wait(bar.s_full + rs.st, rs.ph, abort_flag);
        tc_fence_after();
        float p[kCols];
        tmem_ld_cols(t_s, p);
#pragma unroll
        for (int c = 0; c < kCols / 4; ++c) {
          const float4 l = *reinterpret_cast<const float4*>(lse + 4 * c);
          const float2 e0 = ex2_pair<T, kDkvPoly<D>>(f2_fma(f2_pack(p[4 * c], p[4 * c + 1]), sc2, f2_pack(l.x, l.y)), 2 * c);
          const float2 e1 =
              ex2_pair<T, kDkvPoly<D>>(f2_fma(f2_pack(p[4 * c + 2], p[4 * c + 3]), sc2, f2_pack(l.z, l.w)), 2 * c + 1);
          p[4 * c] = e0.x;
          p[4 * c + 1] = e0.y;
          p[4 * c + 2] = e1.x;
          p[4 * c + 3] = e1.y;
        }
        if (diag) keep_bits(p, behind);
        uint32_t pk[kCols / 2];
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) pk[i] = Elem<T>::pack(p[2 * i], p[2 * i + 1]);
        tmem_st_weights(t_s, pk);
        tc_fence_before();
        warp_arrive(bar.p_full + rs.st, lane);

        ok = warp_ok(ok && mbar_wait(bar.q_full + rq.st, rq.ph, abort_flag) && mbar_wait(bar.dp_full, ph, abort_flag));
        tc_fence_after();
        float dp[kCols];
        tmem_ld_cols(t_dp, dp);
#pragma unroll
        for (int c = 0; c < kCols / 4; ++c) {
          const float4 dl = *reinterpret_cast<const float4*>(delta + 4 * c);
          const float2 d0 = f2_unpack(f2_mul(f2_pack(p[4 * c], p[4 * c + 1]),
                                             f2_add(f2_pack(dp[4 * c], dp[4 * c + 1]), f2_pack(dl.x, dl.y))));
          const float2 d1 = f2_unpack(f2_mul(f2_pack(p[4 * c + 2], p[4 * c + 3]),
                                             f2_add(f2_pack(dp[4 * c + 2], dp[4 * c + 3]), f2_pack(dl.z, dl.w))));
          dp[4 * c] = d0.x;
          dp[4 * c + 1] = d0.y;
          dp[4 * c + 2] = d1.x;
          dp[4 * c + 3] = d1.y;
        }
        if (diag) keep_bits(dp, behind);  // a masked place stays 0 whatever dP holds there
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {
          if constexpr (kScaleDs<T>) {
            const float2 d = f2_unpack(f2_mul(f2_pack(dp[2 * i], dp[2 * i + 1]), f2_pack(up, up)));
            pk[i] = Elem<T>::pack(d.x, d.y);
          } else {
            pk[i] = Elem<T>::pack(dp[2 * i], dp[2 * i + 1]);
          }
        }
        tmem_st_weights(C::DS_IN_S ? t_s + kCols / 2 : t_dp, pk);
        tc_fence_before();
        warp_arrive(bar.ds_full, lane);
        rq.next();
        ro.next();
        rs.next();
        ph ^= 1;
      }
    }
  }
}

// ---------------------------------------------------------------------- dQ
struct DqArgs {
  const Slot* slots;
  int n_items, Hq, G;
  int n_tiles;
  const float *ld, *peak_do, *peak_v;  // as DkvArgs
  View dq;
  float scale, scale_log2;
};

// Exponent of an item's factor of dS: dO of the tile's rows, v of the rows that they see.
template <typename T>
__device__ __forceinline__ int ds_exponent(const DqArgs& a, const Slot& s, int h, int lane) {
  if constexpr (!kScaleDs<T>) return 0;
  return ds_exponent(a.peak_do + static_cast<long long>(h) * a.n_tiles + s.base + s.tile, 1, 1, 0,
                     a.peak_v + static_cast<long long>(h / a.G) * a.n_tiles + s.base, s.tile + 1, lane);
}

template <int D>
struct DqCfg {
  using G = TileGeo<D>;
  static constexpr int QB = D >= 128 ? 1 : 2;   // Q/dO buffers
  static constexpr int KST = D >= 128 ? 3 : 5;  // K stages
  static constexpr int VST = D >= 128 ? 2 : 4;  // V stages
  static constexpr int OB = D >= 128 ? 1 : 2;   // dQ buffers in TMEM
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_DO = OFF_Q + QB * G::BYTES;
  static constexpr int OFF_K = OFF_DO + QB * G::BYTES;
  static constexpr int OFF_V = OFF_K + KST * G::BYTES;
  static constexpr int END = OFF_V + VST * G::BYTES;  // of the tiles
  static constexpr int N_BARS = 2 * QB + 2 * KST + 2 * VST + 2 + 2 + 2 * OB + 1;
  static constexpr int OFF_BAR = BwdSmem<D>::OFF_BARS + 8 * BwdSmem<D>::BARS;
  static constexpr int COL_DP = 256, COL_DQ = 384;  // S: two buffers from 0; dQ + b * D
  static_assert(END <= BwdSmem<D>::OFF_BARS && N_BARS <= BwdSmem<D>::BARS && COL_DQ + OB * D <= 512,
                "shared memory and TMEM");
};

template <int D>
struct DqBars {
  using C = DqCfg<D>;
  uint64_t *q_full, *q_free, *k_full, *k_free, *v_full, *v_free, *s_full, *dp_full, *ds_full, *out_full, *out_free, *drain;
  __device__ __forceinline__ explicit DqBars(uint8_t* smem) {
    q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [QB] Q and dO of an item
    q_free = q_full + C::QB;                                  // [QB]
    k_full = q_free + C::QB;                                  // [KST]
    k_free = k_full + C::KST;                                 // [KST]
    v_full = k_free + C::KST;                                 // [VST]
    v_free = v_full + C::VST;                                 // [VST]
    s_full = v_free + C::VST;                                 // [2]
    dp_full = s_full + 2;
    ds_full = dp_full + 1;
    out_full = ds_full + 1;                                   // [OB]
    out_free = out_full + C::OB;                              // [OB]
    drain = out_free + C::OB;
  }
  __device__ __forceinline__ void init() const {
    for (uint64_t* b = q_full; b < ds_full; ++b) mbar_init(b, 1);
    mbar_init(ds_full, kBwdComputeWarps);
    for (int b = 0; b < C::OB; ++b) {
      mbar_init(out_full + b, 1);
      mbar_init(out_free + b, 4);
    }
    mbar_init(drain, 1);
  }
};

template <typename T, int D>
__device__ __forceinline__ void dq_part(uint8_t* smem, const uint32_t tmem, int* abort_flag, const CUtensorMap& mq,
                                        const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo,
                                        const DqArgs& a) {
  using C = DqCfg<D>;
  using G = TileGeo<D>;
  const DqBars<D> bar(smem);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  // the CTAs in opposite order to the other part's: a few items of both run side by side
  const int cta = gridDim.x - 1 - blockIdx.x, n_ctas = gridDim.x;
  const SlotWalk walk(a.slots, a.n_items, a.Hq, cta);

  if (warp == kBwdComputeWarps + 4) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      bool ok = true;
      int g = 0, ni = 0, nv = 0;
      for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
        const int h = item % a.Hq;
        const Slot s = walk.take(item, k);
        const int qb = ni % C::QB;
        if (ni >= C::QB && !mbar_wait(bar.q_free + qb, (ni / C::QB - 1) & 1, abort_flag)) break;
        if (!PA_WITHHELD(kHoldDqQ, ni)) {
          mbar_arrive_expect_tx(bar.q_full + qb, 2 * G::BYTES);
          load_tile<D>(smem + C::OFF_Q + qb * G::BYTES, &mq, bar.q_full + qb, h, s.start + s.tile * kTile);
          load_tile<D>(smem + C::OFF_DO + qb * G::BYTES, &mdo, bar.q_full + qb, h, s.start + s.tile * kTile);
        }
        ++ni;
        for (int j = 0; ok && j <= s.tile; ++j) {
          const int row = s.start + j * kTile, sk = g % C::KST;
          if (g >= C::KST && !mbar_wait(bar.k_free + sk, (g / C::KST - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar.k_full + sk, G::BYTES);
          load_tile<D>(smem + C::OFF_K + sk * G::BYTES, &mk, bar.k_full + sk, h / a.G, row);
          ++g;
          const int sv = nv % C::VST;
          if (nv >= C::VST && !mbar_wait(bar.v_free + sv, (nv / C::VST - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          if (!PA_WITHHELD(kHoldDqV, nv)) {
            mbar_arrive_expect_tx(bar.v_full + sv, G::BYTES);
            load_tile<D>(smem + C::OFF_V + sv * G::BYTES, &mv, bar.v_full + sv, h / a.G, row);
          }
          ++nv;
        }
      }
      // no copy may land after the CTA has gone, whichever role gives up, and when
      for (int i = ni > C::QB ? ni - C::QB : 0; i < ni; ++i) mbar_wait_drain(bar.q_full + i % C::QB, (i / C::QB) & 1);
      for (int i = g > C::KST ? g - C::KST : 0; i < g; ++i) mbar_wait_drain(bar.k_full + i % C::KST, (i / C::KST) & 1);
      for (int i = nv > C::VST ? nv - C::VST : 0; i < nv; ++i) mbar_wait_drain(bar.v_full + i % C::VST, (i / C::VST) & 1);
    }
  } else if (warp == kBwdComputeWarps + 5) {
    // ------------------------------------------------------------------ MMAs
    constexpr uint32_t id_s = make_idesc<T>(128, 128, false, false);
    constexpr uint32_t id_o = make_idesc<T>(128, D, false, true);
    bool ok = true;
    int ni = 0;
    Ring<C::KST> ik, rk;  // next S to issue; the step whose weights are awaited
    Ring<C::VST> iv;
    Ring<2> is, rs;
    Ring<C::QB> rq;
    Ring<C::OB> rb;
    uint32_t ph = 0;
    for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas), ++ni) {
      const Slot s = uniform(walk.take(item, k));
      const int n = s.tile + 1, qb = rq.st, ob = rb.st;
      ok = mbar_wait_warp(bar.q_full + qb, rq.ph, abort_flag);
      if (!ok) break;
      const Desc q_k = G::kmajor(smem_u32(smem + C::OFF_Q) + qb * G::BYTES);
      const Desc do_k = G::kmajor(smem_u32(smem + C::OFF_DO) + qb * G::BYTES);
      auto has_k = [&]() { return mbar_wait_warp(bar.k_full + ik.st, ik.ph, abort_flag); };
      auto has_v = [&]() { return mbar_wait_warp(bar.v_full + iv.st, iv.ph, abort_flag); };
      auto issue_s = [&](int j) {
        const int st = ik.st;
        // keys behind the sequence's last: masked in S, but dS = 0 must not meet a NaN in dS K
        if (s.len - j * kTile < kTile) zero_rows<D>(smem + C::OFF_K + st * G::BYTES, s.len - j * kTile, lane);
        tc_fence_after();
        const Desc k_k = G::kmajor(smem_u32(smem + C::OFF_K) + st * G::BYTES);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(tmem + is.st * 128, q_k.at(G::kstep(kk)), k_k.at(G::kstep(kk)), id_s, kk > 0);
          mma_commit(bar.s_full + is.st);
        }
        __syncwarp();
        ik.next();
        is.next();
      };
      auto issue_dp = [&]() {
        const int st = iv.st;
        tc_fence_after();
        const Desc v_k = G::kmajor(smem_u32(smem + C::OFF_V) + st * G::BYTES);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(tmem + C::COL_DP, do_k.at(G::kstep(kk)), v_k.at(G::kstep(kk)), id_s, kk > 0);
          mma_commit(bar.dp_full);
          mma_commit(bar.v_free + st);
        }
        __syncwarp();
        iv.next();
      };
      if (!(ok = has_k())) break;
      issue_s(0);
      if (!(ok = has_v())) break;
      issue_dp();
      if (n > 1) {
        if (!(ok = has_k())) break;
        issue_s(1);
      }
      for (int j = 0; ok && j < n; ++j) {
        if (kTilesAhead<D>) ok = (j + 1 >= n || has_v()) && (j + 2 >= n || has_k());
        ok = ok && mbar_wait_warp(bar.ds_full, ph, abort_flag);
        if (ok && j == 0 && ni >= C::OB) ok = mbar_wait_warp(bar.out_free + ob, rb.ph ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (j + 1 < n) {
          if (!kTilesAhead<D> && !(ok = has_v())) break;
          issue_dp();
        }
        const Desc k_mn = G::mnmajor(smem_u32(smem + C::OFF_K) + rk.st * G::BYTES);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_bf16_ts(tmem + C::COL_DQ + ob * D, tmem + rs.st * 128 + weight_col(kk), k_mn.at(G::mnstep(kk)),
                        id_o, j > 0 || kk > 0);
          mma_commit(bar.k_free + rk.st);
        }
        __syncwarp();
        rk.next();
        rs.next();
        ph ^= 1;
        if (j + 2 < n) {  // over dS, behind its product
          if (!kTilesAhead<D> && !(ok = has_k())) break;
          issue_s(j + 2);
        }
      }
      if (ok && elect_one()) {
        mma_commit(bar.q_free + qb);
        mma_commit(bar.out_full + ob);
      }
      rq.next();
      rb.next();
    }
    if (elect_one()) {  // every MMA has completed before TMEM is released
      mma_commit(bar.drain);
      mbar_wait_drain(bar.drain, 0);
    }
    __syncwarp();
  } else if (warp >= kBwdComputeWarps) {
    // ------------------------------------------------------ read-out of dQ
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    bool ok = true;
    int ni = 0;
    for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas), ++ni) {
      const int h = item % a.Hq, ob = ni % C::OB;
      const Slot s = walk.take(item, k);
      const float unscale = pow2(-ds_exponent<T>(a, s, h, lane));
      ok = warp_ok(mbar_wait_steps(bar.out_full + ob, (ni / C::OB) & 1, abort_flag, s.tile + 1));
      if (!ok) break;
      tc_fence_after();
      const int i = s.tile * kTile + row;
      row_out<T, D>(static_cast<T*>(const_cast<void*>(a.dq.p)) + (static_cast<long long>(s.start) + i) * a.dq.rs + h * a.dq.hs,
                    tmem + lane_base + C::COL_DQ + ob * D, i < s.len, a.scale * unscale);
      tc_fence_before();
      warp_arrive(bar.out_free + ob, lane);
    }
  } else {
    // ---------------------------------------------------------- P and dS
    const int w = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;  // w: which kCols keys
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + w * kCols;
    const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2);
    uint32_t before[kCols / 32];  // on the diagonal: the keys that the query sees
#pragma unroll
    for (int c = 0; c < kCols / 32; ++c) {
      const int last = row - w * kCols - c * 32;
      before[c] = last < 0 ? 0u : (last >= 31 ? 0xffffffffu : (2u << last) - 1u);
    }
    bool ok = true;
    Ring<2> rs;
    uint32_t ph = 0;
    for (int k = 0, item = cta; ok && item < a.n_items; item = zigzag(++k, cta, n_ctas)) {
      const int h = item % a.Hq;
      const Slot s = walk.take(item, k);
      const float* ld = a.ld + (static_cast<long long>(h) * a.n_tiles + s.base + s.tile) * 2 * kTile;
      const float neg_lse = ld[row], neg_delta = ld[kTile + row];
      const float up = pow2(ds_exponent<T>(a, s, h, lane) - kWeightBits<T>);  // dS up = P (dP up - delta up)
      const uint64_t l2 = f2_pack(neg_lse, neg_lse), d2 = f2_pack(neg_delta * up, neg_delta * up);
      for (int j = 0; ok && j <= s.tile; ++j) {
        const bool diag = j == s.tile;
        const uint32_t t_s = t_row + rs.st * 128;
        ok = mbar_wait(bar.s_full + rs.st, rs.ph, abort_flag);
        tc_fence_after();
        float p[kCols];
        tmem_ld_cols(t_s, p);
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {
          const float2 e = ex2_pair<T, kDqPoly<D>>(f2_fma(f2_pack(p[2 * i], p[2 * i + 1]), sc2, l2), i);
          p[2 * i] = e.x;
          p[2 * i + 1] = e.y;
        }
        ok = warp_ok(ok && mbar_wait(bar.dp_full, ph, abort_flag));
        tc_fence_after();
        float dp[kCols];
        tmem_ld_cols(t_row + C::COL_DP, dp);
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {
          const uint64_t t = f2_pack(dp[2 * i], dp[2 * i + 1]);
          const uint64_t diff = kScaleDs<T> ? f2_fma(t, f2_pack(up, up), d2) : f2_add(t, d2);
          const float2 v = f2_unpack(f2_mul(f2_pack(p[2 * i], p[2 * i + 1]), diff));
          dp[2 * i] = v.x;
          dp[2 * i + 1] = v.y;
        }
        if (diag) keep_bits(dp, before);  // a masked place is 0 whatever S and dP hold there
        uint32_t pk[kCols / 2];
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) pk[i] = Elem<T>::pack(dp[2 * i], dp[2 * i + 1]);
        tmem_st_weights(t_s, pk);
        tc_fence_before();
        warp_arrive(bar.ds_full, lane);
        rs.next();
        ph ^= 1;
      }
    }
  }
}

// Both parts: a CTA's share of the dK/dV items, then of the dQ items, which
// start as soon as it has none of the first kind left.  The parts share the
// tile buffers and TMEM; their barriers lie side by side.
template <typename T, int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
    pa_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo, const DkvArgs a,
                  const DqArgs b) {
  using C = BwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(smem + C::OFF_MISC + 4);
  const int warp = uniform(threadIdx.x >> 5);
  if (threadIdx.x == 0) {
    DkvBars<D>(smem).init();
    DqBars<D>(smem).init();
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kBwdComputeWarps + 5) tmem_alloc<512>(tmem_slot);
  pdl_wait();  // lse and delta of the kernel before
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  dkv_part<T, D>(smem, tmem, abort_flag, mq, mk, mv, mdo, a);
  tc_fence_before();
  const bool gave_up = __syncthreads_or(*(volatile int*)abort_flag);  // one answer for the block
  tc_fence_after();
  if (!gave_up) dq_part<T, D>(smem, tmem, abort_flag, mq, mk, mv, mdo, b);
  tc_fence_before();
  __syncthreads();
  if (warp == kBwdComputeWarps + 5) {
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

}  // namespace pa
