// Device helpers shared by the packed attention kernels: element types,
// operand descriptors of 128-row tiles, the diagonal mask.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pa_internal.h"
#include "sa_device.cuh"

namespace pa {

using namespace sa;  // mbarrier, TMA, tcgen05 and fp32-pair helpers

// Rows of a tensor: first element, distance of rows and heads in elements.
struct View {
  const void* p;
  long long rs, hs;
};

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1;  // instruction descriptor: bf16
  static constexpr float kBias = 0.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16(lo, hi); }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  }
};
template <>
struct Elem<__half> {
  static constexpr uint32_t kFormat = 0;  // f16
  // The forward's P is at most 2^8 (its running maximum trails by up to 8 in
  // the exponent); 2^7 on top keeps it below fp16's 2^16 and moves the
  // subnormals, which lose relative precision, from 2^-14 down to 2^-21 of
  // the row's largest weight.  The factor cancels in o = sum P v / sum P.
  static constexpr float kBias = 7.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
};

// Instruction descriptor, kind::f16, float32 accumulator (make_idesc_bf16 with the element type).
template <typename T>
__host__ __device__ constexpr uint32_t make_idesc(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (Elem<T>::kFormat << 7) | (Elem<T>::kFormat << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// A shared-memory matrix descriptor (fields as make_desc) as two words: a
// k-step is one 32-bit addition to the low word.  One thread issues every MMA
// of a CTA, and what it spends between two of them is time the tensor core
// waits, so the descriptors are built once per operand and not per MMA.
struct Desc {
  uint32_t lo, hi;
  __device__ __forceinline__ Desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint64_t swz)
      : lo(((saddr >> 4) & 0x3FFF) | ((lbo >> 4) << 16)),
        hi((sbo >> 4) | (1u << 14) | (static_cast<uint32_t>(swz) << 29)) {}
  __device__ __forceinline__ uint64_t at(uint32_t bytes) const {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo + (bytes >> 4)), "r"(hi));
    return d;
  }
};

// One thread of the (converged) warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// mbar_wait by a whole warp, with one answer for all lanes that the compiler
// knows to be one: what follows it stays in uniform registers, which the
// MMA instructions take their operands from.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  uint32_t spins = 0;
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_wait_hint(bar, parity, 20000u))) return true;
    if (((++spins) & 15u) == 0) {
      bool stop = *(volatile int*)abort || *(volatile int*)&g_status == kStatusTimeout;
      if (!stop && clock64() - t0 > kWaitCycles) {
        atomicExch(&g_status, kStatusTimeout);
        stop = true;
      }
      if (__any_sync(0xffffffffu, stop)) {
        *(volatile int*)abort = 1;
        return false;
      }
    }
  }
}

// One answer for a warp whose lanes waited each for itself (they may part ways
// where a wait runs out): what follows, collective instructions and the roles'
// loops, is for the whole warp.
__device__ __forceinline__ bool warp_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

#ifdef SA_TEST_HOOKS
// Test build: whether a producer withholds load number n (its first one) of
// kind `what` in the CTA that takes a part's first item, so that a wait runs out.
enum Withhold : int { kHoldQ = 1, kHoldV = 2, kHoldDkvDO = 3, kHoldDkvK = 4, kHoldDqV = 5, kHoldDqQ = 6 };
__device__ __forceinline__ bool withheld(int what, int n, int cta) {
  return n == 0 && cta == 0 && *(volatile int*)&g_test_withhold == what;
}
#define PA_WITHHELD(what, n) withheld(what, n, cta)
#else
#define PA_WITHHELD(what, n) false
#endif

// mbar_wait for something that takes `steps` steps of a kernel's inner loop:
// an item of a very long sequence may run for more than mbar_wait's second.
__device__ __forceinline__ bool mbar_wait_steps(uint64_t* bar, uint32_t parity, int* abort, int steps) {
  const long long t0 = clock64(), limit = kWaitCycles * (1 + steps / 16384);
  uint32_t spins = 0;
  while (!mbar_try_wait_hint(bar, parity, 20000u)) {
    if (((++spins) & 15u) == 0) {
      if (*(volatile int*)abort || *(volatile int*)&g_status == kStatusTimeout) {
        *(volatile int*)abort = 1;
        return false;
      }
      if (clock64() - t0 > limit) {
        atomicExch(&g_status, kStatusTimeout);
        *(volatile int*)abort = 1;
        return false;
      }
    }
  }
  return true;
}

__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ Slot uniform(const Slot& s) {
  return Slot{uniform(s.start), uniform(s.len), uniform(s.tile), uniform(s.base)};
}

// One arrival for a warp, behind what every lane did before it (an arrival of
// every lane would be 32 updates of one word in shared memory, one by one).
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// A tile of 128 rows of D elements in shared memory: panels of up to 64
// columns, a row of a panel 128 (D = 32: 64) bytes, swizzled over its width.
template <int D>
struct TileGeo {
  static constexpr int ROWB = D >= 64 ? 128 : 64;
  static constexpr int PANELS = D >= 64 ? D / 64 : 1;
  static constexpr int BOXW = D >= 64 ? 64 : D;
  static constexpr uint64_t SWZ = D >= 64 ? kSwizzle128 : kSwizzle64;
  static constexpr int PANEL_BYTES = kTile * ROWB;
  static constexpr int BYTES = kTile * D * 2;
  // Operands of a tile at shared address `base`: the rows as M or N with the
  // D columns as K, and the D columns as N with the rows as K.
  static __device__ __forceinline__ Desc kmajor(uint32_t base) { return Desc(base, 16, 8 * ROWB, SWZ); }
  static __device__ __forceinline__ Desc mnmajor(uint32_t base) { return Desc(base, PANEL_BYTES, 8 * ROWB, SWZ); }
  // byte offset of k-step kk (16 columns, 16 rows)
  static __device__ constexpr uint32_t kstep(int kk) { return (kk / (ROWB / 32)) * PANEL_BYTES + (kk % (ROWB / 32)) * 32; }
  static __device__ constexpr uint32_t mnstep(int kk) { return kk * 16 * ROWB; }
};

// The 128 rows from `row` of head h (rows past the tensor's end read as zero).
template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int h, int row) {
  using G = TileGeo<D>;
#pragma unroll
  for (int p = 0; p < G::PANELS; ++p) tma_load_3d(dst + p * G::PANEL_BYTES, m, bar, p * 64, h, row);
}

// Zeroes rows [r0, 128) of a tile, by a whole warp: rows that a TMA box took
// from the next sequence must not meet a weight of zero (0 * NaN).
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int lane) {
  using G = TileGeo<D>;
#pragma unroll
  for (int p = 0; p < G::PANELS; ++p)
    for (int i = r0 * G::ROWB + lane * 16; i < kTile * G::ROWB; i += 32 * 16)
      *reinterpret_cast<uint4*>(tile + p * G::PANEL_BYTES + i) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// 32 lanes x 32 bit, 32 consecutive columns: thread t gets lane (base + t).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 2^x of a pair on the FMA pipe: x = n + f with n the nearest integer, |f| <=
// 1/2, and 2^f by the polynomial of least relative error (Remez) of degree 3
// for bf16 weights (7.5e-5, next to their rounding of 2^-8) and 4 for fp16
// (2.6e-6, next to 2^-11).  n + 127 sits in the low bits of x + 1.5 2^23 + 127,
// which shifted up are the float 2^n; at n = -127 they are 0, so everything
// below 2^-126.5, and a masked -inf, gives exactly 0.  NaN stays NaN.
template <typename T>
__device__ __forceinline__ float2 ex2_fma(uint64_t x2) {
  constexpr float kMagic = 12582912.f + 127.f;
  const float2 xi = f2_unpack(x2);
  float2 x;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(x.x) : "f"(xi.x), "f"(-127.f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(x.y) : "f"(xi.y), "f"(-127.f));
  const uint64_t xp = f2_pack(x.x, x.y);
  const uint64_t t = f2_add(xp, f2_pack(kMagic, kMagic));
  const uint64_t r = f2_add(t, f2_pack(-kMagic, -kMagic));
  const uint64_t f = f2_fma(r, f2_pack(-1.f, -1.f), xp);
  auto c = [](float v) { return f2_pack(v, v); };
  uint64_t p;
  if constexpr (std::is_same<T, __half>::value) {
    p = f2_fma(f, c(0.009570102207362652f), c(0.05591785907745361f));
    p = f2_fma(p, f, c(0.240247443318367f));
    p = f2_fma(p, f, c(0.6931217908859253f));
    p = f2_fma(p, f, c(0.9999992847442627f));
  } else {
    p = f2_fma(f, c(0.0551716685295105f), c(0.2426111251115799f));
    p = f2_fma(p, f, c(0.6932609677314758f));
    p = f2_fma(p, f, c(0.9999280571937561f));
  }
  const float2 tf = f2_unpack(t);
  const float s0 = __uint_as_float(__float_as_uint(tf.x) << 23), s1 = __uint_as_float(__float_as_uint(tf.y) << 23);
  return f2_unpack(f2_mul(p, f2_pack(s0, s1)));
}

// 2^x of pair i of a row's run of pairs: POLY of every 8 pairs on the FMA
// pipe, the others by ex2 (16 a clock and SM).
template <typename T, int POLY>
__device__ __forceinline__ float2 ex2_pair(uint64_t x2, int i) {
  constexpr uint32_t kPick = POLY == 0 ? 0u : (POLY == 1 ? 0x10u : (POLY == 2 ? 0x44u : (POLY == 3 ? 0x92u : 0xaau)));
  if ((kPick >> (i & 7)) & 1u) return ex2_fma<T>(x2);
  const float2 x = f2_unpack(x2);
  return make_float2(ex2(x.x), ex2(x.y));
}

// Keeps v[i] for i <= last (i in [0, 32)), sets the others to `fill`.
__device__ __forceinline__ void mask_after32(float* v, int last, float fill) {
  const uint32_t m = last < 0 ? 0u : (last >= 31 ? 0xffffffffu : ((2u << last) - 1u));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = ((m >> i) & 1u) ? v[i] : fill;
}

// Item k of a CTA's share: rounds alternate direction, so that long and short
// items pair up (the slots are sorted longest first).
__device__ __forceinline__ int zigzag(int k, int cta, int n_ctas) {
  return k * n_ctas + ((k & 1) ? (n_ctas - 1 - cta) : cta);
}

// Position in a ring of N stages: the stage and its phase's parity.
template <int N>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) st = 0, ph ^= 1;
  }
};

// The slots of a CTA's items in order, the next one requested into L1 while
// this one is worked on: a slot comes from global memory, and every role would
// wait for it at every item.  (Held in registers one item ahead it cost the
// forward spills: 2 x 12288 rows, 8 heads of 64, 404 -> 474 us.)
struct SlotWalk {
  const Slot* slots;
  int n_items, per, cta;  // items, items a slot, this CTA's number
  __device__ __forceinline__ SlotWalk(const Slot* p, int items, int per_slot) : SlotWalk(p, items, per_slot, blockIdx.x) {}
  __device__ __forceinline__ SlotWalk(const Slot* p, int items, int per_slot, int cta_)
      : slots(p), n_items(items), per(per_slot), cta(cta_) {}
  // the slot of item k of the share, item number `item`
  __device__ __forceinline__ Slot take(int item, int k) const {
    const int4 v = __ldg(reinterpret_cast<const int4*>(slots + item / per));
    const int next = zigzag(k + 1, cta, gridDim.x);
    if (next < n_items) asm volatile("prefetch.global.L1 [%0];" ::"l"(slots + next / per));
    return Slot{v.x, v.y, v.z, v.w};
  }
};

}  // namespace pa
