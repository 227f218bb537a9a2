// Plain kernels of packed causal attention: one warp per row, straight from
// the formulas of include/packed_attn.h.
#pragma once

#include "pa_device.cuh"

namespace pa {

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  return static_cast<float>(x);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
  return v;
}

// A lane holds elements lane + 32 u of a D-wide row.
template <typename T, int D>
__device__ __forceinline__ void row_in(float* r, const View& t, long long row, int h, int lane) {
  const T* p = static_cast<const T*>(t.p) + row * t.rs + h * t.hs;
#pragma unroll
  for (int u = 0; u < D / 32; ++u) r[u] = to_f(p[lane + 32 * u]);
}
template <typename T, int D>
__device__ __forceinline__ void row_out(const float* r, const View& t, long long row, int h, int lane, float f) {
  T* p = static_cast<T*>(const_cast<void*>(t.p)) + row * t.rs + h * t.hs;
#pragma unroll
  for (int u = 0; u < D / 32; ++u) p[lane + 32 * u] = static_cast<T>(r[u] * f);
}
template <int D>
__device__ __forceinline__ float row_dot(const float* a, const float* b) {
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < D / 32; ++u) s += a[u] * b[u];
  return warp_sum(s);
}

// delta_i = <dO_i, o_i>, [Hq][rows].
template <typename T, int D>
__global__ void simple_delta_kernel(View o, View dO, float* delta, long long rows) {
  const int h = blockIdx.y, lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (i >= rows) return;
  float a[D / 32], b[D / 32];
  row_in<T, D>(a, o, i, h, lane);
  row_in<T, D>(b, dO, i, h, lane);
  const float d = row_dot<D>(a, b);
  if (lane == 0) delta[h * rows + i] = d;
}

template <typename T, int D>
__global__ void simple_dq_kernel(const Slot* slots, View q, View k, View v, View dO, View dq, const float* lse,
                                 long long ls, const float* delta, long long rows, int G, float scale) {
  const Slot s = slots[blockIdx.x];
  const int h = blockIdx.y, lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < kTile; r += blockDim.x >> 5) {
    const int i = s.tile * kTile + r;
    if (i >= s.len) break;
    const long long row = (long long)s.start + i;
    float qr[D / 32], gr[D / 32], acc[D / 32] = {};
    row_in<T, D>(qr, q, row, h, lane);
    row_in<T, D>(gr, dO, row, h, lane);
    const float L = lse[h * ls + row], de = delta[h * rows + row];
    for (int j = 0; j <= i; ++j) {
      float kr[D / 32], vr[D / 32];
      row_in<T, D>(kr, k, (long long)s.start + j, h / G, lane);
      row_in<T, D>(vr, v, (long long)s.start + j, h / G, lane);
      const float p = __expf(row_dot<D>(qr, kr) * scale - L);
      const float ds = p * (row_dot<D>(gr, vr) - de);
#pragma unroll
      for (int u = 0; u < D / 32; ++u) acc[u] += ds * kr[u];
    }
    row_out<T, D>(acc, dq, row, h, lane, scale);
  }
}

// gridDim.y: K/V heads.
template <typename T, int D>
__global__ void simple_dkv_kernel(const Slot* slots, View q, View k, View v, View dO, View dk, View dv,
                                  const float* lse, long long ls, const float* delta, long long rows, int G,
                                  float scale) {
  const Slot s = slots[blockIdx.x];
  const int hk = blockIdx.y, lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < kTile; r += blockDim.x >> 5) {
    const int j = s.tile * kTile + r;
    if (j >= s.len) break;
    float kr[D / 32], vr[D / 32], ak[D / 32] = {}, av[D / 32] = {};
    row_in<T, D>(kr, k, (long long)s.start + j, hk, lane);
    row_in<T, D>(vr, v, (long long)s.start + j, hk, lane);
    for (int h = hk * G; h < hk * G + G; ++h)
      for (int i = j; i < s.len; ++i) {
        const long long row = (long long)s.start + i;
        float qr[D / 32], gr[D / 32];
        row_in<T, D>(qr, q, row, h, lane);
        row_in<T, D>(gr, dO, row, h, lane);
        const float p = __expf(row_dot<D>(qr, kr) * scale - lse[h * ls + row]);
        const float ds = p * (row_dot<D>(gr, vr) - delta[h * rows + row]);
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
          ak[u] += ds * qr[u];
          av[u] += p * gr[u];
        }
      }
    row_out<T, D>(ak, dk, (long long)s.start + j, hk, lane, scale);
    row_out<T, D>(av, dv, (long long)s.start + j, hk, lane, 1.f);
  }
}

}  // namespace pa
