// Layer norm forward and backward and the clipping of gradients by their
// global norm as calls of their own (include/sparse_block.h).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <type_traits>
#include <vector>

#include "sparse_block.h"

namespace sbt {

constexpr int kMaxC = 16384;

// ------------------------------------------------------------------ types
template <typename T>
__device__ __forceinline__ float to_f(T v) {
  return static_cast<float>(v);
}

// VEC consecutive elements as one word: 16 bytes, or one element.
template <typename T, int VEC>
struct Word {
  using type = uint4;
};
template <typename T>
struct Word<T, 1> {
  using type = T;
};

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const typename Word<T, VEC>::type& w, float* f) {
  const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
  for (int u = 0; u < VEC; ++u) f[u] = to_f(e[u]);
}
template <typename T, int VEC>
__device__ __forceinline__ typename Word<T, VEC>::type pack(const float* f) {
  typename Word<T, VEC>::type w;
  T* e = reinterpret_cast<T*>(&w);
#pragma unroll
  for (int u = 0; u < VEC; ++u) e[u] = static_cast<T>(f[u]);
  return w;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
  return v;
}

// Sum over the threads of a row: a warp, or the block (slots: 2 x 32 floats
// used in turn, so that one barrier a sum is enough).
template <bool WARP, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* slots, int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
  if constexpr (!WARP) {
    float* s = slots + turn * 32 * N;
    turn ^= 1;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) s[k * 32 + w] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum(lane < nw ? s[k * 32 + lane] : 0.f);
  }
}

// A row is cut into words of VEC elements; thread i of the row's n threads
// (a warp's 32, or the block's) holds words i, i + n, ..., NV of them at most.
template <typename T, int VEC, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512)
    norm_fwd_kernel(const T* x, long long ldx, const float* __restrict__ g, const float* __restrict__ b, T* y,
                    long long ldy, float* mean_out, float* rstd_out, long long M, int C, float eps) {
  using W = typename Word<T, VEC>::type;
  __shared__ float slots[64];
  int turn = 0;
  const int i0 = WARP ? (threadIdx.x & 31) : threadIdx.x, n = WARP ? 32 : blockDim.x;
  const int words = C / VEC;
  const long long r0 = WARP ? ((static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5) : blockIdx.x;
  const long long step = WARP ? ((static_cast<long long>(gridDim.x) * blockDim.x) >> 5) : gridDim.x;
  float gv[NV * VEC], bv[NV * VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int u = 0; u < VEC; ++u) {
      const int w = i0 + j * n;
      gv[j * VEC + u] = w < words ? g[w * VEC + u] : 0.f;
      bv[j * VEC + u] = (b && w < words) ? b[w * VEC + u] : 0.f;
    }
  W cur[NV], nxt[NV];
  auto load = [&](W* raw, long long r) {
    const W* p = reinterpret_cast<const W*>(x + r * ldx);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (i0 + j * n < words) raw[j] = p[i0 + j * n];
  };
  if (r0 < M) load(cur, r0);
  const float inv = 1.f / C;
  for (long long r = r0; r < M; r += step) {
    if (r + step < M) load(nxt, r + step);
    float f[NV * VEC], s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (i0 + j * n < words) unpack<T, VEC>(cur[j], f + j * VEC);
      else
#pragma unroll
        for (int u = 0; u < VEC; ++u) f[j * VEC + u] = 0.f;
#pragma unroll
      for (int u = 0; u < VEC; ++u) s[0] += f[j * VEC + u];
    }
    row_sums<WARP>(s, slots, turn);
    const float mean = s[0] * inv;
    float q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (i0 + j * n < words)
#pragma unroll
        for (int u = 0; u < VEC; ++u) {
          f[j * VEC + u] -= mean;
          q[0] += f[j * VEC + u] * f[j * VEC + u];
        }
    row_sums<WARP>(q, slots, turn);
    const float rstd = 1.f / sqrtf(q[0] * inv + eps);
    if (i0 == 0) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
    W* p = reinterpret_cast<W*>(y + r * ldy);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (i0 + j * n < words) {
        float o[VEC];
#pragma unroll
        for (int u = 0; u < VEC; ++u) o[u] = f[j * VEC + u] * rstd * gv[j * VEC + u] + bv[j * VEC + u];
        p[i0 + j * n] = pack<T, VEC>(o);
      }
#pragma unroll
    for (int j = 0; j < NV; ++j) cur[j] = nxt[j];
  }
}

// Rows too wide for the registers of a block: read again for each pass.
template <typename T>
__global__ void __launch_bounds__(512)
    norm_fwd_wide_kernel(const T* x, long long ldx, const float* g, const float* b, T* y, long long ldy,
                         float* mean_out, float* rstd_out, long long M, int C, float eps) {
  __shared__ float slots[64];
  int turn = 0;
  const float inv = 1.f / C;
  for (long long r = blockIdx.x; r < M; r += gridDim.x) {
    const T* p = x + r * ldx;
    float s[1] = {0.f}, q[1] = {0.f};
    for (int i = threadIdx.x; i < C; i += blockDim.x) s[0] += to_f(p[i]);
    row_sums<false>(s, slots, turn);
    const float mean = s[0] * inv;
    for (int i = threadIdx.x; i < C; i += blockDim.x) q[0] += (to_f(p[i]) - mean) * (to_f(p[i]) - mean);
    row_sums<false>(q, slots, turn);
    const float rstd = 1.f / sqrtf(q[0] * inv + eps);
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
    for (int i = threadIdx.x; i < C; i += blockDim.x)
      y[r * ldy + i] = static_cast<T>((to_f(p[i]) - mean) * rstd * g[i] + (b ? b[i] : 0.f));
  }
}

// dx per row, and this block's sums of dy xh and dy per channel into
// part[blockIdx.x][2][C].
template <typename T, int VEC, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512)
    norm_bwd_kernel(const T* x, long long ldx, const float* __restrict__ g, const T* dy, long long lddy,
                    const float* __restrict__ mean_in, const float* __restrict__ rstd_in, T* dx, long long lddx,
                    float* part, long long M, int C) {
  using W = typename Word<T, VEC>::type;
  extern __shared__ float sums[];  // WARP: [8 warps][2][C], else none
  __shared__ float slots[128];
  int turn = 0;
  const int i0 = WARP ? (threadIdx.x & 31) : threadIdx.x, n = WARP ? 32 : blockDim.x;
  const int words = C / VEC;
  const long long r0 = WARP ? ((static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5) : blockIdx.x;
  const long long step = WARP ? ((static_cast<long long>(gridDim.x) * blockDim.x) >> 5) : gridDim.x;
  float gv[NV * VEC], sg[NV * VEC] = {}, sb[NV * VEC] = {};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int u = 0; u < VEC; ++u) gv[j * VEC + u] = i0 + j * n < words ? g[(i0 + j * n) * VEC + u] : 0.f;
  W xc[NV], dc[NV], xn[NV], dn[NV];
  float mc = 0.f, rc = 0.f, mn = 0.f, rn = 0.f;
  auto load = [&](W* xr, W* dr, float& m, float& rs, long long r) {
    const W* px = reinterpret_cast<const W*>(x + r * ldx);
    const W* pd = reinterpret_cast<const W*>(dy + r * lddy);
    m = mean_in[r];
    rs = rstd_in[r];
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (i0 + j * n < words) {
        xr[j] = px[i0 + j * n];
        dr[j] = pd[i0 + j * n];
      }
  };
  if (r0 < M) load(xc, dc, mc, rc, r0);
  const float inv = 1.f / C;
  for (long long r = r0; r < M; r += step) {
    if (r + step < M) load(xn, dn, mn, rn, r + step);
    float xh[NV * VEC], t[NV * VEC], s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (i0 + j * n < words) {
        float d[VEC];
        unpack<T, VEC>(xc[j], xh + j * VEC);
        unpack<T, VEC>(dc[j], d);
#pragma unroll
        for (int u = 0; u < VEC; ++u) {
          const int k = j * VEC + u;
          xh[k] = (xh[k] - mc) * rc;
          t[k] = d[u] * gv[k];
          s[0] += t[k];
          s[1] += t[k] * xh[k];
          sg[k] += d[u] * xh[k];
          sb[k] += d[u];
        }
      }
    row_sums<WARP>(s, slots, turn);
    s[0] *= inv;
    s[1] *= inv;
    W* p = reinterpret_cast<W*>(dx + r * lddx);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (i0 + j * n < words) {
        float o[VEC];
#pragma unroll
        for (int u = 0; u < VEC; ++u) o[u] = rc * (t[j * VEC + u] - s[0] - xh[j * VEC + u] * s[1]);
        p[i0 + j * n] = pack<T, VEC>(o);
      }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xc[j] = xn[j];
      dc[j] = dn[j];
    }
    mc = mn;
    rc = rn;
  }
  float* out = part + static_cast<long long>(blockIdx.x) * 2 * C;
  if constexpr (WARP) {
    float* mine = sums + (threadIdx.x >> 5) * 2 * C;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (i0 + j * n < words)
#pragma unroll
        for (int u = 0; u < VEC; ++u) {
          mine[(i0 + j * n) * VEC + u] = sg[j * VEC + u];
          mine[C + (i0 + j * n) * VEC + u] = sb[j * VEC + u];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * C; i += blockDim.x) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) a += sums[w * 2 * C + i];
      out[i] = a;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (i0 + j * n < words)
#pragma unroll
        for (int u = 0; u < VEC; ++u) {
          out[(i0 + j * n) * VEC + u] = sg[j * VEC + u];
          out[C + (i0 + j * n) * VEC + u] = sb[j * VEC + u];
        }
  }
}

template <typename T>
__global__ void __launch_bounds__(512)
    norm_bwd_wide_kernel(const T* x, long long ldx, const float* g, const T* dy, long long lddy, const float* mean_in,
                         const float* rstd_in, T* dx, long long lddx, float* part, long long M, int C) {
  extern __shared__ float sums[];  // [2][C]; a channel belongs to one thread
  __shared__ float slots[128];
  int turn = 0;
  for (int i = threadIdx.x; i < C; i += blockDim.x) sums[i] = sums[C + i] = 0.f;
  const float inv = 1.f / C;
  for (long long r = blockIdx.x; r < M; r += gridDim.x) {
    const T *px = x + r * ldx, *pd = dy + r * lddy;
    const float m = mean_in[r], rs = rstd_in[r];
    float s[2] = {0.f, 0.f};
    for (int i = threadIdx.x; i < C; i += blockDim.x) {
      const float xh = (to_f(px[i]) - m) * rs, d = to_f(pd[i]);
      s[0] += d * g[i];
      s[1] += d * g[i] * xh;
      sums[i] += d * xh;
      sums[C + i] += d;
    }
    row_sums<false>(s, slots, turn);
    for (int i = threadIdx.x; i < C; i += blockDim.x) {
      const float xh = (to_f(px[i]) - m) * rs, t = to_f(pd[i]) * g[i];
      dx[r * lddx + i] = static_cast<T>(rs * (t - s[0] * inv - xh * (s[1] * inv)));
    }
  }
  for (int i = threadIdx.x; i < C; i += blockDim.x) {
    part[static_cast<long long>(blockIdx.x) * 2 * C + i] = sums[i];
    part[static_cast<long long>(blockIdx.x) * 2 * C + C + i] = sums[C + i];
  }
}

// dg, db: the blocks' partial sums added in order.  32 columns a block, 32
// groups of rows of the partials.
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float* part, int P, int C, float* dg, float* db) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (i < 2 * C)
    for (int p = grp; p < P; p += 32) a += part[static_cast<long long>(p) * 2 * C + i];
  s[grp][lane] = a;
  __syncthreads();
  if (grp == 0 && i < 2 * C) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += s[k][lane];
    if (i < C) dg[i] = t;
    else if (db) db[i - C] = t;
  }
}

// --------------------------------------------------------------- clipping
constexpr int kTensors = 120;   // tensors a launch (their table is a kernel argument)
constexpr int kChunk = 16384;   // elements a block takes at a time
constexpr int kClipBlocks = 592;

struct ClipTensor {
  const void* g;
  void* out;
  unsigned long long n;
  int dtype;
  int pad;
};
struct ClipTable {
  ClipTensor t[kTensors];
  unsigned first[kTensors + 1];  // first chunk of each tensor
  int n;
};

template <typename T>
__device__ double sum_squares(const T* p, unsigned long long n) {
  double s = 0.;
  for (unsigned long long i = threadIdx.x; i < n; i += blockDim.x) {
    const double v = to_f(p[i]);
    s += v * v;
  }
  return s;
}
template <typename T>
__device__ void scale_to(const T* p, T* o, unsigned long long n, float c) {
  for (unsigned long long i = threadIdx.x; i < n; i += blockDim.x) o[i] = static_cast<T>(to_f(p[i]) * c);
}

__device__ __forceinline__ int tensor_of(const ClipTable& t, unsigned chunk) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ double block_sum(double v) {
  __shared__ double s[32];
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < (blockDim.x >> 5) ? s[threadIdx.x & 31] : 0.;
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
  return v;
}

__global__ void __launch_bounds__(512) clip_norm_kernel(const __grid_constant__ ClipTable t, double* part, int add) {
  double s = 0.;
  for (unsigned c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const unsigned long long at = static_cast<unsigned long long>(c - t.first[i]) * kChunk;
    const unsigned long long n = min(static_cast<unsigned long long>(kChunk), t.t[i].n - at);
    if (t.t[i].dtype == SB_BF16) s += sum_squares(static_cast<const __nv_bfloat16*>(t.t[i].g) + at, n);
    else if (t.t[i].dtype == SB_FP16) s += sum_squares(static_cast<const __half*>(t.t[i].g) + at, n);
    else s += sum_squares(static_cast<const float*>(t.t[i].g) + at, n);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = (add ? part[blockIdx.x] : 0.) + s;
}

__global__ void __launch_bounds__(512)
    clip_scale_kernel(const __grid_constant__ ClipTable t, const double* part, double max_norm, float* norm) {
  double s = 0.;
  for (int i = threadIdx.x; i < kClipBlocks; i += blockDim.x) s += part[i];
  const double total = sqrt(block_sum(s));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  if (t.n == 0) return;
  double cd = max_norm / (total + 1e-6);
  if (cd > 1.) cd = 1.;
  const float c = static_cast<float>(cd);
  for (unsigned k = blockIdx.x; k < t.first[t.n]; k += gridDim.x) {
    const int i = tensor_of(t, k);
    const unsigned long long at = static_cast<unsigned long long>(k - t.first[i]) * kChunk;
    const unsigned long long n = min(static_cast<unsigned long long>(kChunk), t.t[i].n - at);
    if (t.t[i].g == t.t[i].out && c == 1.f) continue;
    if (t.t[i].dtype == SB_BF16)
      scale_to(static_cast<const __nv_bfloat16*>(t.t[i].g) + at, static_cast<__nv_bfloat16*>(t.t[i].out) + at, n, c);
    else if (t.t[i].dtype == SB_FP16)
      scale_to(static_cast<const __half*>(t.t[i].g) + at, static_cast<__half*>(t.t[i].out) + at, n, c);
    else scale_to(static_cast<const float*>(t.t[i].g) + at, static_cast<float*>(t.t[i].out) + at, n, c);
  }
}

// ------------------------------------------------------------------ host
int launched() { return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA; }

int sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n;
}

template <typename F>
int by_type(int dtype, F&& f) {
  if (dtype == SB_BF16) return f(__nv_bfloat16{});
  if (dtype == SB_FP16) return f(__half{});
  return f(float{});
}

int esize(int dtype) { return dtype == SB_FP32 ? 4 : 2; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool rows16(const void* p, int64_t ld, int es) { return aligned(p, 16) && (ld * es) % 16 == 0; }

constexpr int kParts = 592;  // blocks of a backward launch, at most

template <typename K>
int resident(K kernel, int threads, size_t smem) {
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem) != cudaSuccess || per < 1) return 1;
  return per;
}

}  // namespace sbt

using namespace sbt;

extern "C" {

int sparse_block_layer_norm_fwd(const void* x, int64_t ldx, const float* g, const float* b, void* y, int64_t ldy,
                                float* mean, float* rstd, int64_t M, int C, float eps, int dtype, void* stream) {
  if (!x || !g || !y || M < 0 || C < 1 || ldx < C || ldy < C || dtype < SB_BF16 || dtype > SB_FP32 || !(eps >= 0.f) ||
      !std::isfinite(eps) || (x == y && ldx != ldy))
    return SA_ERR_INVALID_ARG;
  const int es = esize(dtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(g, 4) || !aligned(b, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return SA_ERR_INVALID_ARG;
  if (C > kMaxC) return SA_ERR_UNSUPPORTED;
  if (M == 0) return SA_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = rows16(x, ldx, es) && rows16(y, ldy, es) && (C * es) % 16 == 0;
  const int n_sm = sms();
  return by_type(dtype, [&](auto t) -> int {
    using T = decltype(t);
    const T* xp = static_cast<const T*>(x);
    T* yp = static_cast<T*>(y);
    auto go = [&](auto kernel, int threads, int rows_per_block) -> int {
      const long long blocks = (M + rows_per_block - 1) / rows_per_block;
      const int grid = static_cast<int>(std::min<long long>(blocks, static_cast<long long>(n_sm) * resident(kernel, threads, 0)));
      kernel<<<grid, threads, 0, s>>>(xp, ldx, g, b, yp, ldy, mean, rstd, M, C, eps);
      return launched();
    };
    auto pick = [&](auto v) -> int {
      constexpr int V = v.value;
      const int words = C / V;
      if (words <= 32) return go(norm_fwd_kernel<T, V, 1, true>, 256, 8);
      if (words <= 64) return go(norm_fwd_kernel<T, V, 2, true>, 256, 8);
      if (words <= 128) return go(norm_fwd_kernel<T, V, 4, true>, 256, 8);
      auto threads = [&](int nv) { return std::min(512, (words + 32 * nv - 1) / (32 * nv) * 32); };
      if (words <= 1024) return go(norm_fwd_kernel<T, V, 2, false>, threads(2), 1);
      if (words <= 2048) return go(norm_fwd_kernel<T, V, 4, false>, threads(4), 1);
      if constexpr (V == 1) {
        if (words <= 6144) return go(norm_fwd_kernel<T, V, 12, false>, threads(12), 1);
      }
      return go(norm_fwd_wide_kernel<T>, 512, 1);
    };
    if (vec) return pick(std::integral_constant<int, 16 / sizeof(T)>{});
    return pick(std::integral_constant<int, 1>{});
  });
}

size_t sparse_block_layer_norm_bwd_workspace_size(int64_t M, int C) {
  if (M < 0 || C < 1 || C > kMaxC) return 0;
  return static_cast<size_t>(std::max<int64_t>(1, std::min<int64_t>(M, kParts))) * 2 * C * sizeof(float);
}

int sparse_block_layer_norm_bwd(const void* x, int64_t ldx, const float* g, const void* dy, int64_t lddy,
                                const float* mean, const float* rstd, void* dx, int64_t lddx, float* dg, float* db,
                                int64_t M, int C, int dtype, void* ws, size_t ws_bytes, void* stream) {
  if (!x || !g || !dy || !mean || !rstd || !dx || !dg || M < 0 || C < 1 || ldx < C || lddy < C || lddx < C ||
      dtype < SB_BF16 || dtype > SB_FP32 || (dx == x && lddx != ldx) || (dx == dy && lddx != lddy) || dg == db)
    return SA_ERR_INVALID_ARG;
  const int es = esize(dtype);
  if (!aligned(x, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(g, 4) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(dg, 4) || !aligned(db, 4))
    return SA_ERR_INVALID_ARG;
  if (C > kMaxC) return SA_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256) || ws_bytes < sparse_block_layer_norm_bwd_workspace_size(M, C)) return SA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(ws);
  const int n_sm = sms();
  int P = 0;
  const bool vec = rows16(x, ldx, es) && rows16(dy, lddy, es) && rows16(dx, lddx, es) && (C * es) % 16 == 0;
  if (M > 0) {
    const int st = by_type(dtype, [&](auto t) -> int {
      using T = decltype(t);
      auto go = [&](auto kernel, int threads, int rows_per_block, size_t smem) -> int {
        if (smem > 48 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(smem)) != cudaSuccess)
          return SA_ERR_CUDA;
        const long long blocks = (M + rows_per_block - 1) / rows_per_block;
        P = static_cast<int>(std::min<long long>(
            std::min<long long>(blocks, kParts), static_cast<long long>(n_sm) * resident(kernel, threads, smem)));
        kernel<<<P, threads, smem, s>>>(static_cast<const T*>(x), ldx, g, static_cast<const T*>(dy), lddy, mean, rstd,
                                        static_cast<T*>(dx), lddx, part, M, C);
        return launched();
      };
      auto pick = [&](auto v) -> int {
        constexpr int V = v.value;
        const int words = C / V;
        const size_t sums = 8 * 2 * static_cast<size_t>(C) * sizeof(float);
        if (words <= 32) return go(norm_bwd_kernel<T, V, 1, true>, 256, 8, sums);
        if (words <= 64) return go(norm_bwd_kernel<T, V, 2, true>, 256, 8, sums);
        auto threads = [&](int nv) { return std::min(512, (words + 32 * nv - 1) / (32 * nv) * 32); };
        if (words <= 1024) return go(norm_bwd_kernel<T, V, 2, false>, threads(2), 1, 0);
        if constexpr (V <= 4) {
          if (words <= 2048) return go(norm_bwd_kernel<T, V, 4, false>, threads(4), 1, 0);
        }
        if constexpr (V == 1) {
          if (words <= 6144) return go(norm_bwd_kernel<T, V, 12, false>, threads(12), 1, 0);
        }
        return go(norm_bwd_wide_kernel<T>, 512, 1, 2 * static_cast<size_t>(C) * sizeof(float));
      };
      if (vec) return pick(std::integral_constant<int, 16 / sizeof(T)>{});
      return pick(std::integral_constant<int, 1>{});
    });
    if (st) return st;
  }
  norm_bwd_sum_kernel<<<(2 * C + 31) / 32, 1024, 0, s>>>(part, P, C, dg, db);
  return launched();
}

size_t sparse_block_clip_workspace_size(void) { return kClipBlocks * sizeof(double); }

int sparse_block_clip_grads(int n, const void* const* grads, void* const* outs, const size_t* numel,
                            const int* dtypes, double max_norm, float* norm, void* ws, size_t ws_bytes, void* stream) {
  if (n < 0 || !norm || (n > 0 && (!grads || !numel || !dtypes)) || !(max_norm >= 0.) || !aligned(norm, 4))
    return SA_ERR_INVALID_ARG;
  struct Range {
    uintptr_t a, b;
    int i;
    bool out;
  };
  std::vector<ClipTensor> ts;
  std::vector<Range> rs;
  try {
    for (int i = 0; i < n; ++i) {
      if (dtypes[i] < SB_BF16 || dtypes[i] > SB_FP32) return SA_ERR_INVALID_ARG;
      if (numel[i] == 0) continue;
      if (numel[i] > (size_t(1) << 40)) return SA_ERR_INVALID_ARG;
      const size_t es = esize(dtypes[i]);
      void* o = outs ? outs[i] : nullptr;
      if (!grads[i] || !aligned(grads[i], es) || (outs && (!o || !aligned(o, es)))) return SA_ERR_INVALID_ARG;
      ts.push_back(ClipTensor{grads[i], o, numel[i], dtypes[i], 0});
      if (outs) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i]), b = reinterpret_cast<uintptr_t>(o);
        rs.push_back(Range{b, b + numel[i] * es, i, true});
        if (a != b) rs.push_back(Range{a, a + numel[i] * es, i, false});
      }
    }
    // an output overlaps nothing else: in address order, no range may begin inside an earlier one when either is an output
    std::sort(rs.begin(), rs.end(), [](const Range& p, const Range& q) { return p.a < q.a; });
    uintptr_t end_any = 0, end_out = 0;
    for (const Range& r : rs) {
      if (r.a < end_out || (r.out && r.a < end_any)) return SA_ERR_INVALID_ARG;
      end_any = std::max(end_any, r.b);
      if (r.out) end_out = std::max(end_out, r.b);
    }
  } catch (...) {
    return SA_ERR_INVALID_ARG;
  }
  if (!ws || !aligned(ws, 256) || ws_bytes < sparse_block_clip_workspace_size()) return SA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  ClipTable t;
  // `norm` pass over the tensors, then the scaling pass; kTensors of them a launch
  for (int pass = 0; pass < 2; ++pass) {
    size_t at = 0;
    bool first = true;
    do {
      t.n = 0;
      t.first[0] = 0;
      if (pass == 0 || outs)
        while (at < ts.size() && t.n < kTensors) {
          const size_t chunks = (ts[at].n + kChunk - 1) / kChunk;
          if (t.first[t.n] + chunks > 0x7fffffffu) break;
          t.t[t.n] = ts[at++];
          t.first[t.n + 1] = t.first[t.n] + static_cast<unsigned>(chunks);
          ++t.n;
        }
      if (pass == 0) clip_norm_kernel<<<kClipBlocks, 512, 0, s>>>(t, part, first ? 0 : 1);
      else clip_scale_kernel<<<t.n ? kClipBlocks : 1, 512, 0, s>>>(t, part, max_norm, norm);
      if (cudaGetLastError() != cudaSuccess) return SA_ERR_CUDA;
      first = false;
    } while ((pass == 0 || outs) && at < ts.size());
  }
  return SA_OK;
}

}  // extern "C"
