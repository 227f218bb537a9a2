// Layer norm forward and backward and the clipping of gradients by their
// global norm as calls of their own (include/sparse_block.h).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <new>
#include <type_traits>
#include <utility>
#include <vector>

#include "sparse_block.h"

namespace sbt {

constexpr int kMaxC = 16384;

// ------------------------------------------------------------------ types
template <typename T>
__device__ __forceinline__ float to_f(T v) {
  return static_cast<float>(v);
}

// Pairs of float32 in a 64-bit register: one instruction for two elements.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_get(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float f2_sum(uint64_t v) {
  const float2 t = f2_get(v);
  return t.x + t.y;
}

// The N elements of a 16-byte word, two of a 2-byte type from each 32-bit
// register (taken and cast one by one they were a third of the backward
// kernel's instructions).
template <typename T, int N>
__device__ __forceinline__ void unpack(const uint4& w, float* f) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      f[2 * i] = __uint_as_float(r[i] << 16);
      f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    } else if constexpr (std::is_same_v<T, __half>) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    } else {
      f[i] = __uint_as_float(r[i]);
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ uint4 pack(const float* f) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      r[i] = *reinterpret_cast<const uint32_t*>(&t);
    } else if constexpr (std::is_same_v<T, __half>) {
      const __half2 t = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      r[i] = *reinterpret_cast<const uint32_t*>(&t);
    } else {
      r[i] = __float_as_uint(f[i]);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Sums over the threads of a row: TPR lanes of a warp, or the block (TPR = 0;
// slots: 2 x 32 N floats used in turn, so that one barrier a sum is enough).
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* slots, int& turn) {
#pragma unroll
  for (int w = (TPR ? TPR : 32) / 2; w >= 1; w >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], w);
  if constexpr (TPR == 0) {
    float* s = slots + turn * 32 * N;
    turn ^= 1;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) s[k * 32 + w] = v[k];
    if (w == 0 && lane >= nw)  // every sum takes whole groups of four
#pragma unroll
      for (int k = 0; k < N; ++k) s[k * 32 + lane] = 0.f;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float4 a = reinterpret_cast<const float4*>(s + k * 32)[0];
      for (int i = 4; i < nw; i += 4) {
        const float4 b = *reinterpret_cast<const float4*>(s + k * 32 + i);
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
      }
      v[k] = (a.x + a.y) + (a.z + a.w);
    }
  }
}

// ------------------------------------------- rows as aligned 16-byte words
// A row is the words that it overlaps, the first and last one perhaps in
// part: word w holds channels w N - shift .. w N - shift + N - 1.  A thread
// visits rows a multiple of 8 apart, so its shift, and with it the channels of
// its words, are the same in every row whatever the stride (8 rows of 2-byte
// elements are a multiple of 16 bytes): gains and sums stay in registers.
// Words come through a ring in shared memory of the thread's own (cp.async, kDepth
// groups of rows, no barrier); a word is read whole where it lies inside the
// tensor's first and last byte, and written element by element where it
// holds another row's elements.
constexpr int kDepth = 3;

// Rows a thread takes at a time in the forward pass: their sums share a
// barrier, their words the gains in registers (65536 x 2048 bf16, two words a
// thread: 88 us, 95 one row at a time; three and more words leave no registers
// for a second row: 16384 x 6144 70 us, 72 with two).
__host__ __device__ constexpr int rows_at_once(int nv) { return nv >= 3 ? 1 : 2; }

// 1 / sqrt(v) to float32's last bit or so: the hardware's approximation and
// one step of Newton's method (0 and infinity pass through).
__device__ __forceinline__ float rsqrt_newton(float v) {
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.f);
  return fabsf(e) < 1.f ? fmaf(0.5f * r, e, r) : r;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The library's second kernels start while the first one drains (programmatic
// stream serialisation) and wait here before they read what it wrote.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The words of a thread: w = i0 + j n of a row, j < NV.  EDGE: words may hold
// other rows' elements (else rows begin and end on 16 bytes).
template <typename T, int NV, bool EDGE>
struct Words {
  static constexpr int N = 16 / sizeof(T);
  int i0, n, words, shift, C;
  uint32_t part = 0;  // bit j: word j holds other rows' elements too
  __device__ __forceinline__ Words(const T* row, int C_, int i0_, int n_) : i0(i0_), n(n_), C(C_) {
    shift = EDGE ? static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / static_cast<int>(sizeof(T)) : 0;
    words = (shift + C + N - 1) / N;
    if (EDGE)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (has(j) && (channel(j, 0) < 0 || channel(j, N - 1) >= C)) part |= 1u << j;
  }
  __device__ __forceinline__ bool has(int j) const { return i0 + j * n < words; }
  __device__ __forceinline__ int channel(int j, int u) const { return (i0 + j * n) * N - shift + u; }
  __device__ __forceinline__ bool in(int j, int u) const {
    return EDGE ? static_cast<unsigned>(channel(j, u)) < static_cast<unsigned>(C) : has(j);
  }
  __device__ __forceinline__ bool whole(int j) const { return !EDGE || !((part >> j) & 1); }
  // zeroes what is not of the row in the thread's words of a ring slot (the other rows' elements may be NaN)
  __device__ __forceinline__ void clean(uint4* slot) const {
    if (!EDGE || part == 0) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (!whole(j)) {
        T* e = reinterpret_cast<T*>(slot + j * blockDim.x);
        for (int u = 0; u < N; ++u)
          if (!in(j, u)) e[u] = static_cast<T>(0.f);
      }
  }
  // values of word j in pairs
  __device__ __forceinline__ void values(const uint4* slot, int j, uint64_t* v) const {
    const uint4 w = slot[j * blockDim.x];
    float f[N];
    unpack<T, N>(w, f);
#pragma unroll
    for (int u = 0; u < N / 2; ++u) v[u] = f2(f[2 * u], f[2 * u + 1]);
  }
};

// A tensor's rows as a thread visits them: its first word of the next row, and the tensor's bytes.
template <typename T, int NV, bool EDGE>
struct Feed {
  const char *p, *base, *end;
  long long step;
  __device__ __forceinline__ Feed(const T* t, long long ld, long long M, long long row, long long rows,
                                  const Words<T, NV, EDGE>& w)
      : p(reinterpret_cast<const char*>(t + row * ld + w.channel(0, 0))),
        base(reinterpret_cast<const char*>(t)),
        end(reinterpret_cast<const char*>(t + (M - 1) * ld + w.C)),
        step(rows * ld * static_cast<long long>(sizeof(T))) {}
  // the next row's words on their way into the thread's words of a ring slot
  __device__ __forceinline__ void request(uint4* slot, const Words<T, NV, EDGE>& w) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!w.has(j)) continue;
      const char* q = p + j * w.n * 16;
      uint4* d = slot + j * blockDim.x;
      if (!EDGE || (q >= base && q + 16 <= end)) {
        cp_async16(d, q);
      } else {  // at the tensor's very ends
        T* e = reinterpret_cast<T*>(d);
        for (int u = 0; u < Words<T, NV, EDGE>::N; ++u)
          if (w.in(j, u)) e[u] = reinterpret_cast<const T*>(q)[u];
      }
    }
    p += step;
  }
};

template <typename T, int NV, bool EDGE>
__device__ __forceinline__ void store_word(char* row, const Words<T, NV, EDGE>& w, int j, const uint64_t* v) {
  constexpr int N = 16 / sizeof(T);
  float f[N];
#pragma unroll
  for (int u = 0; u < N / 2; ++u) {
    const float2 t = f2_get(v[u]);
    f[2 * u] = t.x;
    f[2 * u + 1] = t.y;
  }
  T* p = reinterpret_cast<T*>(row + j * w.n * 16);
  if (w.whole(j)) {
    *reinterpret_cast<uint4*>(p) = pack<T, N>(f);
  } else {
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (w.in(j, u)) p[u] = static_cast<T>(f[u]);
  }
}

// Rows of a thread: the first, the distance, how many, and how many its warp (block) goes round.
template <int TPR>
struct Share {
  static constexpr int kPer = TPR ? TPR : 1;
  long long first, step;
  int mine, all, i0, n;
  __device__ __forceinline__ explicit Share(long long M) {
    first = TPR ? (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / kPer : blockIdx.x;
    step = TPR ? static_cast<long long>(gridDim.x) * blockDim.x / kPer : gridDim.x;
    const long long warp0 = TPR ? first - (threadIdx.x & 31) / kPer : first;
    mine = first < M ? static_cast<int>((M - first - 1) / step) + 1 : 0;
    all = warp0 < M ? static_cast<int>((M - warp0 - 1) / step) + 1 : 0;
    i0 = TPR ? threadIdx.x % kPer : threadIdx.x;
    n = TPR ? kPer : blockDim.x;
  }
};

// Blocks an SM that a kernel's registers are to allow: gains, biases and the row (column sums) of NV words.
__host__ __device__ constexpr int min_blocks(int nv, int maxt, bool bwd, bool edge) {
  if (maxt <= 128) return nv <= 2 ? 4 : 3;
  if (maxt <= 256) return nv == 1 ? (bwd ? 3 : 4) - edge : nv <= 3 || !edge ? 2 : 1;
  return 1;
}

// y = (x - mean) rstd g + b, and the row's mean and rstd.  TPR threads a row (0: the block, of at most MAXT).
// Bound by HBM where rows lie on 16 bytes: x is read and y written once, the row stays in registers between its two
// sums.  bf16: 2^17 x 1024 88 us, 65536 x 2048 87, 16384 x 6144 74 (94, 94 and 83 % of the copy rate); 24576 x 512
// 11.5 us (67 %: filling and emptying the rings).  With EDGE about half of that (16384 x 6143 144 us): the words at a
// row's ends hold up the block at its barriers, and registers leave fewer warps.
template <typename T, int NV, int TPR, bool EDGE, int MAXT>
__global__ void __launch_bounds__(MAXT, min_blocks(NV, MAXT, false, EDGE))
    norm_fwd_kernel(const T* x, long long ldx, const float* __restrict__ g, const float* __restrict__ b, T* y,
                    long long ldy, float* mean_out, float* rstd_out, long long M, int C, float eps) {
  constexpr int N = 16 / sizeof(T);
  extern __shared__ uint4 ring_[];  // [kDepth][rows at once][NV][threads]
  __shared__ __align__(16) float slots[128];
  int turn = 0;
  const Share<TPR> sh(M);
  const Words<T, NV, EDGE> ws(x + sh.first * ldx, C, sh.i0, sh.n);
  Feed<T, NV, EDGE> xs(x, ldx, M, sh.first, sh.step, ws);
  uint4* ring = ring_ + threadIdx.x;
  constexpr int R = rows_at_once(NV);
  const int row_words = NV * blockDim.x, slot_words = R * row_words;
  int asked = 0;
  auto request = [&](uint4* slot) {
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (asked + k < sh.mine) xs.request(slot + k * row_words, ws);
    asked += R;
    cp_commit();
  };
#pragma unroll
  for (int d = 0; d < kDepth - 1; ++d) request(ring + d * slot_words);
  constexpr int H = N / 2;  // pairs of a word
  uint64_t gv[NV * H], bv[NV * H];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int u = 0; u < H; ++u) {
      auto at_channel = [&](const float* p, int e) { return p && ws.in(j, e) ? p[ws.channel(j, e)] : 0.f; };
      gv[j * H + u] = f2(at_channel(g, 2 * u), at_channel(g, 2 * u + 1));
      bv[j * H + u] = f2(at_channel(b, 2 * u), at_channel(b, 2 * u + 1));
    }
  const float inv = 1.f / C;
  char* out = reinterpret_cast<char*>(y + sh.first * ldy + ws.channel(0, 0));
  const long long out_step = sh.step * ldy * static_cast<long long>(sizeof(T));
  int at = 0;
  for (int i = 0; i < sh.all; i += R) {
    request(ring + (at == 0 ? kDepth - 1 : at - 1) * slot_words);
    cp_wait<kDepth - 1>();
    uint64_t f[R][NV * H];
    float s[R], q[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      uint64_t sum = 0;
      if (i + k < sh.mine) ws.clean(ring + at * slot_words + k * row_words);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (i + k < sh.mine && ws.has(j)) ws.values(ring + at * slot_words + k * row_words, j, f[k] + j * H);
        else
#pragma unroll
          for (int u = 0; u < H; ++u) f[k][j * H + u] = 0;
#pragma unroll
        for (int u = 0; u < H; ++u) sum = f2_add(sum, f[k][j * H + u]);
      }
      s[k] = f2_sum(sum);
    }
    row_sums<TPR>(s, slots, turn);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      s[k] *= inv;  // the mean
      const uint64_t neg = f2(-s[k], -s[k]);
      uint64_t sum = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int u = 0; u < H; ++u) {
          uint64_t& v = f[k][j * H + u];
          v = f2_add(v, neg);
          if (!ws.has(j)) v = 0;  // outside the row there is no deviation
        }
      if (EDGE && ws.part != 0)
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (!ws.whole(j))
#pragma unroll
            for (int u = 0; u < H; ++u) {
              const float2 t = f2_get(f[k][j * H + u]);
              f[k][j * H + u] = f2(ws.in(j, 2 * u) ? t.x : 0.f, ws.in(j, 2 * u + 1) ? t.y : 0.f);
            }
#pragma unroll
      for (int c = 0; c < NV * H; ++c) sum = f2_fma(f[k][c], f[k][c], sum);
      q[k] = f2_sum(sum);
    }
    row_sums<TPR>(q, slots, turn);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float rstd = rsqrt_newton(q[k] * inv + eps);
      const uint64_t r2 = f2(rstd, rstd);
      if (i + k < sh.mine) {
        if (sh.i0 == 0) {
          const long long r = sh.first + (i + k) * sh.step;
          if (mean_out) mean_out[r] = s[k];
          if (rstd_out) rstd_out[r] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (ws.has(j)) {
            uint64_t o[H];
#pragma unroll
            for (int u = 0; u < H; ++u) o[u] = f2_fma(f2_mul(f[k][j * H + u], r2), gv[j * H + u], bv[j * H + u]);
            store_word(out, ws, j, o);
          }
      }
      out += out_step;
    }
    at = at + 1 == kDepth ? 0 : at + 1;
  }
}

// Rows too wide for the registers of a block, and tensors whose rows lie at
// different offsets from 16 bytes: one element at a time, read again for each
// pass.  Bound by the loads in flight: bf16 16384 x 6144 with x at an odd element
// and y not, 347 us forward and 1176 backward (74 and 121 where both lie on 16
// bytes); 24576 x 512, 98 and 156; float32 4096 x 9000, 143 and 437.
template <typename T>
__global__ void __launch_bounds__(512)
    norm_fwd_wide_kernel(const T* x, long long ldx, const float* g, const float* b, T* y, long long ldy,
                         float* mean_out, float* rstd_out, long long M, int C, float eps) {
  __shared__ __align__(16) float slots[64];
  int turn = 0;
  const float inv = 1.f / C;
  for (long long r = blockIdx.x; r < M; r += gridDim.x) {
    const T* p = x + r * ldx;
    float s[1] = {0.f}, q[1] = {0.f};
    for (int i = threadIdx.x; i < C; i += blockDim.x) s[0] += to_f(p[i]);
    row_sums<0>(s, slots, turn);
    const float mean = s[0] * inv;
    for (int i = threadIdx.x; i < C; i += blockDim.x) q[0] += (to_f(p[i]) - mean) * (to_f(p[i]) - mean);
    row_sums<0>(q, slots, turn);
    const float rstd = rsqrt_newton(q[0] * inv + eps);
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
    for (int i = threadIdx.x; i < C; i += blockDim.x)
      y[r * ldy + i] = static_cast<T>((to_f(p[i]) - mean) * rstd * g[i] + (b ? b[i] : 0.f));
  }
}

// Rows in flight of the backward kernel (x and dy; four words a thread fill shared memory with two).
__host__ __device__ constexpr int bwd_depth(int nv, int maxt) { return nv >= 4 ? (maxt <= 256 ? 3 : 2) : 4; }

// dx per row, and this block's sums of dy xh and dy per channel into
// part[blockIdx.x][2][C].
// x and dy are read from the ring twice, before and after the row's two sums,
// so that only the gains and the column sums stay in registers.  Bound by HBM and,
// next to it, by the issue of its instructions (about 25 an element pair): bf16
// 2^18 x 512 129 us, 65536 x 2048 142, 16384 x 6144 119 (96, 87 and 77 % of the
// copy rate), float32 16384 x 4096 132 (93 %); with EDGE 16384 x 6143 203 us.
// EDGE in place of the exact variant, measured on one state of both: 262144 x 512 217 us for 133.
template <typename T, int NV, int TPR, bool EDGE, int MAXT>
__global__ void __launch_bounds__(MAXT, min_blocks(NV, MAXT, true, EDGE))
    norm_bwd_kernel(const T* x, long long ldx, const float* __restrict__ g, const T* dy, long long lddy,
                    const float* __restrict__ mean_in, const float* __restrict__ rstd_in, T* dx, long long lddx,
                    float* part, long long M, int C) {
  constexpr int N = 16 / sizeof(T);
  constexpr int kRing = bwd_depth(NV, MAXT);
  extern __shared__ uint4 ring_[];  // [kRing][rows at once][x, dy][NV][threads]; then the row groups' sums [groups][2][C]
  __shared__ __align__(16) float slots[256];
  pdl_trigger();
  int turn = 0;
  const Share<TPR> sh(M);
  const Words<T, NV, EDGE> ws(x + sh.first * ldx, C, sh.i0, sh.n);
  Feed<T, NV, EDGE> xs(x, ldx, M, sh.first, sh.step, ws), ds(dy, lddy, M, sh.first, sh.step, ws);
  uint4* ring = ring_ + threadIdx.x;
  constexpr int R = 1;  // (two at a time: the ring leaves room for one block an SM, 192 us for 158 when that was measured)
  const int row_words = NV * blockDim.x, slot_words = 2 * R * row_words;
  float m_next[kRing - 1][R], r_next[kRing - 1][R];  // statistics of the rows in flight
  const float *pm = mean_in + sh.first, *pr = rstd_in + sh.first;
  int asked = 0;
  auto request = [&](uint4* slot, float (&m)[R], float (&rs)[R]) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      m[k] = rs[k] = 0.f;
      if (asked + k < sh.mine) {
        xs.request(slot + 2 * k * row_words, ws);
        ds.request(slot + (2 * k + 1) * row_words, ws);
        m[k] = *pm;
        rs[k] = *pr;
        pm += sh.step;
        pr += sh.step;
      }
    }
    asked += R;
    cp_commit();
  };
#pragma unroll
  for (int d = 0; d < kRing - 1; ++d) request(ring + d * slot_words, m_next[d], r_next[d]);
  constexpr int H = N / 2;  // pairs of a word
  uint64_t gv[NV * H], sg[NV * H] = {}, sb[NV * H] = {};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int u = 0; u < H; ++u) {
      auto gain = [&](int e) { return ws.in(j, e) ? g[ws.channel(j, e)] : 0.f; };
      gv[j * H + u] = f2(gain(2 * u), gain(2 * u + 1));
    }
  const float inv = 1.f / C;
  char* out = reinterpret_cast<char*>(dx + sh.first * lddx + ws.channel(0, 0));
  const long long out_step = sh.step * lddx * static_cast<long long>(sizeof(T));
  int at = 0;
  for (int i = 0; i < sh.all; i += R) {
    float mc[R], rc[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mc[k] = m_next[0][k];
      rc[k] = r_next[0][k];
#pragma unroll
      for (int d = 0; d + 1 < kRing - 1; ++d) {
        m_next[d][k] = m_next[d + 1][k];
        r_next[d][k] = r_next[d + 1][k];
      }
    }
    request(ring + (at == 0 ? kRing - 1 : at - 1) * slot_words, m_next[kRing - 2], r_next[kRing - 2]);
    cp_wait<kRing - 1>();
    uint4* xw = ring + at * slot_words;
#pragma unroll
    for (int k = 0; k < 2 * R; ++k)
      if (i + k / 2 < sh.mine) ws.clean(xw + k * row_words);
    float s[2 * R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const uint64_t neg = f2(-mc[k], -mc[k]), r2 = f2(rc[k], rc[k]);
      uint64_t s0 = 0, s1 = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (i + k < sh.mine && ws.has(j)) {
          uint64_t x2[H], d2[H];
          ws.values(xw + 2 * k * row_words, j, x2);
          ws.values(xw + (2 * k + 1) * row_words, j, d2);
#pragma unroll
          for (int u = 0; u < H; ++u) {
            const int c = j * H + u;
            const uint64_t xh = f2_mul(f2_add(x2[u], neg), r2);  // (not x r - m r, which cancels where the mean is large)
            sg[c] = f2_fma(d2[u], xh, sg[c]);
            sb[c] = f2_add(sb[c], d2[u]);
            const uint64_t t = f2_mul(d2[u], gv[c]);
            s0 = f2_add(s0, t);
            s1 = f2_fma(t, xh, s1);
          }
        }
      s[2 * k] = f2_sum(s0);
      s[2 * k + 1] = f2_sum(s1);
    }
    row_sums<TPR>(s, slots, turn);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      // dx = r t - r mean(t) - xh r mean(t xh)
      const float a0 = -rc[k] * (s[2 * k] * inv), a1 = -rc[k] * (s[2 * k + 1] * inv);
      const uint64_t c0 = f2(a0, a0), c1 = f2(a1, a1), neg = f2(-mc[k], -mc[k]), r2 = f2(rc[k], rc[k]);
      if (i + k < sh.mine)
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (ws.has(j)) {
            uint64_t x2[H], d2[H];
            ws.values(xw + 2 * k * row_words, j, x2);
            ws.values(xw + (2 * k + 1) * row_words, j, d2);
#pragma unroll
            for (int u = 0; u < H; ++u)
              d2[u] = f2_fma(r2, f2_mul(d2[u], gv[j * H + u]), f2_fma(f2_mul(f2_add(x2[u], neg), r2), c1, c0));
            store_word(out, ws, j, d2);
          }
      out += out_step;
    }
    at = at + 1 == kRing ? 0 : at + 1;
  }
  float* dst = part + static_cast<long long>(blockIdx.x) * 2 * C;
  auto put = [&](float* to) {  // the thread's column sums
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int u = 0; u < N; ++u)
        if (ws.in(j, u)) {
          const float2 a = f2_get(sg[j * H + u / 2]), b = f2_get(sb[j * H + u / 2]);
          to[ws.channel(j, u)] = u & 1 ? a.y : a.x;
          to[C + ws.channel(j, u)] = u & 1 ? b.y : b.x;
        }
  };
  if constexpr (TPR != 0) {
    constexpr int kPer = TPR ? TPR : 1;
    float* sums = reinterpret_cast<float*>(ring_);
    float* mine = sums + threadIdx.x / kPer * 2 * C;
    cp_wait<0>();
    __syncthreads();
    put(mine);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * C; i += blockDim.x) {
      float a = 0.f;
#pragma unroll 8
      for (int w = 0; w < 256 / kPer; ++w) a += sums[w * 2 * C + i];
      dst[i] = a;
    }
  } else {
    put(dst);
  }
}

template <typename T>
__global__ void __launch_bounds__(512)
    norm_bwd_wide_kernel(const T* x, long long ldx, const float* g, const T* dy, long long lddy, const float* mean_in,
                         const float* rstd_in, T* dx, long long lddx, float* part, long long M, int C) {
  extern __shared__ float sums[];  // [2][C]; a channel belongs to one thread
  __shared__ __align__(16) float slots[128];
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
    row_sums<0>(s, slots, turn);
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
  pdl_wait();
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (i < 2 * C)
#pragma unroll 8
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
// Three blocks an SM are what the kernels' registers allow, and one wave of them shares the chunks evenly (352 M bf16
// elements, norm and clip: 106 and 351 us; 592 blocks 127 and 367, 296 blocks 110 and 386).
constexpr int kClipBlocks = 444;

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
  unsigned chunk;  // elements a block takes at a time, a multiple of 8
};

// The squares of a word: each half's summed in float32 by a tree, the halves
// in float64; all in float64 where one is too large or too small for that
// (2^-40 .. 2^60 keeps squares and sums inside float32); zeros are the common
// small values.  A half's sum takes two roundings of 2^-24 whatever its values
// (2-byte types: their squares are exact, two additions; float32: a square and
// an addition), one in the norm, which with its own rounding is good to 2^-23.
// A word summed in one float32 chain would lose up to 3.5 2^-24 of the norm.
template <typename T>
__device__ __forceinline__ double word_squares(const uint4& w) {
  constexpr int N = 16 / sizeof(T);
  float f[N], big = 0.f, pair[N / 2];
  unpack<T, N>(w, f);
#pragma unroll
  for (int u = 0; u < N; u += 2) {
    pair[u / 2] = fmaf(f[u], f[u], f[u + 1] * f[u + 1]);
    big = fmaxf(big, fmaxf(fabsf(f[u]), fabsf(f[u + 1])));
  }
  if (big == 0.f || (big > 9.1e-13f && big < 1.1e18f)) {  // (a NaN beside numbers passes: the sum is NaN)
    if constexpr (N == 8) return static_cast<double>(pair[0] + pair[1]) + static_cast<double>(pair[2] + pair[3]);
    else return static_cast<double>(pair[0]) + static_cast<double>(pair[1]);
  }
  double d = 0.;
#pragma unroll
  for (int u = 0; u < N; ++u) d += static_cast<double>(f[u]) * f[u];
  return d;
}

template <typename T>
__device__ __forceinline__ double sum_squares(const T* p, unsigned n) {
  constexpr unsigned N = 16 / sizeof(T);
  double s = 0.;
  unsigned done = 0;
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const uint4* w = reinterpret_cast<const uint4*>(p);
    const unsigned words = n / N;
    unsigned i = threadIdx.x;
    for (; i + 3 * blockDim.x < words; i += 4 * blockDim.x) {  // four words in flight
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = w[i + k * blockDim.x];
#pragma unroll
      for (int k = 0; k < 4; ++k) s += word_squares<T>(v[k]);
    }
    for (; i < words; i += blockDim.x) s += word_squares<T>(w[i]);
    done = words * N;
  }
  for (unsigned i = done + threadIdx.x; i < n; i += blockDim.x) {
    const double v = to_f(p[i]);
    s += v * v;
  }
  return s;
}

template <typename T>
__device__ __forceinline__ void scale_to(const T* p, T* o, unsigned n, float c) {
  constexpr unsigned N = 16 / sizeof(T);
  unsigned done = 0;
  if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(o)) & 15) == 0) {
    const uint4* w = reinterpret_cast<const uint4*>(p);
    uint4* q = reinterpret_cast<uint4*>(o);
    const unsigned words = n / N;
    auto scaled = [&](const uint4& v) {
      float f[N];
      unpack<T, N>(v, f);
#pragma unroll
      for (unsigned u = 0; u < N; ++u) f[u] *= c;
      return pack<T, N>(f);
    };
    unsigned i = threadIdx.x;
    for (; i + 3 * blockDim.x < words; i += 4 * blockDim.x) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = w[i + k * blockDim.x];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[i + k * blockDim.x] = scaled(v[k]);
    }
    for (; i < words; i += blockDim.x) q[i] = scaled(w[i]);
    done = words * N;
  }
  for (unsigned i = done + threadIdx.x; i < n; i += blockDim.x) o[i] = static_cast<T>(to_f(p[i]) * c);
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
  pdl_trigger();
  double s = 0.;
  for (unsigned c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const unsigned long long at = static_cast<unsigned long long>(c - t.first[i]) * t.chunk;
    const unsigned n = static_cast<unsigned>(min(static_cast<unsigned long long>(t.chunk), t.t[i].n - at));
    if (t.t[i].dtype == SB_BF16) s += sum_squares(static_cast<const __nv_bfloat16*>(t.t[i].g) + at, n);
    else if (t.t[i].dtype == SB_FP16) s += sum_squares(static_cast<const __half*>(t.t[i].g) + at, n);
    else s += sum_squares(static_cast<const float*>(t.t[i].g) + at, n);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = (add ? part[blockIdx.x] : 0.) + s;
}

__global__ void __launch_bounds__(512)
    clip_scale_kernel(const __grid_constant__ ClipTable t, const double* part, double max_norm, float* norm) {
  pdl_wait();
  double s = 0.;
  for (int i = threadIdx.x; i < kClipBlocks; i += blockDim.x) s += part[i];
  const double total = sqrt(block_sum(s));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  if (t.n == 0) return;
  double cd = max_norm / (total + 1e-6);
  if (cd > 1.) cd = 1.;
  const float c = static_cast<float>(cd);
  // from the last chunk back: the norm's pass has left those in L2
  for (unsigned b = blockIdx.x; b < t.first[t.n]; b += gridDim.x) {
    const unsigned k = t.first[t.n] - 1 - b;
    const int i = tensor_of(t, k);
    const unsigned long long at = static_cast<unsigned long long>(k - t.first[i]) * t.chunk;
    const unsigned n = static_cast<unsigned>(min(static_cast<unsigned long long>(t.chunk), t.t[i].n - at));
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

constexpr int kMaxDevices = 64;

int device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices ? dev : -1;
}

// SMs of a device, asked once.
int sms(int dev) {
  static std::atomic<int> known[kMaxDevices];
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 148;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Blocks of a kernel that an SM holds, asked once a device and block size (the
// dynamic shared memory goes with the block size); also allows the memory.
template <auto Kernel>
int resident(int dev, int threads, size_t smem) {
  static std::atomic<int> known[kMaxDevices][17];
  std::atomic<int>& k = known[dev][threads / 32 <= 16 ? threads / 32 : 0];
  int per = k.load(std::memory_order_relaxed);
  if (per == 0) {
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, Kernel, threads, smem) != cudaSuccess || per < 1)
      return 0;
    k.store(per, std::memory_order_relaxed);
  }
  return per;
}

// A launch that may begin while the kernel before it in the stream drains.
template <class... P, class... A>
int launch_behind(void (*kernel)(P...), unsigned grid, unsigned block, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

template <typename F>
int by_type(int dtype, F&& f) {
  if (dtype == SB_BF16) return f(__nv_bfloat16{});
  if (dtype == SB_FP16) return f(__half{});
  return f(float{});
}

int esize(int dtype) { return dtype == SB_FP32 ? 4 : 2; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// go(words a thread, threads a row, EDGE, block's threads at most) for a row of
// `words` words; -1 above the widest.  Narrow rows share a warp, up to 96 words
// a warp takes a row, above that a block of 128 to 512 threads.  Measured (bf16,
// forward and backward, the other side in brackets):
//   2^20 x 64, 8 lanes a row: 49 and 77 us [a warp a row: 190 and 293];
//   2^18 x 512, a warp a row: 99 and 129 us [a block: 115 and 253];
//   2^17 x 768, a warp, three words a thread: 75 and 102 us [a block: 87 and 135; with EDGE the backward spills
//   there: 349 us, 216 in a block];
//   65536 x 2048, 128 threads of two words: 88 and 142 us [256 of one: 120 and 189];
//   16384 x 6144, 256 threads of three words: 70 and 119 us [384 of two: 87 and 143];
//   32768 x 4095 (EDGE), forward 192 threads of three words: 172 us [512 of two: 247], backward the other way: 318 [410];
//   16384 x 8192, forward 256 threads of four words: 86 us [512 of two: 120], backward the other way: 170 [177].
// A row's sums cost a thread the same whatever its words, so more words a
// thread are better until their registers leave too few warps.
template <bool BWD, typename F, typename E>
int by_width(int words, F&& go, E edge) {
  using std::integral_constant;
  using I1 = integral_constant<int, 1>;
  using I2 = integral_constant<int, 2>;
  using I3 = integral_constant<int, 3>;
  using I4 = integral_constant<int, 4>;
  using Warp = integral_constant<int, 32>;
  using Block = integral_constant<int, 0>;
  using T128 = integral_constant<int, 128>;
  using T256 = integral_constant<int, 256>;
  using T512 = integral_constant<int, 512>;
  if (words <= 8) return go(I1{}, integral_constant<int, 8>{}, edge, T256{});
  if (words <= 16) return go(I1{}, integral_constant<int, 16>{}, edge, T256{});
  if (words <= 32) return go(I1{}, Warp{}, edge, T256{});
  if (words <= 64) return go(I2{}, Warp{}, edge, T256{});
  if constexpr (!BWD || !E::value)
    if (words <= 96) return go(I3{}, Warp{}, edge, T256{});
  if (words <= 256) return go(I2{}, Block{}, edge, T128{});
  if (words <= 384) return go(I3{}, Block{}, edge, T128{});
  if (words <= 512) return go(I2{}, Block{}, edge, T256{});
  if constexpr (!BWD || !E::value)
    if (words <= 768) return go(I3{}, Block{}, edge, T256{});
  if constexpr (!BWD && !E::value)
    if (words <= 1024) return go(I4{}, Block{}, edge, T256{});
  if (words <= 1024) return go(I2{}, Block{}, edge, T512{});
  if (words <= 2048) return go(I4{}, Block{}, edge, T512{});
  return -1;
}

// Whether the rows of two tensors lie at the same offsets from 16 bytes.
bool alike(const void* a, int64_t lda, const void* b, int64_t ldb, int es) {
  return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0 && ((lda - ldb) * es) % 16 == 0;
}

// Blocks of a backward launch at most, each with 2 C float32 sums in the workspace: eight an SM where blocks are of 64
// threads (2^17 x 1024 bf16: 139 us, 169 with four), no more than an SM holds of the wider ones.
int64_t parts(int C) { return C <= 2048 ? 1184 : C <= 4096 ? 592 : 296; }

// The words of a row, at most (it may begin anywhere in its first one).
int words_of(const void* p, int64_t ld, int C, int es) {
  const bool even = aligned(p, 16) && (ld * es) % 16 == 0;
  return (C * es + 15) / 16 + (even ? 0 : 1);
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
  const int dev = device();
  if (dev < 0) return SA_ERR_CUDA;
  const int n_sm = sms(dev), words = words_of(x, ldx, C, es);
  const bool same = alike(x, ldx, y, ldy, es);
  const bool edge = !aligned(x, 16) || (ldx * es) % 16 != 0 || (C * es) % 16 != 0;
  return by_type(dtype, [&](auto t) -> int {
    using T = decltype(t);
    auto go = [&](auto nv, auto tpr, auto edge, auto maxt) -> int {
      constexpr int NV = nv.value, TPR = tpr.value;
      constexpr auto K = norm_fwd_kernel<T, NV, TPR, edge.value, maxt.value>;
      const int threads = TPR ? 256 : (words + 32 * NV - 1) / (32 * NV) * 32;
      const int rows = TPR ? 256 / (TPR ? TPR : 1) : 1;  // rows of a block at a time
      const size_t smem = static_cast<size_t>(kDepth) * rows_at_once(NV) * NV * threads * 16;
      const int per = resident<K>(dev, threads, smem);
      if (per == 0) return SA_ERR_CUDA;
      long long grid = std::min<long long>((M + rows - 1) / rows, static_cast<long long>(n_sm) * per);
      if (TPR == 0 && grid < M) grid = std::max<long long>(grid / 8 * 8, 8);  // rows of a thread: a multiple of 8 apart
      K<<<static_cast<unsigned>(grid), threads, smem, s>>>(static_cast<const T*>(x), ldx, g, b, static_cast<T*>(y), ldy,
                                                           mean, rstd, M, C, eps);
      return launched();
    };
    if (same) {
      const int st = edge ? by_width<false>(words, go, std::true_type{}) : by_width<false>(words, go, std::false_type{});
      if (st >= 0) return st;
    }
    const int grid = static_cast<int>(std::min<long long>(M, static_cast<long long>(n_sm) * 4));
    norm_fwd_wide_kernel<T><<<grid, 512, 0, s>>>(static_cast<const T*>(x), ldx, g, b, static_cast<T*>(y), ldy, mean, rstd, M,
                                                 C, eps);
    return launched();
  });
}

size_t sparse_block_layer_norm_bwd_workspace_size(int64_t M, int C) {
  if (M < 0 || C < 1 || C > kMaxC) return 0;
  return static_cast<size_t>(std::max<int64_t>(1, std::min<int64_t>(M, parts(C)))) * 2 * C * sizeof(float);
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
  const int dev = device();
  if (dev < 0) return SA_ERR_CUDA;
  const int n_sm = sms(dev);
  int P = 0;
  if (M > 0) {
    const int words = words_of(x, ldx, C, es);
    const bool same = alike(x, ldx, dy, lddy, es) && alike(x, ldx, dx, lddx, es);
    const bool edge = !aligned(x, 16) || (ldx * es) % 16 != 0 || (C * es) % 16 != 0;
    const int st = by_type(dtype, [&](auto t) -> int {
      using T = decltype(t);
      auto go = [&](auto nv, auto tpr, auto edge, auto maxt) -> int {
        constexpr int NV = nv.value, TPR = tpr.value;
        constexpr auto K = norm_bwd_kernel<T, NV, TPR, edge.value, maxt.value>;
        const int threads = TPR ? 256 : (words + 32 * NV - 1) / (32 * NV) * 32;
        const int rows = TPR ? 256 / (TPR ? TPR : 1) : 1;
        // the ring, and in its place afterwards the row groups' sums of up to NV TPR words
        const size_t ring = 2 * static_cast<size_t>(bwd_depth(NV, maxt.value)) * NV * threads * 16;
        const size_t sums = TPR ? static_cast<size_t>(rows) * 2 * (NV * TPR * 16 / sizeof(T)) * sizeof(float) : 0;
        const size_t smem = std::max(ring, sums);
        const int per = resident<K>(dev, threads, smem);
        if (per == 0) return SA_ERR_CUDA;
        long long grid = std::min<long long>(std::min<long long>((M + rows - 1) / rows, parts(C)), static_cast<long long>(n_sm) * per);
        if (TPR == 0 && grid < M) grid = std::max<long long>(grid / 8 * 8, 8);
        P = static_cast<int>(grid);
        K<<<P, threads, smem, s>>>(static_cast<const T*>(x), ldx, g, static_cast<const T*>(dy), lddy, mean, rstd,
                                   static_cast<T*>(dx), lddx, part, M, C);
        return launched();
      };
      if (same) {
        const int r = edge ? by_width<true>(words, go, std::true_type{}) : by_width<true>(words, go, std::false_type{});
        if (r >= 0) return r;
      }
      constexpr auto K = norm_bwd_wide_kernel<T>;
      const size_t smem = 2 * static_cast<size_t>(C) * sizeof(float);
      if (resident<K>(dev, 512, smem) == 0) return SA_ERR_CUDA;
      P = static_cast<int>(std::min<long long>(std::min<long long>(M, parts(C)), n_sm));
      K<<<P, 512, smem, s>>>(static_cast<const T*>(x), ldx, g, static_cast<const T*>(dy), lddy, mean, rstd,
                             static_cast<T*>(dx), lddx, part, M, C);
      return launched();
    });
    if (st) return st;
  }
  return launch_behind(norm_bwd_sum_kernel, (2 * C + 31) / 32, 1024, s, static_cast<const float*>(part), P, C, dg, db);
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
  // A chunk is 2048 elements (one word a thread and more) to 65536: small enough that every block has one, large
  // enough that finding its tensor costs nothing.
  size_t total = 0;
  for (const ClipTensor& x : ts) total += x.n;
  t.chunk = static_cast<unsigned>(std::min<size_t>(std::max<size_t>((total / (2 * kClipBlocks) + 2047) / 2048 * 2048, 2048), 65536));
  // `norm` pass over the tensors, then the scaling pass; kTensors of them a launch
  for (int pass = 0; pass < 2; ++pass) {
    size_t at = 0;
    bool first = true;
    do {
      t.n = 0;
      t.first[0] = 0;
      if (pass == 0 || outs)
        while (at < ts.size() && t.n < kTensors) {
          const size_t chunks = (ts[at].n + t.chunk - 1) / t.chunk;
          if (t.first[t.n] + chunks > 0x7fffffffu) break;
          t.t[t.n] = ts[at++];
          t.first[t.n + 1] = t.first[t.n] + static_cast<unsigned>(chunks);
          ++t.n;
        }
      if (pass == 0) {
        clip_norm_kernel<<<kClipBlocks, 512, 0, s>>>(t, part, first ? 0 : 1);
        if (launched()) return SA_ERR_CUDA;
      } else if (launch_behind(clip_scale_kernel, t.n ? kClipBlocks : 1, 512, s, t, static_cast<const double*>(part), max_norm,
                               norm)) {
        return SA_ERR_CUDA;
      }
      first = false;
    } while ((pass == 0 || outs) && at < ts.size());
  }
  return SA_OK;
}

}  // extern "C"
