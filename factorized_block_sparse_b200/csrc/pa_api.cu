// C ABI of libpacked_attn.so (include/packed_attn.h): argument checks, the
// device copies of a packing's tables, and the launches.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <new>
#include <type_traits>

#include "pa_internal.h"
#include "pa_bwd.cuh"
#include "pa_fwd.cuh"

namespace pa {
namespace {

// Calls that a capture on another thread must not be broken by.
struct RelaxedCapture {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// The tables on the current device: found, or copied there (not inside a
// capture of `s`, whose graph would hold an allocation that it cannot replay).
int to_device(const pa_layout* L, cudaStream_t s, DeviceTables* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SA_ERR_CUDA;
  std::lock_guard<std::mutex> g(L->mu);
  for (auto& d : L->dev)
    if (d.device == dev) {
      *out = d;
      return SA_OK;
    }
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) return SA_ERR_CUDA;
  if (cap != cudaStreamCaptureStatusNone) return SA_ERR_INVALID_ARG;
  RelaxedCapture relaxed;
  const std::vector<Slot>* tabs[3] = {&L->fwd, &L->fwd2, &L->bwd};
  size_t n = 0;
  for (auto* t : tabs) n += t->size();
  Slot* dptr = nullptr;
  if (cudaMalloc(reinterpret_cast<void**>(&dptr), (n ? n : 1) * sizeof(Slot)) != cudaSuccess) return SA_ERR_CUDA;
  DeviceTables d;
  d.device = dev;
  d.blob = dptr;
  const Slot** fields[3] = {&d.fwd, &d.fwd2, &d.bwd};
  size_t at = 0;
  bool ok = true;
  for (int i = 0; i < 3; ++i) {
    *fields[i] = dptr + at;
    const size_t bytes = tabs[i]->size() * sizeof(Slot);
    if (bytes)
      ok = ok && cudaMemcpyAsync(dptr + at, tabs[i]->data(), bytes, cudaMemcpyHostToDevice, cudaStreamPerThread) ==
                     cudaSuccess;
    at += tabs[i]->size();
  }
  // on the device before any stream may read it
  ok = cudaStreamSynchronize(cudaStreamPerThread) == cudaSuccess && ok;
  if (!ok) {
    cudaFree(dptr);
    return SA_ERR_CUDA;
  }
  try {
    L->dev.push_back(d);
  } catch (...) {
    cudaFree(dptr);
    return SA_ERR_CUDA;
  }
  *out = d;
  return SA_OK;
}

struct Call {
  long long rows;
  int Hq, Hkv, D, dtype;
  float scale;
  cudaStream_t s;
};

bool stride_ok(int64_t st, int64_t extent) { return extent <= 1 || (st > 0 && st % 8 == 0 && st < (int64_t(1) << 38)); }

bool tensor_ok(const pa_tensor* t, const Call& c, int heads) {
  if (!t || !t->data || (reinterpret_cast<uintptr_t>(t->data) & 15)) return false;
  return stride_ok(t->row_stride, c.rows) && stride_ok(t->head_stride, heads);
}

// An output's (row, head) vectors must not overlap: heads inside a row, or rows inside a head.
bool output_ok(const pa_tensor* t, const Call& c, int heads) {
  if (!tensor_ok(t, c, heads)) return false;
  const int64_t rs = c.rows > 1 ? t->row_stride : 0, hs = heads > 1 ? t->head_stride : 0;
  if (c.rows > 1 && rs < c.D) return false;
  if (heads > 1 && hs < c.D) return false;
  if (c.rows <= 1 || heads <= 1) return true;
  return (heads - 1) * hs + c.D <= rs || (c.rows - 1) <= (hs - c.D) / rs;
}

bool lse_ok(const float* lse) { return lse && (reinterpret_cast<uintptr_t>(lse) & 3) == 0; }

int check_call(const Call& c, const pa_layout* L) {
  if (!L || c.Hq < 1 || c.Hkv < 1 || c.Hq > 65535 || c.Hq % c.Hkv || c.rows < L->rows ||
      c.rows > (int64_t(1) << 31) - 1024 || (c.dtype != PA_BF16 && c.dtype != PA_FP16))
    return SA_ERR_INVALID_ARG;
  if (!(c.scale > 0.f) || !std::isfinite(c.scale)) return SA_ERR_INVALID_ARG;
  if (c.D != 32 && c.D != 64 && c.D != 128) return SA_ERR_UNSUPPORTED;
  return SA_OK;
}

View view(const pa_tensor* t) { return View{t->data, t->row_stride, t->head_stride}; }

int launched() { return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA; }

// ------------------------------------------------------------ tensor maps
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool have_encode() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

// {D, heads, rows}, box: up to 64 columns of `box_rows` rows of one head.
// `rows` ends with the last sequence, so nothing behind it is ever read.
int map_rows(CUtensorMap* m, const pa_tensor* t, const Call& c, int heads, long long rows, int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)c.D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? t->head_stride : c.D) * 2,
                                 (cuuint64_t)(c.rows > 1 ? t->row_stride : c.D) * 2};
  const cuuint32_t box[3] = {(cuuint32_t)std::min(c.D, 64), 1, (cuuint32_t)box_rows};
  const cuuint32_t es[3] = {1, 1, 1};
  const auto type = c.dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const auto swz = c.D >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  return g_encode(m, type, 3, t->data, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? SA_OK
             : SA_ERR_CUDA;
}

constexpr int kMaxDevices = 64;

// SMs of the current device (asked once a device).
int sm_count(int* out) {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SA_ERR_CUDA;
  n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return SA_ERR_CUDA;
    known[dev].store(n, std::memory_order_relaxed);
  }
  *out = n;
  return SA_OK;
}

// Allows a kernel its dynamic shared memory (once a kernel and device).
template <auto Kernel, int Bytes>
int allow_smem() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SA_ERR_CUDA;
  if ((done.load(std::memory_order_acquire) >> dev) & 1u) return SA_OK;
  if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Bytes) != cudaSuccess) return SA_ERR_CUDA;
  done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  return SA_OK;
}

template <typename T, int D>
int run_fwd(const Call& c, const pa_tensor* q, const pa_tensor* k, const pa_tensor* v, const pa_tensor* o, float* lse,
            int64_t ls, const pa_layout* L, const DeviceTables& dc) {
  CUtensorMap mq, mk, mv;
  int st, sms;
  if ((st = map_rows(&mq, q, c, c.Hq, L->rows, kTile)) || (st = map_rows(&mk, k, c, c.Hkv, L->rows, kTile)) ||
      (st = map_rows(&mv, v, c, c.Hkv, L->rows, kTile)) || (st = sm_count(&sms)) ||
      (st = allow_smem<pa_fwd_kernel<T, D>, FwdCfg<D>::SMEM>()))
    return st;
  FwdArgs a;
  a.G = c.Hq / c.Hkv;
  a.o = view(o);
  a.lse = lse;
  a.ls = ls;
  a.scale_log2 = static_cast<float>(static_cast<double>(c.scale) * 1.4426950408889634);
  const long long tiles = static_cast<long long>(L->fwd.size());
  long long items;
  // A CTA for every tile where there are no more than SMs: nothing to pair (one sequence of 2048, 8 heads of 64: 25 us,
  // 32 in pairs).  Else two heads of a K/V head share its tiles where the group is even, which leaves no item half
  // empty (128 sequences of 128, 16 / 8 heads of 64: 45 us, 50 by row tiles; ten ragged sequences, 32 / 8 of 128: 412 and
  // 423), and two row tiles of a head otherwise.
  if (tiles * c.Hq <= sms) {
    a.pairing = kSingle;
    a.slots = dc.fwd;
    a.heads = c.Hq;
    items = tiles * c.Hq;
  } else if (a.G % 2 == 0) {
    a.pairing = kHeads;
    a.slots = dc.fwd;
    a.heads = c.Hq / 2;
    items = tiles * a.heads;
  } else {
    a.pairing = kTiles;
    a.slots = dc.fwd2;
    a.heads = c.Hq;
    items = static_cast<long long>(L->fwd2.size()) * a.heads;
  }
  if (items > (1ll << 30)) return SA_ERR_UNSUPPORTED;  // item numbers stay in 31 bits
  a.n_items = static_cast<int>(items);
  pa_fwd_kernel<T, D><<<std::min(a.n_items, sms), FwdCfg<D>::THREADS, FwdCfg<D>::SMEM, c.s>>>(mq, mk, mv, a);
  return launched();
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// Parts that a dK/dV item's steps are cut into.  An item is a key tile of a
// K/V head with the query tiles of its whole group; where a few items are much
// longer than an SM's share of all steps (but 8 steps at least, below which
// the parts' own cost shows), the longest of them is the pass's time.
// Measured, in one piece and in parts: one sequence of 4096, 4 heads on one
// K/V head of 64, 141 and 54 us; one of 2048, 8 on 8 of 64 (longest 16 steps, share
// 7), 29 and (forced) 52 us.  The parts' sums take the workspace of `parts`
// float32 copies of dK and dV: more parts go with fewer tiles, at most 0.23 GB
// at D = 128 (two parts, 850 key tiles on one K/V head, 40 of them one sequence).
int bwd_split(int Hq, int Hkv, const pa_layout* L) {
  constexpr int kSms = 148;  // (a size rule: the workspace must not depend on the device)
  if (L->bwd.empty()) return 1;
  const int64_t longest = static_cast<int64_t>(Hq / Hkv) * ((L->longest + kTile - 1) / kTile);
  const int64_t share = std::max<int64_t>(8, L->steps * Hq / kSms);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(longest / (2 * share), 16)));
}

// Workspace of the backward pass: packed lse and delta of every (head, tile),
// the largest squared norms of its rows of dO and v, then the float32 dV and
// dK of items in parts.
size_t bwd_ws_ld(int Hq, const pa_layout* L) {
  return align256(static_cast<size_t>(Hq) * L->fwd.size() * 2 * kTile * sizeof(float));
}
size_t bwd_ws_peak(int Hq, int Hkv, const pa_layout* L) {
  return align256(static_cast<size_t>(Hq + Hkv) * L->fwd.size() * sizeof(float));
}
size_t bwd_ws(int Hq, int Hkv, int D, const pa_layout* L) {
  const int split = bwd_split(Hq, Hkv, L);
  return bwd_ws_ld(Hq, L) + bwd_ws_peak(Hq, Hkv, L) +
         (split > 1 ? static_cast<size_t>(split) * 2 * Hkv * L->rows * D * sizeof(float) : 0) + 256;
}

template <typename T, int D>
int run_bwd(const Call& c, const pa_tensor* q, const pa_tensor* k, const pa_tensor* v, const pa_tensor* o,
            const float* lse, int64_t ls, const pa_tensor* dO, const pa_tensor* dq, const pa_tensor* dk,
            const pa_tensor* dv, const pa_layout* L, const DeviceTables& dc, void* ws) {
  CUtensorMap mq, mk, mv, mdo;
  int st, sms;
  if ((st = map_rows(&mq, q, c, c.Hq, L->rows, kTile)) || (st = map_rows(&mk, k, c, c.Hkv, L->rows, kTile)) ||
      (st = map_rows(&mv, v, c, c.Hkv, L->rows, kTile)) || (st = map_rows(&mdo, dO, c, c.Hq, L->rows, kTile)) ||
      (st = sm_count(&sms)) || (st = allow_smem<pa_bwd_kernel<T, D>, BwdCfg<D>::SMEM>()))
    return st;
  const unsigned tiles = static_cast<unsigned>(L->fwd.size());
  if (static_cast<long long>(tiles) * c.Hq > (1ll << 30)) return SA_ERR_UNSUPPORTED;  // item numbers stay in 31 bits
  float* ld = static_cast<float*>(ws);
  uint8_t* behind_ld = static_cast<uint8_t*>(ws) + bwd_ws_ld(c.Hq, L);
  float* peak = reinterpret_cast<float*>(behind_ld);
  const float scale_log2 = static_cast<float>(static_cast<double>(c.scale) * 1.4426950408889634);
  DkvArgs a;
  a.slots = dc.bwd;
  a.Hkv = c.Hkv;
  a.G = c.Hq / c.Hkv;
  a.split = bwd_split(c.Hq, c.Hkv, L);
  a.n_items = static_cast<int>(tiles) * c.Hkv * a.split;
  a.part = a.split > 1 ? reinterpret_cast<float*>(behind_ld + bwd_ws_peak(c.Hq, c.Hkv, L)) : nullptr;
  a.rows = L->rows;
  a.n_tiles = static_cast<int>(tiles);
  a.ld = ld;
  a.peak_do = peak;
  a.peak_v = peak + static_cast<size_t>(c.Hq) * tiles;
  a.dk = view(dk);
  a.dv = view(dv);
  a.scale = c.scale;
  a.scale_log2 = scale_log2;
  DqArgs b;
  b.slots = dc.fwd;
  b.Hq = c.Hq;
  b.G = a.G;
  b.n_items = static_cast<int>(tiles) * c.Hq;
  b.n_tiles = a.n_tiles;
  b.ld = ld;
  b.peak_do = a.peak_do;
  b.peak_v = a.peak_v;
  b.dq = view(dq);
  b.scale = c.scale;
  b.scale_log2 = scale_log2;
  pa_bwd_pre_kernel<T, D><<<dim3(tiles, c.Hq), 256, 0, c.s>>>(dc.fwd, view(o), view(dO), view(v), lse, ls, ld, peak, a.n_tiles,
                                                              c.Hkv);
  if ((st = launched())) return st;
  // The main kernel sets itself up while the one before it drains (programmatic stream serialisation).
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(static_cast<long long>(a.n_items) + b.n_items, sms)));
  cfg.blockDim = dim3(kBwdThreads);
  cfg.dynamicSmemBytes = BwdCfg<D>::SMEM;
  cfg.stream = c.s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, pa_bwd_kernel<T, D>, mq, mk, mv, mdo, a, b) != cudaSuccess) return SA_ERR_CUDA;
  if (a.split == 1) return SA_OK;
  cfg.gridDim = dim3(tiles, c.Hkv, kTile / kSumRows);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, pa_bwd_sum_kernel<T, D>, dc.bwd, static_cast<const float*>(a.part), a.split, c.Hkv, a.G,
                            a.rows, a.dk, a.dv, c.scale) == cudaSuccess
             ? SA_OK
             : SA_ERR_CUDA;
}

template <typename F>
int dispatch(const Call& c, F&& f) {
  auto by_d = [&](auto t) -> int {
    switch (c.D) {
      case 32: return f(t, std::integral_constant<int, 32>{});
      case 64: return f(t, std::integral_constant<int, 64>{});
      default: return f(t, std::integral_constant<int, 128>{});
    }
  };
  return c.dtype == PA_BF16 ? by_d(__nv_bfloat16{}) : by_d(__half{});
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

void packed_attn_layout_free(pa_layout* L) {
  if (!L) return;
  int cur = -1;
  const bool have = !L->dev.empty() && cudaGetDevice(&cur) == cudaSuccess;
  {
    RelaxedCapture relaxed;
    for (auto& d : L->dev)
      if (cudaSetDevice(d.device) == cudaSuccess) cudaFree(d.blob);
  }
  if (have) cudaSetDevice(cur);
  delete L;
}

int packed_attn_layout_upload(const pa_layout* L, void* stream) {
  if (!L) return SA_ERR_INVALID_ARG;
  DeviceTables dc;
  return to_device(L, static_cast<cudaStream_t>(stream), &dc);
}

int packed_attn_fwd(const pa_tensor* q, const pa_tensor* k, const pa_tensor* v, const pa_tensor* o, float* lse,
                    int64_t lse_stride, int64_t rows, int Hq, int Hkv, int D, int dtype, float scale,
                    const pa_layout* L, void* stream) {
  const Call c{rows, Hq, Hkv, D, dtype, scale, static_cast<cudaStream_t>(stream)};
  int st = check_call(c, L);
  if (st) return st;
  if (L->rows == 0) return SA_OK;
  if (!tensor_ok(q, c, Hq) || !tensor_ok(k, c, Hkv) || !tensor_ok(v, c, Hkv) || !output_ok(o, c, Hq) || !lse_ok(lse) ||
      lse_stride < rows || o->data == q->data || o->data == k->data || o->data == v->data)
    return SA_ERR_INVALID_ARG;
  if (!have_encode()) return SA_ERR_CUDA;
  DeviceTables dc;
  if ((st = to_device(L, c.s, &dc))) return st;
  return dispatch(c, [&](auto t, auto d) -> int {
    return run_fwd<decltype(t), d.value>(c, q, k, v, o, lse, lse_stride, L, dc);
  });
}

size_t packed_attn_bwd_workspace_size(int Hq, int Hkv, int D, const pa_layout* L) {
  const Call c{L ? static_cast<long long>(L->rows) : 0, Hq, Hkv, D, PA_BF16, 1.f, nullptr};
  if (check_call(c, L)) return 0;
  return bwd_ws(Hq, Hkv, D, L);
}

int packed_attn_bwd(const pa_tensor* q, const pa_tensor* k, const pa_tensor* v, const pa_tensor* o, const float* lse,
                    int64_t lse_stride, const pa_tensor* dO, const pa_tensor* dq, const pa_tensor* dk,
                    const pa_tensor* dv, int64_t rows, int Hq, int Hkv, int D, int dtype, float scale,
                    const pa_layout* L, void* ws, size_t ws_bytes, void* stream) {
  const Call c{rows, Hq, Hkv, D, dtype, scale, static_cast<cudaStream_t>(stream)};
  int st = check_call(c, L);
  if (st) return st;
  if (L->rows == 0) return SA_OK;
  if (!tensor_ok(q, c, Hq) || !tensor_ok(k, c, Hkv) || !tensor_ok(v, c, Hkv) || !tensor_ok(o, c, Hq) ||
      !tensor_ok(dO, c, Hq) || !output_ok(dq, c, Hq) || !output_ok(dk, c, Hkv) || !output_ok(dv, c, Hkv) || !lse_ok(lse) ||
      lse_stride < rows)
    return SA_ERR_INVALID_ARG;
  const pa_tensor* outs[3] = {dq, dk, dv};
  const pa_tensor* ins[5] = {q, k, v, o, dO};
  for (int i = 0; i < 3; ++i) {
    for (auto* t : ins)
      if (outs[i]->data == t->data) return SA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[i]->data == outs[j]->data) return SA_ERR_INVALID_ARG;
  }
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < packed_attn_bwd_workspace_size(Hq, Hkv, D, L))
    return SA_ERR_WORKSPACE;
  DeviceTables dc;
  if ((st = to_device(L, c.s, &dc))) return st;
  return dispatch(c, [&](auto t, auto d) -> int {
    return run_bwd<decltype(t), d.value>(c, q, k, v, o, lse, lse_stride, dO, dq, dk, dv, L, dc, ws);
  });
}

int packed_attn_status(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return SA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, sa::g_status, sizeof(int)) != cudaSuccess) return SA_ERR_CUDA;
  if (v != 0) {
    const int zero = 0;
    cudaMemcpyToSymbol(sa::g_status, &zero, sizeof(int));
    return v;
  }
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

#ifdef SA_TEST_HOOKS
// Test build only (not declared in the header): which first load the producers withhold (pa::Withhold; 0: none).
int packed_attn_test_withhold(int what) {
  return cudaMemcpyToSymbol(sa::g_test_withhold, &what, sizeof(int)) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
#endif

}  // extern "C"
