// Global norm of many gradient tensors and clipping by it (svconv_clip_grads).
//
// HBM-bound: the norm reads every value once, the scaling reads and writes it once more (from L2
// where the set fits).  The tensors travel as a table in the kernel parameters, cut into chunks of
// kClipChunk values; each CTA takes one run of the chunks of all tensors, so many small tensors cost no
// launches of their own.  Squares are summed in fp64: a finite set of gradients has a finite
// norm, and one conversion per value stays below the time of its load.  CTA sums are added in a
// fixed order by every CTA of the second kernel (deterministic, no atomics).
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "svconv_internal.h"
#include "svconv_ptx.cuh"

namespace svc {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipCtas = 592;      // 4 per SM on 148 SMs
constexpr int kClipChunk = 4096;    // values of one tensor per step of a CTA
constexpr int kClipBatch = 4;       // 16-byte loads in flight per thread
constexpr int kClipSmall = 64;      // tensors in the small table (2.2 KB of parameters)
constexpr int kClipMedium = 256;    // in the medium one (8.5 KB: a launch copies its parameters, ~3 us for the large one)
constexpr int kClipLarge = 800;     // in the large one (under the 32,764 bytes a launch may carry)

template <int N>
struct ClipTable {
  const void* src[N];
  void* dst[N];
  int64_t numel[N];
  int32_t first[N + 1];   // chunks before tensor i
  uint8_t bf16[N];
  int count;
  double* part;           // every launch's CTA sums
  int part_at, parts;     // this launch's first slot; slots of all launches
  float max_norm;
  float* norm;
};

template <int N>
__device__ __forceinline__ int tensor_of(const ClipTable<N>& t, int chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// CTA b takes chunks first_of(b) .. first_of(b + 1) - 1: one run of the table, found once.
template <int N>
__device__ __forceinline__ int first_of(const ClipTable<N>& t, int b) {
  return (int)((int64_t)t.first[t.count] * b / (int)gridDim.x);
}

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }

template <typename T>
__device__ __forceinline__ void widen16(const uint4& u, float (&f)[16 / sizeof(T)]) {
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(v[i]);
    } else {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
}

// Values before p's first 16-byte boundary, at most n.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
  const int h = (int)(((16u - (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T));
  return h < n ? h : n;
}

template <typename T>
__device__ __forceinline__ double squares(const T* p, int n) {
  constexpr int V = 16 / sizeof(T);
  const int head = head_of(p, n), vecs = (n - head) / V;
  double a = 0.0, b = 0.0;
  for (int i = threadIdx.x; i < head; i += kClipThreads) {
    const double x = value(p + i);
    a = fma(x, x, a);
  }
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kClipBatch * kClipThreads) {
    uint4 u[kClipBatch];
#pragma unroll
    for (int k = 0; k < kClipBatch; ++k) u[k] = i0 + k * kClipThreads < vecs ? q[i0 + k * kClipThreads] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int k = 0; k < kClipBatch; ++k) {
      float f[V];
      widen16<T>(u[k], f);
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const double x = f[j], y = f[j + 1];
        a = fma(x, x, a);
        b = fma(y, y, b);
      }
    }
  }
  for (int i = head + vecs * V + threadIdx.x; i < n; i += kClipThreads) {
    const double x = value(p + i);
    b = fma(x, x, b);
  }
  return a + b;
}

__device__ __forceinline__ double block_sum(double v, double* s) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kClipThreads / 32; ++i) v += s[i];
  return v;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, 4) clip_norm_kernel(const __grid_constant__ ClipTable<N> t) {
  __shared__ double s[kClipThreads / 32];
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  const int lo = first_of(t, blockIdx.x), hi = first_of(t, blockIdx.x + 1);
  int i = lo < hi ? tensor_of(t, lo) : 0;
  for (int c = lo; c < hi; ++c) {
    while (c >= t.first[i + 1]) ++i;
    const int64_t at = (int64_t)(c - t.first[i]) * kClipChunk;
    const int n = (int)min((int64_t)kClipChunk, t.numel[i] - at);
    sum += t.bf16[i] ? squares(static_cast<const __nv_bfloat16*>(t.src[i]) + at, n)
                     : squares(static_cast<const float*>(t.src[i]) + at, n);
  }
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) t.part[t.part_at + blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void scaled(T* dst, const T* src, int n, float f) {
  constexpr int V = 16 / sizeof(T);
  const bool same = ((reinterpret_cast<uintptr_t>(dst) ^ reinterpret_cast<uintptr_t>(src)) & 15u) == 0;
  const int head = same ? head_of(src, n) : n, vecs = (n - head) / V;
  for (int i = threadIdx.x; i < head; i += kClipThreads) put(dst + i, value(src + i) * f);
  const uint4* q = reinterpret_cast<const uint4*>(src + head);
  uint4* o = reinterpret_cast<uint4*>(dst + head);
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kClipBatch * kClipThreads) {
    uint4 u[kClipBatch];
#pragma unroll
    for (int k = 0; k < kClipBatch; ++k)
      if (i0 + k * kClipThreads < vecs) u[k] = q[i0 + k * kClipThreads];
#pragma unroll
    for (int k = 0; k < kClipBatch; ++k) {
      if (i0 + k * kClipThreads >= vecs) break;
      float x[V];
      widen16<T>(u[k], x);
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          v[j] = __float_as_uint(x[j] * f);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j] * f, x[2 * j + 1] * f);
          v[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      __stcs(o + i0 + k * kClipThreads, make_uint4(v[0], v[1], v[2], v[3]));  // not read again here: leave L2 to the sources
    }
  }
  for (int i = head + vecs * V + threadIdx.x; i < n; i += kClipThreads) put(dst + i, value(src + i) * f);
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, 4) clip_scale_kernel(const __grid_constant__ ClipTable<N> t) {
  __shared__ double s[kClipThreads / 32];
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  for (int i = threadIdx.x; i < t.parts; i += kClipThreads) sum += t.part[i];
  const float norm = (float)sqrt(block_sum(sum, s));
  if (blockIdx.x == 0 && threadIdx.x == 0) *t.norm = norm;
  float f = t.max_norm / (norm + 1e-6f);
  if (!(f < 1.f) || !(norm < INFINITY)) f = 1.f;
  const int lo = first_of(t, blockIdx.x), hi = first_of(t, blockIdx.x + 1);
  int i = lo < hi ? tensor_of(t, hi - 1) : 0;
  for (int c = hi - 1; c >= lo; --c) {  // backwards: what the norm read last is still in L2
    while (c < t.first[i]) --i;
    if (f == 1.f && t.dst[i] == t.src[i]) continue;
    const int64_t at = (int64_t)(c - t.first[i]) * kClipChunk;
    const int n = (int)min((int64_t)kClipChunk, t.numel[i] - at);
    if (t.bf16[i])
      scaled(static_cast<__nv_bfloat16*>(t.dst[i]) + at, static_cast<const __nv_bfloat16*>(t.src[i]) + at, n, f);
    else
      scaled(static_cast<float*>(t.dst[i]) + at, static_cast<const float*>(t.src[i]) + at, n, f);
  }
}

int check_grads(const svconv_grad* g, int count) {
  if (count < 0 || count > (1 << 20)) return SVCONV_ERR_SIZE;
  if (count > 0 && !g) return SVCONV_ERR_NULL;
  for (int i = 0; i < count; ++i) {
    if (g[i].numel < 0 || g[i].numel > (1ll << 40)) return SVCONV_ERR_SIZE;
    if (g[i].dtype != SVCONV_F32 && g[i].dtype != SVCONV_BF16) return SVCONV_ERR_UNSUPPORTED;
    if (g[i].numel > 0 && (!g[i].src || !g[i].dst)) return SVCONV_ERR_NULL;
    const uintptr_t e = g[i].dtype == SVCONV_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(g[i].src) % e || reinterpret_cast<uintptr_t>(g[i].dst) % e) return SVCONV_ERR_ALIGN;
  }
  return SVCONV_OK;
}

// Fills a table with tensors from `from` on; returns how many entries of g it covers.  An empty
// tensor takes no slot.
template <int N>
int fill(ClipTable<N>& t, const svconv_grad* g, int from, int count) {
  t.count = 0;
  t.first[0] = 0;
  int i = from;
  for (; i < count && t.count < N; ++i) {
    if (g[i].numel == 0) continue;
    const int64_t chunks = (g[i].numel + kClipChunk - 1) / kClipChunk;
    if (t.first[t.count] + chunks > 0x7fffffff - 2 * kClipCtas) break;
    t.src[t.count] = g[i].src;
    t.dst[t.count] = g[i].dst;
    t.numel[t.count] = g[i].numel;
    t.bf16[t.count] = g[i].dtype == SVCONV_BF16;
    t.first[t.count + 1] = t.first[t.count] + (int)chunks;
    ++t.count;
  }
  return i - from;
}

template <int N>
int grid_of(const ClipTable<N>& t) {
  const int c = t.first[t.count];
  return c < 1 ? 1 : c > kClipCtas ? kClipCtas : c;
}

int launches_of(const svconv_grad* g, int count) {
  int tensors = 0;
  for (int i = 0; i < count; ++i) tensors += g[i].numel > 0;
  return tensors <= kClipSmall ? 1 : (tensors + kClipLarge - 1) / kClipLarge;
}

template <int N>
cudaError_t clip_run(const svconv_grad* g, int count, float max_norm, float* norm, double* part, cudaStream_t s) {
  ClipTable<N> t;
  t.part = part;
  t.max_norm = max_norm;
  t.norm = norm;
  const int launches = launches_of(g, count);
  int parts[2] = {0, 0};  // slots used; tables
  for (int pass = 0; pass < 2; ++pass) {
    t.part_at = 0;
    t.parts = parts[0];
    int from = 0, tables = 0;
    do {
      from += fill(t, g, from, count);
      const int grid = grid_of(t);
      const cudaError_t e = pass == 0 ? launch_pdl(clip_norm_kernel<N>, dim3(grid), dim3(kClipThreads), 0, s, t)
                                      : launch_pdl(clip_scale_kernel<N>, dim3(grid), dim3(kClipThreads), 0, s, t);
      if (e != cudaSuccess) return e;
      t.part_at += grid;
      ++tables;
    } while (from < count && tables < launches);
    parts[0] = t.part_at;
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace svc

using namespace svc;

extern "C" {

size_t svconv_clip_grads_workspace_size(const svconv_grad* grads, int count) {
  if (check_grads(grads, count)) return 0;
  return (size_t)launches_of(grads, count) * kClipCtas * sizeof(double);
}

int svconv_clip_grads(const svconv_grad* grads, int count, float max_norm, float* norm, void* workspace, size_t ws_bytes,
                      void* stream) {
  int rc = check_grads(grads, count);
  if (rc) return rc;
  if (!(max_norm >= 0.f)) return SVCONV_ERR_SIZE;
  if (!norm) return SVCONV_ERR_NULL;
  if (!workspace || ws_bytes < svconv_clip_grads_workspace_size(grads, count)) return SVCONV_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return SVCONV_ERR_ALIGN;
  if ((rc = check_device())) return rc;
  int tensors = 0;
  for (int i = 0; i < count; ++i) tensors += grads[i].numel > 0;
  double* part = static_cast<double*>(workspace);
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = tensors <= kClipSmall    ? clip_run<kClipSmall>(grads, count, max_norm, norm, part, s)
                        : tensors <= kClipMedium ? clip_run<kClipMedium>(grads, count, max_norm, norm, part, s)
                                                 : clip_run<kClipLarge>(grads, count, max_norm, norm, part, s);
  return e == cudaSuccess ? SVCONV_OK : SVCONV_ERR_CUDA;
}

}  // extern "C"
