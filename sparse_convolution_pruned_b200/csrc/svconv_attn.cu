// Cross-attention of packed groups, forward and backward: every query row attends over the kept
// keys of its group (see svconv_cross_attn_fwd in svconv.h for the definition).
//
// CUDA-core form: one warp per (query row, head) forward and for dQ, one warp per (key row, key
// head) for dK and dV.  Scores are in base 2 (scale * log2 e folded into one factor).
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "svconv_internal.h"
#include "svconv_ptx.cuh"

namespace svc {
namespace {

constexpr int kMaxD = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 8;

struct AttnParams {
  const __nv_bfloat16 *Q, *K, *V, *O, *dO;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;
  int nq, nkv, Hq, Hkv, r, d, G;
  const int32_t *q_off, *kv_off;
  int max_q, max_kv;
  const uint8_t* keep;
  float scale;
  __nv_bfloat16 *Oout, *dQ, *dK, *dV;
  float* lse_out;
  const float* lse;
  float* D;
  int* status;
};

// Rows lo .. hi-1 of group g, clipped to the bound; flags for the status word.
__device__ __forceinline__ int group_range(const int32_t* off, int g, int n, int bound, int& lo, int& hi) {
  lo = off[g];
  hi = off[g + 1];
  if (lo < 0 || hi < lo || hi > n) {
    lo = hi = 0;
    return SVCONV_STATUS_BAD_OFFSETS;
  }
  if (hi - lo > bound) {
    hi = lo + bound;
    return SVCONV_STATUS_CHUNK_OVERFLOW;
  }
  return 0;
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
__device__ __forceinline__ float dot_row(const float* a, const __nv_bfloat16* b, int d) {
  float s = 0.f;
  for (int c = 0; c < d; c += 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(b + c);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      s = fmaf(a[c + 2 * i], f.x, s);
      s = fmaf(a[c + 2 * i + 1], f.y, s);
    }
  }
  return s;
}

__global__ void __launch_bounds__(kWarps * 32) attn_fwd_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float sq[kWarps][kMaxD];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = blockIdx.z, h = blockIdx.y;
  int q0, q1, k0, k1;
  const int flags = group_range(p.q_off, g, p.nq, p.max_q, q0, q1) | group_range(p.kv_off, g, p.nkv, p.max_kv, k0, k1);
  if (flags && threadIdx.x == 0 && blockIdx.x == 0 && h == 0) atomicOr(p.status, flags);
  if (flags & SVCONV_STATUS_BAD_OFFSETS) return;
  const int row = q0 + blockIdx.x * kWarps + w;
  if (row >= q1) return;
  for (int c = lane; c < p.d; c += 32)
    sq[w][c] = __bfloat162float(p.Q[row * p.q_row + h * p.q_head + c]) * (p.scale * kLog2e);
  __syncwarp();
  const int hk = h / p.r;
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = k0; j0 < k1; j0 += 32) {
    const int j = j0 + lane;
    const bool ok = j < k1 && (!p.keep || p.keep[j]);
    const float s = ok ? dot_row(sq[w], p.K + j * p.k_row + hk * p.k_head, p.d) : -INFINITY;
    const float mx = fmaxf(m, warp_max(s));
    if (mx == -INFINITY) continue;
    const float a = exp2f(m - mx), pr = ok ? exp2f(s - mx) : 0.f;
    l = l * a + warp_sum(pr);
    m = mx;
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] *= a;
    const unsigned kept = __ballot_sync(~0u, ok);
    for (int u = 0; u < 32; ++u) {
      const float pu = __shfl_sync(~0u, pr, u);
      if (!(kept >> u & 1)) continue;
      const __nv_bfloat16* v = p.V + (j0 + u) * p.v_row + hk * p.v_head;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (lane + 32 * c < p.d) acc[c] = fmaf(pu, __bfloat162float(v[lane + 32 * c]), acc[c]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* o = p.Oout + ((int64_t)row * p.Hq + h) * p.d;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < p.d) o[lane + 32 * c] = __float2bfloat16(l == 0.f ? 0.f : acc[c] * inv);
  if (lane == 0) p.lse_out[(int64_t)row * p.Hq + h] = (m == -INFINITY) ? -INFINITY : (m + log2f(l)) * kLn2;
}

__global__ void __launch_bounds__(kWarps * 32) attn_dq_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float sq[kWarps][kMaxD], sdo[kWarps][kMaxD];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = blockIdx.z, h = blockIdx.y;
  int q0, q1, k0, k1;
  const int flags = group_range(p.q_off, g, p.nq, p.max_q, q0, q1) | group_range(p.kv_off, g, p.nkv, p.max_kv, k0, k1);
  if (flags && threadIdx.x == 0 && blockIdx.x == 0 && h == 0) atomicOr(p.status, flags);
  if (flags & SVCONV_STATUS_BAD_OFFSETS) return;
  const int row = q0 + blockIdx.x * kWarps + w;
  if (row >= q1) return;
  const int64_t at = ((int64_t)row * p.Hq + h);
  float D = 0.f;
  for (int c = lane; c < p.d; c += 32) {
    sq[w][c] = __bfloat162float(p.Q[row * p.q_row + h * p.q_head + c]) * (p.scale * kLog2e);
    const float go = __bfloat162float(p.dO[at * p.d + c]);
    sdo[w][c] = go;
    D = fmaf(go, __bfloat162float(p.O[at * p.d + c]), D);
  }
  D = warp_sum(D);
  __syncwarp();
  if (lane == 0) p.D[at] = D;
  const int hk = h / p.r;
  const float lse2 = p.lse[at] * kLog2e;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = k0; j0 < k1; j0 += 32) {
    const int j = j0 + lane;
    const bool ok = j < k1 && (!p.keep || p.keep[j]);
    float ds = 0.f;
    if (ok) {
      const float s = dot_row(sq[w], p.K + j * p.k_row + hk * p.k_head, p.d);
      ds = exp2f(s - lse2) * (dot_row(sdo[w], p.V + j * p.v_row + hk * p.v_head, p.d) - D);
    }
    const unsigned kept = __ballot_sync(~0u, ok);
    for (int u = 0; u < 32; ++u) {
      const float du = __shfl_sync(~0u, ds, u);
      if (!(kept >> u & 1)) continue;
      const __nv_bfloat16* k = p.K + (j0 + u) * p.k_row + hk * p.k_head;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (lane + 32 * c < p.d) acc[c] = fmaf(du, __bfloat162float(k[lane + 32 * c]), acc[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < p.d) p.dQ[at * p.d + lane + 32 * c] = __float2bfloat16(acc[c] * p.scale);
}

__global__ void __launch_bounds__(kWarps * 32) attn_dkv_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float sk[kWarps][kMaxD], sv[kWarps][kMaxD];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = blockIdx.z, hk = blockIdx.y;
  int q0, q1, k0, k1;
  const int flags = group_range(p.q_off, g, p.nq, p.max_q, q0, q1) | group_range(p.kv_off, g, p.nkv, p.max_kv, k0, k1);
  if (flags & SVCONV_STATUS_BAD_OFFSETS) return;
  const int row = k0 + blockIdx.x * kWarps + w;
  if (row >= k1) return;
  const bool on = !p.keep || p.keep[row];
  float dk[4] = {0.f, 0.f, 0.f, 0.f}, dv[4] = {0.f, 0.f, 0.f, 0.f};
  if (on) {
    for (int c = lane; c < p.d; c += 32) {
      sk[w][c] = __bfloat162float(p.K[row * p.k_row + hk * p.k_head + c]) * (p.scale * kLog2e);
      sv[w][c] = __bfloat162float(p.V[row * p.v_row + hk * p.v_head + c]);
    }
    __syncwarp();
    const int n = (q1 - q0) * p.r;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      float pr = 0.f, ds = 0.f;
      if (i < n) {
        const int qi = q0 + i / p.r, h = hk * p.r + i % p.r;
        const int64_t at = (int64_t)qi * p.Hq + h;
        pr = exp2f(dot_row(sk[w], p.Q + qi * p.q_row + h * p.q_head, p.d) - p.lse[at] * kLog2e);
        ds = pr * (dot_row(sv[w], p.dO + at * p.d, p.d) - p.D[at]);
      }
      for (int u = 0; u < 32 && i0 + u < n; ++u) {
        const float pu = __shfl_sync(~0u, pr, u), du = __shfl_sync(~0u, ds, u);
        const int qi = q0 + (i0 + u) / p.r, h = hk * p.r + (i0 + u) % p.r;
        const __nv_bfloat16* q = p.Q + qi * p.q_row + h * p.q_head;
        const __nv_bfloat16* go = p.dO + ((int64_t)qi * p.Hq + h) * p.d;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (lane + 32 * c < p.d) {
            dk[c] = fmaf(du, __bfloat162float(q[lane + 32 * c]), dk[c]);
            dv[c] = fmaf(pu, __bfloat162float(go[lane + 32 * c]), dv[c]);
          }
      }
    }
  }
  const int64_t at = ((int64_t)row * p.Hkv + hk) * p.d;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < p.d) {
      p.dK[at + lane + 32 * c] = __float2bfloat16(dk[c] * p.scale);
      p.dV[at + lane + 32 * c] = __float2bfloat16(dv[c]);
    }
}

// ---------------------------------------------------------------------------- host side
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Strides of an operand with `heads` heads and `n` rows: the ones that are never used (a single
// head or row) are replaced, so whatever a caller's view carries there is accepted.
bool fix_strides(int64_t& row, int64_t& head, int n, int heads, int d) {
  if (heads == 1) head = d;
  if (n <= 1) row = (int64_t)heads * (head > d ? head : d);
  return row > 0 && head > 0 && row % 8 == 0 && head % 8 == 0 && row < (1ll << 38) && head < (1ll << 38);
}

int check_desc(const svconv_cross_attn_desc* c, svconv_cross_attn_desc& o) {
  if (!c) return SVCONV_ERR_NULL;
  o = *c;
  if (o.nq < 0 || o.nkv < 0 || o.G < 0 || o.max_q < 0 || o.max_kv < 0) return SVCONV_ERR_SIZE;
  if (o.Hq < 1 || o.Hkv < 1 || o.Hq > 65535 || o.G > 65535) return SVCONV_ERR_SIZE;
  if (o.d < 8 || o.d > kMaxD || o.d % 8 != 0 || o.Hq % o.Hkv != 0 || o.Hq / o.Hkv > 128) return SVCONV_ERR_UNSUPPORTED;
  if (!std::isfinite(o.scale)) return SVCONV_ERR_SIZE;
  if (o.G > 0 && (!o.q_off || !o.kv_off)) return SVCONV_ERR_NULL;
  if (!fix_strides(o.q_row, o.q_head, o.nq, o.Hq, o.d) || !fix_strides(o.k_row, o.k_head, o.nkv, o.Hkv, o.d) ||
      !fix_strides(o.v_row, o.v_head, o.nkv, o.Hkv, o.d))
    return SVCONV_ERR_ALIGN;
  if (o.max_q > o.nq) o.max_q = o.nq;
  if (o.max_kv > o.nkv) o.max_kv = o.nkv;
  return SVCONV_OK;
}

AttnParams make_params(const svconv_cross_attn_desc& c, const void* Q, const void* K, const void* V, int* status) {
  AttnParams p{};
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.K = static_cast<const __nv_bfloat16*>(K);
  p.V = static_cast<const __nv_bfloat16*>(V);
  p.q_row = c.q_row, p.q_head = c.q_head, p.k_row = c.k_row, p.k_head = c.k_head, p.v_row = c.v_row, p.v_head = c.v_head;
  p.nq = c.nq, p.nkv = c.nkv, p.Hq = c.Hq, p.Hkv = c.Hkv, p.r = c.Hq / c.Hkv, p.d = c.d, p.G = c.G;
  p.q_off = c.q_off, p.kv_off = c.kv_off, p.max_q = c.max_q, p.max_kv = c.max_kv, p.keep = c.kv_keep, p.scale = c.scale;
  p.status = status ? status : device_error_word();
  return p;
}

int cdiv(int a, int b) { return (int)(((long long)a + b - 1) / b); }

}  // namespace
}  // namespace svc

using namespace svc;

extern "C" {

size_t svconv_cross_attn_fwd_workspace_size(const svconv_cross_attn_desc*) { return 0; }

size_t svconv_cross_attn_bwd_workspace_size(const svconv_cross_attn_desc* desc) {
  svconv_cross_attn_desc c;
  if (check_desc(desc, c)) return 0;
  return ((size_t)c.nq * c.Hq * sizeof(float) + 15) / 16 * 16;
}

int svconv_cross_attn_fwd(const svconv_cross_attn_desc* desc, const void* Q, const void* K, const void* V, void* O,
                          float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  svconv_cross_attn_desc c;
  int rc = check_desc(desc, c);
  if (rc) return rc;
  if (c.G == 0 || c.max_q == 0) return SVCONV_OK;
  if (!Q || !O || !lse || (c.nkv > 0 && (!K || !V))) return SVCONV_ERR_NULL;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned16(workspace)) return SVCONV_ERR_ALIGN;
  const size_t need = svconv_cross_attn_fwd_workspace_size(desc);
  if (need && (!workspace || ws_bytes < need)) return SVCONV_ERR_WORKSPACE;
  if ((rc = check_device())) return rc;
  AttnParams p = make_params(c, Q, K, V, dev_status);
  p.Oout = static_cast<__nv_bfloat16*>(O);
  p.lse_out = lse;
  attn_fwd_kernel<<<dim3(cdiv(c.max_q, kWarps), c.Hq, c.G), kWarps * 32, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SVCONV_OK : SVCONV_ERR_CUDA;
}

int svconv_cross_attn_bwd(const svconv_cross_attn_desc* desc, const void* dO, const void* Q, const void* K,
                          const void* V, const void* O, const float* lse, void* dQ, void* dK, void* dV,
                          void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  svconv_cross_attn_desc c;
  int rc = check_desc(desc, c);
  if (rc) return rc;
  if (c.G == 0 || (c.max_q == 0 && c.max_kv == 0)) return SVCONV_OK;
  if (c.nq > 0 && (!dO || !Q || !O || !lse || !dQ)) return SVCONV_ERR_NULL;
  if (c.nkv > 0 && (!K || !V || !dK || !dV)) return SVCONV_ERR_NULL;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned16(dO) || !aligned16(dQ) ||
      !aligned16(dK) || !aligned16(dV) || !aligned16(workspace))
    return SVCONV_ERR_ALIGN;
  const size_t need = svconv_cross_attn_bwd_workspace_size(desc);
  if (need && (!workspace || ws_bytes < need)) return SVCONV_ERR_WORKSPACE;
  if ((rc = check_device())) return rc;
  AttnParams p = make_params(c, Q, K, V, dev_status);
  p.O = static_cast<const __nv_bfloat16*>(O);
  p.dO = static_cast<const __nv_bfloat16*>(dO);
  p.lse = lse;
  p.dQ = static_cast<__nv_bfloat16*>(dQ);
  p.dK = static_cast<__nv_bfloat16*>(dK);
  p.dV = static_cast<__nv_bfloat16*>(dV);
  p.D = static_cast<float*>(workspace);
  cudaStream_t s = (cudaStream_t)stream;
  if (c.max_q > 0) attn_dq_kernel<<<dim3(cdiv(c.max_q, kWarps), c.Hq, c.G), kWarps * 32, 0, s>>>(p);
  if (c.max_kv > 0) attn_dkv_kernel<<<dim3(cdiv(c.max_kv, kWarps), c.Hkv, c.G), kWarps * 32, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? SVCONV_OK : SVCONV_ERR_CUDA;
}

}  // extern "C"
