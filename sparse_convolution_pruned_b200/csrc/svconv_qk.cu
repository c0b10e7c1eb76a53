// Per-head RMS norm with rotary positions, forward and backward (svconv_qk_norm_rope_fwd / _bwd).
//
// HBM-bound: each value is read once and written once (backward: two reads, one write) for ~10
// flops, so the work is to keep the instructions per value below what the loads take.  Both sides
// (queries and keys) share one launch, split over the CTAs by their bytes.  A warp owns whole tokens: its
// lanes form the sines and cosines of a token's pairs once and share them over all heads through shared
// memory.  A head's d channels lie in d / 8 lanes (padded to a power of two), each lane holding both members
// of its four pairs, so a norm is a few shuffles and a rotation none.  Four chunks per lane are in
// flight before the trigonometry starts.
//
// Angles: a pair's frequency in turns per position is kept as a 64-bit binary fraction; its product with the
// position, modulo one turn, is three integer operations and off by less than 2^-33 turns at any position.
// All other arithmetic is fp32 and rounds once, at the store.  The bf16 forms take sin.approx /
// cos.approx (error below 2^-20.9 on one turn, 2^-12 of a bf16 rounding), the fp32 forms sincospif.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "svconv_internal.h"
#include "svconv_ptx.cuh"

namespace svc {
namespace {

constexpr int kQkWarps = 8;
constexpr int kQkSms = 148;     // fixed numbers, so that the partial sums of dw need no device query
constexpr int kQkCtas = 4 * kQkSms;
constexpr int kQkMaxD = 256;
constexpr int kQkBatch = 4;     // chunks (8 channels a lane) in flight
constexpr int kQkMaxPairs = kQkMaxD / 2;

struct QkSide {
  const void *x, *dy;
  void* out;              // y (forward) or dx (backward)
  const int32_t* pos;
  const float* w;
  int64_t x_row;
  int n, H, ctas;
  int chunks;             // passes of a warp over a token's heads
};

struct QkParams {
  QkSide side[2];
  const double* freq;
  int d, pairs, axes, cut1, cut2;  // pairs below cut1 follow axis 0, below cut2 axis 1, the rest axis 2
  int lanes;                       // lanes per head (a power of two, 8 channels each)
  float eps;
  float* part;                     // backward: [ctas][d] partial sums of dw
};

// A lane's 8 channels of a head as loaded, from channels a and b on, four each: bf16 in 4 words, fp32 in 8
template <typename T>
struct Raw {
  uint32_t v[sizeof(T) * 2];
};

template <typename T, bool HALF>
__device__ __forceinline__ Raw<T> load8(const T* p, int a, int b) {
  Raw<T> r;
  if constexpr (sizeof(T) == 4) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p + a)), w = __ldcs(reinterpret_cast<const uint4*>(p + b));
    r.v[0] = u.x, r.v[1] = u.y, r.v[2] = u.z, r.v[3] = u.w, r.v[4] = w.x, r.v[5] = w.y, r.v[6] = w.z, r.v[7] = w.w;
  } else if constexpr (HALF) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p + a)), w = __ldcs(reinterpret_cast<const uint2*>(p + b));
    r.v[0] = u.x, r.v[1] = u.y, r.v[2] = w.x, r.v[3] = w.y;
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p + a));
    r.v[0] = u.x, r.v[1] = u.y, r.v[2] = u.z, r.v[3] = u.w;
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void widen(const Raw<T>& r, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(r.v[i] << 16);
      f[2 * i + 1] = __uint_as_float(r.v[i] & 0xffff0000u);
    }
  }
}

template <typename T, bool HALF>
__device__ __forceinline__ void store8(T* p, int a, int b, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4*>(p + a), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p + b), make_float4(f[4], f[5], f[6], f[7]));
  } else {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      v[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (HALF) {
      __stcs(reinterpret_cast<uint2*>(p + a), make_uint2(v[0], v[1]));
      __stcs(reinterpret_cast<uint2*>(p + b), make_uint2(v[2], v[3]));
    } else {
      __stcs(reinterpret_cast<uint4*>(p + a), make_uint4(v[0], v[1], v[2], v[3]));
    }
  }
}

__device__ __forceinline__ float sum_lanes(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Turn (INVERSE: back) the lane's four pairs by the angles at cs / sn: channels i and 4 + i, or 2i and 2i + 1.
template <bool HALF, bool INVERSE>
__device__ __forceinline__ void rotate(float (&f)[8], const float* cs, const float* sn) {
  const float4 c4 = *reinterpret_cast<const float4*>(cs), s4 = *reinterpret_cast<const float4*>(sn);
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float& a = f[HALF ? i : 2 * i];
    float& b = f[HALF ? 4 + i : 2 * i + 1];
    const float z = INVERSE ? -s[i] : s[i];
    const float t = a * c[i] - b * z;
    b = a * z + b * c[i];
    a = t;
  }
}

// One warp's share of a side: TPB tokens of kQkBatch / TPB chunks each per step (TPB = 1: as many
// steps per token as its chunks need).  dw gathers the lane's 8 channels of the weight gradient.
template <typename T, bool HALF, bool BWD, int TPB>
__device__ __forceinline__ void qk_tokens(const QkParams& p, const QkSide& sd, int cta, const unsigned long long* turn, float* cs,
                                          float* sn, float (&dw)[8]) {
  constexpr int CPB = kQkBatch / TPB;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (p.lanes - 1), hsub = lane / p.lanes, heads_per = 32 / p.lanes;
  const bool on = sub * 8 < p.d, turned = sub * 4 < p.pairs;
  const int a = HALF && turned ? sub * 4 : sub * 8, b = HALF && turned ? a + p.pairs : a + 4;
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = on ? (sd.w ? sd.w[i < 4 ? a + i : b + i - 4] : 1.f) : 0.f;
  const float inv_d = 1.f / (float)p.d;
  const T* x = static_cast<const T*>(sd.x);
  const T* dy = static_cast<const T*>(sd.dy);
  T* out = static_cast<T*>(sd.out);
  const int64_t step = (int64_t)sd.ctas * kQkWarps * TPB;
  for (int64_t t0 = ((int64_t)cta * kQkWarps + warp) * TPB; t0 < sd.n; t0 += step) {
    for (int ch0 = 0; ch0 < sd.chunks; ch0 += CPB) {
      Raw<T> rx[kQkBatch], rg[BWD ? kQkBatch : 1];
#pragma unroll
      for (int u = 0; u < kQkBatch; ++u) {
        const int64_t t = t0 + u / CPB;
        const int h = (ch0 + u % CPB) * heads_per + hsub;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) * 2; ++i) {
          rx[u].v[i] = 0u;
          if constexpr (BWD) rg[u].v[i] = 0u;
        }
        if (on && t < sd.n && h < sd.H) {
          rx[u] = load8<T, HALF>(x + t * sd.x_row + h * p.d, a, b);
          if constexpr (BWD) rg[u] = load8<T, HALF>(dy + (t * sd.H + h) * p.d, a, b);
        }
      }
      if (ch0 == 0) {
        __syncwarp();  // the previous step's readers are done
        const int total = TPB * p.pairs;
        for (int i = lane; i < total; i += 32) {
          const int tt = TPB == 1 ? 0 : i / p.pairs, pr = TPB == 1 ? i : i - tt * p.pairs;
          if (t0 + tt < sd.n) {
            const int axis = pr < p.cut1 ? 0 : pr < p.cut2 ? 1 : 2;
            const int pos = sd.pos[(t0 + tt) * p.axes + axis];
            const unsigned long long f = turn[pr];
            const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32);
            const uint32_t frac = hi * (uint32_t)pos + __umulhi(lo, (uint32_t)pos) - (pos < 0 ? lo : 0u);
            const float turns = (float)(int)frac * 2.3283064365386963e-10f;  // 2^-32: -1/2 .. 1/2
            if constexpr (sizeof(T) == 4) {
              sincospif(2.f * turns, &sn[i], &cs[i]);
            } else {
              sn[i] = __sinf(6.283185307179586f * turns);
              cs[i] = __cosf(6.283185307179586f * turns);
            }
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < kQkBatch; ++u) {
        const int64_t t = t0 + u / CPB;
        const int h = (ch0 + u % CPB) * heads_per + hsub;
        if (t >= sd.n || ch0 + u % CPB >= sd.chunks) continue;  // uniform over the warp
        const bool ok = on && h < sd.H;
        float f[8];
        widen(rx[u], f);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
        const float rstd = rsqrtf(sum_lanes(ss, p.lanes) * inv_d + p.eps);
        const float* tcs = cs + (u / CPB) * p.pairs + sub * 4;
        const float* tsn = sn + (u / CPB) * p.pairs + sub * 4;
        if constexpr (!BWD) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = f[i] * rstd * w[i];
          if (turned) rotate<HALF, false>(f, tcs, tsn);
          if (ok) store8<T, HALF>(out + (t * sd.H + h) * p.d, a, b, f);
        } else {
          float g[8];
          widen(rg[u], g);
          if (turned) rotate<HALF, true>(g, tcs, tsn);
          float dot = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[i] *= rstd;  // the normalised channel
            if (ok) dw[i] = fmaf(g[i], f[i], dw[i]);
            g[i] *= w[i];
            dot = fmaf(g[i], f[i], dot);
          }
          dot = sum_lanes(dot, p.lanes) * inv_d;
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = rstd * (g[i] - f[i] * dot);
          if (ok) store8<T, HALF>(out + (t * sd.H + h) * p.d, a, b, g);
        }
      }
    }
  }
}

// CTAs resident on an SM: as many as the registers of a variant allow without spills.
template <typename T, bool BWD>
constexpr int kQkPerSm = BWD ? (sizeof(T) == 4 ? 2 : 3) : (sizeof(T) == 4 ? 3 : 4);

// CTAs 0 .. side[0].ctas-1 take the queries, the rest the keys; a side's warps stride over its tokens.
template <typename T, bool HALF, bool BWD>
__global__ void __launch_bounds__(kQkWarps * 32, kQkPerSm<T, BWD>) qk_kernel(const __grid_constant__ QkParams p) {
  __shared__ __align__(16) float s_cs[kQkWarps][kQkBatch * kQkMaxPairs];
  __shared__ __align__(16) float s_sn[kQkWarps][kQkBatch * kQkMaxPairs];
  __shared__ unsigned long long s_turn[kQkMaxPairs];
  const int warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  if ((int)threadIdx.x < p.pairs) {
    const double t = p.freq[threadIdx.x] * 0.15915494309189533577;
    s_turn[threadIdx.x] = (unsigned long long)__double2ll_rn((t - rint(t)) * 18446744073709551616.0);
  }
  __syncthreads();
  const bool is_k = (int)blockIdx.x >= p.side[0].ctas;
  const QkSide& sd = p.side[is_k ? 1 : 0];
  const int cta = (int)blockIdx.x - (is_k ? p.side[0].ctas : 0);
  float dw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;
  if (sd.chunks == 1)
    qk_tokens<T, HALF, BWD, 4>(p, sd, cta, s_turn, s_cs[warp], s_sn[warp], dw);
  else if (sd.chunks == 2)
    qk_tokens<T, HALF, BWD, 2>(p, sd, cta, s_turn, s_cs[warp], s_sn[warp], dw);
  else
    qk_tokens<T, HALF, BWD, 1>(p, sd, cta, s_turn, s_cs[warp], s_sn[warp], dw);
  if constexpr (BWD) {
    // dw of this CTA: warps and head slots in a fixed order
    __shared__ float s_dw[kQkWarps][32][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s_dw[warp][threadIdx.x & 31][i] = dw[i];
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += kQkWarps * 32) {
      // the lane and place that held channel c
      int sub = c / 8, at = c % 8;
      if (HALF && c < 2 * p.pairs) {
        const int m = c < p.pairs ? c : c - p.pairs;
        sub = m / 4, at = m % 4 + (c < p.pairs ? 0 : 4);
      }
      float s = 0.f;
      for (int v = 0; v < kQkWarps; ++v)
        for (int h = 0; h < 32 / p.lanes; ++h) s += s_dw[v][h * p.lanes + sub][at];
      p.part[(size_t)blockIdx.x * p.d + c] = s;
    }
  }
}

// dw[c] of both sides: the CTAs' partial sums in a fixed order, in fp64.  Block b: side b / (d / 8), 8 channels.
__global__ void __launch_bounds__(256) qk_dw_kernel(const float* part, int d, int ctas_q, int ctas_k, float* dwq, float* dwk) {
  __shared__ double s[32][8];
  const int per = d / 8;
  const bool is_k = (int)blockIdx.x >= per;
  float* dw = is_k ? dwk : dwq;
  const int lo = is_k ? ctas_q : 0, hi = is_k ? ctas_q + ctas_k : ctas_q;
  const int c = ((int)blockIdx.x - (is_k ? per : 0)) * 8 + (threadIdx.x & 7), r = threadIdx.x >> 3;
  pdl_wait();
  pdl_trigger();
  double v = 0.0;
  for (int i = lo + r; i < hi; i += 32) v += (double)part[(size_t)i * d + c];
  s[r][threadIdx.x & 7] = v;
  __syncthreads();
  if (r == 0 && dw) {
    for (int i = 1; i < 32; ++i) v += s[i][threadIdx.x & 7];
    dw[c] = (float)v;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// CTAs of each side: as many as its tokens can use, at most `cap` in all, shared by bytes.
void split_ctas(QkParams& p, int cap) {
  int need[2];
  double bytes[2];
  for (int i = 0; i < 2; ++i) {
    const QkSide& s = p.side[i];
    const int tpb = s.chunks == 1 ? 4 : s.chunks == 2 ? 2 : 1;
    const int64_t c = ((int64_t)s.n + kQkWarps * tpb - 1) / (kQkWarps * tpb);
    need[i] = c > cap ? cap : (int)c;
    bytes[i] = (double)s.n * s.H;
  }
  if (need[0] + need[1] > cap) {
    int a = (int)(cap * (bytes[0] / (bytes[0] + bytes[1])) + 0.5);
    if (a < 1 && need[0] > 0) a = 1;
    if (a > cap - 1 && need[1] > 0) a = cap - 1;
    if (a > need[0]) a = need[0];
    need[0] = a;
    if (need[1] > cap - a) need[1] = cap - a;
  }
  p.side[0].ctas = need[0];
  p.side[1].ctas = need[1];
}

template <typename T, bool HALF, bool BWD>
cudaError_t launch_qk(QkParams& p, cudaStream_t s) {
  static_assert(kQkSms * kQkPerSm<T, BWD> <= kQkCtas, "the partial sums have kQkCtas slots");
  split_ctas(p, kQkSms * kQkPerSm<T, BWD>);
  const int grid = p.side[0].ctas + p.side[1].ctas;
  return grid == 0 ? cudaSuccess : launch_pdl(qk_kernel<T, HALF, BWD>, dim3(grid), dim3(kQkWarps * 32), 0, s, p);
}

int check_side(const svconv_qk_side& s, int dtype, int d, bool bwd) {
  if (s.n < 0 || s.H < 1 || s.H > 65535) return SVCONV_ERR_SIZE;
  if (s.n == 0) return SVCONV_OK;
  if (!s.x || !s.pos || (bwd ? (!s.dy || !s.dx) : !s.y)) return SVCONV_ERR_NULL;
  if (s.n > 1 && (s.x_row < (int64_t)s.H * d || s.x_row % 8 != 0)) return SVCONV_ERR_ALIGN;
  if (!aligned16(s.x) || !aligned16(s.y) || !aligned16(s.dy) || !aligned16(s.dx)) return SVCONV_ERR_ALIGN;
  if (!bwd && s.y == s.x && s.n > 1 && s.x_row != (int64_t)s.H * d) return SVCONV_ERR_ALIGN;  // in place: contiguous
  return SVCONV_OK;
}

int qk_run(bool bwd, int dtype, int d, int rot, int layout, const double* freq, int axes, const int32_t* axis_pairs,
           float eps, const svconv_qk_side* q, const svconv_qk_side* k, void* workspace, size_t ws_bytes,
           cudaStream_t s) {
  if (!q || !k || !axis_pairs) return SVCONV_ERR_NULL;
  if (dtype != SVCONV_F32 && dtype != SVCONV_BF16) return SVCONV_ERR_UNSUPPORTED;
  if (d < 8 || d > kQkMaxD || d % 8 != 0 || rot < 0 || rot > d || rot % 16 != 0) return SVCONV_ERR_UNSUPPORTED;
  if (layout != SVCONV_ROPE_HALF && layout != SVCONV_ROPE_INTERLEAVED) return SVCONV_ERR_UNSUPPORTED;
  if (axes < 1 || axes > 3 || !(eps >= 0.f) || std::isinf(eps)) return SVCONV_ERR_SIZE;
  int64_t pairs = 0;
  for (int a = 0; a < axes; ++a) {
    if (axis_pairs[a] < 0) return SVCONV_ERR_SIZE;
    pairs += axis_pairs[a];
  }
  if (pairs != rot / 2) return SVCONV_ERR_SIZE;
  const svconv_qk_side* sides[2] = {q, k};
  QkParams p{};
  for (int i = 0; i < 2; ++i) {
    const int rc = check_side(*sides[i], dtype, d, bwd);
    if (rc) return rc;
    const svconv_qk_side& c = *sides[i];
    p.side[i] = QkSide{c.x, c.dy, bwd ? c.dx : c.y, c.pos, c.w, c.x_row, c.n, c.H, 0, 0};
  }
  if (rot > 0 && !freq && q->n + (int64_t)k->n > 0) return SVCONV_ERR_NULL;
  if (bwd) {
    const size_t need = svconv_qk_norm_rope_bwd_workspace_size(d);
    if (!workspace || ws_bytes < need) return SVCONV_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SVCONV_ERR_ALIGN;
  }
  const int rc = check_device();
  if (rc) return rc;
  p.freq = freq;
  p.d = d;
  p.pairs = rot / 2;
  p.axes = axes;
  p.cut1 = axes > 1 ? axis_pairs[0] : p.pairs;
  p.cut2 = axes > 2 ? p.cut1 + axis_pairs[1] : p.pairs;
  p.lanes = 1;
  while (p.lanes < d / 8) p.lanes *= 2;
  const int heads_per = 32 / p.lanes;
  for (QkSide& sd : p.side) sd.chunks = (sd.H + heads_per - 1) / heads_per;
  p.eps = eps;
  p.part = static_cast<float*>(workspace);
  cudaError_t e;
  const bool half = layout == SVCONV_ROPE_HALF, f32 = dtype == SVCONV_F32;
  if (bwd)
    e = f32 ? (half ? launch_qk<float, true, true>(p, s) : launch_qk<float, false, true>(p, s))
            : (half ? launch_qk<__nv_bfloat16, true, true>(p, s) : launch_qk<__nv_bfloat16, false, true>(p, s));
  else
    e = f32 ? (half ? launch_qk<float, true, false>(p, s) : launch_qk<float, false, false>(p, s))
            : (half ? launch_qk<__nv_bfloat16, true, false>(p, s) : launch_qk<__nv_bfloat16, false, false>(p, s));
  if (e != cudaSuccess) return SVCONV_ERR_CUDA;
  if (bwd && (q->dw || k->dw))
    e = launch_pdl(qk_dw_kernel, dim3(2 * (d / 8)), dim3(256), 0, s, static_cast<const float*>(workspace), d, p.side[0].ctas,
                   p.side[1].ctas, q->dw, k->dw);
  return e == cudaSuccess ? SVCONV_OK : SVCONV_ERR_CUDA;
}

}  // namespace
}  // namespace svc

using namespace svc;

extern "C" {

size_t svconv_qk_norm_rope_bwd_workspace_size(int d) {
  if (d < 8 || d > kQkMaxD || d % 8 != 0) return 0;
  return (size_t)kQkCtas * d * sizeof(float);
}

int svconv_qk_norm_rope_fwd(int dtype, int d, int rot, int layout, const double* freq, int axes, const int32_t* axis_pairs,
                            float eps, const svconv_qk_side* q, const svconv_qk_side* k, void* stream) {
  return qk_run(false, dtype, d, rot, layout, freq, axes, axis_pairs, eps, q, k, nullptr, 0, (cudaStream_t)stream);
}

int svconv_qk_norm_rope_bwd(int dtype, int d, int rot, int layout, const double* freq, int axes, const int32_t* axis_pairs,
                            float eps, const svconv_qk_side* q, const svconv_qk_side* k, void* workspace, size_t ws_bytes,
                            void* stream) {
  return qk_run(true, dtype, d, rot, layout, freq, axes, axis_pairs, eps, q, k, workspace, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
