// Per-head RMS norm with rotary positions, forward and backward (svconv_qk_norm_rope_fwd / _bwd).
//
// HBM-bound: each value is read once and written once (backward: two reads, one write) for ~10
// flops, so the work is to keep the instructions per value below what the loads take.  Both sides
// (queries and keys) share one launch, split over the CTAs by their bytes.  A warp owns whole tokens: its
// lanes form the sines and cosines of a token's pairs once and share them over all heads through shared
// memory.  A head's d channels lie in d / 8 lanes (padded to a power of two), each lane holding both members
// of its four pairs, so a norm is a few shuffles and a rotation none.  Tokens of fewer than 256 channels in all leave lanes
// idle: one head of 64 runs at a third of the bytes per second of four (1.3 and 4.1 TB/s forward).  Four chunks per lane are in
// flight before the trigonometry starts.
//
// Angles: a pair's frequency in turns per position, formed in two doubles, is kept as a 64-bit binary fraction (off by
// 2^-64); its product with the position, modulo one turn and rounded to 32 bits, is three integer operations and off by
// less than 2^-32 turns + 2^-64 turns a position, 2^-31 at the farthest.  The fp32 forms take the quarter turn off as an
// integer, so that 24 bits hold the rest (2^-27 of half a turn), and sincospif; the bf16 forms round the
// whole fraction to 24 bits and take sin.approx / cos.approx (error below 2^-20.9 on one turn, 2^-12 of a bf16 rounding).
// All other arithmetic is fp32 and rounds once, at the store.
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
constexpr double kTwo64 = 18446744073709551616.0;
constexpr double kInvTwoPi = 0.15915494309189535, kInvTwoPiRest = -9.839338337591243e-18;  // 1 / (2 pi) in two doubles

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

// Two fp32 values that one instruction handles together
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A lane's four pairs of a head: first members in a[0], a[1], second ones in b[0], b[1].
struct Pairs {
  f2 a[2], b[2];
};

// The same as loaded (bf16 in 4 words, fp32 in 8): for the half layout four channels from a and four from b on,
// for the interleaved one the eight channels from a on.
template <typename T>
struct Raw {
  uint32_t v[sizeof(T) * 2];
};

template <typename T, bool HALF>
__device__ __forceinline__ Raw<T> load8(const T* p, int b_off) {
  Raw<T> r;
  if constexpr (sizeof(T) == 4) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p)), w = __ldcs(reinterpret_cast<const uint4*>(p + b_off));
    r.v[0] = u.x, r.v[1] = u.y, r.v[2] = u.z, r.v[3] = u.w, r.v[4] = w.x, r.v[5] = w.y, r.v[6] = w.z, r.v[7] = w.w;
  } else if constexpr (HALF) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p)), w = __ldcs(reinterpret_cast<const uint2*>(p + b_off));
    r.v[0] = u.x, r.v[1] = u.y, r.v[2] = w.x, r.v[3] = w.y;
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    r.v[0] = u.x, r.v[1] = u.y, r.v[2] = u.z, r.v[3] = u.w;
  }
  return r;
}

template <typename T, bool HALF>
__device__ __forceinline__ Pairs widen(const Raw<T>& r) {
  float f[8];
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
  Pairs v;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v.a[i] = HALF ? pack2(f[2 * i], f[2 * i + 1]) : pack2(f[4 * i], f[4 * i + 2]);
    v.b[i] = HALF ? pack2(f[4 + 2 * i], f[5 + 2 * i]) : pack2(f[4 * i + 1], f[4 * i + 3]);
  }
  return v;
}

template <typename T, bool HALF>
__device__ __forceinline__ void store8(T* p, int b_off, const Pairs& v) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    unpack2(v.a[i], f[HALF ? 2 * i : 4 * i], f[HALF ? 2 * i + 1 : 4 * i + 2]);
    unpack2(v.b[i], f[HALF ? 4 + 2 * i : 4 * i + 1], f[HALF ? 5 + 2 * i : 4 * i + 3]);
  }
  if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p + b_off), make_float4(f[4], f[5], f[6], f[7]));
  } else {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (HALF) {
      __stcs(reinterpret_cast<uint2*>(p), make_uint2(u[0], u[1]));
      __stcs(reinterpret_cast<uint2*>(p + b_off), make_uint2(u[2], u[3]));
    } else {
      __stcs(reinterpret_cast<uint4*>(p), make_uint4(u[0], u[1], u[2], u[3]));
    }
  }
}

// Sum over the lanes of a head; LANES: known when compiling, or 0.
template <int LANES>
__device__ __forceinline__ float sum_lanes(float v, int lanes) {
  if constexpr (LANES > 0) {
#pragma unroll
    for (int o = LANES >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  } else {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

__device__ __forceinline__ float dot8(const Pairs& x, const Pairs& y) {
  f2 s = mul2(x.a[0], y.a[0]);
  s = fma2(x.a[1], y.a[1], s);
  s = fma2(x.b[0], y.b[0], s);
  s = fma2(x.b[1], y.b[1], s);
  float lo, hi;
  unpack2(s, lo, hi);
  return lo + hi;
}

// Turn (INVERSE: back) the lane's four pairs by the angles at cs / sn.
template <bool INVERSE>
__device__ __forceinline__ void rotate(Pairs& v, const float* cs, const float* sn) {
  const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(cs), s = *reinterpret_cast<const ulonglong2*>(sn);
  const f2 minus = pack2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f2 ci = i ? c.y : c.x, si = i ? s.y : s.x, ni = mul2(si, minus);
    const f2 a = v.a[i];
    v.a[i] = fma2(a, ci, mul2(v.b[i], INVERSE ? si : ni));
    v.b[i] = fma2(v.b[i], ci, mul2(a, INVERSE ? ni : si));
  }
}

// sine and cosine of pos times a frequency (a binary fraction of a turn per position)
template <typename T>
__device__ __forceinline__ void turn_by(unsigned long long f, int pos, float& s, float& c) {
  const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32);
  const uint32_t low = (uint32_t)(((unsigned long long)lo * (uint32_t)pos + 0x80000000ull) >> 32);  // rounded
  const uint32_t frac = hi * (uint32_t)pos + low - (pos < 0 ? lo : 0u);
  if constexpr (sizeof(T) == 4) {
    const uint32_t q = frac + 0x20000000u;  // the nearest quarter turn in the top two bits
    float sr, cr;
    sincospif((float)(int)(frac - (q & 0xc0000000u)) * 4.656612873077393e-10f, &sr, &cr);  // 2^-31: over pi, -1/4 .. 1/4
    s = q & 0x40000000u ? cr : sr;
    c = q & 0x40000000u ? sr : cr;
    if (q & 0x80000000u) s = -s;
    if ((q + 0x40000000u) & 0x80000000u) c = -c;
  } else {
    const float x = (float)(int)frac * 1.4629180792671596e-9f;  // 2 pi 2^-32
    s = __sinf(x);
    c = __cosf(x);
  }
}

// One warp's share of a side: TPB tokens of kQkBatch / TPB chunks each per step (TPB = 1: as many
// steps per token as its chunks need).  dw gathers the lane's share of the weight gradient.
template <typename T, bool HALF, bool BWD, int LANES, int TPB>
__device__ __forceinline__ void qk_tokens(const QkParams& p, const QkSide& side, int cta, const unsigned long long* turn, float* cs,
                                          float* sn, Pairs& dw) {
  constexpr int CPB = kQkBatch / TPB;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = LANES > 0 ? LANES : p.lanes;
  const int sub = lane & (lanes - 1), hsub = lane / lanes, heads_per = 32 / lanes;
  const int n = side.n, H = side.H, d = p.d, pairs = p.pairs, axes = p.axes, chunks = side.chunks;
  const bool on = sub * 8 < d, turned = sub * 4 < pairs;
  const int a = on ? (HALF && turned ? sub * 4 : sub * 8) : 0, b_off = HALF && turned ? pairs : 4;
  Pairs w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = 2 * i + k;
      f[k] = side.w ? side.w[HALF ? a + at : a + 2 * at] : 1.f;
      f[2 + k] = side.w ? side.w[HALF ? a + b_off + at : a + 2 * at + 1] : 1.f;
    }
    w.a[i] = pack2(f[0], f[1]);
    w.b[i] = pack2(f[2], f[3]);
  }
  const float inv_d = 1.f / (float)d, eps = p.eps;
  const int64_t x_row = side.x_row, row = (int64_t)H * d;
  const int64_t first = (int64_t)(cta * kQkWarps + warp) * TPB, step = (int64_t)side.ctas * kQkWarps * TPB;
  // lanes without a channel, a head or a token of their own load another's (in bounds) and store nothing
  const T* x = static_cast<const T*>(side.x) + first * x_row + a;
  const T* dy = BWD ? static_cast<const T*>(side.dy) + first * row + a : nullptr;
  T* out = static_cast<T*>(side.out) + first * row + a;
  const int32_t* pos = side.pos + first * axes;
  const unsigned long long turn0 = lane < pairs ? turn[lane] : 0;
  const int axis0 = lane < p.cut1 ? 0 : lane < p.cut2 ? 1 : 2;
  for (int64_t t0 = first; t0 < n; t0 += step, x += step * x_row, out += step * row, pos += step * axes) {
    const int last = (int)min((int64_t)TPB, n - t0) - 1;  // the last token of the step
    for (int ch0 = 0; ch0 < chunks; ch0 += CPB) {
      Raw<T> rx[kQkBatch], rg[BWD ? kQkBatch : 1];
      {
        const T *px = x, *pg = dy;
#pragma unroll
        for (int u = 0; u < TPB; ++u) {
#pragma unroll
          for (int c = 0; c < CPB; ++c) {
            const int at = min((ch0 + c) * heads_per + hsub, H - 1) * d;
            rx[u * CPB + c] = load8<T, HALF>(px + at, b_off);
            if constexpr (BWD) rg[u * CPB + c] = load8<T, HALF>(pg + at, b_off);
          }
          if (u < last) {
            px += x_row;
            if constexpr (BWD) pg += row;
          }
        }
      }
      if (ch0 == 0) {
        __syncwarp();  // the previous step's readers are done
        const int32_t* pp = pos;
#pragma unroll
        for (int u = 0; u < TPB; ++u) {
          if (lane < pairs) turn_by<T>(turn0, pp[axis0], sn[u * pairs + lane], cs[u * pairs + lane]);
          for (int i = lane + 32; i < pairs; i += 32)
            turn_by<T>(turn[i], pp[i < p.cut1 ? 0 : i < p.cut2 ? 1 : 2], sn[u * pairs + i], cs[u * pairs + i]);
          if (u < last) pp += axes;
        }
        __syncwarp();
      }
      T* po = out;
#pragma unroll
      for (int u = 0; u < TPB; ++u) {
        if (u > last) break;  // uniform over the warp
        const float* tcs = cs + u * pairs + sub * 4;
        const float* tsn = sn + u * pairs + sub * 4;
#pragma unroll
        for (int c = 0; c < CPB; ++c) {
          if (CPB > 1 && ch0 + c >= chunks) break;  // uniform over the warp
          const int h = (ch0 + c) * heads_per + hsub;
          const bool ok = on && h < H;
          Pairs f = widen<T, HALF>(rx[u * CPB + c]);
          const float ss = dot8(f, f);
          const float rstd = rsqrtf(fmaf(sum_lanes<LANES>(LANES > 0 || on ? ss : 0.f, lanes), inv_d, eps));
          const f2 r2 = pack2(rstd, rstd);
#pragma unroll
          for (int i = 0; i < 2; ++i) f.a[i] = mul2(f.a[i], r2), f.b[i] = mul2(f.b[i], r2);  // the normalised channels
          if constexpr (!BWD) {
#pragma unroll
            for (int i = 0; i < 2; ++i) f.a[i] = mul2(f.a[i], w.a[i]), f.b[i] = mul2(f.b[i], w.b[i]);
            if (turned) rotate<false>(f, tcs, tsn);
            if (ok) store8<T, HALF>(po + h * d, b_off, f);
          } else {
            Pairs g = widen<T, HALF>(rg[u * CPB + c]);
            if (turned) rotate<true>(g, tcs, tsn);
            if (ok) {
#pragma unroll
              for (int i = 0; i < 2; ++i) dw.a[i] = fma2(g.a[i], f.a[i], dw.a[i]), dw.b[i] = fma2(g.b[i], f.b[i], dw.b[i]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) g.a[i] = mul2(g.a[i], w.a[i]), g.b[i] = mul2(g.b[i], w.b[i]);
            const float dot = dot8(g, f);
            const float m = -sum_lanes<LANES>(LANES > 0 || on ? dot : 0.f, lanes) * inv_d;
            const f2 m2 = pack2(m, m);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              g.a[i] = mul2(r2, fma2(f.a[i], m2, g.a[i]));
              g.b[i] = mul2(r2, fma2(f.b[i], m2, g.b[i]));
            }
            if (ok) store8<T, HALF>(po + h * d, b_off, g);
          }
        }
        po += row;
      }
    }
    if constexpr (BWD) dy += step * row;
  }
}

// CTAs resident on an SM.  Two for the fp32 backward, whose registers allow no third without spills.  The bf16 backward
// spills 150 to 280 bytes a thread at three: 112 us against 126 with two for 49,152 x 8 and 98,317 x 2 heads of 128 (interleaved),
// 64 against 58 at 4 heads of 64, 124 against 111 at 80 (half).
template <typename T, bool BWD>
constexpr int kQkPerSm = BWD && sizeof(T) == 4 ? 2 : 3;

// CTAs 0 .. side[0].ctas-1 take the queries, the rest the keys; a side's warps stride over its tokens.
template <typename T, bool HALF, bool BWD, int LANES>
__global__ void __launch_bounds__(kQkWarps * 32, kQkPerSm<T, BWD>) qk_kernel(const __grid_constant__ QkParams p) {
  __shared__ __align__(16) float s_cs[kQkWarps][kQkBatch * kQkMaxPairs];
  __shared__ __align__(16) float s_sn[kQkWarps][kQkBatch * kQkMaxPairs];
  __shared__ unsigned long long s_turn[kQkMaxPairs];
  const int warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  if ((int)threadIdx.x < p.pairs) {
    // freq / (2 pi) as t + rest: the product's rounding error, and the part of 1 / (2 pi) that one double leaves out
    const double f = p.freq[threadIdx.x], t = f * kInvTwoPi, rest = fma(f, kInvTwoPi, -t) + f * kInvTwoPiRest;
    s_turn[threadIdx.x] = (unsigned long long)__double2ll_rn((t - rint(t)) * kTwo64) + (unsigned long long)__double2ll_rn(rest * kTwo64);
  }
  __syncthreads();
  const bool is_k = (int)blockIdx.x >= p.side[0].ctas;
  const QkSide& sd = p.side[is_k ? 1 : 0];
  const int cta = (int)blockIdx.x - (is_k ? p.side[0].ctas : 0);
  Pairs dw = {{0ull, 0ull}, {0ull, 0ull}};
  if (sd.chunks == 1)
    qk_tokens<T, HALF, BWD, LANES, 4>(p, sd, cta, s_turn, s_cs[warp], s_sn[warp], dw);
  else if (sd.chunks == 2)
    qk_tokens<T, HALF, BWD, LANES, 2>(p, sd, cta, s_turn, s_cs[warp], s_sn[warp], dw);
  else
    qk_tokens<T, HALF, BWD, LANES, 1>(p, sd, cta, s_turn, s_cs[warp], s_sn[warp], dw);
  if constexpr (BWD) {
    // dw of this CTA: warps and head slots in a fixed order
    __shared__ float s_dw[kQkWarps][32][8];
    float* mine = s_dw[warp][threadIdx.x & 31];  // first members, then second ones
#pragma unroll
    for (int i = 0; i < 2; ++i) unpack2(dw.a[i], mine[2 * i], mine[2 * i + 1]), unpack2(dw.b[i], mine[4 + 2 * i], mine[5 + 2 * i]);
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += kQkWarps * 32) {
      // the lane and place that held channel c
      int sub = c / 8, at = HALF ? c % 8 : c % 8 / 2 + c % 2 * 4;
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
  if (grid == 0) return cudaSuccess;
  const dim3 g(grid), b(kQkWarps * 32);
  // 64 and 128 channels (whole lane groups of a known size) have loops without a runtime bound
  if (p.d == 64) return launch_pdl(qk_kernel<T, HALF, BWD, 8>, g, b, 0, s, p);
  if (p.d == 128) return launch_pdl(qk_kernel<T, HALF, BWD, 16>, g, b, 0, s, p);
  return launch_pdl(qk_kernel<T, HALF, BWD, 0>, g, b, 0, s, p);
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
