// Cross-attention of packed groups, forward and backward: every query row attends over the kept
// keys of its group (see svconv_cross_attn_fwd in svconv.h for the definition).
//
// CUDA-core form: one warp per (query row, head) forward and for dQ, one warp per (key row, key
// head) for dK and dV.  Scores are in base 2 (scale * log2 e folded into one factor).
#include <cuda.h>
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
  __nv_bfloat16 *dQ, *dK, *dV;
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

// ============================================================================ tensor-core building blocks
constexpr int kTile = 128;             // query rows (query tokens x their r heads) and keys of a tile
constexpr int kBlockBytes = kTile * 128;  // 128 rows of 64 bf16 channels, 128-byte swizzled
constexpr int kSoftWarps = 8;          // two softmax warpgroups, one per stream
constexpr int kFwdThreads = (kSoftWarps + 2) * 32;
constexpr int kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          dst),
      "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The whole warp waits: lane 0 polls, the verdict is broadcast (control flow stays warp-uniform).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_flag, err, kDefaultTimeoutNs);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// 32 lanes x 16 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Zero the rows of a tile that must not reach a product (0 x NaN): bit j of drop[w] is row 32 w + j.
// One warp; a row is 128 contiguous bytes of each 64-channel block whatever the swizzle.
__device__ __forceinline__ void scrub_rows(uint32_t tile, int blocks, const uint32_t (&drop)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (drop[w] >> lane & 1u)
      for (int b = 0; b < blocks; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) st_shared_16(tile + b * kBlockBytes + (32 * w + lane) * 128 + ((i + lane) & 7) * 16, 0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Keys of the tile starting at row j0 of the group (k0 .. k1-1) that take part, as four words.  The whole warp calls.
__device__ __forceinline__ void kept_words(const uint8_t* keep, int j0, int k1, uint32_t (&word)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int j = j0 + 32 * w + lane;
    word[w] = __ballot_sync(0xffffffffu, j < k1 && (!keep || __ldg(keep + j) != 0));
  }
}

// ============================================================================ forward
// Two streams of 128-row score tiles run through one CTA, a softmax warpgroup each, so that one
// stream's exponentials overlap the other's matrix products:
//   pair form   (many queries)  the streams are two query tiles and share every key tile;
//   split form  (few queries)   one query tile; the streams take alternate key tiles and are
//                               merged through shared memory at the end.
// A row of a tile is one (query token, head of the key head's group), so heads that share a key
// head share its loads.  Per stream and key tile: S = Q K^T into tensor memory, one thread per row
// reads its 128 scores, updates the running maximum, writes P = exp2(S - m) as bf16 to tensor
// memory, and O += P V follows with P as the A operand.  O stays in tensor memory and is rescaled
// only when a row's maximum has risen by more than 2^kRescaleLog2.
constexpr float kRescaleLog2 = 8.f;

struct FwdParams {
  CUtensorMap tq, tk, tv;
  const int32_t *q_off, *kv_off;
  const uint8_t* keep;
  int nq, nkv, max_q, max_kv, Hq, Hkv, r, d;
  int tokens;       // query tokens of a tile: 128 / r
  int qblocks, splits, pair;
  float c;          // scale * log2(e)
  __nv_bfloat16* O;
  float* lse;
  float* part_o;    // [splits][nq * Hq][d] unnormalised, and
  float* part_ml;   // [splits][nq * Hq][2] (maximum in base 2, sum), when splits > 1
  int* status;
};

struct FwdBarriers {
  uint64_t qfull, kvfull[12], kvempty[12], sfull[2], pfull[2], odone[2], fin;
  uint32_t tmem;
  int abort_flag;
};

template <int DB>  // 64-channel blocks: 1 (d <= 64) or 2
struct FwdShape {
  static constexpr int kTileBytes = DB * kBlockBytes;
  static constexpr int kStages = DB == 1 ? 10 : 4;
  static constexpr size_t kSmem = 1024 + (2 + kStages) * (size_t)kTileBytes + sizeof(FwdBarriers);
  // tensor memory: at 64 channels P has columns of its own, so the next S can be issued before P V; at 128 it takes S's
  static constexpr int kS(int s) { return s * 128; }
  static constexpr int kP(int s) { return DB == 1 ? 256 + s * 64 : s * 128; }
  static constexpr int kO(int s) { return DB == 1 ? 384 + s * 64 : 256 + s * 128; }
};

template <int DB>
__global__ void __launch_bounds__(kFwdThreads, 1) attn_fwd_kernel(const __grid_constant__ FwdParams p) {
  using Sh = FwdShape<DB>;
  constexpr int NS = Sh::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* aligned = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t sq = base, skv = base + 2 * Sh::kTileBytes;
  FwdBarriers* bar = reinterpret_cast<FwdBarriers*>(aligned + (2 + NS) * (size_t)Sh::kTileBytes);
  volatile int* abort_flag = &bar->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // work item: query block fastest, so CTAs that run together share keys in L2
  int item = blockIdx.x;
  const int qb = item % p.qblocks;
  item /= p.qblocks;
  const int split = item % p.splits;
  item /= p.splits;
  const int hk = item % p.Hkv, g = item / p.Hkv;

  if (threadIdx.x == 0) {
    mbar_init(&bar->qfull, 1);
    for (int i = 0; i < NS; ++i) mbar_init(&bar->kvfull[i], 1), mbar_init(&bar->kvempty[i], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&bar->sfull[s], 1), mbar_init(&bar->pfull[s], 4), mbar_init(&bar->odone[s], 1);
    mbar_init(&bar->fin, 1);
    bar->abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&p.tq), prefetch_tmap(&p.tk), prefetch_tmap(&p.tv);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  pdl_wait();
  pdl_trigger();
  int* err = p.status;

  int q0, q1, k0, k1;
  const int flags = group_range(p.q_off, g, p.nq, p.max_q, q0, q1) | group_range(p.kv_off, g, p.nkv, p.max_kv, k0, k1);
  if (flags && threadIdx.x == 0 && qb == 0 && split == 0 && hk == 0) atomicOr(p.status, flags);
  // the first token of each stream's tile, the rows that exist, and this split's key tiles
  const int tok0 = q0 + qb * p.tokens * (p.pair ? 2 : 1);
  const bool work = !(flags & SVCONV_STATUS_BAD_OFFSETS) && tok0 < q1;
  const int tiles = (k1 - k0 + kTile - 1) / kTile;
  const int t_lo = (int)((int64_t)tiles * split / p.splits), t_hi = work ? (int)((int64_t)tiles * (split + 1) / p.splits) : 0;
  const int nt = work ? t_hi - t_lo : 0;
  // tiles of stream s, and the tile of its step i (counted from t_lo)
  auto steps_of = [&](int s) { return p.pair ? (tok0 + s * p.tokens < q1 ? nt : 0) : (nt + 1 - s) / 2; };
  auto tile_of = [&](int s, int i) { return p.pair ? i : 2 * i + s; };

  int loaded = 0;  // K / V tiles whose loads were issued (the loader's count)
  if (warp == kLoadWarp) {
    if (lane == 0 && nt > 0) {
      const uint32_t q_bytes = (uint32_t)(p.tokens * p.r) * 128u * DB;
      const int nq_tiles = steps_of(1) > 0 && p.pair ? 2 : 1;
      mbar_arrive_expect_tx(&bar->qfull, q_bytes * nq_tiles);
      for (int s = 0; s < nq_tiles; ++s)
        for (int b = 0; b < DB; ++b)
          tma_load_4d(sq + s * Sh::kTileBytes + b * kBlockBytes, &p.tq, &bar->qfull, b * 64, 0, hk, tok0 + s * p.tokens);
      for (; loaded < 2 * nt; ++loaded) {  // K, V of each tile in turn
        const int slot = loaded % NS;
        if (loaded >= NS && !mbar_wait(&bar->kvempty[slot], ((loaded / NS) & 1) ^ 1, abort_flag, err, kDefaultTimeoutNs)) break;
        mbar_arrive_expect_tx(&bar->kvfull[slot], Sh::kTileBytes);
        for (int b = 0; b < DB; ++b)
          tma_load_3d(skv + slot * Sh::kTileBytes + b * kBlockBytes, (loaded & 1) ? &p.tv : &p.tk, &bar->kvfull[slot], b * 64, hk,
                      k0 + (t_lo + loaded / 2) * kTile);
      }
    }
  } else if (warp == kMmaWarp) {
    if (nt > 0) {
      const int dn = (p.d + 15) / 16 * 16, ks = dn / 16;
      const uint32_t idesc_s = idesc_bf16_f32(kTile, kTile, 0, 0), idesc_o = idesc_bf16_f32(kTile, dn, 0, 1);
      int k_seen = -1, v_seen = -1;  // newest K / V tile known to have landed
      auto seen = [&](int& newest, int tile, int which) {
        if (tile <= newest) return true;
        const int n = 2 * tile + which;
        if (!warp_wait(&bar->kvfull[n % NS], (n / NS) & 1, abort_flag, err)) return false;
        newest = tile;
        if (which) {  // rows of V behind the group's end or dropped by the mask must be zero: their weights are
          const int j0 = k0 + (t_lo + tile) * kTile;
          if (p.keep || j0 + kTile > k1) {
            uint32_t w[4];
            kept_words(p.keep, j0, k1, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ~w[i];
            scrub_rows(skv + (n % NS) * Sh::kTileBytes, DB, w);
          }
        }
        return true;
      };
      auto issue_s = [&](int s, int i) {
        const int tile = tile_of(s, i);
        if (!seen(k_seen, tile, 0)) return false;
        if (lane == 0) {
          tc_fence_after();
          const uint64_t a0 = smem_desc_sw128(sq + (p.pair ? s : 0) * Sh::kTileBytes, 16, 1024);
          const uint64_t b0 = smem_desc_sw128(skv + (2 * tile % NS) * Sh::kTileBytes, 16, 1024);
          for (int k = 0; k < ks; ++k) {
            const uint64_t at = (uint64_t)((k >> 2) * (kBlockBytes >> 4) + (k & 3) * 2);
            tc_mma_bf16(tmem + Sh::kS(s), a0 + at, b0 + at, idesc_s, k ? 1u : 0u);
          }
          tc_commit(&bar->sfull[s]);
          // the tile's last reader frees it (pair form: the second stream, where it has rows)
          if (!p.pair || s == 1 || steps_of(1) == 0) tc_commit(&bar->kvempty[2 * tile % NS]);
        }
        __syncwarp();
        return true;
      };
      auto issue_o = [&](int s, int i) {
        const int tile = tile_of(s, i);
        if (!seen(v_seen, tile, 1)) return false;
        if (lane == 0) {
          tc_fence_after();
          const int slot = (2 * tile + 1) % NS;
          const uint64_t b0 = smem_desc_sw128(skv + slot * Sh::kTileBytes, kBlockBytes, 1024);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            tc_mma_bf16_ts(tmem + Sh::kO(s), tmem + Sh::kP(s) + k * 8, b0 + (uint64_t)(k * (2048 >> 4)), idesc_o, (i | k) ? 1u : 0u);
          tc_commit(&bar->odone[s]);
          if (!p.pair || s == 1 || steps_of(1) == 0) tc_commit(&bar->kvempty[slot]);
        }
        __syncwarp();
        return true;
      };
      bool ok = warp_wait(&bar->qfull, 0, abort_flag, err);
      for (int s = 0; s < 2 && ok; ++s)
        if (steps_of(s) > 0) ok = issue_s(s, 0);
      const int steps = steps_of(0);
      for (int i = 0; i < steps && ok; ++i)
        for (int s = 0; s < 2 && ok; ++s) {
          if (i >= steps_of(s)) continue;
          ok = warp_wait(&bar->pfull[s], i & 1, abort_flag, err);
          const bool more = i + 1 < steps_of(s);
          if constexpr (DB == 1) {
            if (ok && more) ok = issue_s(s, i + 1);
            if (ok) ok = issue_o(s, i);
          } else {
            if (ok) ok = issue_o(s, i);
            if (ok && more) {
              ok = warp_wait(&bar->odone[s], i & 1, abort_flag, err);  // P shares S's columns
              if (ok) ok = issue_s(s, i + 1);
            }
          }
        }
      if (lane == 0) {  // every issued product is complete before tensor memory is released
        tc_commit(&bar->fin);
        volatile int never = 0;
        mbar_wait(&bar->fin, 0, &never, err, kDefaultTimeoutNs);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax: one thread per row
    const int s = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int stok0 = tok0 + (p.pair ? s * p.tokens : 0);
    const int left = work ? min(p.tokens, q1 - stok0) * p.r : 0;
    const bool warp_on = (warp & 3) * 32 < left, row_on = row < left;
    const int steps = steps_of(s);
    const float ca = fmaxf(fabsf(p.c), 1e-30f);  // never 0: a masked score stays -inf when scaled
    float m = -INFINITY, l = 0.f;  // running maximum (of the raw scores, negated for a negative scale) and sum
    bool ok = true;
    for (int i = 0; i < steps; ++i) {
      const int j0 = k0 + (t_lo + tile_of(s, i)) * kTile;
      const bool masked = p.keep || j0 + kTile > k1;
      uint32_t kept[4];
      if (masked) kept_words(p.keep, j0, k1, kept);
      if (!(ok = warp_wait(&bar->sfull[s], i & 1, abort_flag, err))) break;
      tc_fence_after();
      if (warp_on) {
        uint32_t v[4][32];
#pragma unroll
        for (int b = 0; b < 4; ++b) tmem_ld_32x32b_x32(tmem + lanes + Sh::kS(s) + b * 32, v[b]);
        tmem_ld_wait();
        if (p.c < 0.f) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int k = 0; k < 32; ++k) v[b][k] ^= 0x80000000u;
        }
        if (masked) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(kept[b] >> k & 1u)) v[b][k] = 0xff800000u;
        }
        float mx[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          mx[b] = __uint_as_float(v[b][0]);
#pragma unroll
          for (int k = 1; k < 32; ++k) mx[b] = fmaxf(mx[b], __uint_as_float(v[b][k]));
        }
        const float tile_max = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // a row that has seen no key yet takes the tile's maximum; later ones only a clear rise
        const float m_old = m;
        if (m == -INFINITY || (tile_max - m) * ca > kRescaleLog2) m = fmaxf(m, tile_max);
        const float mm = m == -INFINITY ? 0.f : m * ca;
        if (i > 0) {
          ok = warp_wait(&bar->odone[s], (i - 1) & 1, abort_flag, err);
          if (!ok) break;
          tc_fence_after();
          const float a = m == m_old ? 1.f : ex2(m_old * ca - mm);
          l *= a;
          if (__any_sync(0xffffffffu, m != m_old && m_old != -INFINITY)) {
            for (int b = 0; b < 4 * DB; ++b) {
              uint32_t o[16];
              tmem_ld_x16(tmem + lanes + Sh::kO(s) + b * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
              tmem_st_x16(tmem + lanes + Sh::kO(s) + b * 16, o);
            }
          }
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float x = ex2(fmaf(__uint_as_float(v[2 * h + k / 16][2 * (k & 15)]), ca, -mm));
            const float y = ex2(fmaf(__uint_as_float(v[2 * h + k / 16][2 * (k & 15) + 1]), ca, -mm));
            sum[k & 3] += x + y;
            w[k] = pack_bf16(x, y);
          }
          tmem_st_32x32b_x32(tmem + lanes + Sh::kP(s) + h * 32, w);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st_wait();
      }
      tc_fence_before();
      warp_arrive(&bar->pfull[s]);
    }
    if (ok && steps > 0) {
      ok = warp_wait(&bar->odone[s], (steps - 1) & 1, abort_flag, err);
      tc_fence_after();
    }
    float m2 = l > 0.f ? m * ca : -INFINITY;  // the maximum in base 2; -inf: no key
    if (!(l > 0.f) && !(l == 0.f)) m2 = l;    // NaN scores: carried along
    float* so = reinterpret_cast<float*>(aligned + 2 * Sh::kTileBytes);  // split form: the second stream's state, [column][row]
    constexpr int kCols = DB * 64;
    const bool merge = !p.pair && nt > 1;
    if (merge) {
      // both streams' last products, and with them every load into the ring, are done before it is reused
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (s == 1 && warp_on && ok) {
        so[kCols * kTile + row] = m2;
        so[(kCols + 1) * kTile + row] = l;
#pragma unroll
        for (int b = 0; b < 2 * DB; ++b) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tmem + lanes + Sh::kO(s) + b * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) so[(b * 32 + k) * kTile + row] = __uint_as_float(o[k]);
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    const bool writer = p.pair || s == 0;
    if (warp_on && ok && writer) {
      float f0 = 1.f, f1 = 0.f;
      if (merge) {
        const float m1 = so[kCols * kTile + row], l1 = so[(kCols + 1) * kTile + row];
        const float top = fmaxf(m2, m1);
        f0 = m2 == -INFINITY ? 0.f : ex2(m2 - top);
        f1 = m1 == -INFINITY ? 0.f : ex2(m1 - top);
        l = l * f0 + l1 * f1;
        m2 = (l == l) ? top : l;
      }
      const int token = stok0 + row / p.r, head = hk * p.r + row % p.r;
      const int64_t at = (int64_t)token * p.Hq + head;
      const float inv = p.splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
      const int64_t rows = (int64_t)p.nq * p.Hq;
#pragma unroll
      for (int b = 0; b < 2 * DB; ++b) {
        if (b * 32 >= p.d) break;
        uint32_t o[32];
        if (steps > 0) {
          tmem_ld_32x32b_x32(tmem + lanes + Sh::kO(s) + b * 32, o);
          tmem_ld_wait();
        }
        if (!row_on) continue;
        float f[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          f[k] = steps > 0 && l != 0.f ? __uint_as_float(o[k]) : 0.f;
          if (merge) f[k] = f[k] * f0 + (f1 != 0.f ? so[(b * 32 + k) * kTile + row] * f1 : 0.f);
          f[k] *= inv;
        }
        if (p.splits > 1) {
          float* dst = p.part_o + (split * rows + at) * p.d + b * 32;
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            if (b * 32 + k < p.d) *reinterpret_cast<float4*>(dst + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
        } else {
          __nv_bfloat16* dst = p.O + at * p.d + b * 32;
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            if (b * 32 + k < p.d)
              *reinterpret_cast<uint4*>(dst + k) = make_uint4(pack_bf16(f[k], f[k + 1]), pack_bf16(f[k + 2], f[k + 3]),
                                                              pack_bf16(f[k + 4], f[k + 5]), pack_bf16(f[k + 6], f[k + 7]));
        }
      }
      if (row_on) {
        if (p.splits > 1)
          *reinterpret_cast<float2*>(p.part_ml + (split * rows + at) * 2) = make_float2(m2, l);
        else
          p.lse[at] = l == 0.f ? -INFINITY : (m2 + log2f(l)) * kLn2;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (bar->abort_flag && warp == kLoadWarp && lane == 0 && nt > 0) {
    // a wait ran out somewhere: let the copies in flight land before the CTA gives its memory back
    volatile int never = 0;
    mbar_wait(&bar->qfull, 0, &never, err, kDefaultTimeoutNs);
    for (int i = loaded > NS ? loaded - NS : 0; i < loaded; ++i)
      mbar_wait(&bar->kvfull[i % NS], (i / NS) & 1, &never, err, kDefaultTimeoutNs);
  }
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The splits of each (row, head) merged in a fixed order: a warp takes every 8th split, then the
// warps' states are folded in order.
__global__ void __launch_bounds__(256) attn_combine_kernel(const __grid_constant__ FwdParams p) {
  __shared__ float s_ml[8][2], s_o[8][kMaxD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.z, h = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  int q0, q1, k0, k1;
  const int flags = group_range(p.q_off, g, p.nq, p.max_q, q0, q1) | group_range(p.kv_off, g, p.nkv, p.max_kv, k0, k1);
  const int row = q0 + blockIdx.x;
  if ((flags & SVCONV_STATUS_BAD_OFFSETS) || row >= q1) return;
  const int64_t at = (int64_t)row * p.Hq + h, rows = (int64_t)p.nq * p.Hq;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  auto fold = [&](float m1, float l1, const float (&o1)[4]) {
    if (l1 == 0.f) return;
    const float top = fmaxf(m, m1);
    const float a = m == -INFINITY ? 0.f : ex2(m - top), b = ex2(m1 - top);
    l = l * a + l1 * b;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = o[c] * a + o1[c] * b;
    m = top;
  };
  for (int sp = warp; sp < p.splits; sp += 8) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (sp * rows + at) * 2);
    float o1[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) o1[c] = lane + 32 * c < p.d ? p.part_o[(sp * rows + at) * p.d + lane + 32 * c] : 0.f;
    fold(ml.x, ml.y, o1);
  }
  if (lane == 0) s_ml[warp][0] = m, s_ml[warp][1] = l;
#pragma unroll
  for (int c = 0; c < 4; ++c) s_o[warp][lane + 32 * c] = o[c];
  __syncthreads();
  if (warp != 0) return;
  m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] = 0.f;
  for (int w = 0; w < 8; ++w) {
    float o1[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) o1[c] = s_o[w][lane + 32 * c];
    fold(s_ml[w][0], s_ml[w][1], o1);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < p.d) p.O[at * p.d + lane + 32 * c] = __float2bfloat16(o[c] * inv);
  if (lane == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
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

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// bf16 map with 128-byte swizzle and zero fill outside the tensor; dims and strides (elements) innermost first.
bool make_map(CUtensorMap* m, const void* base, int rank, const int64_t* dims, const int64_t* strides, const uint32_t* box) {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(f)
               : nullptr;
  }();
  if (!fn) return false;
  cuuint64_t gd[5], gs[4];
  cuuint32_t bx[5], es[5];
  for (int i = 0; i < rank; ++i) gd[i] = (cuuint64_t)dims[i], bx[i] = box[i], es[i] = 1;
  for (int i = 0; i < rank - 1; ++i) gs[i] = (cuuint64_t)strides[i] * 2;
  auto encode = [&] {
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), gd, gs, bx, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  if (encode() == CUDA_SUCCESS) return true;
  // a host thread whose first CUDA work is this call has no current context yet: bind the device's and try again
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode() == CUDA_SUCCESS;
}

// [n][heads][d] in boxes of one head x `rows` rows x 64 channels
bool make_rows_map(CUtensorMap* m, const void* base, int n, int heads, int d, int64_t row, int64_t head, int rows) {
  const int64_t dims[3] = {d, heads, n > 0 ? n : 1}, strides[2] = {head, row};
  const uint32_t box[3] = {64, 1, (uint32_t)rows};
  return make_map(m, base, 3, dims, strides, box);
}

// [n][Hkv][r][d] in boxes of `tokens` rows x the r heads of one key head x 64 channels
bool make_packed_map(CUtensorMap* m, const void* base, int n, int Hkv, int r, int d, int64_t row, int64_t head, int tokens) {
  const int64_t dims[4] = {d, r, Hkv, n > 0 ? n : 1}, strides[3] = {head, head * r, row};
  const uint32_t box[4] = {64, (uint32_t)r, 1, (uint32_t)tokens};
  return make_map(m, base, 4, dims, strides, box);
}

int cdiv(int a, int b) { return (int)(((long long)a + b - 1) / b); }

// How a forward call is cut.  Pair form where a group can have more query tokens than one tile holds.  Keys are
// split where the query blocks leave SMs idle, down to kMinTiles key tiles a split; the counts use fixed numbers
// (148 SMs), so the workspace size needs no device query.
constexpr int kSms = 148, kMinTiles = 4;
struct FwdPlan {
  int pair, qblocks, splits;
};
FwdPlan plan_fwd(const svconv_cross_attn_desc& c) {
  FwdPlan f;
  const int tokens = kTile / (c.Hq / c.Hkv);
  f.pair = c.max_q > tokens;
  f.qblocks = f.pair ? cdiv(c.max_q, 2 * tokens) : 1;
  const long long units = (long long)c.G * c.Hkv * f.qblocks;
  const int most = cdiv(cdiv(c.max_kv, kTile), kMinTiles);
  f.splits = units >= kSms ? 1 : (int)(kSms / units);
  if (f.splits > most) f.splits = most;
  if (f.splits < 1) f.splits = 1;
  return f;
}

template <int DB>
cudaError_t launch_fwd(const FwdParams& p, int grid, cudaStream_t s) {
  static int done[64];
  cudaError_t e = ensure_smem_attr(attn_fwd_kernel<DB>, FwdShape<DB>::kSmem, done);
  return e == cudaSuccess ? launch_pdl(attn_fwd_kernel<DB>, dim3(grid), dim3(kFwdThreads), FwdShape<DB>::kSmem, s, p) : e;
}

}  // namespace
}  // namespace svc

using namespace svc;

extern "C" {

size_t svconv_cross_attn_fwd_workspace_size(const svconv_cross_attn_desc* desc) {
  svconv_cross_attn_desc c;
  if (check_desc(desc, c) || c.G == 0 || c.max_q == 0) return 0;
  const FwdPlan f = plan_fwd(c);
  return f.splits > 1 ? (size_t)f.splits * c.nq * c.Hq * (c.d + 2) * sizeof(float) : 0;
}

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
  const FwdPlan f = plan_fwd(c);
  const long long grid = (long long)c.G * c.Hkv * f.qblocks * f.splits;
  if (grid > 0x7fffffffLL) return SVCONV_ERR_SIZE;
  FwdParams p{};
  p.q_off = c.q_off, p.kv_off = c.kv_off, p.keep = c.kv_keep;
  p.nq = c.nq, p.nkv = c.nkv, p.max_q = c.max_q, p.max_kv = c.max_kv, p.Hq = c.Hq, p.Hkv = c.Hkv, p.r = c.Hq / c.Hkv, p.d = c.d;
  p.tokens = kTile / p.r;
  p.qblocks = f.qblocks, p.splits = f.splits, p.pair = f.pair;
  p.c = c.scale * kLog2e;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = p.part_o + (size_t)f.splits * c.nq * c.Hq * c.d;
  p.status = dev_status ? dev_status : device_error_word();
  // no keys at all: the maps only have to be well formed
  if (!make_packed_map(&p.tq, Q, c.nq, c.Hkv, p.r, c.d, c.q_row, c.q_head, p.tokens) ||
      !make_rows_map(&p.tk, c.nkv ? K : Q, c.nkv, c.Hkv, c.d, c.k_row, c.k_head, kTile) ||
      !make_rows_map(&p.tv, c.nkv ? V : Q, c.nkv, c.Hkv, c.d, c.v_row, c.v_head, kTile))
    return SVCONV_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = c.d <= 64 ? launch_fwd<1>(p, (int)grid, s) : launch_fwd<2>(p, (int)grid, s);
  if (e == cudaSuccess && f.splits > 1)
    e = launch_pdl(attn_combine_kernel, dim3(c.max_q, c.Hq, c.G), dim3(256), 0, s, p);
  return e == cudaSuccess ? SVCONV_OK : SVCONV_ERR_CUDA;
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
