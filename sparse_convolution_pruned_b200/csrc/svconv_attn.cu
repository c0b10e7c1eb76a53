// Cross-attention of packed groups, forward and backward: every query row attends over the kept
// keys of its group (see svconv_cross_attn_fwd in svconv.h for the definition).
// Scores are in base 2: scale * log2(e) is one factor, and every exponential is one ex2.
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

// ============================================================================ tensor-core building blocks
constexpr int kTile = 128;             // query rows (query tokens x their r heads) and keys of a tile
constexpr int kBlockBytes = kTile * 128;  // 128 rows of 64 bf16 channels, 128-byte swizzled
constexpr int kSoftWarps = 16;         // four softmax warpgroups: two per stream, half of a tile's columns each
constexpr int kLoadWarp = kSoftWarps;
constexpr int kCheckWarp = kSoftWarps + 1;  // zeroes rows that take no part, ahead of the products
// Two warps issue products, one the scores and one the sums (P V; dS K and the like): a warp's first shared-memory
// access after a batch of products waits ~200 cycles for them, which then overlaps the other warp's.
constexpr int kScoreWarp = kSoftWarps + 2, kSumWarp = kSoftWarps + 3;
constexpr int kThreads = (kSoftWarps + 4) * 32;

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

// Two fp32 values that one instruction handles together
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 pack2(uint32_t lo, uint32_t hi) { return pack2(__uint_as_float(lo), __uint_as_float(hi)); }
__device__ __forceinline__ void unpack2(f2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Bounded waits.  The waits between products and softmax follow each other every few hundred cycles:
// every thread polls, without a sleep hint (a thread put to sleep wakes late), in a loop of three instructions, and
// nothing branches on the outcome: a call, a result to carry through the loops or one polling lane with a
// broadcast each cost 10 to 25% of the kernels.  A wait that runs out raises the abort flag, after which every wait
// returns at once and the loops run to their ends on whatever is there (in bounds; the status word tells).
__device__ __forceinline__ uint32_t try_wait_many(uint64_t* bar, uint32_t parity) {
  uint32_t left;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mov.u32 %0, 256;\n\t"
      "ATTN_WAIT:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra ATTN_DONE;\n\t"
      "sub.u32 %0, %0, 1;\n\t"
      "setp.ne.u32 q, %0, 0;\n\t"
      "@q bra ATTN_WAIT;\n\t"
      "ATTN_DONE:\n\t}"
      : "=&r"(left)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return left;
}
__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  if (try_wait_many(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!*abort_flag && !try_wait_many(bar, parity)) {
    if (globaltimer_ns() - t0 > kDefaultTimeoutNs) {
      *abort_flag = 1;
      atomicOr(err, SVCONV_STATUS_TIMEOUT);
    }
  }
}
// The whole warp waits, and is converged afterwards; mostly the first try succeeds, and a vote is all it takes.
__device__ __forceinline__ void wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
  wait_for(bar, parity, abort_flag, err);
  __syncwarp();
}
// A value that is the same in every lane, told to the compiler as such: what depends on it stays in uniform registers.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Products and commits issued by the one lane with e != 0 of a converged warp.  Predicated instead of branched
// around, so that descriptors and addresses are warp-uniform and sit in uniform registers when the instruction
// wants them there (in a branch of one lane each operand was moved over first: ~100 cycles a product).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t e) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(e)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t e) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(e)
      : "memory");
}
__device__ __forceinline__ void commit_to(uint64_t* bar, uint32_t e) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(e)
      : "memory");
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

// 32 consecutive values of a row, of which `n` exist (a multiple of 8), by 32-byte stores where the row allows it
__device__ __forceinline__ void store_row(float* dst, const float (&f)[32], int n) {
#pragma unroll
  for (int k = 0; k < 32; k += 8)
    if (k < n) st_global_32(dst + k, reinterpret_cast<const uint32_t*>(f) + k);  // rows of 8 k floats: 32-byte aligned
}
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, const float (&f)[32], int n, bool wide) {
  uint32_t v[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = pack_bf16(f[2 * k], f[2 * k + 1]);
  if (wide && n >= 32) {
    st_global_32(dst, v);
    st_global_32(dst + 16, v + 8);
  } else {
#pragma unroll
    for (int k = 0; k < 16; k += 4)
      if (2 * k < n) *reinterpret_cast<uint4*>(dst + 2 * k) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
  }
}

// Zero the rows of a tile that must not reach a product (0 x NaN): bit j of drop[w] is row 32 w + j.
// One warp; a row is 128 contiguous bytes of each 64-channel block whatever the swizzle.
template <int WORDS>
__device__ __forceinline__ void scrub_rows(uint32_t tile, int blocks, uint32_t block_bytes, const uint32_t (&drop)[WORDS]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    if (drop[w] >> lane & 1u)
      for (int b = 0; b < blocks; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) st_shared_16(tile + b * block_bytes + (32 * w + lane) * 128 + ((i + lane) & 7) * 16, 0, 0, 0, 0);
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
  int wide;         // rows of O start on 32-byte boundaries
  __nv_bfloat16* O;
  float* lse;
  float* part_o;    // [splits][nq * Hq][d] unnormalised, and
  float* part_ml;   // [splits][nq * Hq][2] (maximum in base 2, sum), when splits > 1
  int* status;
};

struct FwdBarriers {
  uint64_t qfull, kvfull[10], kvempty[10], vready[10], sfull[2], sread[2], pfull[2], odone[2], fin[2];
  uint32_t kept[10][4];  // keys that take part, of the tile whose V lies in this slot
  float rowmax[2][2][2][kTile];  // [step parity][stream][half of the columns][row], exchanged between the halves
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
__global__ void __launch_bounds__(kThreads, 1) attn_fwd_kernel(const __grid_constant__ FwdParams p) {
  using Sh = FwdShape<DB>;
  constexpr int NS = Sh::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* aligned = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t sq = base, skv = base + 2 * Sh::kTileBytes;
  FwdBarriers* bar = reinterpret_cast<FwdBarriers*>(aligned + (2 + NS) * (size_t)Sh::kTileBytes);
  volatile int* abort_flag = &bar->abort_flag;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  // work item: query block fastest, so CTAs that run together share keys in L2
  int item = blockIdx.x;
  const int qb = item % p.qblocks;
  item /= p.qblocks;
  const int split = item % p.splits;
  item /= p.splits;
  const int hk = item % p.Hkv, g = item / p.Hkv;

  // Set-up in parallel: the loader makes the barriers and issues the first loads itself, another warp takes
  // the tensor memory, everyone reads the offsets; one barrier then joins them.
  if (warp == kLoadWarp && lane == 0) {
    mbar_init(&bar->qfull, 1);
    for (int i = 0; i < NS; ++i) mbar_init(&bar->kvfull[i], 1), mbar_init(&bar->kvempty[i], 1), mbar_init(&bar->vready[i], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&bar->sfull[s], 1), mbar_init(&bar->sread[s], 8), mbar_init(&bar->pfull[s], 8), mbar_init(&bar->odone[s], 1);
    mbar_init(&bar->fin[0], 1), mbar_init(&bar->fin[1], 1);
    bar->abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&p.tq), prefetch_tmap(&p.tk), prefetch_tmap(&p.tv);
  }
  if (warp == kSumWarp) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  pdl_wait();
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
  auto masked = [&](int tile) { return p.keep || k0 + (t_lo + tile + 1) * kTile > k1; };

  int loaded = 0;  // K / V tiles whose loads were issued (the loader's count): K, V of each tile in turn
  auto load_kv = [&] {
    const int slot = loaded % NS;
    mbar_arrive_expect_tx(&bar->kvfull[slot], Sh::kTileBytes);
    for (int b = 0; b < DB; ++b)
      tma_load_3d(skv + slot * Sh::kTileBytes + b * kBlockBytes, (loaded & 1) ? &p.tv : &p.tk, &bar->kvfull[slot], b * 64, hk,
                  k0 + (t_lo + loaded / 2) * kTile);
    ++loaded;
  };
  if (warp == kLoadWarp && lane == 0 && nt > 0) {
    const uint32_t q_bytes = (uint32_t)(p.tokens * p.r) * 128u * DB;
    const int nq_tiles = steps_of(1) > 0 && p.pair ? 2 : 1;
    mbar_arrive_expect_tx(&bar->qfull, q_bytes * nq_tiles);
    for (int s = 0; s < nq_tiles; ++s)
      for (int b = 0; b < DB; ++b)
        tma_load_4d(sq + s * Sh::kTileBytes + b * kBlockBytes, &p.tq, &bar->qfull, b * 64, 0, hk, tok0 + s * p.tokens);
    while (loaded < min(2 * nt, NS)) load_kv();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now may the next kernel's CTAs come and ask for tensor memory: this one has its own
  pdl_trigger();
  const uint32_t tmem = bar->tmem;

  if (warp == kLoadWarp) {
    if (lane == 0)
      while (loaded < 2 * nt) {
        wait_for(&bar->kvempty[loaded % NS], ((loaded / NS) & 1) ^ 1, abort_flag, err);
        if (*abort_flag) break;
        load_kv();
      }
  } else if (warp == kScoreWarp) {
    if (nt > 0) {
      const uint32_t e = lane == 0;
      const int ks = (p.d + 15) / 16;
      const uint32_t idesc = idesc_bf16_f32(kTile, kTile, 0, 0), tm = uniform(tmem);
      const int steps0 = uniform(steps_of(0)), steps1 = uniform(steps_of(1));
      const bool pair = p.pair, lone = steps1 == 0;
      const uint64_t dq = smem_desc_sw128(sq, 16, 1024), dk = smem_desc_sw128(skv, 16, 1024);
      wait_warp(&bar->qfull, 0, abort_flag, err);
      for (int i = 0; i < steps0; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (i >= (s ? steps1 : steps0)) continue;
          const int tile = pair ? i : 2 * i + s, n = 2 * tile, slot = n % NS;
          // S is free once its scores have been read; where P lies in its columns, once P V is done too
          if (i > 0) wait_warp(DB == 1 ? &bar->sread[s] : &bar->odone[s], (i - 1) & 1, abort_flag, err);
          if (!pair || s == 0) wait_warp(&bar->kvfull[slot], (n / NS) & 1, abort_flag, err);
          tc_fence_after();
          const uint64_t a0 = dq + (uint64_t)(pair && s ? Sh::kTileBytes >> 4 : 0), b0 = dk + (uint64_t)(slot * (Sh::kTileBytes >> 4));
#pragma unroll
          for (int k = 0; k < 4 * DB; ++k) {
            const uint64_t at = (uint64_t)((k >> 2) * (kBlockBytes >> 4) + (k & 3) * 2);
            if (k < ks) mma_ss(tm + Sh::kS(s), a0 + at, b0 + at, idesc, k ? 1u : 0u, e);
          }
          commit_to(&bar->sfull[s], e);
          // the tile's last reader frees it (pair form: the second stream, where it has rows)
          if (!pair || s == 1 || lone) commit_to(&bar->kvempty[slot], e);
        }
      commit_to(&bar->fin[0], e);  // every issued product is complete before tensor memory is released
      wait_warp(&bar->fin[0], 0, abort_flag, err);
    }
  } else if (warp == kSumWarp) {
    if (nt > 0) {
      const uint32_t e = lane == 0;
      const uint32_t idesc = idesc_bf16_f32(kTile, (p.d + 15) / 16 * 16, 0, 1), tm = uniform(tmem);
      const int steps0 = uniform(steps_of(0)), steps1 = uniform(steps_of(1));
      const bool pair = p.pair, lone = steps1 == 0;
      const uint64_t dv = smem_desc_sw128(skv, kBlockBytes, 1024);
      for (int i = 0; i < steps0; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (i >= (s ? steps1 : steps0)) continue;
          const int tile = pair ? i : 2 * i + s, n = 2 * tile + 1, slot = n % NS;
          // rows of V behind the group's end or dropped by the mask must be zero: their weights are
          if (!pair || s == 0) wait_warp(masked(tile) ? &bar->vready[slot] : &bar->kvfull[slot], (n / NS) & 1, abort_flag, err);
          // Where the next scores wait for P V, they go first: O_0, S_0, O_1, S_1 in turn keeps the streams half a
          // period apart, one's softmax under the other's products (left alone they fall into step: 4,700 cycles
          // for both streams' tiles instead of 3,500)
          if constexpr (DB == 2) {
            if (s == 0 && i > 0 && i < steps1) wait_warp(&bar->sfull[1], i & 1, abort_flag, err);
            if (s == 1 && i + 1 < steps0) wait_warp(&bar->sfull[0], (i + 1) & 1, abort_flag, err);
          }
          wait_warp(&bar->pfull[s], i & 1, abort_flag, err);
          tc_fence_after();
          const uint64_t b0 = dv + (uint64_t)(slot * (Sh::kTileBytes >> 4));
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_ts(tm + Sh::kO(s), tm + Sh::kP(s) + k * 8, b0 + (uint64_t)(k * (2048 >> 4)), idesc, (i | k) ? 1u : 0u, e);
          commit_to(&bar->odone[s], e);
          if (!pair || s == 1 || lone) commit_to(&bar->kvempty[slot], e);
        }
      commit_to(&bar->fin[1], e);
      wait_warp(&bar->fin[1], 0, abort_flag, err);
    }
  } else if (warp == kCheckWarp) {
    for (int tile = 0; tile < nt; ++tile) {
      const int n = 2 * tile + 1, slot = n % NS;
      wait_warp(&bar->kvfull[slot], (n / NS) & 1, abort_flag, err);
      if (masked(tile)) {
        uint32_t w[4];
        kept_words(p.keep, k0 + (t_lo + tile) * kTile, k1, w);
        if (lane < 4) bar->kept[slot][lane] = lane == 0 ? w[0] : lane == 1 ? w[1] : lane == 2 ? w[2] : w[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ~w[i];
        scrub_rows(skv + slot * Sh::kTileBytes, DB, kBlockBytes, w);
      }
      warp_arrive(&bar->vready[slot]);
    }
  } else {
    // ------------------------------------------------------------ softmax: two threads per row, 64 scores each
    const int s = warp >> 3, half = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int pair_bar = 1 + s * 4 + (warp & 3);  // named barrier of the two warps that hold the same rows
    const int stok0 = tok0 + (p.pair ? s * p.tokens : 0);
    const int left = work ? min(p.tokens, q1 - stok0) * p.r : 0;
    const bool warp_on = (warp & 3) * 32 < left, row_on = row < left;
    const int steps = steps_of(s);
    const float ca = fmaxf(fabsf(p.c), 1e-30f);  // never 0: a masked score stays -inf when scaled
    float m = -INFINITY, l = 0.f;  // running maximum (of the raw scores, negated for a negative scale), and sum of this half
    for (int i = 0; i < steps; ++i) {
      const int tile = tile_of(s, i);
      const bool some = masked(tile);
      wait_warp(&bar->sfull[s], i & 1, abort_flag, err);
      tc_fence_after();
      uint32_t v[2][32];
      if (warp_on) {
#pragma unroll
        for (int b = 0; b < 2; ++b) tmem_ld_32x32b_x32(tmem + lanes + Sh::kS(s) + half * 64 + b * 32, v[b]);
      }
      if constexpr (DB == 1) {
        // P's columns and O are free again; at 128 channels these scores already waited for that
        if (i > 0) wait_warp(&bar->odone[s], (i - 1) & 1, abort_flag, err);
      }
      tmem_ld_wait();
      if constexpr (DB == 1) {
        // the scores are in registers: the next ones may be computed over them
        tc_fence_before();
        warp_arrive(&bar->sread[s]);
      }
      if (warp_on) {
        if (p.c < 0.f) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < 32; ++k) v[b][k] ^= 0x80000000u;
        }
        if (some) {
          const int n = 2 * tile + 1;
          wait_warp(&bar->vready[n % NS], (n / NS) & 1, abort_flag, err);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t w = bar->kept[n % NS][half * 2 + b];
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(w >> k & 1u)) v[b][k] = 0xff800000u;
          }
        }
        float mx[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t* u = &v[b >> 1][(b & 1) * 16];
          mx[b] = fmaxf(__uint_as_float(u[0]), __uint_as_float(u[1]));
#pragma unroll
          for (int k = 2; k < 16; k += 2) mx[b] = max3(mx[b], __uint_as_float(u[k]), __uint_as_float(u[k + 1]));
        }
        const float own = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        bar->rowmax[i & 1][s][half][row] = own;
        tc_fence_before();
        asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");  // also: both halves hold their scores in registers
        tc_fence_after();
        const float tile_max = fmaxf(own, bar->rowmax[i & 1][s][half ^ 1][row]);
        // a row that has seen no key yet takes the tile's maximum; later ones only a clear rise
        const float m_old = m;
        if (m == -INFINITY || (tile_max - m) * ca > kRescaleLog2) m = fmaxf(m, tile_max);
        const float mm = m == -INFINITY ? 0.f : m * ca;
        if (i > 0 && __any_sync(0xffffffffu, m != m_old)) {
          tc_fence_after();
          const float a = m == m_old ? 1.f : ex2(m_old * ca - mm);
          l *= a;
          for (int b = 0; b < 2 * DB; ++b) {  // each half rescales half of O's columns
            const uint32_t at = tmem + lanes + Sh::kO(s) + half * 32 * DB + b * 16;
            uint32_t o[16];
            tmem_ld_x16(at, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
            tmem_st_x16(at, o);
          }
        }
        const f2 c2 = pack2(ca, ca), m2 = pack2(-mm, -mm);
        f2 sum[2] = {0ull, 0ull};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float x, y;
            unpack2(fma2(pack2(v[b][2 * k], v[b][2 * k + 1]), c2, m2), x, y);
            x = ex2(x);
            y = ex2(y);
            sum[k & 1] = add2(sum[k & 1], pack2(x, y));
            w[k] = pack_bf16(x, y);
          }
          tmem_st_x16(tmem + lanes + Sh::kP(s) + half * 32 + b * 16, w);
        }
        float x, y;
        unpack2(add2(sum[0], sum[1]), x, y);
        l += x + y;
        tmem_st_wait();
      }
      tc_fence_before();
      warp_arrive(&bar->pfull[s]);
    }
    if (steps > 0) {
      wait_warp(&bar->odone[s], (steps - 1) & 1, abort_flag, err);
      tc_fence_after();
    }
    if (warp_on) {  // the sum of both halves (the buffer of the step before last: its readers are done)
      bar->rowmax[steps & 1][s][half][row] = l;
      asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
      const float other = bar->rowmax[steps & 1][s][half ^ 1][row];
      l = half ? other + l : l + other;
    }
    float m2 = l > 0.f ? m * ca : -INFINITY;  // the maximum in base 2; -inf: no key
    if (!(l > 0.f) && !(l == 0.f)) m2 = l;    // NaN scores: carried along
    float* so = reinterpret_cast<float*>(aligned + 2 * Sh::kTileBytes);  // split form: the second stream's state, [column][row]
    constexpr int kCols = DB * 64;
    const bool merge = !p.pair && nt > 1;
    if (merge) {
      // both streams' last products, and with them every load into the ring, are done before it is reused
      asm volatile("bar.sync 9, 512;" ::: "memory");
      if (s == 1 && warp_on) {
        so[kCols * kTile + row] = m2;
        so[(kCols + 1) * kTile + row] = l;
#pragma unroll
        for (int b = half * DB; b < half * DB + DB; ++b) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tmem + lanes + Sh::kO(s) + b * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) so[(b * 32 + k) * kTile + row] = __uint_as_float(o[k]);
        }
      }
      asm volatile("bar.sync 9, 512;" ::: "memory");
    }
    const bool writer = p.pair || s == 0;
    if (warp_on && writer) {
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
      for (int b = half * DB; b < half * DB + DB; ++b) {  // each half writes half of the channels
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
        if (p.splits > 1) store_row(p.part_o + (split * rows + at) * p.d + b * 32, f, p.d - b * 32);
        else store_row(p.O + at * p.d + b * 32, f, p.d - b * 32, p.wide);
      }
      if (row_on && half == 0) {
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
  if (warp == kSumWarp) tmem_dealloc(tmem, 512);
}

// Few splits: a warp merges the splits of a (row, head) one after the other, 4 channels a lane.
__global__ void __launch_bounds__(256) attn_merge_kernel(const __grid_constant__ FwdParams p) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  int q0, q1, k0, k1;
  const int flags = group_range(p.q_off, blockIdx.y, p.nq, p.max_q, q0, q1) | group_range(p.kv_off, blockIdx.y, p.nkv, p.max_kv, k0, k1);
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if ((flags & SVCONV_STATUS_BAD_OFFSETS) || i >= (q1 - q0) * p.Hq) return;
  const int64_t at = (int64_t)q0 * p.Hq + i, rows = (int64_t)p.nq * p.Hq;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int sp = 0; sp < p.splits; ++sp) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (sp * rows + at) * 2);
    const float4 x = lane * 4 < p.d ? *reinterpret_cast<const float4*>(p.part_o + (sp * rows + at) * p.d + lane * 4) : o;
    if (ml.y == 0.f) continue;
    const float top = fmaxf(m, ml.x);
    const float a = m == -INFINITY ? 0.f : ex2(m - top), b = ex2(ml.x - top);
    l = l * a + ml.y * b;
    o = make_float4(o.x * a + x.x * b, o.y * a + x.y * b, o.z * a + x.z * b, o.w * a + x.w * b);
    m = top;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (lane * 4 < p.d)
    *reinterpret_cast<uint2*>(p.O + at * p.d + lane * 4) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (lane == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Many splits: a warp takes every 8th split of a (row, head), then the warps' states are folded in order.
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

// ============================================================================ backward
// Two passes over the scores, both of one form: a CTA holds a fixed tile of 128 rows (two operands F1,
// F2) and runs over moving tiles of 64 rows (M1, M2), its two softmax warpgroups taking alternate
// moving tiles (streams) while both add to the same accumulators in tensor memory.
//                   fixed F1, F2   moving M1, M2   scores          accumulates
//   key pass        K, V           Q, dO           S^T, dP^T       dV += P^T dO, dK += dS^T Q
//   query pass      Q, dO          K, V            S, dP           dQ += dS K
// With the scores transposed in the key pass, P^T and dS^T are written row by row as A operands in
// tensor memory, and M1, M2 serve both as K-major operands of the scores and as MN-major operands of the
// sums: nothing is transposed and nothing passes through shared memory.  No atomics: each output
// row has one owner, or one per split with the splits added in a fixed order.  That costs 7 products
// per tile where one pass with atomics on dQ would take 5.
constexpr int kMove = 64;                  // rows of a moving tile
constexpr int kMoveBlock = kMove * 128;    // bytes of its 64-channel block
constexpr int kStat = 2 * kMove;           // a tile's statistics: -lse in base 2 of its 64 rows, then -D
constexpr int kStatBytes = kStat * 4;

struct BwdParams {
  CUtensorMap fq, fdo, fk, fv;   // boxes of the fixed tiles
  CUtensorMap mq, mdo, mk, mv;   // boxes of the moving tiles
  const int32_t *q_off, *kv_off;
  const uint8_t* keep;
  int nq, nkv, max_q, max_kv, Hq, Hkv, r, d;
  int qblocks, qsplits, kblocks, ksplits;
  int q_items, k_items;          // CTAs of the two passes
  int keys_first;                // the pass with the longer items comes first
  float c, scale;
  int wide;                      // rows of the gradients start on 32-byte boundaries
  const float* stat;             // [Hkv][stat_tiles][kStat], see attn_stat_kernel
  int stat_tiles;
  __nv_bfloat16 *dQ, *dK, *dV;
  float *part_q, *part_k, *part_v;  // [splits][rows][d] where a pass is split
  int* status;
};

struct BwdBarriers {
  uint64_t ffull, mfull[8], mempty[8], mready[8], sfull[2], pfull[2], pdone[2], adone[2], fin[2];
  uint32_t kept[8][2];  // query pass: keys of the slot's tile that take part
  uint32_t tmem;
  int abort_flag;
};

template <int DB>
struct BwdShape {
  static constexpr int kFixedBytes = DB * kBlockBytes, kMoveBytes = DB * kMoveBlock;
  static constexpr int kStages = DB == 1 ? 8 : 4;
  static constexpr int kStageBytes = 2 * kMoveBytes;
  static constexpr size_t kSmem = 1024 + 2 * kFixedBytes + kStages * (size_t)(kStageBytes + kStatBytes) + sizeof(BwdBarriers);
};

// Tensor-memory columns.  P and dS have columns of their own except in the key pass at 128
// channels, where the accumulators leave room for the scores alone and P, dS take their place.
template <int DB, bool KEYS>
struct BwdTmem {
  static constexpr bool kShared = DB == 2 && KEYS;
  static constexpr int kStride = DB == 1 ? 192 : KEYS ? 128 : 160;
  static constexpr int S(int s) { return s * kStride; }
  static constexpr int dP(int s) { return s * kStride + 64; }
  static constexpr int P(int s) { return DB == 1 ? s * kStride + 128 : s * kStride; }
  static constexpr int dS(int s) { return DB == 1 ? s * kStride + 160 : KEYS ? s * kStride + 64 : s * kStride + 128; }
  static constexpr int kAcc1 = DB == 1 ? 384 : 256;   // dV
  static constexpr int kAcc2 = DB == 1 ? 448 : 384;   // dK or dQ
};

template <int DB, bool KEYS>
__device__ __forceinline__ void bwd_pass(const BwdParams& p, int item, uint32_t base, BwdBarriers* bar, const uint8_t* stats) {
  using Sh = BwdShape<DB>;
  using Tm = BwdTmem<DB, KEYS>;
  constexpr int NS = Sh::kStages;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* abort_flag = &bar->abort_flag;
  int* err = p.status;
  const uint32_t sf = base, sm = base + 2 * Sh::kFixedBytes;
  const uint32_t sstat = sm + NS * Sh::kStageBytes;

  const int blocks = KEYS ? p.kblocks : p.qblocks, splits = KEYS ? p.ksplits : p.qsplits;
  const int block = item % blocks;
  item /= blocks;
  const int split = item % splits;
  item /= splits;
  const int hk = item % p.Hkv, g = item / p.Hkv;
  int q0, q1, k0, k1;
  const int flags = group_range(p.q_off, g, p.nq, p.max_q, q0, q1) | group_range(p.kv_off, g, p.nkv, p.max_kv, k0, k1);
  if (flags && threadIdx.x == 0 && block == 0 && split == 0 && hk == 0) atomicOr(p.status, flags);
  const int ftok = kTile / p.r, mtok = kMove / p.r;  // query tokens of a fixed and of a moving tile
  const int f0 = KEYS ? k0 + block * kTile : q0 + block * ftok;
  const int f1 = KEYS ? k1 : q1;
  const int left = (flags & SVCONV_STATUS_BAD_OFFSETS) ? 0 : KEYS ? min(kTile, f1 - f0) : min(ftok, f1 - f0) * p.r;  // rows
  const int mstep = KEYS ? mtok : kMove;
  const int tiles = KEYS ? (q1 - q0 + mtok - 1) / mtok : (k1 - k0 + kMove - 1) / kMove;
  const int t_lo = (int)((int64_t)tiles * split / splits), t_hi = (int)((int64_t)tiles * (split + 1) / splits);
  const int nt = left > 0 ? t_hi - t_lo : 0;
  const int m0 = (KEYS ? q0 : k0) + t_lo * mstep;  // first row of the first moving tile
  auto steps_of = [&](int s) { return (nt + 1 - s) / 2; };
  // rows of moving tile t that take part (two words), and whether any is missing
  auto partial = [&](int t) {
    return KEYS ? (mtok * p.r < kMove || m0 + (t + 1) * mtok > q1) : (p.keep || m0 + (t + 1) * kMove > k1);
  };
  auto kept = [&](int t, uint32_t (&w)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = 32 * i + lane;
      bool on;
      if constexpr (KEYS) {
        on = at < min(mtok, q1 - m0 - t * mtok) * p.r;
      } else {
        const int j = m0 + t * kMove + at;
        on = j < k1 && (!p.keep || __ldg(p.keep + j) != 0);
      }
      w[i] = __ballot_sync(0xffffffffu, on);
    }
  };
  // the statistics of query tile t of the group
  auto stat_of = [&](int t) { return p.stat + ((int64_t)hk * p.stat_tiles + q0 / mtok + g + t) * kStat; };

  int loaded = 0;  // moving tiles whose loads were issued (the loader's count)
  auto load_moving = [&] {
    const CUtensorMap* m[2] = {KEYS ? &p.mq : &p.mk, KEYS ? &p.mdo : &p.mv};
    const int slot = loaded % NS;
    mbar_arrive_expect_tx(&bar->mfull[slot], 2 * DB * (uint32_t)(KEYS ? mtok * p.r : kMove) * 128u + (KEYS ? (uint32_t)kStatBytes : 0u));
    for (int o = 0; o < 2; ++o)
      for (int b = 0; b < DB; ++b) {
        const uint32_t dst = sm + slot * Sh::kStageBytes + o * Sh::kMoveBytes + b * kMoveBlock;
        if constexpr (KEYS) tma_load_4d(dst, m[o], &bar->mfull[slot], b * 64, 0, hk, m0 + loaded * mtok);
        else tma_load_3d(dst, m[o], &bar->mfull[slot], b * 64, hk, m0 + loaded * kMove);
      }
    if constexpr (KEYS) bulk_copy_g2s(sstat + slot * kStatBytes, stat_of(t_lo + loaded), kStatBytes, &bar->mfull[slot]);
    ++loaded;
  };
  if (warp == kLoadWarp && lane == 0 && nt > 0) {
    const CUtensorMap* f[2] = {KEYS ? &p.fk : &p.fq, KEYS ? &p.fv : &p.fdo};
    mbar_arrive_expect_tx(&bar->ffull, 2 * DB * (uint32_t)(KEYS ? kTile : ftok * p.r) * 128u);
    for (int o = 0; o < 2; ++o)
      for (int b = 0; b < DB; ++b) {
        const uint32_t dst = sf + o * Sh::kFixedBytes + b * kBlockBytes;
        if constexpr (KEYS) tma_load_3d(dst, f[o], &bar->ffull, b * 64, hk, f0);
        else tma_load_4d(dst, f[o], &bar->ffull, b * 64, 0, hk, f0);
      }
    while (loaded < min(nt, NS)) load_moving();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now may the next kernel's CTAs come and ask for tensor memory: this one has its own
  pdl_trigger();
  const uint32_t tmem = bar->tmem;

  if (warp == kLoadWarp) {
    if (lane == 0)
      while (loaded < nt) {
        wait_for(&bar->mempty[loaded % NS], ((loaded / NS) & 1) ^ 1, abort_flag, err);
        if (*abort_flag) break;
        load_moving();
      }
  } else if (warp == kScoreWarp) {
    if (nt > 0) {
      const uint32_t e = lane == 0;
      const int ks = (p.d + 15) / 16, n = uniform(nt);
      const uint32_t idesc = idesc_bf16_f32(kTile, kMove, 0, 0), tm = uniform(tmem);
      const uint64_t df = smem_desc_sw128(sf, 16, 1024), dm = smem_desc_sw128(sm, 16, 1024);
      // operand o (0: F1 M1, 1: F2 M2) of the tile in this slot
      auto scores = [&](int o, int slot, uint32_t d) {
        const uint64_t a0 = df + (uint64_t)(o * (Sh::kFixedBytes >> 4)), b0 = dm + (uint64_t)(slot * (Sh::kStageBytes >> 4) + o * (Sh::kMoveBytes >> 4));
#pragma unroll
        for (int k = 0; k < 4 * DB; ++k)
          if (k < ks)
            mma_ss(d, a0 + (uint64_t)((k >> 2) * (kBlockBytes >> 4) + (k & 3) * 2), b0 + (uint64_t)((k >> 2) * (kMoveBlock >> 4) + (k & 3) * 2),
                   idesc, k ? 1u : 0u, e);
      };
      wait_warp(&bar->ffull, 0, abort_flag, err);
      for (int t0 = 0; t0 < n; t0 += 2)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int t = t0 + s, ph = ((t0 >> 1) - 1) & 1, slot = t % NS;
          if (t >= n) continue;
          // rows that take no part are zero by then: they meet zero weights
          wait_warp(partial(t) ? &bar->mready[slot] : &bar->mfull[slot], (t / NS) & 1, abort_flag, err);
          // the scores' columns are free once they have been read; where P and dS lie in them, once the sums
          // that read those are done
          if (t0 > 0) wait_warp(Tm::kShared ? &bar->pdone[s] : &bar->pfull[s], ph, abort_flag, err);
          tc_fence_after();
          scores(0, slot, tm + Tm::S(s));
          if (Tm::kShared && t0 > 0) {
            wait_warp(&bar->adone[s], ph, abort_flag, err);
            tc_fence_after();
          }
          scores(1, slot, tm + Tm::dP(s));
          commit_to(&bar->sfull[s], e);
        }
      commit_to(&bar->fin[0], e);  // every issued product is complete before tensor memory is released
      wait_warp(&bar->fin[0], 0, abort_flag, err);
    }
  } else if (warp == kSumWarp) {
    if (nt > 0) {
      const uint32_t e = lane == 0;
      const int n = uniform(nt);
      const uint32_t idesc = idesc_bf16_f32(kTile, (p.d + 15) / 16 * 16, 0, 1), tm = uniform(tmem);
      const uint64_t dt = smem_desc_sw128(sm, kMoveBlock, 1024);
      // acc += A (tensor memory) x operand o of the tile in this slot
      auto sums = [&](int o, int slot, uint32_t a_col, uint32_t acc, bool more) {
        const uint64_t b0 = dt + (uint64_t)(slot * (Sh::kStageBytes >> 4) + o * (Sh::kMoveBytes >> 4));
#pragma unroll
        for (int k = 0; k < kMove / 16; ++k) mma_ts(acc, a_col + k * 8, b0 + (uint64_t)(k * (2048 >> 4)), idesc, more || k ? 1u : 0u, e);
      };
      for (int t0 = 0; t0 < n; t0 += 2)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int t = t0 + s, slot = t % NS;
          if (t >= n) continue;
          wait_warp(&bar->pfull[s], (t0 >> 1) & 1, abort_flag, err);  // the tile itself landed before its scores
          tc_fence_after();
          if constexpr (KEYS) {
            sums(1, slot, tm + Tm::P(s), tm + Tm::kAcc1, t > 0);
            if constexpr (Tm::kShared) commit_to(&bar->pdone[s], e);
          }
          sums(0, slot, tm + Tm::dS(s), tm + Tm::kAcc2, t > 0);
          commit_to(&bar->adone[s], e);
          commit_to(&bar->mempty[slot], e);
        }
      commit_to(&bar->fin[1], e);
      wait_warp(&bar->fin[1], 0, abort_flag, err);
    }
  } else if (warp == kCheckWarp) {
    for (int t = 0; t < nt; ++t) {
      const int slot = t % NS;
      wait_warp(&bar->mfull[slot], (t / NS) & 1, abort_flag, err);
      if (partial(t)) {
        uint32_t w[2];
        kept(t, w);
        if (lane < 2) bar->kept[slot][lane] = lane == 0 ? w[0] : w[1];
        w[0] = ~w[0], w[1] = ~w[1];
        scrub_rows(sm + slot * Sh::kStageBytes, 2 * DB, kMoveBlock, w);
      }
      warp_arrive(&bar->mready[slot]);
    }
  } else {
    // ------------------------------------------------------------ P and dS: two threads per fixed row, 32 columns each
    const int s = warp >> 3, h = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const bool warp_on = (warp & 3) * 32 < left, row_on = row < left;
    const int steps = steps_of(s);
    const f2 c2 = pack2(p.c, p.c);
    f2 row_lse = pack2(-INFINITY, -INFINITY), row_d = 0ull;
    if (!KEYS && row_on) {
      const int token = f0 - q0 + row / p.r;
      const float* st = stat_of(token / mtok) + (token % mtok) * p.r + row % p.r;
      row_lse = pack2(st[0], st[0]);
      row_d = pack2(st[kMove], st[kMove]);
    }
    for (int i = 0; i < steps; ++i) {
      const int t = 2 * i + s;
      if (KEYS) wait_warp(&bar->mfull[t % NS], (t / NS) & 1, abort_flag, err);
      wait_warp(&bar->sfull[s], i & 1, abort_flag, err);
      if (i > 0) wait_warp(&bar->adone[s], (i - 1) & 1, abort_flag, err);  // P and dS are free again
      tc_fence_after();
      if (warp_on) {
        const float* st = reinterpret_cast<const float*>(stats + (t % NS) * kStatBytes);
        uint32_t a[32], b[32], u[16];
        tmem_ld_32x32b_x32(tmem + lanes + Tm::S(s) + h * 32, a);
        tmem_ld_32x32b_x32(tmem + lanes + Tm::dP(s) + h * 32, b);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          ulonglong2 nl = make_ulonglong2(row_lse, row_lse), nd = make_ulonglong2(row_d, row_d);
          if constexpr (KEYS) {  // a row that takes no part has -lse = -inf there: weight 0
            nl = *reinterpret_cast<const ulonglong2*>(st + h * 32 + k);
            nd = *reinterpret_cast<const ulonglong2*>(st + kMove + h * 32 + k);
          }
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            float x, y;
            unpack2(fma2(pack2(a[k + j], a[k + j + 1]), c2, j ? nl.y : nl.x), x, y);
            x = ex2(x);
            y = ex2(y);
            const f2 w = pack2(x, y);
            const f2 z = mul2(w, add2(pack2(b[k + j], b[k + j + 1]), j ? nd.y : nd.x));
            if constexpr (KEYS) a[(k + j) / 2] = pack_bf16(x, y);
            unpack2(z, x, y);
            u[(k + j) / 2] = pack_bf16(x, y);
          }
        }
        if constexpr (KEYS) {
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = a[k];
          tmem_st_x16(tmem + lanes + Tm::P(s) + h * 16, v);
        } else if (partial(t)) {
          // keys that take no part: weight 0 whatever the products left there
          wait_warp(&bar->mready[t % NS], (t / NS) & 1, abort_flag, err);
          const uint32_t w = bar->kept[t % NS][h];
#pragma unroll
          for (int k = 0; k < 16; ++k) u[k] &= (w >> (2 * k) & 1u ? 0xffffu : 0u) | (w >> (2 * k + 1) & 1u ? 0xffff0000u : 0u);
        }
        tmem_st_x16(tmem + lanes + Tm::dS(s) + h * 16, u);
        tmem_st_wait();
      }
      tc_fence_before();
      warp_arrive(&bar->pfull[s]);
    }
    if (nt > 0) wait_warp(&bar->fin[1], 0, abort_flag, err);  // both streams' sums are complete
    tc_fence_after();
    // key pass: warpgroups 0, 1 write dV and 2, 3 dK, half of the channels each; query pass: a quarter of dQ's each,
    // at up to 64 channels by the first two
    if (warp_on) {
      const int64_t rows = KEYS ? (int64_t)p.nkv * p.Hkv : (int64_t)p.nq * p.Hq;
      const int64_t at = KEYS ? (int64_t)(f0 + row) * p.Hkv + hk : (int64_t)(f0 + row / p.r) * p.Hq + hk * p.r + row % p.r;
      const bool live = nt > 0 && !(KEYS && p.keep && row_on && p.keep[f0 + row] == 0);
      const float f = KEYS && s == 0 ? 1.f : p.scale;
      __nv_bfloat16* out = KEYS ? (s == 0 ? p.dV : p.dK) : p.dQ;
      float* part = KEYS ? (s == 0 ? p.part_v : p.part_k) : p.part_q;
      const int acc = KEYS && s == 0 ? Tm::kAcc1 : Tm::kAcc2;
      const int b_lo = KEYS ? h * DB : DB == 1 ? (s == 0 ? h : 2) : s * 2 + h, b_hi = KEYS ? h * DB + DB : DB == 1 && s == 1 ? 2 : b_lo + 1;
      for (int b = b_lo; b < b_hi; ++b) {
        if (b * 32 >= p.d) break;
        uint32_t o[32];
        if (nt > 0) {
          tmem_ld_32x32b_x32(tmem + lanes + acc + b * 32, o);
          tmem_ld_wait();
        }
        if (!row_on) continue;
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = live ? __uint_as_float(o[k]) * f : 0.f;
        if (splits > 1) store_row(part + (split * rows + at) * p.d + b * 32, v, p.d - b * 32);
        else store_row(out + at * p.d + b * 32, v, p.d - b * 32, p.wide);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (bar->abort_flag && warp == kLoadWarp && lane == 0 && nt > 0) {
    // a wait ran out somewhere: let the copies in flight land before the CTA gives its memory back
    volatile int never = 0;
    mbar_wait(&bar->ffull, 0, &never, err, kDefaultTimeoutNs);
    for (int i = loaded > NS ? loaded - NS : 0; i < loaded; ++i)
      mbar_wait(&bar->mfull[i % NS], (i / NS) & 1, &never, err, kDefaultTimeoutNs);
  }
}

template <int DB>
__global__ void __launch_bounds__(kThreads, 1) attn_bwd_kernel(const __grid_constant__ BwdParams p) {
  using Sh = BwdShape<DB>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* aligned = smem_raw + (base - smem_u32(smem_raw));
  const uint8_t* stats = aligned + 2 * Sh::kFixedBytes + Sh::kStages * (size_t)Sh::kStageBytes;
  BwdBarriers* bar = reinterpret_cast<BwdBarriers*>(aligned + 2 * Sh::kFixedBytes + Sh::kStages * (size_t)(Sh::kStageBytes + kStatBytes));
  const int warp = uniform(threadIdx.x >> 5);
  // set-up as in the forward kernel: the loader's barriers and first loads beside the tensor-memory allocation
  if (warp == kLoadWarp && (threadIdx.x & 31) == 0) {
    mbar_init(&bar->ffull, 1);
    for (int i = 0; i < Sh::kStages; ++i) mbar_init(&bar->mfull[i], 1), mbar_init(&bar->mempty[i], 1), mbar_init(&bar->mready[i], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->sfull[s], 1), mbar_init(&bar->pfull[s], 8);
      mbar_init(&bar->pdone[s], 1), mbar_init(&bar->adone[s], 1);
    }
    mbar_init(&bar->fin[0], 1), mbar_init(&bar->fin[1], 1);
    bar->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kSumWarp) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  pdl_wait();
  const int first = p.keys_first ? p.k_items : p.q_items, item = (int)blockIdx.x < first ? blockIdx.x : blockIdx.x - first;
  if (((int)blockIdx.x < first) == (p.keys_first != 0)) bwd_pass<DB, true>(p, item, base, bar, stats);
  else bwd_pass<DB, false>(p, item, base, bar, stats);
  if (warp == kSumWarp) tmem_dealloc(bar->tmem, 512);
}

// -lse in base 2 and -D = -dO . O of every (query token, head), 64 packed rows of a key head to a tile as the
// key pass reads them: group g's tiles start at tile q_off[g] / tokens + g, which leaves room for each
// group's last, partly filled one.  Rows that do not exist, and rows without any key, get -inf and 0, so
// that their weights vanish.  CTA (x, g): a tile and key head of group g; 2^k lanes a row, 8 channels a lane.
__global__ void __launch_bounds__(256) attn_stat_kernel(const __nv_bfloat16* __restrict__ dO, const __nv_bfloat16* __restrict__ O,
                                                        const float* __restrict__ lse, const int32_t* __restrict__ q_off, int nq,
                                                        int max_q, int Hq, int Hkv, int d, int lanes, int tiles,
                                                        float* __restrict__ stat) {
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, hk = blockIdx.x % Hkv, t = blockIdx.x / Hkv, r = Hq / Hkv, tokens = kMove / r;
  int q0, q1;
  if (group_range(q_off, g, nq, max_q, q0, q1) & SVCONV_STATUS_BAD_OFFSETS) return;
  if (t * tokens >= q1 - q0) return;
  float* out = stat + ((int64_t)hk * tiles + q0 / tokens + g + t) * kStat;
  const int sub = threadIdx.x & (lanes - 1);
  for (int row = threadIdx.x / lanes; row < kMove; row += 256 / lanes) {
    const int token = q0 + t * tokens + row / r;
    const bool on = row < tokens * r && token < q1;
    const int64_t at = (int64_t)token * Hq + hk * r + row % r;
    float v = 0.f;
    if (on && sub * 8 < d) {
      const uint4 a = *reinterpret_cast<const uint4*>(dO + at * d + sub * 8), b = *reinterpret_cast<const uint4*>(O + at * d + sub * 8);
      const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), v);
        v = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), v);
      }
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (sub == 0) {
      const float l = on ? lse[at] : -INFINITY;
      out[row] = l == -INFINITY ? -INFINITY : -l * kLog2e;
      out[kMove + row] = on ? -v : 0.f;
    }
  }
}

// The splits of a gradient added in order: 8 channels a thread over the rows of group blockIdx.y.
__global__ void __launch_bounds__(256) attn_sum_kernel(const float* __restrict__ part, int splits, const int32_t* off, const int32_t* off2,
                                                       int n, int n2, int bound, int H, int d, __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  int lo, hi, lo2, hi2;
  const int flags = group_range(off, blockIdx.y, n, bound, lo, hi) | group_range(off2, blockIdx.y, n2, n2, lo2, hi2);
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if ((flags & SVCONV_STATUS_BAD_OFFSETS) || i >= (int64_t)(hi - lo) * H * d) return;
  const int64_t at = (int64_t)lo * H * d + i, step = (int64_t)n * H * d;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4 a = *reinterpret_cast<const float4*>(part + s * step + at), b = *reinterpret_cast<const float4*>(part + s * step + at + 4);
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
  }
  *reinterpret_cast<uint4*>(out + at) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// ---------------------------------------------------------------------------- host side
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

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
  if (o.d < 8 || o.d > kMaxD || o.d % 8 != 0 || o.Hq % o.Hkv != 0 || o.Hq / o.Hkv > kMove) return SVCONV_ERR_UNSUPPORTED;
  if (!std::isfinite(o.scale)) return SVCONV_ERR_SIZE;
  if (o.G > 0 && (!o.q_off || !o.kv_off)) return SVCONV_ERR_NULL;
  if (!fix_strides(o.q_row, o.q_head, o.nq, o.Hq, o.d) || !fix_strides(o.k_row, o.k_head, o.nkv, o.Hkv, o.d) ||
      !fix_strides(o.v_row, o.v_head, o.nkv, o.Hkv, o.d))
    return SVCONV_ERR_ALIGN;
  if (o.max_q > o.nq) o.max_q = o.nq;
  if (o.max_kv > o.nkv) o.max_kv = o.nkv;
  return SVCONV_OK;
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

// How a forward call is cut: pair or split form, and over how many splits of the keys.  The candidates are
// compared by the time of whole rounds of CTAs over 148 SMs (a fixed number, so the workspace size needs no device
// query), with the group lengths known only by their sum and bound.  In units of one key tile for both streams (about
// 1.1 us): a tile costs 1 in the pair form and 1/2 in the split form, a CTA kFixed besides, and splits their
// partial results.  Measured with 184 units of 64 key tiles of 128 channels: one split of the pair form 331 us.
constexpr int kSms = 148, kMinTiles = 4;
constexpr double kFixed = 3.5, kMerge = 3.0, kMergeBytes = 5.5e6;  // merge: a launch, and bytes a unit
struct FwdPlan {
  int pair, qblocks, splits;
};
double blocks_est(int n, int longest, int G, int rows) {  // blocks of `rows` rows over all groups
  const double most = (double)G * cdiv(longest, rows);
  double est = (double)n / rows + 0.5 * G;  // a group's last block is half full
  if (est < G) est = G;
  return est < most ? est : most;
}
FwdPlan plan_fwd(const svconv_cross_attn_desc& c) {
  const int tokens = kTile / (c.Hq / c.Hkv), tiles = cdiv(c.max_kv, kTile);
  const double merge_bytes = (double)c.nq * c.Hq * c.d * 8.0;
  FwdPlan best{};
  double best_t = 0.0;
  for (int pair = c.max_q > tokens ? 1 : 0; pair >= 0; --pair) {
    const int rows = tokens * (pair ? 2 : 1);
    const double units = c.Hkv * blocks_est(c.nq, c.max_q, c.G, rows);
    for (int s = 1; s == 1 || (s * kMinTiles <= tiles && units * s <= 8.0 * kSms); ++s) {
      const double rounds = units * s <= kSms ? 1.0 : std::ceil(units * s / kSms);
      const double t = rounds * ((double)cdiv(tiles, s) * (pair ? 1.0 : 0.5) + kFixed) + (s > 1 ? kMerge + merge_bytes * s / kMergeBytes : 0.0);
      if (best_t == 0.0 || t < best_t * 0.98) best_t = t, best = FwdPlan{pair, cdiv(c.max_q, rows), s};
    }
  }
  return best;
}

// The same for the two passes of the backward call, which share one launch.  A pass whose single item would take
// more than kLong of an SM's share of all work is split until it does not; the pass with the longer items goes first.
// In units of one moving tile of the query pass.
constexpr double kBwdFixed = 5.0, kKeyTile = 1.3, kLong = 0.5;
struct BwdPlan {
  int qblocks, qsplits, kblocks, ksplits, keys_first;
  int tiles;            // of statistics, for each key head
  size_t stat, pq, pk;  // floats: statistics, split partials of dQ, of dK (and again of dV)
  size_t floats() const { return stat + pq + 2 * pk; }
};
BwdPlan plan_bwd(const svconv_cross_attn_desc& c) {
  BwdPlan b;
  const int r = c.Hq / c.Hkv, G = c.G > 0 ? c.G : 1;
  const int tq = cdiv(c.max_kv, kMove), tk = cdiv(c.max_q, kMove / r);  // moving tiles of an item of the query / key pass
  b.qblocks = cdiv(c.max_q, kTile / r);
  b.kblocks = cdiv(c.max_kv, kTile);
  const double all = c.Hkv * (blocks_est(c.nq, c.max_q, G, kTile / r) * (cdiv(c.nkv, G * kMove) + kBwdFixed) +
                              blocks_est(c.nkv, c.max_kv, G, kTile) * (cdiv(c.nq, G * (kMove / r)) * kKeyTile + kBwdFixed));
  const double share = all / kSms;
  auto splits = [&](int tiles, double tile) {
    int s = (int)std::ceil(tiles * tile / (kLong * share));
    const int most = tiles / (2 * kMinTiles);
    if (s > most) s = most;
    return s < 1 ? 1 : s;
  };
  b.qsplits = b.qblocks ? splits(tq, 1.0) : 1;
  b.ksplits = b.kblocks ? splits(tk, kKeyTile) : 1;
  b.keys_first = (double)tk * kKeyTile / b.ksplits > (double)tq / b.qsplits;
  const size_t nq = (size_t)c.nq * c.Hq, nk = (size_t)c.nkv * c.Hkv;
  b.tiles = c.nq / (kMove / r) + c.G + 1;
  b.stat = (size_t)b.tiles * c.Hkv * kStat;
  b.pq = b.qsplits > 1 ? b.qsplits * nq * c.d : 0;
  b.pk = b.ksplits > 1 ? b.ksplits * nk * c.d : 0;
  return b;
}

template <int DB>
cudaError_t launch_bwd(const BwdParams& p, int grid, cudaStream_t s) {
  static int done[64];
  cudaError_t e = ensure_smem_attr(attn_bwd_kernel<DB>, BwdShape<DB>::kSmem, done);
  return e == cudaSuccess ? launch_pdl(attn_bwd_kernel<DB>, dim3(grid), dim3(kThreads), BwdShape<DB>::kSmem, s, p) : e;
}

template <int DB>
cudaError_t launch_fwd(const FwdParams& p, int grid, cudaStream_t s) {
  static int done[64];
  cudaError_t e = ensure_smem_attr(attn_fwd_kernel<DB>, FwdShape<DB>::kSmem, done);
  return e == cudaSuccess ? launch_pdl(attn_fwd_kernel<DB>, dim3(grid), dim3(kThreads), FwdShape<DB>::kSmem, s, p) : e;
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
  if (check_desc(desc, c) || c.G == 0) return 0;
  return plan_bwd(c).floats() * sizeof(float);
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
  p.wide = c.d % 16 == 0 && aligned32(O);
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
  // a CTA a row hides the chain of many splits; it is wasteful for few (170 us against 20 at 47k rows of 2 splits)
  if (e == cudaSuccess && f.splits > 8)
    e = launch_pdl(attn_combine_kernel, dim3(c.max_q, c.Hq, c.G), dim3(256), 0, s, p);
  else if (e == cudaSuccess && f.splits > 1)
    e = launch_pdl(attn_merge_kernel, dim3((unsigned)(((int64_t)c.max_q * c.Hq + 7) / 8), c.G), dim3(256), 0, s, p);
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
  const BwdPlan b = plan_bwd(c);
  const long long heads = (long long)c.G * c.Hkv;
  const long long q_items = heads * b.qblocks * b.qsplits, k_items = heads * b.kblocks * b.ksplits;
  const int r = c.Hq / c.Hkv;
  int lanes = 1;
  while (lanes < c.d / 8) lanes *= 2;
  const long long stat_grid = (long long)cdiv(c.max_q, kMove / r) * c.Hkv;
  if (q_items + k_items > 0x7fffffffLL || stat_grid > 0x7fffffffLL) return SVCONV_ERR_SIZE;
  float* ws = static_cast<float*>(workspace);
  BwdParams p{};
  p.q_off = c.q_off, p.kv_off = c.kv_off, p.keep = c.kv_keep;
  p.nq = c.nq, p.nkv = c.nkv, p.max_q = c.max_q, p.max_kv = c.max_kv, p.Hq = c.Hq, p.Hkv = c.Hkv, p.r = r, p.d = c.d;
  p.qblocks = b.qblocks, p.qsplits = b.qsplits, p.kblocks = b.kblocks, p.ksplits = b.ksplits;
  p.q_items = (int)q_items;
  p.k_items = (int)k_items;
  p.keys_first = b.keys_first;
  p.c = c.scale * kLog2e;
  p.scale = c.scale;
  p.stat = ws;
  p.stat_tiles = b.tiles;
  p.part_q = ws + b.stat;
  p.part_k = p.part_q + b.pq;
  p.part_v = p.part_k + b.pk;
  p.dQ = static_cast<__nv_bfloat16*>(dQ);
  p.dK = static_cast<__nv_bfloat16*>(dK);
  p.dV = static_cast<__nv_bfloat16*>(dV);
  p.wide = c.d % 16 == 0 && aligned32(dQ) && aligned32(dK) && aligned32(dV);
  p.status = dev_status ? dev_status : device_error_word();
  // a side without rows: its maps only have to be well formed
  const void *q = c.nq ? Q : K, *go = c.nq ? dO : K, *k = c.nkv ? K : Q, *v = c.nkv ? V : Q;
  const int64_t go_row = (int64_t)c.Hq * c.d, go_head = c.d;
  if (!make_packed_map(&p.fq, q, c.nq, c.Hkv, r, c.d, c.q_row, c.q_head, kTile / r) ||
      !make_packed_map(&p.mq, q, c.nq, c.Hkv, r, c.d, c.q_row, c.q_head, kMove / r) ||
      !make_packed_map(&p.fdo, go, c.nq, c.Hkv, r, c.d, go_row, go_head, kTile / r) ||
      !make_packed_map(&p.mdo, go, c.nq, c.Hkv, r, c.d, go_row, go_head, kMove / r) ||
      !make_rows_map(&p.fk, k, c.nkv, c.Hkv, c.d, c.k_row, c.k_head, kTile) ||
      !make_rows_map(&p.mk, k, c.nkv, c.Hkv, c.d, c.k_row, c.k_head, kMove) ||
      !make_rows_map(&p.fv, v, c.nkv, c.Hkv, c.d, c.v_row, c.v_head, kTile) ||
      !make_rows_map(&p.mv, v, c.nkv, c.Hkv, c.d, c.v_row, c.v_head, kMove))
    return SVCONV_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (c.max_q > 0)
    e = launch_pdl(attn_stat_kernel, dim3((unsigned)stat_grid, c.G), dim3(256), 0, s, static_cast<const __nv_bfloat16*>(dO),
                   static_cast<const __nv_bfloat16*>(O), lse, c.q_off, c.nq, c.max_q, c.Hq, c.Hkv, c.d, lanes, b.tiles, ws);
  if (e == cudaSuccess)
    e = c.d <= 64 ? launch_bwd<1>(p, (int)(q_items + k_items), s) : launch_bwd<2>(p, (int)(q_items + k_items), s);
  auto add = [&](const float* part, int splits, const int32_t* off, const int32_t* off2, int n, int n2, int bound, int H,
                 __nv_bfloat16* out) {
    if (e != cudaSuccess || splits < 2) return;
    const long long grid = ((long long)bound * H * c.d / 8 + 255) / 256;
    e = launch_pdl(attn_sum_kernel, dim3((unsigned)grid, c.G), dim3(256), 0, s, part, splits, off, off2, n, n2, bound, H, c.d, out);
  };
  add(p.part_q, b.qsplits, c.q_off, c.kv_off, c.nq, c.nkv, c.max_q, c.Hq, p.dQ);
  add(p.part_k, b.ksplits, c.kv_off, c.q_off, c.nkv, c.nq, c.max_kv, c.Hkv, p.dK);
  add(p.part_v, b.ksplits, c.kv_off, c.q_off, c.nkv, c.nq, c.max_kv, c.Hkv, p.dV);
  return e == cudaSuccess ? SVCONV_OK : SVCONV_ERR_CUDA;
}

}  // extern "C"
