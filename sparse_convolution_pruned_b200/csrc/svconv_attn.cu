// Cross-attention of packed groups, forward and backward: every query row attends over the kept
// keys of its group (see svconv_cross_attn_fwd in svconv.h for the definition).
// Scores are in base 2: scale * log2(e) is one factor, and every exponential is one ex2.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>
#include <cstddef>
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
__device__ __forceinline__ uint32_t try_wait_many(uint32_t bar, uint32_t parity) {
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
      : "r"(bar), "r"(parity)
      : "memory");
  return left;
}
__device__ __forceinline__ void wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
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
__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  wait_for(smem_u32(bar), parity, abort_flag, err);
}
// The whole warp waits, and is converged afterwards; mostly the first try succeeds, and a vote is all it takes.
__device__ __forceinline__ void wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
  wait_for(bar, parity, abort_flag, err);
  __syncwarp();
}
// The same with the barrier at a fixed offset from a shared-memory address that the loop holds anyway: the softmax
// loops are short of registers, and one for each barrier's address is spilled.
template <int OFF>
__device__ __forceinline__ void wait_at(uint32_t at, uint32_t parity, volatile int* abort_flag, int* err) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1 + %3], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(at), "r"(parity), "n"(OFF)
      : "memory");
  if (__all_sync(0xffffffffu, ok != 0)) return;
  wait_for(at + OFF, parity, abort_flag, err);
  __syncwarp();
}
template <int OFF>
__device__ __forceinline__ void arrive_at(uint32_t at) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0 + %1];" ::"r"(at), "n"(OFF) : "memory");
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

// What rounding a pair to bf16 left behind, as bf16 again
__device__ __forceinline__ uint32_t rest_bf16(float lo, float hi, uint32_t rounded) {
  return pack_bf16(lo - __uint_as_float(rounded << 16), hi - __uint_as_float(rounded & 0xffff0000u));
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

// 16 consecutive values of a row, of which `n` exist (a multiple of 8), by 32-byte stores where the row allows it
__device__ __forceinline__ void store_row(float* dst, const float (&f)[16], int n) {
#pragma unroll
  for (int k = 0; k < 16; k += 8)
    if (k < n) st_global_32(dst + k, reinterpret_cast<const uint32_t*>(f) + k);  // rows of 8 k floats from a 32-byte boundary (ws_floats)
}
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, const float (&f)[16], int n, bool wide) {
  uint32_t v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = pack_bf16(f[2 * k], f[2 * k + 1]);
  if (wide && n >= 16) {
    st_global_32(dst, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; k += 4)
      if (2 * k < n) *reinterpret_cast<uint4*>(dst + 2 * k) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
  }
}

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
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
  int nq, nkv, max_q, max_kv, Hq, Hkv, r, d, G;
  int tokens;       // query tokens of a tile: 128 / r
  int splits, pair;
  float c;          // scale * log2(e)
  int wide;         // rows of O start on 32-byte boundaries
  __nv_bfloat16* O;
  float* lse;
  float* part_o;    // [splits][nq * Hq][d] unnormalised, and
  float* part_ml;   // [splits][nq * Hq][2] (maximum in base 2, sum), when splits > 1
  int* status;
};

// One piece of work: a query block of a key head of a group, over one split of the keys.
struct FwdItem {
  int nt;                    // key tiles; -1: no more items
  int steps0, steps1;        // of them, the steps of each stream
  int tok0, q1;              // first query token of the block, end of the group
  int k0, k1;                // first key of the split, end of the group
  int hk, split;
};

// Walks the items of the whole call in order.  A warp keeps 32 groups at a time, one per lane, so finding an
// item is a vote and some shuffles, and groups without queries take no item.
struct FwdCursor {
  int chunk, base, incl, q0, q1, k0, k1;

  __device__ __forceinline__ void load(const FwdParams& p) {
    const int g = chunk * 32 + (threadIdx.x & 31);
    int cnt = 0;
    q0 = q1 = k0 = k1 = 0;
    if (g < p.G) {
      const int f = group_range(p.q_off, g, p.nq, p.max_q, q0, q1) | group_range(p.kv_off, g, p.nkv, p.max_kv, k0, k1);
      const int rows = p.tokens * (p.pair ? 2 : 1);
      if (!(f & SVCONV_STATUS_BAD_OFFSETS)) cnt = (q1 - q0 + rows - 1) / rows * p.splits * p.Hkv;
    }
    incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if ((int)(threadIdx.x & 31) >= o) incl += v;
    }
  }
  __device__ __forceinline__ bool find(const FwdParams& p, int v, FwdItem& it) {
    int total = __shfl_sync(0xffffffffu, incl, 31);
    while (v >= base + total) {
      base += total;
      if (++chunk * 32 >= p.G) return false;
      load(p);
      total = __shfl_sync(0xffffffffu, incl, 31);
    }
    const int j = __ffs(__ballot_sync(0xffffffffu, v - base < incl)) - 1;
    const int before = __shfl_sync(0xffffffffu, incl, j > 0 ? j - 1 : 0);
    int i = v - base - (j > 0 ? before : 0);
    const int a0 = __shfl_sync(0xffffffffu, q0, j), b0 = __shfl_sync(0xffffffffu, k0, j);
    it.q1 = __shfl_sync(0xffffffffu, q1, j);
    it.k1 = __shfl_sync(0xffffffffu, k1, j);
    // query block fastest, so CTAs that run together share keys in L2
    const int rows = p.tokens * (p.pair ? 2 : 1), blocks = (it.q1 - a0 + rows - 1) / rows;
    it.tok0 = a0 + i % blocks * rows;
    i /= blocks;
    it.split = i % p.splits;
    it.hk = i / p.splits;
    const int tiles = (it.k1 - b0 + kTile - 1) / kTile;
    const int lo = (int)((int64_t)tiles * it.split / p.splits), hi = (int)((int64_t)tiles * (it.split + 1) / p.splits);
    it.nt = hi - lo;
    it.k0 = b0 + lo * kTile;
    it.steps0 = p.pair ? it.nt : (it.nt + 1) / 2;
    it.steps1 = p.pair ? (it.tok0 + p.tokens < it.q1 ? it.nt : 0) : it.nt / 2;
    return true;
  }
};

constexpr int kItems = 4;  // items the loader may be ahead
// Named barriers of the forward kernel: 1 to 8 the two warps of a row quarter (stream x 4 + quarter), 9 to 12 the
// streams' merge, and the start; 0 is __syncthreads.
constexpr int kPairBarrier = 1, kMergeBarrier = 9, kStartBarrier = 13;

struct FwdBarriers {
  uint64_t ifull[kItems], iempty[kItems], qfull[2], qempty[2], kvfull[8], kvempty[8], vready[8];
  uint64_t sfull[2], sread[2], pfull[2], odone[2], oread[2], fin[2];
  FwdItem item[kItems];
  uint32_t kept[8][4];           // keys that take part, of the tile whose V lies in this slot
  float rowmax[2][2][2][kTile];  // [step parity][stream][half of the columns][row], exchanged between the halves
  float rowsum[2][2][kTile];     // the same for the sums at an item's end
  float state[2][2][kTile];      // split form: [half][maximum, sum][row] of the second stream
  uint32_t tmem;
  int abort_flag;
};

template <int DB>  // 64-channel blocks: 1 (d <= 64) or 2
struct FwdShape {
  static constexpr int kTileBytes = DB * kBlockBytes;
  static constexpr int kQSets = DB == 1 ? 2 : 1;  // looping, the next item's query tiles are loaded ahead
  static constexpr int kStages = DB == 1 ? 8 : 4;
  static constexpr size_t kSmem = 1024 + (2 * kQSets + kStages) * (size_t)kTileBytes + sizeof(FwdBarriers);
  static constexpr int kQ(int set, int s) { return (s * kQSets + set) * kTileBytes; }
  static constexpr int kExchange = kQSets * kTileBytes;  // split form: the unused second stream's query tiles, 32 KB
  // tensor memory: at 64 channels P has columns of its own, so the next S can be issued before P V; at 128 it takes S's
  static constexpr int kS(int s) { return s * 128; }
  static constexpr int kP(int s) { return DB == 1 ? 256 + s * 64 : s * 128; }
  static constexpr int kO(int s) { return DB == 1 ? 384 + s * 64 : 256 + s * 128; }
};

// The end of an item: the streams' states merged (split form), O divided by the sum and written, or kept as a
// split's partial result.
template <int DB, bool PAIR>
__device__ __forceinline__ void fwd_output(const FwdParams& p, const FwdItem* it, FwdBarriers* bar, uint32_t tmem, float* exchange, int s,
                                        int half, int row, int steps, float m2, float l) {
  using Sh = FwdShape<DB>;
  const int left = min(p.tokens, it->q1 - it->tok0 - (PAIR ? s * p.tokens : 0)) * p.r;
  const bool warp_on = (row & ~31) < left;
  const int merge_bar = kMergeBarrier + half * 2 + (row >> 6);  // named barrier of the two streams' warps of two quarters and this half
  m2 = l > 0.f ? m2 : -INFINITY;  // no key
  if (!(l > 0.f) && !(l == 0.f)) m2 = l;    // NaN scores: carried along
  // split form: the second stream hands its state over, 32 columns of each half at a time
  float* ex = exchange + half * 32 * kTile + row;
  const bool merge = !PAIR && it->steps1 > 0;
  if (merge && s == 1) {
    bar->state[half][0][row] = m2;
    bar->state[half][1][row] = l;
#pragma unroll
    for (int b = 0; b < DB; ++b) {
      if (warp_on) {
#pragma unroll 1
        for (int c = 0; c < 32; c += 16) {
          uint32_t o[16];
          tmem_ld_x16(tmem + Sh::kO(s) + (half * DB + b) * 32 + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) ex[(c + k) * kTile] = __uint_as_float(o[k]);
        }
      }
      asm volatile("bar.sync %0, 128;" ::"r"(merge_bar) : "memory");  // written
      asm volatile("bar.sync %0, 128;" ::"r"(merge_bar) : "memory");  // read
    }
  }
  if (PAIR || s == 0) {
    const int token = it->tok0 + (PAIR ? s * p.tokens : 0) + row / p.r, head = it->hk * p.r + row % p.r;
    const int64_t out = (int64_t)token * p.Hq + head, part = it->split * (int64_t)p.nq * p.Hq + out;
    float f0 = 1.f, f1 = 0.f, inv = 1.f;
#pragma unroll
    for (int b = 0; b < DB; ++b) {  // each half writes half of the channels
      const int c0 = (half * DB + b) * 32;
      if (merge) asm volatile("bar.sync %0, 128;" ::"r"(merge_bar) : "memory");
      if (b == 0) {
        if (merge) {
          const float m1 = bar->state[half][0][row], l1 = bar->state[half][1][row];
          const float top = fmaxf(m2, m1);
          f0 = m2 == -INFINITY ? 0.f : ex2(m2 - top);
          f1 = m1 == -INFINITY ? 0.f : ex2(m1 - top);
          l = l * f0 + l1 * f1;
          m2 = (l == l) ? top : l;
        }
        inv = p.splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
      }
      if (warp_on) {
#pragma unroll 1
        for (int c = c0; c < c0 + 32; c += 16) {
          uint32_t o[16];
          if (steps > 0) {
            tmem_ld_x16(tmem + Sh::kO(s) + c, o);
            tmem_ld_wait();
          }
          float f[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            f[k] = steps > 0 && l != 0.f ? __uint_as_float(o[k]) : 0.f;
            if (merge) f[k] = f[k] * f0 + (f1 != 0.f ? ex[(c - c0 + k) * kTile] * f1 : 0.f);
            f[k] *= inv;
          }
          if (row < left && c < p.d) {
            if (p.splits > 1) store_row(p.part_o + part * p.d + c, f, p.d - c);
            else store_row(p.O + out * p.d + c, f, p.d - c, p.wide);
          }
        }
      }
      if (merge) asm volatile("bar.sync %0, 128;" ::"r"(merge_bar) : "memory");
    }
    if (row < left && half == 0) {
      if (p.splits > 1) *reinterpret_cast<float2*>(p.part_ml + part * 2) = make_float2(m2, l);
      else p.lse[out] = l == 0.f ? -INFINITY : (m2 + log2f(l)) * kLn2;
    }
  }
}

// LOOP: a CTA takes every gridDim.x-th item.  Set-up, tensor memory and descriptors are paid once, and the warps
// run ahead of each other from item to item: the loader by the rings' depth, the products by a tile, so one stream's
// output and the next item's first tiles overlap (a CTA per item takes 8.7 us for one tile of keys, of which 3 us are
// set-up and release, and 2 us loads with nothing to do beside them).  Otherwise a CTA takes one item: with many key
// tiles an item that is the faster form, because in the loop the output's registers spill the softmax's (kLoopTiles).
template <int DB, bool PAIR, bool LOOP>
__global__ void __launch_bounds__(kThreads, 1) attn_fwd_kernel(const __grid_constant__ FwdParams p) {
  using Sh = FwdShape<DB>;
  constexpr int NS = Sh::kStages, NQ = Sh::kQSets;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* aligned = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t skv = base + 2 * NQ * Sh::kTileBytes;
  FwdBarriers* bar = reinterpret_cast<FwdBarriers*>(aligned + (2 * NQ + NS) * (size_t)Sh::kTileBytes);
  volatile int* abort_flag = &bar->abort_flag;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  int* err = p.status;

  if (warp == kLoadWarp && lane == 0) {
    for (int i = 0; i < kItems; ++i) mbar_init(&bar->ifull[i], 1), mbar_init(&bar->iempty[i], kSoftWarps + 3);
    // K and V tiles alternate, so V's slots are the odd ones: the check warp has to be done with those too
    for (int i = 0; i < NS; ++i) mbar_init(&bar->kvfull[i], 1), mbar_init(&bar->kvempty[i], 1 + (i & 1)), mbar_init(&bar->vready[i], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->qfull[s], 1), mbar_init(&bar->qempty[s], 1), mbar_init(&bar->sfull[s], 1), mbar_init(&bar->sread[s], 8);
      mbar_init(&bar->pfull[s], 8), mbar_init(&bar->odone[s], 1), mbar_init(&bar->oread[s], 8), mbar_init(&bar->fin[s], 1);
    }
    bar->abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&p.tq), prefetch_tmap(&p.tk), prefetch_tmap(&p.tv);
  }
  if (warp == kSumWarp) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  // The loader made the barriers itself and needs no tensor memory: it goes ahead.  On a barrier of its own: the loader may
  // be at the kernel's last __syncthreads before tensor memory is there, and must not be counted twice.
  if (warp == kLoadWarp) asm volatile("bar.arrive %0, %1;" ::"n"(kStartBarrier), "n"(kThreads) : "memory");
  else asm volatile("bar.sync %0, %1;" ::"n"(kStartBarrier), "n"(kThreads) : "memory");
  tc_fence_after();
  pdl_wait();
  // After the tensor memory is there: the next kernel's CTAs may come and ask for theirs.  So not from the loader, which does
  // not wait for it.
  if (warp != kLoadWarp) pdl_trigger();

  int loaded = 0, qloaded = 0;  // K / V tiles and query sets whose loads were issued
  if (warp == kLoadWarp) {
    FwdCursor cur{};
    cur.load(p);
    int n = 0;
    for (int v = blockIdx.x;; v += gridDim.x, ++n) {
      const int slot = n % kItems;
      if (n >= kItems) wait_warp(&bar->iempty[slot], ((n / kItems) & 1) ^ 1, abort_flag, err);
      FwdItem it;
      it.nt = -1;
      const bool have = cur.find(p, v, it);
      if (lane == 0) {
        bar->item[slot] = it;
        mbar_arrive(&bar->ifull[slot]);
      }
      if (!have) break;
      if (lane == 0)
        for (int j = 0; j < 2 * it.nt; ++j) {  // K, V of each tile in turn
          const int kv = loaded % NS;
          if (loaded >= NS) wait_for(&bar->kvempty[kv], ((loaded / NS) & 1) ^ 1, abort_flag, err);
          if (*abort_flag) break;
          mbar_arrive_expect_tx(&bar->kvfull[kv], Sh::kTileBytes);
          for (int b = 0; b < DB; ++b)
            tma_load_3d(skv + kv * Sh::kTileBytes + b * kBlockBytes, (j & 1) ? &p.tv : &p.tk, &bar->kvfull[kv], b * 64, it.hk, it.k0 + j / 2 * kTile);
          ++loaded;
          if (j == 0) {
            const int set = qloaded % NQ, tiles = PAIR && it.steps1 > 0 ? 2 : 1;
            if (qloaded >= NQ) wait_for(&bar->qempty[set], ((qloaded / NQ) & 1) ^ 1, abort_flag, err);
            if (*abort_flag) break;
            mbar_arrive_expect_tx(&bar->qfull[set], (uint32_t)(p.tokens * p.r * tiles) * 128u * DB);
            for (int s = 0; s < tiles; ++s)
              for (int b = 0; b < DB; ++b)
                tma_load_4d(base + Sh::kQ(set, s) + b * kBlockBytes, &p.tq, &bar->qfull[set], b * 64, 0, it.hk, it.tok0 + s * p.tokens);
            ++qloaded;
          }
        }
      if (!LOOP) break;
    }
    if (blockIdx.x == 0) {  // every group is looked at once for the status word
      for (int g = lane; g < p.G; g += 32) {
        int a0, a1;
        const int f = group_range(p.q_off, g, p.nq, p.max_q, a0, a1) | group_range(p.kv_off, g, p.nkv, p.max_kv, a0, a1);
        if (f) atomicOr(err, f);
      }
    }
  } else if (warp == kScoreWarp) {
    const uint32_t e = lane == 0;
    const int ks = (p.d + 15) / 16;
    const uint32_t idesc = idesc_bf16_f32(kTile, kTile, 0, 0), tm = uniform(bar->tmem);
    constexpr bool pair = PAIR;
    const uint64_t dq = smem_desc_sw128(base, 16, 1024), dk = smem_desc_sw128(skv, 16, 1024);
    int done0 = 0, done1 = 0, seq = 0, sets = 0;  // steps of each stream, K / V tiles and query sets before this item
    for (int n = 0;; ++n) {
      const int at = n % kItems;
      wait_warp(&bar->ifull[at], (n / kItems) & 1, abort_flag, err);
      const int nt = uniform(bar->item[at].nt), steps0 = uniform(bar->item[at].steps0), steps1 = uniform(bar->item[at].steps1);
      warp_arrive(&bar->iempty[at]);
      if (nt < 0) break;
      if (nt == 0) {
        if (LOOP) continue;
        break;
      }
      const bool lone = steps1 == 0;
      const int set = sets % NQ;
      wait_warp(&bar->qfull[set], (sets / NQ) & 1, abort_flag, err);
      for (int i = 0; i < steps0; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (i >= (s ? steps1 : steps0)) continue;
          const int tile = pair ? i : 2 * i + s, k = seq + 2 * tile, slot = k % NS, step = (s ? done1 : done0) + i;
          // S is free once its scores have been read; where P lies in its columns, once P V is done too
          if (step > 0) wait_warp(DB == 1 ? &bar->sread[s] : &bar->odone[s], (step - 1) & 1, abort_flag, err);
          if (!pair || s == 0) wait_warp(&bar->kvfull[slot], (k / NS) & 1, abort_flag, err);
          tc_fence_after();
          const uint64_t a0 = dq + (uint64_t)((set + (pair && s ? NQ : 0)) * (Sh::kTileBytes >> 4)), b0 = dk + (uint64_t)(slot * (Sh::kTileBytes >> 4));
#pragma unroll
          for (int c = 0; c < 4 * DB; ++c) {
            const uint64_t off = (uint64_t)((c >> 2) * (kBlockBytes >> 4) + (c & 3) * 2);
            if (c < ks) mma_ss(tm + Sh::kS(s), a0 + off, b0 + off, idesc, c ? 1u : 0u, e);
          }
          commit_to(&bar->sfull[s], e);
          // the tile's last reader frees it (pair form: the second stream, where it has rows)
          if (!pair || s == 1 || lone) commit_to(&bar->kvempty[slot], e);
        }
      commit_to(&bar->qempty[set], e);
      done0 += steps0, done1 += steps1, seq += 2 * nt, ++sets;
      if (!LOOP) break;
    }
    commit_to(&bar->fin[0], e);  // every issued product is complete before tensor memory is released
    wait_warp(&bar->fin[0], 0, abort_flag, err);
  } else if (warp == kSumWarp) {
    const uint32_t e = lane == 0;
    const uint32_t idesc = idesc_bf16_f32(kTile, (p.d + 15) / 16 * 16, 0, 1), tm = uniform(bar->tmem);
    constexpr bool pair = PAIR;
    const uint64_t dv = smem_desc_sw128(skv, kBlockBytes, 1024);
    int done0 = 0, done1 = 0, seq = 0, outs0 = 0, outs1 = 0;  // outs: items in which the stream had an output before this one
    for (int n = 0;; ++n) {
      const int at = n % kItems;
      wait_warp(&bar->ifull[at], (n / kItems) & 1, abort_flag, err);
      const int nt = uniform(bar->item[at].nt), steps0 = uniform(bar->item[at].steps0), steps1 = uniform(bar->item[at].steps1);
      const int k0 = uniform(bar->item[at].k0), k1 = uniform(bar->item[at].k1);
      warp_arrive(&bar->iempty[at]);
      if (nt < 0) break;
      const bool lone = steps1 == 0;
      for (int i = 0; i < steps0; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (i >= (s ? steps1 : steps0)) continue;
          const int tile = pair ? i : 2 * i + s, k = seq + 2 * tile + 1, slot = k % NS, step = (s ? done1 : done0) + i;
          // rows of V behind the group's end or dropped by the mask must be zero: their weights are
          if (!pair || s == 0)
            wait_warp(p.keep || k0 + (tile + 1) * kTile > k1 ? &bar->vready[slot] : &bar->kvfull[slot], (k / NS) & 1, abort_flag, err);
          // Where the next scores wait for P V, they go first: O_0, S_0, O_1, S_1 in turn keeps the streams half a
          // period apart, one's softmax under the other's products (left alone they fall into step: 4,700 cycles
          // for both streams' tiles instead of 4,000)
          if constexpr (DB == 2) {
            if (s == 0 && i > 0 && i < steps1) wait_warp(&bar->sfull[1], (done1 + i) & 1, abort_flag, err);
            if (s == 1 && i + 1 < steps0) wait_warp(&bar->sfull[0], (done0 + i + 1) & 1, abort_flag, err);
          }
          if (i == 0 && (s ? outs1 : outs0) > 0) wait_warp(&bar->oread[s], ((s ? outs1 : outs0) - 1) & 1, abort_flag, err);
          wait_warp(&bar->pfull[s], step & 1, abort_flag, err);
          tc_fence_after();
          const uint64_t b0 = dv + (uint64_t)(slot * (Sh::kTileBytes >> 4));
#pragma unroll
          for (int c = 0; c < kTile / 16; ++c)
            mma_ts(tm + Sh::kO(s), tm + Sh::kP(s) + c * 8, b0 + (uint64_t)(c * (2048 >> 4)), idesc, (i | c) ? 1u : 0u, e);
          commit_to(&bar->odone[s], e);
          if (!pair || s == 1 || lone) commit_to(&bar->kvempty[slot], e);
        }
      done0 += steps0, done1 += steps1, seq += 2 * nt, outs0 += steps0 > 0, outs1 += steps1 > 0;
      if (!LOOP) break;
    }
    commit_to(&bar->fin[1], e);
    wait_warp(&bar->fin[1], 0, abort_flag, err);
  } else if (warp == kCheckWarp) {
    int seq = 0;
    for (int n = 0;; ++n) {
      const int at = n % kItems;
      wait_warp(&bar->ifull[at], (n / kItems) & 1, abort_flag, err);
      const int nt = uniform(bar->item[at].nt), k0 = uniform(bar->item[at].k0), k1 = uniform(bar->item[at].k1);
      warp_arrive(&bar->iempty[at]);
      if (nt < 0) break;
      for (int tile = 0; tile < nt; ++tile) {
        const int k = seq + 2 * tile + 1, slot = k % NS;
        wait_warp(&bar->kvfull[slot], (k / NS) & 1, abort_flag, err);
        if (p.keep || k0 + (tile + 1) * kTile > k1) {
          uint32_t w[4];
          kept_words(p.keep, k0 + tile * kTile, k1, w);
          if (lane < 4) bar->kept[slot][lane] = lane == 0 ? w[0] : lane == 1 ? w[1] : lane == 2 ? w[2] : w[3];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = ~w[i];
          scrub_rows(skv + slot * Sh::kTileBytes, DB, kBlockBytes, w);
        }
        warp_arrive(&bar->vready[slot]);
        warp_arrive(&bar->kvempty[slot]);
      }
      seq += 2 * nt;
      if (!LOOP) break;
    }
  } else {
    // ------------------------------------------------------------ softmax: two threads per row, 64 scores each
    const int s = warp >> 3, half = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
    const uint32_t tmem = bar->tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int pair_bar = kPairBarrier + s * 4 + (warp & 3);           // named barrier of the two warps that hold the same rows
    const float ca = fmaxf(fabsf(p.c), 1e-30f);  // never 0: a masked score stays -inf when scaled
    const uint32_t sb = smem_u32(bar) + s * 8;   // this stream's barriers, at fixed offsets
    int done = 0, seq = 0;                       // steps of this stream and K / V tiles before this item
    for (int n = 0;; ++n) {
      const int at = n % kItems;
      const FwdItem* it = &bar->item[at];
      wait_warp(&bar->ifull[at], (n / kItems) & 1, abort_flag, err);
      if (it->nt < 0) break;
      const int steps = s ? it->steps1 : it->steps0;
      const int left = min(p.tokens, it->q1 - it->tok0 - (PAIR ? s * p.tokens : 0)) * p.r;
      const bool warp_on = (warp & 3) * 32 < left;
      float m = -INFINITY, l = 0.f;  // running maximum (of the raw scores, negated for a negative scale), and sum of this half
      for (int i = 0; i < steps; ++i) {
        const int tile = PAIR ? i : 2 * i + s, step = done + i;
        const bool some = p.keep || it->k0 + (tile + 1) * kTile > it->k1;
        wait_at<(int)offsetof(FwdBarriers, sfull)>(sb, step & 1, abort_flag, err);
        tc_fence_after();
        uint32_t v[2][32];
#pragma unroll
        for (int b = 0; b < 2; ++b) tmem_ld_32x32b_x32(tmem + Sh::kS(s) + half * 64 + b * 32, v[b]);
        if constexpr (DB == 1) {
          // P's columns and O are free again; at 128 channels these scores already waited for that
          if (step > 0) wait_at<(int)offsetof(FwdBarriers, odone)>(sb, (step - 1) & 1, abort_flag, err);
        }
        tmem_ld_wait();
        if constexpr (DB == 1) {
          // the scores are in registers: the next ones may be computed over them
          tc_fence_before();
          arrive_at<(int)offsetof(FwdBarriers, sread)>(sb);
        }
        if (warp_on) {
          if (p.c < 0.f) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int k = 0; k < 32; ++k) v[b][k] ^= 0x80000000u;
          }
          if (some) {
            const int k = seq + 2 * tile + 1;
            wait_warp(&bar->vready[k % NS], (k / NS) & 1, abort_flag, err);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t w = bar->kept[k % NS][half * 2 + b];
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
          bar->rowmax[step & 1][s][half][row] = own;
          tc_fence_before();
          asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");  // also: both halves hold their scores in registers
          tc_fence_after();
          const float tile_max = fmaxf(own, bar->rowmax[step & 1][s][half ^ 1][row]);
          // a row that has seen no key yet takes the tile's maximum; later ones only a clear rise
          const float m_old = m;
          if (m == -INFINITY || (tile_max - m) * ca > kRescaleLog2) m = fmaxf(m, tile_max);
          const float mm = m == -INFINITY ? 0.f : m * ca;
          if (i > 0 && __any_sync(0xffffffffu, m != m_old)) {
            tc_fence_after();
            const float a = m == m_old ? 1.f : ex2(m_old * ca - mm);
            l *= a;
#pragma unroll 1
            for (int b = 0; b < 32 * DB; b += 8) {  // each half rescales half of O's columns; few at a time, beside 64 scores
              const uint32_t col = tmem + Sh::kO(s) + half * 32 * DB + b;
              uint32_t o[8];
              tmem_ld_x8(col, o);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
              tmem_st_x8(col, o);
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
            tmem_st_x16(tmem + Sh::kP(s) + half * 32 + b * 16, w);
          }
          float x, y;
          unpack2(add2(sum[0], sum[1]), x, y);
          l += x + y;
          tmem_st_wait();
        }
        tc_fence_before();
        arrive_at<(int)offsetof(FwdBarriers, pfull)>(sb);
      }
      if (steps > 0) {
        if (warp_on) {  // the sum of both halves
          bar->rowsum[s][half][row] = l;
          asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
          l = bar->rowsum[s][0][row] + bar->rowsum[s][1][row];
        }
        wait_at<(int)offsetof(FwdBarriers, odone)>(sb, (done + steps - 1) & 1, abort_flag, err);
        tc_fence_after();
      }
      fwd_output<DB, PAIR>(p, it, bar, tmem, reinterpret_cast<float*>(aligned + Sh::kExchange), s, half, row, steps, m * ca, l);
      if (steps > 0) {  // O may be overwritten
        tc_fence_before();
        arrive_at<(int)offsetof(FwdBarriers, oread)>(sb);
      }
      done += steps, seq += 2 * it->nt;
      warp_arrive(&bar->iempty[at]);
      if (!LOOP) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (bar->abort_flag && warp == kLoadWarp && lane == 0) {
    // a wait ran out somewhere: let the copies in flight land before the CTA gives its memory back
    volatile int never = 0;
    for (int i = qloaded > NQ ? qloaded - NQ : 0; i < qloaded; ++i) mbar_wait(&bar->qfull[i % NQ], (i / NQ) & 1, &never, err, kDefaultTimeoutNs);
    for (int i = loaded > NS ? loaded - NS : 0; i < loaded; ++i)
      mbar_wait(&bar->kvfull[i % NS], (i / NS) & 1, &never, err, kDefaultTimeoutNs);
  }
  if (warp == kSumWarp) tmem_dealloc(bar->tmem, 512);
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
  const __nv_bfloat16 *dO, *O;   // few queries or keys: the kernels take the statistics themselves
  const float* lse;
  __nv_bfloat16 *dQ, *dK, *dV;
  float *part_q, *part_k, *part_v;  // [splits][rows][d] where a pass is split
  int* status;
};

struct BwdBarriers {
  uint64_t ffull, mfull[8], mempty[8], mready[8], sfull[2], sread[2], pfull[2], pdone[2], adone[2], fin[2];
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
// channels, where the accumulators leave room for the scores alone and P, dS take their place: a row's two threads
// load 32 columns of scores each at their own pace, so each packs its 16 columns into its own 32 (kHalf).
template <int DB, bool KEYS>
struct BwdTmem {
  static constexpr bool kShared = DB == 2 && KEYS;
  static constexpr bool kEarly = !kShared;
  static constexpr int kStride = DB == 1 ? 192 : KEYS ? 128 : 160;
  static constexpr int kHalf = kShared ? 32 : 16;  // columns from the first thread's part of P or dS to the second's
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
  const uint32_t tmem = bar->tmem;

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

  int loaded = 0;
  if (warp == kLoadWarp) {
    if (lane == 0 && nt > 0) {
      const CUtensorMap* f[2] = {KEYS ? &p.fk : &p.fq, KEYS ? &p.fv : &p.fdo};
      const CUtensorMap* m[2] = {KEYS ? &p.mq : &p.mk, KEYS ? &p.mdo : &p.mv};
      const uint32_t f_bytes = (uint32_t)(KEYS ? kTile : ftok * p.r) * 128u, m_bytes = (uint32_t)(KEYS ? mtok * p.r : kMove) * 128u;
      mbar_arrive_expect_tx(&bar->ffull, 2 * DB * f_bytes);
      for (int o = 0; o < 2; ++o)
        for (int b = 0; b < DB; ++b) {
          const uint32_t dst = sf + o * Sh::kFixedBytes + b * kBlockBytes;
          if constexpr (KEYS) tma_load_3d(dst, f[o], &bar->ffull, b * 64, hk, f0);
          else tma_load_4d(dst, f[o], &bar->ffull, b * 64, 0, hk, f0);
        }
      for (; loaded < nt; ++loaded) {
        const int slot = loaded % NS;
        if (loaded >= NS) wait_for(&bar->mempty[slot], ((loaded / NS) & 1) ^ 1, abort_flag, err);
        if (*abort_flag) break;
        mbar_arrive_expect_tx(&bar->mfull[slot], 2 * DB * m_bytes + (KEYS ? (uint32_t)kStatBytes : 0u));
        for (int o = 0; o < 2; ++o)
          for (int b = 0; b < DB; ++b) {
            const uint32_t dst = sm + slot * Sh::kStageBytes + o * Sh::kMoveBytes + b * kMoveBlock;
            if constexpr (KEYS) tma_load_4d(dst, m[o], &bar->mfull[slot], b * 64, 0, hk, m0 + loaded * mtok);
            else tma_load_3d(dst, m[o], &bar->mfull[slot], b * 64, hk, m0 + loaded * kMove);
          }
        if constexpr (KEYS)
          bulk_copy_g2s(sstat + slot * kStatBytes, stat_of(t_lo + loaded), kStatBytes, &bar->mfull[slot]);
      }
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
          if (t0 > 0) wait_warp(Tm::kShared ? &bar->pdone[s] : Tm::kEarly ? &bar->sread[s] : &bar->pfull[s], ph, abort_flag, err);
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
        for (int k = 0; k < kMove / 16; ++k)
          mma_ts(acc, a_col + (k >> 1) * Tm::kHalf + (k & 1) * 8, b0 + (uint64_t)(k * (2048 >> 4)), idesc, more || k ? 1u : 0u, e);
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
      warp_arrive(&bar->mempty[slot]);  // the products' last reader is the other arrival
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
      uint32_t a[32], b[32];
      if (warp_on) {
        tmem_ld_32x32b_x32(tmem + lanes + Tm::S(s) + h * 32, a);
        tmem_ld_32x32b_x32(tmem + lanes + Tm::dP(s) + h * 32, b);
      }
      tmem_ld_wait();
      if constexpr (Tm::kEarly) {  // the scores are in registers: the next ones may be computed over them
        tc_fence_before();
        warp_arrive(&bar->sread[s]);
      }
      if (warp_on) {
        const float* st = reinterpret_cast<const float*>(stats + (t % NS) * kStatBytes);
        uint32_t u[16];
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
          tmem_st_x16(tmem + lanes + Tm::P(s) + h * Tm::kHalf, v);
        } else if (partial(t)) {
          // keys that take no part: weight 0 whatever the products left there
          wait_warp(&bar->mready[t % NS], (t / NS) & 1, abort_flag, err);
          const uint32_t w = bar->kept[t % NS][h];
#pragma unroll
          for (int k = 0; k < 16; ++k) u[k] &= (w >> (2 * k) & 1u ? 0xffffu : 0u) | (w >> (2 * k + 1) & 1u ? 0xffff0000u : 0u);
        }
        tmem_st_x16(tmem + lanes + Tm::dS(s) + h * Tm::kHalf, u);
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
#pragma unroll 1
      for (int c = b_lo * 32; c < b_hi * 32; c += 16) {
        if (c >= p.d) break;
        uint32_t o[16];
        if (nt > 0) {
          tmem_ld_x16(tmem + lanes + acc + c, o);
          tmem_ld_wait();
        }
        if (!row_on) continue;
        float v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = live ? __uint_as_float(o[k]) * f : 0.f;
        if (splits > 1) store_row(part + (split * rows + at) * p.d + c, v, p.d - c);
        else store_row(out + at * p.d + c, v, p.d - c, p.wide);
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
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    mbar_init(&bar->ffull, 1);
    for (int i = 0; i < Sh::kStages; ++i) mbar_init(&bar->mfull[i], 1), mbar_init(&bar->mempty[i], 2), mbar_init(&bar->mready[i], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->sfull[s], 1), mbar_init(&bar->sread[s], 8), mbar_init(&bar->pfull[s], 8);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  pdl_wait();
  pdl_trigger();
  const int first = p.keys_first ? p.k_items : p.q_items, item = (int)blockIdx.x < first ? blockIdx.x : blockIdx.x - first;
  if (((int)blockIdx.x < first) == (p.keys_first != 0)) bwd_pass<DB, true>(p, item, base, bar, stats);
  else bwd_pass<DB, false>(p, item, base, bar, stats);
  if (warp == kSumWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------- backward, few queries
// Groups whose queries fit one tile of 32 packed rows (CLS and auxiliary tokens): that tile stays in shared memory and
// the keys stream past it once.  Every key has its gradients from this tile alone, so they are written as they
// come, and dQ is the only sum: K is read once and each score is computed once (5 products a tile; 4 x 16 queries over
// 9,000 keys, 4 heads of 64: 22.6 us against 53.4 by the two passes).
//     S^T = K Q^T, dP^T = V dO^T;  dV = P^T dO, dK = dS^T Q (P^T, dS^T in tensor memory);  dQ^T += K^T dS
// For the last one dS^T goes to shared memory too, one row per key, which makes it an MN-major B operand, and K's
// tile is read as an MN-major A.  The tile's statistics (-lse in base 2 and -D of its rows) are taken in the kernel: a
// launch before it costs more.  Two streams take alternate key tiles; at 128 channels they share the accumulators.
// dS goes into its products as two bf16 values, the second in the unused half of each shared-memory row: a few dozen
// scores average no rounding out (one value: dQ and dK of 13 queries over 107 keys 1.5 times as far off).
constexpr int kFew = 32;
constexpr int kFewBlock = kFew * 128;  // bytes of the tile's 64-channel block

struct FewBarriers {
  uint64_t qfull, qready, kvfull[10], kvempty[10], kready[10], sfull[2], sread[2], pfull[2], adone[2], qdone[2], oread, fin[2];
  uint32_t kept[10][4];  // keys of the slot's tile that take part
  uint32_t tmem;
  int abort_flag;
};

template <int DB>
struct FewShape {
  static constexpr int kTileBytes = DB * kBlockBytes;
  static constexpr int kStages = DB == 1 ? 10 : 4;  // K and V tiles in turn
  static constexpr int kdS = 2 * DB * kFewBlock, kRing = kdS + 2 * kBlockBytes, kStatAt = kRing + kStages * kTileBytes;
  static constexpr size_t kSmem = 1024 + kStatAt + 2 * kFew * sizeof(float) + sizeof(FewBarriers);
  static constexpr int kStride = DB == 1 ? 224 : 96;
  static constexpr int S(int s) { return s * kStride; }
  static constexpr int dP(int s) { return s * kStride + 32; }
  static constexpr int P(int s) { return s * kStride + 64; }
  static constexpr int dS(int s) { return s * kStride + 80; }
  static constexpr int dV(int s) { return DB == 1 ? s * kStride + 96 : 192; }
  static constexpr int dK(int s) { return DB == 1 ? s * kStride + 160 : 320; }
  static constexpr int kQ = 448;  // dQ^T: a channel a lane, a packed row a column; from dS's second values 32 columns on
};

template <int DB>
__global__ void __launch_bounds__(kThreads, 1) attn_bwd_few_kernel(const __grid_constant__ BwdParams p) {
  using Sh = FewShape<DB>;
  constexpr int NS = Sh::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* aligned = smem_raw + (base - smem_u32(smem_raw));
  float* stat = reinterpret_cast<float*>(aligned + Sh::kStatAt);
  FewBarriers* bar = reinterpret_cast<FewBarriers*>(aligned + Sh::kStatAt + 2 * kFew * sizeof(float));
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* abort_flag = &bar->abort_flag;
  int* err = p.status;
  if (threadIdx.x == 0) {
    mbar_init(&bar->qfull, 1), mbar_init(&bar->qready, 1), mbar_init(&bar->oread, 8);
    // K's slots are the even ones: their readers are the products and the check warp
    for (int i = 0; i < NS; ++i) mbar_init(&bar->kvfull[i], 1), mbar_init(&bar->kvempty[i], 2 - (i & 1)), mbar_init(&bar->kready[i], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->sfull[s], 1), mbar_init(&bar->sread[s], 8), mbar_init(&bar->pfull[s], 8);
      mbar_init(&bar->adone[s], 1), mbar_init(&bar->qdone[s], 1), mbar_init(&bar->fin[s], 1);
    }
    bar->abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&p.mq), prefetch_tmap(&p.mdo), prefetch_tmap(&p.fk), prefetch_tmap(&p.fv);
  }
  if (warp == kSumWarp) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  pdl_wait();
  pdl_trigger();

  int item = blockIdx.x;
  const int hk = item % p.Hkv;
  item /= p.Hkv;
  const int split = item % p.qsplits, g = item / p.qsplits;
  int q0, q1, k0, k1;
  const int flags = group_range(p.q_off, g, p.nq, p.max_q, q0, q1) | group_range(p.kv_off, g, p.nkv, p.max_kv, k0, k1);
  if (flags && threadIdx.x == 0 && split == 0 && hk == 0) atomicOr(p.status, flags);
  const bool bad = flags & SVCONV_STATUS_BAD_OFFSETS;
  const int rows = bad ? 0 : (q1 - q0) * p.r, tiles = bad ? 0 : (k1 - k0 + kTile - 1) / kTile;
  const int t_lo = (int)((int64_t)tiles * split / p.qsplits), t_hi = (int)((int64_t)tiles * (split + 1) / p.qsplits);
  const int nt = rows > 0 ? t_hi - t_lo : 0, key0 = k0 + t_lo * kTile;
  auto partial = [&](int t) { return p.keep || key0 + (t + 1) * kTile > k1; };

  int loaded = 0;
  if (warp == kLoadWarp) {
    if (lane == 0 && nt > 0) {
      const int tokens = kFew / p.r;
      mbar_arrive_expect_tx(&bar->qfull, (uint32_t)(tokens * p.r) * 256u * DB);
      for (int b = 0; b < DB; ++b) {
        tma_load_4d(base + b * kFewBlock, &p.mq, &bar->qfull, b * 64, 0, hk, q0);
        tma_load_4d(base + (DB + b) * kFewBlock, &p.mdo, &bar->qfull, b * 64, 0, hk, q0);
      }
      for (; loaded < 2 * nt; ++loaded) {
        const int slot = loaded % NS;
        if (loaded >= NS) wait_for(&bar->kvempty[slot], ((loaded / NS) & 1) ^ 1, abort_flag, err);
        if (*abort_flag) break;
        mbar_arrive_expect_tx(&bar->kvfull[slot], Sh::kTileBytes);
        for (int b = 0; b < DB; ++b)
          tma_load_3d(base + Sh::kRing + slot * Sh::kTileBytes + b * kBlockBytes, (loaded & 1) ? &p.fv : &p.fk, &bar->kvfull[slot], b * 64,
                      hk, key0 + (loaded >> 1) * kTile);
      }
    }
  } else if (warp == kScoreWarp) {
    if (nt > 0) {
      const uint32_t e = lane == 0;
      const int ks = (p.d + 15) / 16, n = uniform(nt);
      const uint32_t idesc = idesc_bf16_f32(kTile, kFew, 0, 0), tm = uniform(tmem);
      const uint64_t dq = smem_desc_sw128(base, 16, 1024), dkv = smem_desc_sw128(base + Sh::kRing, 16, 1024);
      // operand o (0: K Q, 1: V dO)
      auto scores = [&](int o, int slot, uint32_t d) {
        const uint64_t a0 = dkv + (uint64_t)(slot * (Sh::kTileBytes >> 4)), b0 = dq + (uint64_t)(o * DB * (kFewBlock >> 4));
#pragma unroll
        for (int k = 0; k < 4 * DB; ++k)
          if (k < ks)
            mma_ss(d, a0 + (uint64_t)((k >> 2) * (kBlockBytes >> 4) + (k & 3) * 2), b0 + (uint64_t)((k >> 2) * (kFewBlock >> 4) + (k & 3) * 2),
                   idesc, k ? 1u : 0u, e);
      };
      wait_warp(&bar->qready, 0, abort_flag, err);
      for (int t = 0; t < n; ++t) {
        const int s = t & 1, i = t >> 1, k = 2 * t, v = k + 1;
        wait_warp(&bar->kvfull[k % NS], (k / NS) & 1, abort_flag, err);
        if (i > 0) wait_warp(&bar->sread[s], (i - 1) & 1, abort_flag, err);  // the columns are free
        tc_fence_after();
        scores(0, k % NS, tm + Sh::S(s));
        wait_warp(&bar->kvfull[v % NS], (v / NS) & 1, abort_flag, err);
        tc_fence_after();
        scores(1, v % NS, tm + Sh::dP(s));
        commit_to(&bar->sfull[s], e);
        commit_to(&bar->kvempty[v % NS], e);
      }
      commit_to(&bar->fin[0], e);  // every issued product is complete before tensor memory is released
      wait_warp(&bar->fin[0], 0, abort_flag, err);
    }
  } else if (warp == kSumWarp) {
    if (nt > 0) {
      const uint32_t e = lane == 0;
      const int n = uniform(nt);
      const uint32_t tm = uniform(tmem), idesc = idesc_bf16_f32(kTile, (p.d + 15) / 16 * 16, 0, 1), idesc_q = idesc_bf16_f32(kTile, 2 * kFew, 1, 1);
      const uint64_t dq = smem_desc_sw128(base, kFewBlock, 1024), dgo = smem_desc_sw128(base + DB * kFewBlock, kFewBlock, 1024);
      // up to 64 channels A's second half of rows is the next slot's V tile: rows of dQ^T that are not read
      const uint64_t dk = smem_desc_sw128(base + Sh::kRing, kBlockBytes, 1024), dds = smem_desc_sw128(base + Sh::kdS, kBlockBytes, 1024);
      const uint64_t dsa = smem_desc_sw128(base + Sh::kdS + kFew * 2, 16, 1024);  // the second values as an A operand
      for (int t = 0; t < n; ++t) {
        const int s = t & 1, i = t >> 1, slot = 2 * t % NS;
        wait_warp(&bar->pfull[s], i & 1, abort_flag, err);
        if (DB == 2 && t > 0) wait_warp(&bar->oread, (t - 1) & 1, abort_flag, err);  // the accumulators are free
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kFew / 16; ++k) {
          mma_ts(tm + Sh::dV(s), tm + Sh::P(s) + k * 8, dgo + (uint64_t)(k * (2048 >> 4)), idesc, k ? 1u : 0u, e);
          mma_ts(tm + Sh::dK(s), tm + Sh::dS(s) + k * 8, dq + (uint64_t)(k * (2048 >> 4)), idesc, k ? 1u : 0u, e);
        }
#pragma unroll
        for (int k = 0; k < kFew / 16; ++k)
          mma_ss(tm + Sh::dK(s), dsa + (uint64_t)(s * (kBlockBytes >> 4) + k * 2), dq + (uint64_t)(k * (2048 >> 4)), idesc, 1u, e);
        commit_to(&bar->adone[s], e);
        if (partial(t)) wait_warp(&bar->kready[slot], (2 * t / NS) & 1, abort_flag, err);  // keys that take no part are zero
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ss(tm + Sh::kQ, dk + (uint64_t)(slot * (Sh::kTileBytes >> 4) + k * (2048 >> 4)), dds + (uint64_t)(s * (kBlockBytes >> 4) + k * (2048 >> 4)),
                 idesc_q, t || k ? 1u : 0u, e);
        commit_to(&bar->qdone[s], e);
        commit_to(&bar->kvempty[slot], e);
      }
      commit_to(&bar->fin[1], e);
      wait_warp(&bar->fin[1], 0, abort_flag, err);
    }
  } else if (warp == kCheckWarp) {
    if (nt > 0) {
      wait_warp(&bar->qfull, 0, abort_flag, err);
      if (rows < kFew) {
        const uint32_t w[1] = {~0u << rows};
        scrub_rows(base, 2 * DB, kFewBlock, w);
      }
      warp_arrive(&bar->qready);
    }
    for (int t = 0; t < nt; ++t) {
      const int slot = 2 * t % NS;
      wait_warp(&bar->kvfull[slot], (2 * t / NS) & 1, abort_flag, err);
      if (partial(t)) {
        uint32_t w[4];
        kept_words(p.keep, key0 + t * kTile, k1, w);
        if (lane < 4) bar->kept[slot][lane] = lane == 0 ? w[0] : lane == 1 ? w[1] : lane == 2 ? w[2] : w[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ~w[i];
        scrub_rows(base + Sh::kRing + slot * Sh::kTileBytes, DB, kBlockBytes, w);
      }
      warp_arrive(&bar->kready[slot]);
      warp_arrive(&bar->kvempty[slot]);
    }
  } else {
    // ------------------------------------------------------------ P, dS and the outputs: two threads per key
    const int s = warp >> 3, h = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const f2 c2 = pack2(p.c, p.c);
    if (nt > 0) {
      // -lse in base 2 and -D: a warp a row; rows that do not exist or have no key get weight 0
#pragma unroll
      for (int q = warp; q < kFew; q += kSoftWarps) {
        const int64_t at = (int64_t)(q0 + q / p.r) * p.Hq + hk * p.r + q % p.r;
        float v = 0.f;
        if (q < rows && lane * 4 < p.d) {
          const uint2 x = *reinterpret_cast<const uint2*>(p.dO + at * p.d + lane * 4), y = *reinterpret_cast<const uint2*>(p.O + at * p.d + lane * 4);
          v = __uint_as_float(x.x << 16) * __uint_as_float(y.x << 16);
          v = fmaf(__uint_as_float(x.x & 0xffff0000u), __uint_as_float(y.x & 0xffff0000u), v);
          v = fmaf(__uint_as_float(x.y << 16), __uint_as_float(y.y << 16), v);
          v = fmaf(__uint_as_float(x.y & 0xffff0000u), __uint_as_float(y.y & 0xffff0000u), v);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) {
          const float l = q < rows ? p.lse[at] : -INFINITY;
          stat[q] = l == -INFINITY ? -INFINITY : -l * kLog2e;
          stat[kFew + q] = -v;
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory");
    }
    for (int t = s; t < nt; t += 2) {
      const int i = t >> 1, slot = 2 * t % NS;
      wait_warp(&bar->sfull[s], i & 1, abort_flag, err);
      tc_fence_after();
      uint32_t a[16], b[16], w[8], u[8], r[8];
      tmem_ld_x16(tmem + lanes + Sh::S(s) + h * 16, a);
      tmem_ld_x16(tmem + lanes + Sh::dP(s) + h * 16, b);
      tmem_ld_wait();
      tc_fence_before();
      warp_arrive(&bar->sread[s]);
#pragma unroll
      for (int k = 0; k < 16; k += 4) {  // a row that does not exist has -lse = -inf: weight 0
        const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(stat + h * 16 + k);
        const ulonglong2 nd = *reinterpret_cast<const ulonglong2*>(stat + kFew + h * 16 + k);
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          float x, y;
          unpack2(fma2(pack2(a[k + j], a[k + j + 1]), c2, j ? nl.y : nl.x), x, y);
          x = ex2(x);
          y = ex2(y);
          w[(k + j) / 2] = pack_bf16(x, y);
          unpack2(mul2(pack2(x, y), add2(pack2(b[k + j], b[k + j + 1]), j ? nd.y : nd.x)), x, y);
          u[(k + j) / 2] = pack_bf16(x, y);
          r[(k + j) / 2] = rest_bf16(x, y, u[(k + j) / 2]);
        }
      }
      // A key that takes no part has weight 0 in dQ; its own gradients are 0 at the store, since 0 times a query's
      // infinity is not.
      bool live = true;
      if (partial(t)) {
        wait_warp(&bar->kready[slot], (2 * t / NS) & 1, abort_flag, err);
        live = bar->kept[slot][warp & 3] >> lane & 1u;
        if (!live) {
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = u[k] = r[k] = 0u;
        }
      }
      tmem_st_x8(tmem + lanes + Sh::P(s) + h * 8, w);
      tmem_st_x8(tmem + lanes + Sh::dS(s) + h * 8, u);
      if (i > 0) wait_warp(&bar->qdone[s], (i - 1) & 1, abort_flag, err);  // dS in shared memory is free again
      const uint32_t ds = base + Sh::kdS + s * kBlockBytes + row * 128;
      st_shared_16(ds + ((h * 2) ^ (row & 7)) * 16, u[0], u[1], u[2], u[3]);
      st_shared_16(ds + ((h * 2 + 1) ^ (row & 7)) * 16, u[4], u[5], u[6], u[7]);
      st_shared_16(ds + ((4 + h * 2) ^ (row & 7)) * 16, r[0], r[1], r[2], r[3]);
      st_shared_16(ds + ((5 + h * 2) ^ (row & 7)) * 16, r[4], r[5], r[6], r[7]);
      fence_proxy_async_smem();
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&bar->pfull[s]);
      wait_warp(&bar->adone[s], i & 1, abort_flag, err);
      tc_fence_after();
      // half 0 writes dV, half 1 dK
      const int key = key0 + t * kTile + row;
      const float f = h ? p.scale : 1.f;
      __nv_bfloat16* out = (h ? p.dK : p.dV) + ((int64_t)key * p.Hkv + hk) * p.d;
      const int acc = h ? Sh::dK(s) : Sh::dV(s);
#pragma unroll 1
      for (int c = 0; c < p.d; c += 32) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tmem + lanes + acc + c, o);
        tmem_ld_wait();
        if (key < k1) {
          float v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = live ? __uint_as_float(o[k]) * f : 0.f;
          store_row(out + c, v, p.d - c, p.wide);
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = live ? __uint_as_float(o[16 + k]) * f : 0.f;
          store_row(out + c + 16, v, p.d - c - 16, p.wide);
        }
      }
      if (DB == 2) {
        tc_fence_before();
        warp_arrive(&bar->oread);
      }
    }
    if (nt > 0) wait_warp(&bar->fin[1], 0, abort_flag, err);
    tc_fence_after();
    // dQ: 8 packed rows a warpgroup, a channel a thread
    if (rows > 0) {
      const int part = warp >> 2;
      uint32_t o[8], o2[8];
      if (nt > 0) {
        tmem_ld_x8(tmem + lanes + Sh::kQ + part * 8, o);
        tmem_ld_x8(tmem + lanes + Sh::kQ + kFew + part * 8, o2);
        tmem_ld_wait();
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int q = part * 8 + k;
        if (q >= rows || row >= p.d) continue;
        const int64_t at = ((int64_t)(q0 + q / p.r) * p.Hq + hk * p.r + q % p.r) * p.d + row;
        const float v = nt > 0 ? (__uint_as_float(o[k]) + __uint_as_float(o2[k])) * p.scale : 0.f;
        if (p.qsplits > 1) p.part_q[split * ((int64_t)p.nq * p.Hq * p.d) + at] = v;
        else p.dQ[at] = __float2bfloat16(v);
      }
    } else if (!bad) {  // keys without queries
      const int chunks = p.d / 8;
      for (int i = threadIdx.x; i < (min(k1, k0 + t_hi * kTile) - key0) * chunks; i += kSoftWarps * 32) {
        const int64_t at = ((int64_t)(key0 + i / chunks) * p.Hkv + hk) * p.d + i % chunks * 8;
        *reinterpret_cast<uint4*>(p.dK + at) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(p.dV + at) = make_uint4(0u, 0u, 0u, 0u);
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

// ---------------------------------------------------------------------------- backward, few keys
// Groups of at most 96 keys (an encoder's states, a handful of landmarks) under many queries: the keys stay in shared
// memory and the queries stream past them once, 5 products a tile (8 x 6,144 queries over 77 keys, 4 heads of 64: 43 us
// against 77 by the two passes; 4 x 9,000 over 90, 8 heads of 128: 94 against 147; 1,000 over 50: 16.5 either way).  With fewer
// queries the two passes are faster (200 over 50: 10.3 us against 14.4); this form is taken all the same, because it
// rounds less (D, and dS up to kTwoKeys keys).
//     S = Q K^T, dP = dO V^T;  dQ = dS K, written as it comes;  dV^T += dO^T P, dK^T += Q^T dS
// A row's keys are all here, so D is the sum of P dP itself: no product with O, and none of its rounding, which would
// show where few keys leave dP - D small.  With at most 64 keys dS goes into its products as two bf16 values, the
// second in its second block of shared memory, since so few scores average no rounding out.
// P and dS go to shared memory, a row per query: K-major as the A operand of dQ, MN-major as the B operands of the sums,
// whose A operands are the query tiles read MN-major.  Four threads share a query row, so that few registers hold a tile;
// two groups of warps on alternate tiles gained 4% at 64 channels and lost 15% at 128, where P and dS have one place.
constexpr int kFewKeys = 96;
constexpr int kTwoKeys = 64;  // up to so many dS is two bf16 values
constexpr int kFewKeyBlock = kFewKeys * 128;  // bytes of a 64-channel block of the keys

struct FewKeyBarriers {
  uint64_t kfull, kready, full[8], empty[8], ready[8], sfull, sread, pfull, qdone, sdone, fin[2];
  uint32_t kept[4];
  float rowsum[2][4][kTile];  // [tile parity][quarter of the keys][row]: parts of D
  uint32_t tmem;
  int abort_flag;
};

template <int DB>
struct FewKeyShape {
  static constexpr int kTileBytes = DB * kBlockBytes;
  static constexpr int kStages = DB == 1 ? 8 : 3;  // Q and dO tiles in turn
  static constexpr int kRing = 2 * DB * kFewKeyBlock, kP = kRing + kStages * kTileBytes, kdS = kP + 2 * kBlockBytes, kBar = kdS + 2 * kBlockBytes;
  static constexpr size_t kSmem = 1024 + kBar + sizeof(FewKeyBarriers);
  // tensor memory: the scores, dQ, and dV^T, dK^T with a channel a lane and a key a column
  static constexpr int kTmS = 0, kTmdP = 96, kTmdQ = 192, kTmdV = 320, kTmdK = 416;
};

template <int DB, bool TWO>  // TWO: at most kTwoKeys keys, dS in two values
__global__ void __launch_bounds__(kThreads, 1) attn_bwd_few_keys_kernel(const __grid_constant__ BwdParams p) {
  using Sh = FewKeyShape<DB>;
  constexpr int NS = Sh::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* aligned = smem_raw + (base - smem_u32(smem_raw));
  FewKeyBarriers* bar = reinterpret_cast<FewKeyBarriers*>(aligned + Sh::kBar);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* abort_flag = &bar->abort_flag;
  int* err = p.status;
  if (threadIdx.x == 0) {
    mbar_init(&bar->kfull, 1), mbar_init(&bar->kready, 1);
    for (int i = 0; i < NS; ++i) mbar_init(&bar->full[i], 1), mbar_init(&bar->empty[i], 2), mbar_init(&bar->ready[i], 1);
    mbar_init(&bar->sfull, 1), mbar_init(&bar->sread, kSoftWarps), mbar_init(&bar->pfull, kSoftWarps);
    mbar_init(&bar->qdone, 1), mbar_init(&bar->sdone, 1), mbar_init(&bar->fin[0], 1), mbar_init(&bar->fin[1], 1);
    bar->abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&p.mk), prefetch_tmap(&p.mv), prefetch_tmap(&p.fq), prefetch_tmap(&p.fdo);
  }
  if (warp == kSumWarp) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  pdl_wait();
  pdl_trigger();

  int item = blockIdx.x;
  const int hk = item % p.Hkv;
  item /= p.Hkv;
  const int split = item % p.ksplits, g = item / p.ksplits;
  int q0, q1, k0, k1;
  const int flags = group_range(p.q_off, g, p.nq, p.max_q, q0, q1) | group_range(p.kv_off, g, p.nkv, p.max_kv, k0, k1);
  if (flags && threadIdx.x == 0 && split == 0 && hk == 0) atomicOr(p.status, flags);
  const bool bad = flags & SVCONV_STATUS_BAD_OFFSETS;
  const int ftok = kTile / p.r, tiles = bad ? 0 : (q1 - q0 + ftok - 1) / ftok, keys = bad ? 0 : k1 - k0;
  const int t_lo = (int)((int64_t)tiles * split / p.ksplits), t_hi = (int)((int64_t)tiles * (split + 1) / p.ksplits);
  const int nt = keys > 0 ? t_hi - t_lo : 0, tok0 = q0 + t_lo * ftok;
  const int n16 = (p.max_kv + 15) / 16 * 16;  // columns of the scores
  auto rows_of = [&](int t) { return min(ftok, q1 - tok0 - t * ftok) * p.r; };

  int loaded = 0;
  if (warp == kLoadWarp) {
    if (lane == 0 && nt > 0) {
      mbar_arrive_expect_tx(&bar->kfull, 2 * DB * kFewKeyBlock);
      for (int b = 0; b < DB; ++b) {
        tma_load_3d(base + b * kFewKeyBlock, &p.mk, &bar->kfull, b * 64, hk, k0);
        tma_load_3d(base + (DB + b) * kFewKeyBlock, &p.mv, &bar->kfull, b * 64, hk, k0);
      }
      for (; loaded < 2 * nt; ++loaded) {
        const int slot = loaded % NS;
        if (loaded >= NS) wait_for(&bar->empty[slot], ((loaded / NS) & 1) ^ 1, abort_flag, err);
        if (*abort_flag) break;
        mbar_arrive_expect_tx(&bar->full[slot], (uint32_t)(ftok * p.r) * 128u * DB);
        for (int b = 0; b < DB; ++b)
          tma_load_4d(base + Sh::kRing + slot * Sh::kTileBytes + b * kBlockBytes, (loaded & 1) ? &p.fdo : &p.fq, &bar->full[slot], b * 64, 0,
                      hk, tok0 + (loaded >> 1) * ftok);
      }
    }
  } else if (warp == kScoreWarp) {
    if (nt > 0) {
      const uint32_t e = lane == 0;
      const int ks = (p.d + 15) / 16, n = uniform(nt);
      const uint32_t idesc = idesc_bf16_f32(kTile, n16, 0, 0), tm = uniform(tmem);
      const uint64_t dkv = smem_desc_sw128(base, 16, 1024), dq = smem_desc_sw128(base + Sh::kRing, 16, 1024);
      // operand o (0: Q K, 1: dO V) of the tile in this slot
      auto scores = [&](int o, int slot, uint32_t d) {
        const uint64_t a0 = dq + (uint64_t)(slot * (Sh::kTileBytes >> 4)), b0 = dkv + (uint64_t)(o * DB * (kFewKeyBlock >> 4));
#pragma unroll
        for (int k = 0; k < 4 * DB; ++k)
          if (k < ks)
            mma_ss(d, a0 + (uint64_t)((k >> 2) * (kBlockBytes >> 4) + (k & 3) * 2), b0 + (uint64_t)((k >> 2) * (kFewKeyBlock >> 4) + (k & 3) * 2),
                   idesc, k ? 1u : 0u, e);
      };
      wait_warp(&bar->kready, 0, abort_flag, err);
      for (int t = 0; t < n; ++t) {
        const int q = 2 * t, o = q + 1;
        wait_warp(&bar->full[q % NS], (q / NS) & 1, abort_flag, err);
        if (t > 0) wait_warp(&bar->sread, (t - 1) & 1, abort_flag, err);  // the columns are free
        tc_fence_after();
        scores(0, q % NS, tm + Sh::kTmS);
        wait_warp(&bar->full[o % NS], (o / NS) & 1, abort_flag, err);
        tc_fence_after();
        scores(1, o % NS, tm + Sh::kTmdP);
        commit_to(&bar->sfull, e);
      }
      commit_to(&bar->fin[0], e);  // every issued product is complete before tensor memory is released
      wait_warp(&bar->fin[0], 0, abort_flag, err);
    }
  } else if (warp == kSumWarp) {
    if (nt > 0) {
      const uint32_t e = lane == 0;
      const int n = uniform(nt), nk = uniform(n16 / 16);
      const uint32_t tm = uniform(tmem), idesc_q = idesc_bf16_f32(kTile, (p.d + 15) / 16 * 16, 0, 1), idesc_s = idesc_bf16_f32(kTile, n16, 1, 1);
      const uint64_t dk = smem_desc_sw128(base, kFewKeyBlock, 1024), dsa = smem_desc_sw128(base + Sh::kdS, 16, 1024);
      // up to 64 channels A's second half of rows is whatever follows the tile: rows of dV^T and dK^T that are not read
      const uint64_t dt = smem_desc_sw128(base + Sh::kRing, kBlockBytes, 1024);
      const uint64_t dpb = smem_desc_sw128(base + Sh::kP, kBlockBytes, 1024), dsb = smem_desc_sw128(base + Sh::kdS, kBlockBytes, 1024);
      for (int t = 0; t < n; ++t) {
        const int sq = 2 * t % NS, so = (2 * t + 1) % NS;
        wait_warp(&bar->pfull, t & 1, abort_flag, err);  // dQ was read by then, too
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kFewKeys / 16; ++k)
          if (k < nk)
            mma_ss(tm + Sh::kTmdQ, dsa + (uint64_t)((k >> 2) * (kBlockBytes >> 4) + (k & 3) * 2), dk + (uint64_t)(k * (2048 >> 4)), idesc_q, k ? 1u : 0u, e);
        if constexpr (TWO) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < nk) mma_ss(tm + Sh::kTmdQ, dsa + (uint64_t)((kBlockBytes >> 4) + k * 2), dk + (uint64_t)(k * (2048 >> 4)), idesc_q, 1u, e);
        }
        commit_to(&bar->qdone, e);
        if (rows_of(t) < kTile) {  // rows that do not exist are zero by then
          wait_warp(&bar->ready[sq], (2 * t / NS) & 1, abort_flag, err);
          wait_warp(&bar->ready[so], ((2 * t + 1) / NS) & 1, abort_flag, err);
          tc_fence_after();
        }
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k) {
          mma_ss(tm + Sh::kTmdV, dt + (uint64_t)(so * (Sh::kTileBytes >> 4) + k * (2048 >> 4)), dpb + (uint64_t)(k * (2048 >> 4)), idesc_s, t || k ? 1u : 0u, e);
          mma_ss(tm + Sh::kTmdK, dt + (uint64_t)(sq * (Sh::kTileBytes >> 4) + k * (2048 >> 4)), dsb + (uint64_t)(k * (2048 >> 4)), idesc_s, t || k ? 1u : 0u, e);
        }
        if constexpr (TWO) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_ss(tm + Sh::kTmdK, dt + (uint64_t)(sq * (Sh::kTileBytes >> 4) + k * (2048 >> 4)), dsb + (uint64_t)((kBlockBytes >> 4) + k * (2048 >> 4)),
                   idesc_s, 1u, e);
        }
        commit_to(&bar->sdone, e);
        commit_to(&bar->empty[sq], e);
        commit_to(&bar->empty[so], e);
      }
      commit_to(&bar->fin[1], e);
      wait_warp(&bar->fin[1], 0, abort_flag, err);
    }
  } else if (warp == kCheckWarp) {
    if (nt > 0) {
      wait_warp(&bar->kfull, 0, abort_flag, err);
      uint32_t w[4];
      kept_words(p.keep, k0, k1, w);
      if (lane < 4) bar->kept[lane] = lane == 0 ? w[0] : lane == 1 ? w[1] : lane == 2 ? w[2] : w[3];
      const uint32_t drop[3] = {~w[0], ~w[1], ~w[2]};
      scrub_rows(base, 2 * DB, kFewKeyBlock, drop);
      warp_arrive(&bar->kready);
    }
    for (int j = 0; j < 2 * nt; ++j) {
      const int slot = j % NS, rows = rows_of(j >> 1);
      wait_warp(&bar->full[slot], (j / NS) & 1, abort_flag, err);
      if (rows < kTile) {
        uint32_t drop[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) drop[i] = rows <= 32 * i ? ~0u : rows >= 32 * i + 32 ? 0u : ~0u << (rows - 32 * i);
        scrub_rows(base + Sh::kRing + slot * Sh::kTileBytes, DB, kBlockBytes, drop);
      }
      warp_arrive(&bar->ready[slot]);
      warp_arrive(&bar->empty[slot]);
    }
  } else {
    // ------------------------------------------------------------ P, dS and dQ: four threads per query row, 24 keys each
    const int part = warp >> 2, row = (warp & 3) * 32 + lane, col0 = part * 24;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t kept = 0;  // of this part's keys
    bool lone = false;  // a single key has weight 1 and dS = 0, exactly
    if (nt > 0) {
      wait_warp(&bar->kready, 0, abort_flag, err);
      const uint64_t pair = (uint64_t)bar->kept[col0 >> 5] | (uint64_t)bar->kept[(col0 >> 5) + 1] << 32;
      kept = (uint32_t)(pair >> (col0 & 31)) & 0xffffffu;
      lone = __popc(bar->kept[0]) + __popc(bar->kept[1]) + __popc(bar->kept[2]) == 1;
    }
    const f2 c2 = lone ? 0ull : pack2(p.c, p.c);
    const int rq = row / p.r, rh = row - rq * p.r;  // the row's token in its tile, and head
    // -lse in base 2 of this row of tile t
    auto lse_of = [&](int t) {
      if (t >= nt || row >= rows_of(t) || lone) return 0.f;
      const float l = p.lse[(int64_t)(tok0 + t * ftok + rq) * p.Hq + hk * p.r + rh];
      return l == -INFINITY ? -INFINITY : -l * kLog2e;
    };
    float next_l = lse_of(0);
    for (int t = 0; t < nt; ++t) {
      const bool row_on = row < rows_of(t);
      const f2 nl = pack2(next_l, next_l);
      const uint32_t bits = row_on ? kept : 0u;
      next_l = lse_of(t + 1);
      wait_warp(&bar->sfull, t & 1, abort_flag, err);
      tc_fence_after();
      uint32_t a[3][8], b[3][8];
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (col0 + 8 * i < n16) {
          tmem_ld_x8(tmem + lanes + Sh::kTmS + col0 + 8 * i, a[i]);
          tmem_ld_x8(tmem + lanes + Sh::kTmdP + col0 + 8 * i, b[i]);
        }
      tmem_ld_wait();
      tc_fence_before();
      warp_arrive(&bar->sread);
      // P, and this part of D = sum P dP, which the row's four threads share
      f2 dsum = 0ull;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (col0 + 8 * i >= n16) continue;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          float x, y;
          unpack2(fma2(pack2(a[i][k], a[i][k + 1]), c2, nl), x, y);
          a[i][k] = __float_as_uint(ex2(x));
          a[i][k + 1] = __float_as_uint(ex2(y));
        }
        if (!__all_sync(0xffffffffu, (bits >> (8 * i) & 0xffu) == 0xffu)) {  // rows that do not exist and keys that take no part: weight 0
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (!(bits >> (8 * i + k) & 1u)) a[i][k] = b[i][k] = 0u;
        }
#pragma unroll
        for (int k = 0; k < 8; k += 2) dsum = fma2(pack2(a[i][k], a[i][k + 1]), pack2(b[i][k], b[i][k + 1]), dsum);
      }
      float x, y;
      unpack2(dsum, x, y);
      bar->rowsum[t & 1][part][row] = x + y;
      asm volatile("bar.sync %0, 128;" ::"r"(1 + (warp & 3)) : "memory");
      const float dd = -((bar->rowsum[t & 1][0][row] + bar->rowsum[t & 1][1][row]) + (bar->rowsum[t & 1][2][row] + bar->rowsum[t & 1][3][row]));
      const f2 nd = pack2(dd, dd);
      if (t > 0) wait_warp(&bar->sdone, (t - 1) & 1, abort_flag, err);  // P and dS are free again
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int col = col0 + 8 * i;
        if (col >= n16) continue;
        uint32_t w[4], u[4], rest[4];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          w[k / 2] = pack_bf16(__uint_as_float(a[i][k]), __uint_as_float(a[i][k + 1]));
          unpack2(mul2(pack2(a[i][k], a[i][k + 1]), add2(pack2(b[i][k], b[i][k + 1]), nd)), x, y);
          u[k / 2] = pack_bf16(x, y);
          if constexpr (TWO) rest[k / 2] = rest_bf16(x, y, u[k / 2]);
        }
        const uint32_t at = base + (uint32_t)((col >> 6) * kBlockBytes + row * 128 + (((col & 63) >> 3) ^ (row & 7)) * 16);
        st_shared_16(at + Sh::kP, w[0], w[1], w[2], w[3]);
        st_shared_16(at + Sh::kdS, u[0], u[1], u[2], u[3]);
        if constexpr (TWO) st_shared_16(at + Sh::kdS + kBlockBytes, rest[0], rest[1], rest[2], rest[3]);
      }
      fence_proxy_async_smem();
      warp_arrive(&bar->pfull);
      wait_warp(&bar->qdone, t & 1, abort_flag, err);
      tc_fence_after();
#pragma unroll
      for (int b2 = 0; b2 < DB; ++b2) {
        const int c = (part * DB + b2) * 16;
        if (c >= p.d) break;
        uint32_t o[16];
        tmem_ld_x16(tmem + lanes + Sh::kTmdQ + c, o);
        tmem_ld_wait();
        if (!row_on) continue;
        float v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(o[k]) * p.scale;
        store_row(p.dQ + ((int64_t)(tok0 + t * ftok + rq) * p.Hq + hk * p.r + rh) * p.d + c, v, p.d - c, p.wide);
      }
      tc_fence_before();
    }
    if (nt > 0) wait_warp(&bar->fin[1], 0, abort_flag, err);
    tc_fence_after();
    // dV and dK: a channel a thread, 24 keys a warpgroup
#pragma unroll 1
    for (int i = 0; i < 3; ++i) {
      const int key0 = (warp >> 2) * 24 + 8 * i;
      if (key0 >= n16) break;
      uint32_t o[8], w[8];
      if (nt > 0) {
        tmem_ld_x8(tmem + lanes + Sh::kTmdV + key0, o);
        tmem_ld_x8(tmem + lanes + Sh::kTmdK + key0, w);
        tmem_ld_wait();
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int key = key0 + k;
        if (key >= keys || row >= p.d) continue;
        const int64_t at = ((int64_t)(k0 + key) * p.Hkv + hk) * p.d + row, from = split * ((int64_t)p.nkv * p.Hkv * p.d) + at;
        // a key that takes no part: 0 whatever its weights of 0 met in the queries' rows
        const bool live = nt > 0 && (bar->kept[key >> 5] >> (key & 31) & 1u);
        const float dv = live ? __uint_as_float(o[k]) : 0.f, dk = live ? __uint_as_float(w[k]) * p.scale : 0.f;
        if (p.ksplits > 1) p.part_v[from] = dv, p.part_k[from] = dk;
        else p.dV[at] = __float2bfloat16(dv), p.dK[at] = __float2bfloat16(dk);
      }
    }
    if (keys == 0 && !bad) {  // queries without keys
      const int64_t lo = (int64_t)tok0 * p.Hq, chunks = p.d / 8, per = (int64_t)p.r * chunks;
      for (int64_t i = threadIdx.x; i < (min(q1, q0 + t_hi * ftok) - tok0) * per; i += kSoftWarps * 32)
        *reinterpret_cast<uint4*>(p.dQ + (lo + i / per * p.Hq + hk * p.r) * p.d + i % per * 8) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (bar->abort_flag && warp == kLoadWarp && lane == 0 && nt > 0) {
    // a wait ran out somewhere: let the copies in flight land before the CTA gives its memory back
    volatile int never = 0;
    mbar_wait(&bar->kfull, 0, &never, err, kDefaultTimeoutNs);
    for (int i = loaded > NS ? loaded - NS : 0; i < loaded; ++i)
      mbar_wait(&bar->full[i % NS], (i / NS) & 1, &never, err, kDefaultTimeoutNs);
  }
  if (warp == kSumWarp) tmem_dealloc(tmem, 512);
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

// The splits of a gradient added up: 8 channels a thread over the rows of group blockIdx.y, by SLICES warps of the block
// that take every SLICES-th split and whose sums are added in order.  One slice moves the most bytes; eight
// shorten the chain of loads where there are many splits (148 of 32 rows: a call of 22.7 us takes 14.5).
// blockIdx.z: the gradient (dK and dV in one launch).
template <int SLICES>
__global__ void __launch_bounds__(256) attn_sum_kernel(const float* part0, const float* part1, int splits, const int32_t* off, const int32_t* off2,
                                                       int n, int n2, int bound, int H, int d, __nv_bfloat16* out0, __nv_bfloat16* out1) {
  const float* __restrict__ part = blockIdx.z ? part1 : part0;
  __nv_bfloat16* __restrict__ out = blockIdx.z ? out1 : out0;
  constexpr int kThreadsX = 256 / SLICES;
  __shared__ float s_v[SLICES > 1 ? SLICES : 1][SLICES > 1 ? kThreadsX : 1][9];
  const int x = threadIdx.x % kThreadsX, y = threadIdx.x / kThreadsX;
  pdl_wait();
  pdl_trigger();
  int lo, hi, lo2, hi2;
  const int flags = group_range(off, blockIdx.y, n, bound, lo, hi) | group_range(off2, blockIdx.y, n2, n2, lo2, hi2);
  const int64_t i = ((int64_t)blockIdx.x * kThreadsX + x) * 8;
  const bool on = !(flags & SVCONV_STATUS_BAD_OFFSETS) && i < (int64_t)(hi - lo) * H * d;
  const int64_t at = (int64_t)lo * H * d + i, step = (int64_t)n * H * d;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (on) {
#pragma unroll 4
    for (int s = y; s < splits; s += SLICES) {
      const float4 a = *reinterpret_cast<const float4*>(part + s * step + at), b = *reinterpret_cast<const float4*>(part + s * step + at + 4);
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
  }
  if constexpr (SLICES > 1) {
#pragma unroll
    for (int k = 0; k < 8; ++k) s_v[y][x][k] = v[k];
    __syncthreads();
    if (y > 0) return;
#pragma unroll
    for (int w = 1; w < SLICES; ++w)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += s_v[w][x][k];
  }
  if (on)
    *reinterpret_cast<uint4*>(out + at) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// ---------------------------------------------------------------------------- host side
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// Partial results are stored 32 bytes at a time; a workspace is aligned to 16.  Its first 32-byte boundary, and the
// bytes that a size has more for it.
constexpr size_t kWsSlack = 16;
float* ws_floats(void* p) { return reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(p) + 31u) & ~(uintptr_t)31u); }

// Rows, and items of a launch: a row, block or item behind the last one still has a 32-bit number.
constexpr int kMaxRows = 0x7fff0000;

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
  if (o.nq > kMaxRows || o.nkv > kMaxRows) return SVCONV_ERR_SIZE;
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
// query), with the group lengths known only by their sum and bound.  In units of one key tile for both streams (1.5 us
// up to 64 channels, 1.9 at 128: 4,096 queries x 8 heads over 8,192 and 16,384 keys take 102 and 197 us, 132 and 254): a tile
// costs 1 in the pair form and 1/2 in the split form, a CTA kFixed besides, and splits their partial results (kMerge and
// kMergeBytes are the same at either width, so a merge counts for a quarter more at 128 channels).
constexpr int kSms = 148, kMinTiles = 4;
// Up to so many key tiles an item, CTAs loop over items.  24,576 queries x 4 heads of 64: 1 tile 26.7 us a CTA an item
// and 20.6 us looping, 2 tiles 29.2 and 24.7, 4 tiles 37 and 37, 8 tiles 55 and 59; heads of 128, whose query tiles
// cannot be loaded ahead: 1 tile 26.7 and 23.9, 2 tiles 32.9 and 30.9, 3 tiles 39.0 and 37.9.
constexpr int kLoopTiles = 3;
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

// The same for the two passes of the backward call, which share one launch: CTAs take the items of the pass with
// the longer ones first, then the other's, as SMs come free.  Splits are tried around the number that keeps an item under
// half an SM's share of all work, by that schedule's end plus the cost of the partial results.  In units of one
// moving tile of the query pass (about 0.6 us).
constexpr double kBwdFixed = 5.0, kKeyTile = 1.3, kBwdMerge = 5.0, kBwdMergeBytes = 3.0e6;
// Few queries or few keys: microseconds of a tile of 64 channels, of a CTA beside its tiles, and of adding the splits up.
constexpr double kFewTile = 1.5, kFewKeyTile = 2.5, kFewFixed = 8.0, kFewMerge = 5.0;
struct BwdPlan {
  int qblocks, qsplits, kblocks, ksplits, keys_first;
  int few;              // 1: the kernel for few queries, with qsplits cuts of the keys; 2: for few keys, ksplits cuts of the queries
  int tiles;            // of statistics, for each key head
  size_t stat, pq, pk;  // floats: statistics, split partials of dQ, of dK (and again of dV)
  size_t floats() const { return stat + pq + 2 * pk; }
};
// When kSms machines that take na items of la, then nb of lb, as they come free, are done.
double schedule_end(double na, double la, double nb, double lb) {
  if (na + nb > 30.0 * kSms) return (na * la + nb * lb) / kSms + (la > lb ? la : lb) * 0.5;
  struct {
    double t, n;
  } free[80];  // machines by the time they come free, earliest first
  int cnt = 1;
  free[0] = {0.0, (double)kSms};
  double end = 0.0;
  for (int k = 0; k < 2; ++k) {
    double n = k ? nb : na;
    const double l = k ? lb : la;
    while (n > 0.0) {
      const double take = n < free[0].n ? n : free[0].n, t = free[0].t + l;
      n -= take;
      if (t > end) end = t;
      if (take < free[0].n) {
        free[0].n -= take;
      } else {
        --cnt;
        for (int i = 0; i < cnt; ++i) free[i] = free[i + 1];
      }
      int i = cnt++;
      while (i > 0 && free[i - 1].t > t) free[i] = free[i - 1], --i;
      free[i] = {t, take};
    }
  }
  return end;
}
BwdPlan plan_bwd(const svconv_cross_attn_desc& c) {
  BwdPlan b;
  const int r = c.Hq / c.Hkv, G = c.G > 0 ? c.G : 1;
  const int tq = cdiv(c.max_kv, kMove), tk = cdiv(c.max_q, kMove / r);  // moving tiles of an item of the query / key pass
  b.qblocks = cdiv(c.max_q, kTile / r);
  b.kblocks = cdiv(c.max_kv, kTile);
  const double nqb = b.qblocks ? c.Hkv * blocks_est(c.nq, c.max_q, G, kTile / r) : 0.0;
  const double nkb = b.kblocks ? c.Hkv * blocks_est(c.nkv, c.max_kv, G, kTile) : 0.0;
  const double share = (nqb * (cdiv(c.nkv, G * kMove) + kBwdFixed) + nkb * (cdiv(c.nq, G * (kMove / r)) * kKeyTile + kBwdFixed)) / kSms;
  const double bq = (double)c.nq * c.Hq * c.d * 8.0 / kBwdMergeBytes, bk = 2.0 * c.nkv * c.Hkv * c.d * 8.0 / kBwdMergeBytes;
  auto start = [&](int tiles, double tile) { return share > 0.0 ? (int)std::ceil(tiles * tile / (0.5 * share)) : 1; };
  const int mq = tq / (2 * kMinTiles), mk = tk / (2 * kMinTiles);  // most splits
  const int sq0 = start(tq, 1.0), sk0 = start(tk, kKeyTile);
  double best = 0.0;
  for (int i = -3; i < 2; ++i)
    for (int j = -3; j < 2; ++j) {
      int sq = i == -3 ? 1 : sq0 + i, sk = j == -3 ? 1 : sk0 + j;
      sq = sq > mq ? mq : sq, sk = sk > mk ? mk : sk;
      sq = sq < 1 ? 1 : sq, sk = sk < 1 ? 1 : sk;
      const double lq = (double)tq / sq + kBwdFixed, lk = (double)tk * kKeyTile / sk + kBwdFixed;
      const bool kf = lk > lq;
      const double t = (kf ? schedule_end(nkb * sk, lk, nqb * sq, lq) : schedule_end(nqb * sq, lq, nkb * sk, lk)) +
                       (sq > 1 ? kBwdMerge + bq * sq : 0.0) + (sk > 1 ? kBwdMerge + bk * sk : 0.0);
      if (best == 0.0 || t < best) best = t, b.qsplits = sq, b.ksplits = sk, b.keys_first = kf;
    }
  // The forms for few rows, by the bounds.  Where both would do, the one that gives dS two bf16 values: few keys up to
  // kTwoKeys of them, few queries above (also the faster there: 64 x 8 queries over 96 keys, 8 heads of 128, 31 us and 47).
  if (c.max_q == 0 || c.max_kv == 0) b.few = 0;
  else if (c.max_kv <= kTwoKeys) b.few = 2;
  else if ((int64_t)c.max_q * r <= kFew) b.few = 1;
  else b.few = c.max_kv <= kFewKeys ? 2 : 0;
  if (b.few) {  // one item a split of a group's keys (queries) and key head
    const int tiles = b.few == 1 ? cdiv(c.max_kv, kTile) : cdiv(c.max_q, kTile / r);
    const double units = (double)G * c.Hkv, tile = (b.few == 1 ? kFewTile : kFewKeyTile) * (c.d <= 64 ? 1 : 2);
    const double bytes = b.few == 1 ? bq : bk;
    int splits = 1;
    best = 0.0;
    for (int s = 1; s <= tiles && (s == 1 || units * s <= 8.0 * kSms); ++s) {
      const double t = std::ceil(units * s / kSms) * (cdiv(tiles, s) * tile + kFewFixed) + (s > 1 ? kFewMerge + bytes * s : 0.0);
      if (best == 0.0 || t < best) best = t, splits = s;
    }
    b.qsplits = b.few == 1 ? splits : 1;
    b.ksplits = b.few == 2 ? splits : 1;
  }
  const size_t nq = (size_t)c.nq * c.Hq, nk = (size_t)c.nkv * c.Hkv;
  b.tiles = b.few ? 0 : c.nq / (kMove / r) + c.G + 1;
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
cudaError_t launch_few(const BwdParams& p, int grid, cudaStream_t s) {
  static int done[64];
  cudaError_t e = ensure_smem_attr(attn_bwd_few_kernel<DB>, FewShape<DB>::kSmem, done);
  return e == cudaSuccess ? launch_pdl(attn_bwd_few_kernel<DB>, dim3(grid), dim3(kThreads), FewShape<DB>::kSmem, s, p) : e;
}

template <int DB>
cudaError_t launch_few_keys(const BwdParams& p, int grid, cudaStream_t s) {
  static int done[2][64];
  const bool two = p.max_kv <= kTwoKeys;
  auto kernel = two ? attn_bwd_few_keys_kernel<DB, true> : attn_bwd_few_keys_kernel<DB, false>;
  cudaError_t e = ensure_smem_attr(kernel, FewKeyShape<DB>::kSmem, done[two]);
  return e == cudaSuccess ? launch_pdl(kernel, dim3(grid), dim3(kThreads), FewKeyShape<DB>::kSmem, s, p) : e;
}

template <int DB>
cudaError_t launch_fwd(const FwdParams& p, int items, int tiles, cudaStream_t s) {
  static int done[4][64];
  const int ctas = sm_count();
  const bool loop = items > ctas && tiles <= kLoopTiles;
  auto kernel = p.pair ? (loop ? attn_fwd_kernel<DB, true, true> : attn_fwd_kernel<DB, true, false>)
                       : (loop ? attn_fwd_kernel<DB, false, true> : attn_fwd_kernel<DB, false, false>);
  cudaError_t e = ensure_smem_attr(kernel, FwdShape<DB>::kSmem, done[2 * p.pair + loop]);
  return e == cudaSuccess ? launch_pdl(kernel, dim3(loop ? ctas : items), dim3(kThreads), FwdShape<DB>::kSmem, s, p) : e;
}

}  // namespace
}  // namespace svc

using namespace svc;

extern "C" {

size_t svconv_cross_attn_fwd_workspace_size(const svconv_cross_attn_desc* desc) {
  svconv_cross_attn_desc c;
  if (check_desc(desc, c) || c.G == 0 || c.max_q == 0) return 0;
  const FwdPlan f = plan_fwd(c);
  return f.splits > 1 ? (size_t)f.splits * c.nq * c.Hq * (c.d + 2) * sizeof(float) + kWsSlack : 0;
}

size_t svconv_cross_attn_bwd_workspace_size(const svconv_cross_attn_desc* desc) {
  svconv_cross_attn_desc c;
  if (check_desc(desc, c) || c.G == 0) return 0;
  const size_t floats = plan_bwd(c).floats();
  return floats ? floats * sizeof(float) + kWsSlack : 0;
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
  if (grid > kMaxRows) return SVCONV_ERR_SIZE;
  FwdParams p{};
  p.q_off = c.q_off, p.kv_off = c.kv_off, p.keep = c.kv_keep;
  p.nq = c.nq, p.nkv = c.nkv, p.max_q = c.max_q, p.max_kv = c.max_kv, p.Hq = c.Hq, p.Hkv = c.Hkv, p.r = c.Hq / c.Hkv, p.d = c.d;
  p.tokens = kTile / p.r;
  p.G = c.G, p.splits = f.splits, p.pair = f.pair;
  p.c = c.scale * kLog2e;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.wide = c.d % 16 == 0 && aligned32(O);
  p.lse = lse;
  p.part_o = ws_floats(workspace);
  p.part_ml = p.part_o + (size_t)f.splits * c.nq * c.Hq * c.d;
  p.status = dev_status ? dev_status : device_error_word();
  // no keys at all: the maps only have to be well formed
  if (!make_packed_map(&p.tq, Q, c.nq, c.Hkv, p.r, c.d, c.q_row, c.q_head, p.tokens) ||
      !make_rows_map(&p.tk, c.nkv ? K : Q, c.nkv, c.Hkv, c.d, c.k_row, c.k_head, kTile) ||
      !make_rows_map(&p.tv, c.nkv ? V : Q, c.nkv, c.Hkv, c.d, c.v_row, c.v_head, kTile))
    return SVCONV_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  const int tiles = cdiv(cdiv(c.max_kv, kTile), f.splits);
  cudaError_t e = c.d <= 64 ? launch_fwd<1>(p, (int)grid, tiles, s) : launch_fwd<2>(p, (int)grid, tiles, s);
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
  const long long q_items = heads * (b.few ? 1 : b.qblocks) * b.qsplits, k_items = heads * (b.few ? 1 : b.kblocks) * b.ksplits;
  const int r = c.Hq / c.Hkv;
  int lanes = 1;
  while (lanes < c.d / 8) lanes *= 2;
  const long long stat_grid = (long long)cdiv(c.max_q, kMove / r) * c.Hkv;
  if (q_items + k_items > kMaxRows || stat_grid > kMaxRows) return SVCONV_ERR_SIZE;
  float* ws = ws_floats(workspace);
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
  p.dO = static_cast<const __nv_bfloat16*>(dO), p.O = static_cast<const __nv_bfloat16*>(O), p.lse = lse;
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
      !make_packed_map(&p.mq, q, c.nq, c.Hkv, r, c.d, c.q_row, c.q_head, (b.few == 1 ? kFew : kMove) / r) ||
      !make_packed_map(&p.fdo, go, c.nq, c.Hkv, r, c.d, go_row, go_head, kTile / r) ||
      !make_packed_map(&p.mdo, go, c.nq, c.Hkv, r, c.d, go_row, go_head, (b.few == 1 ? kFew : kMove) / r) ||
      !make_rows_map(&p.fk, k, c.nkv, c.Hkv, c.d, c.k_row, c.k_head, kTile) ||
      !make_rows_map(&p.mk, k, c.nkv, c.Hkv, c.d, c.k_row, c.k_head, b.few == 2 ? kFewKeys : kMove) ||
      !make_rows_map(&p.fv, v, c.nkv, c.Hkv, c.d, c.v_row, c.v_head, kTile) ||
      !make_rows_map(&p.mv, v, c.nkv, c.Hkv, c.d, c.v_row, c.v_head, b.few == 2 ? kFewKeys : kMove))
    return SVCONV_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (c.max_q > 0 && !b.few)
    e = launch_pdl(attn_stat_kernel, dim3((unsigned)stat_grid, c.G), dim3(256), 0, s, static_cast<const __nv_bfloat16*>(dO),
                   static_cast<const __nv_bfloat16*>(O), lse, c.q_off, c.nq, c.max_q, c.Hq, c.Hkv, c.d, lanes, b.tiles, ws);
  if (e == cudaSuccess && b.few == 1)
    e = c.d <= 64 ? launch_few<1>(p, (int)q_items, s) : launch_few<2>(p, (int)q_items, s);
  else if (e == cudaSuccess && b.few == 2)
    e = c.d <= 64 ? launch_few_keys<1>(p, (int)k_items, s) : launch_few_keys<2>(p, (int)k_items, s);
  else if (e == cudaSuccess)
    e = c.d <= 64 ? launch_bwd<1>(p, (int)(q_items + k_items), s) : launch_bwd<2>(p, (int)(q_items + k_items), s);
  auto add = [&](const float* part0, const float* part1, int splits, const int32_t* off, const int32_t* off2, int n, int n2, int bound,
                 int H, __nv_bfloat16* out0, __nv_bfloat16* out1) {
    if (e != cudaSuccess || splits < 2) return;
    const long long chunks = (long long)bound * H * c.d / 8;
    const int slices = splits > 8 ? 8 : 1, per = 256 / slices;
    e = launch_pdl(slices > 1 ? attn_sum_kernel<8> : attn_sum_kernel<1>, dim3((unsigned)((chunks + per - 1) / per), c.G, out1 ? 2 : 1), dim3(256), 0,
                   s, part0, part1, splits, off, off2, n, n2, bound, H, c.d, out0, out1);
  };
  add(p.part_q, nullptr, b.qsplits, c.q_off, c.kv_off, c.nq, c.nkv, c.max_q, c.Hq, p.dQ, nullptr);
  add(p.part_k, p.part_v, b.ksplits, c.kv_off, c.q_off, c.nkv, c.nq, c.max_kv, c.Hkv, p.dK, p.dV);
  return e == cudaSuccess ? SVCONV_OK : SVCONV_ERR_CUDA;
}

}  // extern "C"
