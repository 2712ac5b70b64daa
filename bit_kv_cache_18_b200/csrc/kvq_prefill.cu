// kvq_prefill.cu -- attention of whole prompts over their own rows, on the
// fifth-generation tensor cores (tcgen05): the definition is in include/kvq.h.
//
// Rows.  The G query heads of a kv head share its keys and values, so the
// tile of a matrix product is (128 / G tokens) x (G heads): 128 rows, row r =
// token r / G, head r % G.  An item is two such tiles, 256 / G tokens in a
// row; they walk the 128-key tiles that either reads, from the newest to the
// oldest (with a distance bias the largest scores come first).  Packed this
// way an item covers 32 tokens at G = 8, so little of the diagonal is computed
// for nothing, and a prompt of 20 tokens fills its tiles.
//
// Roles.  One CTA a multiprocessor stays and takes items from a list.  Warps
// 0-3 and 4-7 are the softmax of tile 0 and 1, a thread per row; warp 8 issues
// the products, warp 9 the copies (TMA, 128-byte swizzle; K and V tiles of 32
// KB through one ring of four), warp 10 finds the items ahead of the others,
// so the next item's copies and first scores run under the last one's output.
// Tensor memory holds, per tile, the scores S (128 fp32 columns) and the
// output O (128 columns): all 512.
//   S = Q K^T: A and B K-major from shared memory;
//   P = 2^(y - m) overwrites S in 16 bits, O += P V: A from tensor memory, V
//   as it lies ([token][dim]: MN-major).
// While one tile is in its softmax the tensor core works for the other.
//
// Softmax.  y is the base-2 score, m a running max that only moves when a
// score passes it by 8 (then O and l are rescaled in place, by the same
// threads: S(j) is only issued after PV(j-1), so O is at rest when S(j) has
// arrived); p is at most 2^8, l the fp32 sum of the unrounded p, and the sums
// of P V are fp32.  P is rounded to the inputs' type, the only rounding to
// fewer bits before the output's own: half a step, 2^-8 (bf16) or 2^-11 (fp16)
// of p, of either sign, so it averages out over the keys.
//
// Masked places.  A masked score is replaced, not added to, so nothing that
// stands in a masked key reaches a row.  A masked value is multiplied by p = 0,
// which only a NaN or an infinity survives.  So in the tiles that some row of
// the item reads only in part (the diagonal's, the window's older end) the
// products' warp zeroes the values that are not finite and those that no row
// reads, while the softmax runs; where it met one that is not finite, the rows that
// read it get it added to their output (add_cleared): no row is formed twice.
//
// What bounds it.  A step of two tiles and 128 keys is 2048 clocks of the
// tensor core at its full rate (and of shared memory, which S reads at 128
// bytes a clock) and 2048 of the MUFU's exponentials.  Measured it takes about
// 3200: a tile's 2100 from S to P (150 for the loads, 350 for the maximum, 1550
// for 128 exponentials a thread where the MUFU needs 1024, waits for the
// stores), then 1050 for half of PV, the next S and two hand-overs.  One prompt
// of 16384 tokens, 64 and 8 heads, bf16: 3.47 ms, 1267 TFLOP/s, alone, 4.0 ms in
// a row, where the card's power limit lowers the clock (a library product of
// 8192^3 gives 1661 and 1385).  Twelve ragged prompts of 1 to 1500 tokens, 32 and
// 8 heads: 81 us, 643 TFLOP/s.  Tried, and not faster: a part of the
// exponentials on the FMA pipe; two threads a row (16 softmax warps); 64-key
// steps with two S buffers a tile, which hide the hand-overs, but their S reads
// shared memory half again as often (4.4 ms; with a softcap 0.72 against 0.80 at
// 8192 tokens); P formed with the old maximum while the new one is found.
#include <cuda.h>
#include <math_constants.h>

#include <algorithm>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kTile = 128;         // rows of a product, keys of a tile
constexpr int kHalf = kTile / 2;
constexpr int kStages = 4;         // K and V tiles in shared memory
constexpr int kTileBytes = kTile * kHeadDim * 2;
constexpr int kHalfBytes = kTileBytes / 2;  // 64 of the 128 dims: one swizzle width
constexpr int kSoftWarps = 8;      // four a tile
constexpr int kMmaWarp = 8, kLoadWarp = 9, kItemWarp = 10;
constexpr int kThreads = 384;
constexpr int kItems = 2;          // items handed out ahead
constexpr int kItemReaders = kSoftWarps + 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 per tile
constexpr int kEarly = 2;          // quarters of P handed over first (1 and 3 measured no faster)
constexpr float kLazy = 8.0f;      // log2 of the largest p
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // a device-side wait gives up after one second

// The rows of a prompt's 256 / G tokens and one kv head: what a CTA works on.
struct Item {
  int row0, n;     // the prompt's first row and length; n < 0: no more items
  int prefix;      // keys that every query reads
  int t0;          // first token
  int kv_head;
};

struct __align__(1024) Smem {
  uint8_t q[2][kTileBytes];
  uint8_t kv[kStages][kTileBytes];
  uint8_t out[kSoftWarps][32 * kHeadDim];  // per warp: 32 rows of half the output, on their way to memory
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t s_full[2];  // S of the tile is written (and every product before it is complete)
  uint64_t p_early[2], p_full[2];  // P of the tile's first keys, of all, is written (O rescaled)
  uint64_t o_full[2];  // O of the tile is final
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t fin;        // every product issued is complete
  Item item[kItems];
  uint32_t cleared[4];  // number of the last item (from 1, at its remainder by 4) with values that were not finite
  uint32_t tmem_base;
  int abort;           // a wait ran out: every other wait gives up at once
};
constexpr int kSmemBytes = static_cast<int>(sizeof(Smem));
static_assert(kSmemBytes <= 227 * 1024, "one CTA per SM");

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Bounded, warp-uniform wait for a barrier phase: false if it did not come
// within the limit or another warp already gave up.  `abort` may be null (a
// last wait, which ignores the others' failure).
__device__ __forceinline__ bool mbar_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint64_t t0 = global_ns();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((it & 15u) == 0u) {
      if (abort != nullptr && __any_sync(0xffffffffu, *abort != 0)) return false;
      if (__any_sync(0xffffffffu, global_ns() - t0 > kWaitLimitNs)) break;
    }
  }
  if (abort != nullptr) *abort = 1;
  return false;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return mbar_wait_slow(bar, parity, abort);
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// A box of a tensor map into this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// A box of shared memory to memory, in a group of its own (one thread), and the
// warp's waits: until its copies have read their shared memory, and until they
// have written theirs.
__device__ __forceinline__ void tma_store4(const CUtensorMap* map, uint32_t src, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n"
      "cp.async.bulk.commit_group;" ::"l"(map),
      "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void copies_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
__device__ __forceinline__ void copies_done() {
  asm volatile("cp.async.bulk.wait_group 0;\nfence.proxy.async.global;" ::: "memory");
  __syncwarp();
}

// sm_100 shared-memory matrix descriptors with the 128-byte swizzle, version
// 1: 8 rows of 128 bytes are an atom of 1024.  K-major (Q, K): atoms follow
// each other along the rows, the leading offset is not used.  MN-major (V):
// the atoms of the second 64 dims lie kHalfBytes away, those of the next 8
// tokens 1024 bytes.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor, kind::f16: D f32, A and B f16 or bf16, M = N = 128;
// vmajor: B is MN-major.
template <bool kBF16>
constexpr uint32_t idesc(bool vmajor) {
  return (1u << 4) | ((kBF16 ? 1u : 0u) << 7) | ((kBF16 ? 1u : 0u) << 10) | ((vmajor ? 1u : 0u) << 16) |
         ((128u >> 3) << 17) | ((128u >> 4) << 24);
}
// One thread issues the products, but its warp walks them together: the
// instructions are predicated, not branched around, so that descriptors and
// addresses stay in uniform registers (behind `if (lane == 0)` each product
// took about 120 clocks to issue, more than the 64 that it runs).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_ss(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(static_cast<uint32_t>(acc)), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t elected, uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(static_cast<uint32_t>(acc)), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t elected, uint64_t* bar) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {  // 2^x (MUFU.EX2); ex2(-inf) = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
typedef unsigned long long u64x;
__device__ __forceinline__ u64x pk2(float a, float b) {
  u64x r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
// The same value twice, in registers that stay: from a plain constant the
// compiler makes the pair anew, two moves, at every use.
__device__ __forceinline__ u64x twice(float a) {
  u64x r;
  asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ void upk2(u64x v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ u64x add2(u64x a, u64x b) {
  u64x d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64x mul2(u64x a, u64x b) {
  u64x d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64x fma2(u64x a, u64x b, u64x c) {
  u64x d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <bool kBF16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if (kBF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool kBF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (kBF16) return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Softcap: y = cap tanh(s / cap) in base-2 units from the raw product d, by the
// size of x = d cap_inv = s / cap:
//   |x| <= 1/2 or 1: y = d scale T(x^2), T of degree 3 or 6 the interpolation of
//     tanh(sqrt u) / sqrt u at the Chebyshev points of [0, 1/4] or [0, 1], off
//     by 5.5e-7 or 5.2e-8 of itself, so right for caps of any size.  The first
//     form, the usual one, is a polynomial in d^2, powers of cap_inv in its
//     coefficients, five packed operations a pair of scores (six in x^2: 3%
//     of two prompts of 4096 and 2047 tokens); where those powers would leave
//     fp32's range cap_half is 0 and the second form, in x^2, takes over: nine;
//   beyond: y = cap (1 - 2 / (e^2x + 1)), off by 2^-22 cap; four of the MUFU's
//     a pair, 32 clocks a warp where the FMA pipe takes 10 or 18.
// With a cap up to 1000 (kCap = 1) a row's scores in a tile take one form, by the
// largest of them: the highest that a row of the warp needs where every row reads
// every key, else each row its own, found over the scores that it reads, so that
// what stands in the others reaches no bit of it.  With a larger one (kCap = 2),
// for which 2^-22 cap is more than 2.4e-4 of a probability, every score takes
// its own of the last two.
constexpr float kLargeCap = 1442.7f;  // 1000, base 2
__device__ __forceinline__ float capped_far(float d, const PrefillArgs& a) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(d * (a.cap_inv * 2.8853900817779268f)) + 1.0f));  // 2^(2x log2 e)
  return fmaf(-2.0f * a.softcap, r, a.softcap);
}
__device__ __forceinline__ float capped(float d, const PrefillArgs& a) {
  const float x = d * a.cap_inv, u = x * x;
  float p = a.cap_one_coef[6];
#pragma unroll
  for (int k = 5; k >= 0; --k) p = fmaf(p, u, a.cap_one_coef[k]);
  return fabsf(x) > 1.0f ? capped_far(d, a) : d * p;
}
// s times the polynomial in (s unit)^2 or, without kUnit, in s^2
template <bool kUnit, int kN>
__device__ __forceinline__ void capped_near(float (&s)[kTile], const float (&coef)[kN], float unit) {
  u64x c[kN];
#pragma unroll
  for (int x = 0; x < kN; ++x) c[x] = twice(coef[x]);
  const u64x unit2 = twice(unit);
#pragma unroll
  for (int e = 0; e < kTile; e += 2) {
    const u64x d = pk2(s[e], s[e + 1]), x = kUnit ? mul2(d, unit2) : d, u = mul2(x, x);
    u64x p = c[kN - 1];
#pragma unroll
    for (int k = kN - 2; k >= 0; --k) p = fma2(p, u, c[k]);
    upk2(mul2(d, p), s[e], s[e + 1]);
  }
}
// live: my row is one of the prompt's; edge: a row of the tile does not read every key (those scores are 0)
__device__ __forceinline__ void cap_scores(float (&s)[kTile], const PrefillArgs& a, bool live, bool edge) {
  float big[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < kTile; e += 2) big[(e >> 1) & 3] = max3f(big[(e >> 1) & 3], fabsf(s[e]), fabsf(s[e + 1]));
  float x = live ? fmaxf(max3f(big[0], big[1], big[2]), big[3]) * a.cap_inv : 0.0f;
  if (!edge) x = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
  if (x <= a.cap_half) {
    capped_near<false>(s, a.cap_half_coef, 1.0f);
  } else if (x <= 1.0f) {
    capped_near<true>(s, a.cap_one_coef, a.cap_inv);
  } else {
#pragma unroll
    for (int e = 0; e < kTile; ++e) s[e] = capped_far(s[e], a);
  }
}

// The key interval [lo, hi) of the query at position t of a prompt.
struct Span {
  int prefix, window;
  __device__ __forceinline__ int lo(int t) const { return window > 0 ? max(t - window + 1, 0) : 0; }
  __device__ __forceinline__ int hi(int t) const { return max(t + 1, prefix); }
};

// An item's two row tiles and the key tiles that each reads, [klo, khi), walked
// from the newest to the oldest in `steps` steps; the second tile may have no token.
struct Walk {
  Span sp;
  int first[2], last[2];  // tokens of each tile
  int klo[2], khi[2];
  int top, steps;
  int whole0, whole1;  // the key tiles that every row reads wholly: [whole0, whole1)
  int newest;          // keys that some row reads: up to here
  bool two;
  __device__ __forceinline__ Walk(const Item& it, int window, int tile_tokens) {
    sp.prefix = it.prefix;
    sp.window = window;
    two = it.t0 + tile_tokens < it.n;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      first[i] = it.t0 + i * tile_tokens;
      last[i] = min(first[i] + tile_tokens, it.n) - 1;
      klo[i] = sp.lo(first[i]) / kTile;
      khi[i] = (sp.hi(last[i]) + kTile - 1) / kTile;
    }
    if (!two) khi[1] = klo[1] = klo[0];
    top = max(khi[0], khi[1]);
    steps = top - klo[0];
    whole0 = (sp.lo(two ? last[1] : last[0]) + kTile - 1) / kTile;
    whole1 = sp.hi(first[0]) / kTile;
    newest = sp.hi(two ? last[1] : last[0]);
  }
  __device__ __forceinline__ bool whole(int j) const { return j >= whole0 && j < whole1; }
  __device__ __forceinline__ bool active(int i, int c) const { return top - 1 - c >= klo[i] && top - 1 - c < khi[i]; }
};

// Which of a word's two values are not finite: bits 15 and 31 (one more in an
// exponent of all ones carries into the sign, which is cleared before).
template <bool kBF16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & (kBF16 ? 0x7F807F80u : 0x7C007C00u)) + (kBF16 ? 0x00800080u : 0x04000400u)) & 0x80008000u;
}

// acc + 0 x of two values each: not a number once an x was not finite
template <bool kBF16>
__device__ __forceinline__ void add_zero_times(uint32_t& acc, uint32_t x) {
  if (kBF16)
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
}

// A tile of values that some row of the item reads only in part, as it lies in
// shared memory: the keys from `rows` on become 0, and so do values of the keys
// [r0, rows) that are not finite (true if there was one).  One warp, eight lanes
// a key; it has the time until the tile's P is there, so it looks at 16 keys at a
// time with one operation a word, and at single values only where that finds
// something.
template <bool kBF16>
__device__ __forceinline__ bool clear_values(uint8_t* tile, int r0, int rows) {
  const int row = (threadIdx.x & 31) >> 3;
  uint8_t* at = tile + row * 128 + 16 * (threadIdx.x & 7);
  uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
  for (int r = r0; r < rows; r += 16) {
    uint4 v[4][2];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        v[x][hf] = make_uint4(0u, 0u, 0u, 0u);
        if (r + 4 * x + row < rows) v[x][hf] = *reinterpret_cast<const uint4*>(at + (r + 4 * x) * 128 + hf * kHalfBytes);
      }
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        add_zero_times<kBF16>(acc[0], v[x][hf].x);
        add_zero_times<kBF16>(acc[1], v[x][hf].y);
        add_zero_times<kBF16>(acc[2], v[x][hf].z);
        add_zero_times<kBF16>(acc[3], v[x][hf].w);
      }
  }
  const bool found = __any_sync(0xffffffffu, (not_finite<kBF16>(acc[0]) | not_finite<kBF16>(acc[1]) |
                                              not_finite<kBF16>(acc[2]) | not_finite<kBF16>(acc[3])) != 0u);
  if (found) {
#pragma unroll 1
    for (int r = r0 + row; r < rows; r += 4) {
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        uint4* p = reinterpret_cast<uint4*>(at + (r - row) * 128 + hf * kHalfBytes);
        uint4 v = *p;
        v.x &= ~((not_finite<kBF16>(v.x) >> 15) * 0xFFFFu);
        v.y &= ~((not_finite<kBF16>(v.y) >> 15) * 0xFFFFu);
        v.z &= ~((not_finite<kBF16>(v.z) >> 15) * 0xFFFFu);
        v.w &= ~((not_finite<kBF16>(v.w) >> 15) * 0xFFFFu);
        *p = v;
      }
    }
  }
#pragma unroll 4
  for (int r = rows; r < kTile - row; r += 4) {
    *reinterpret_cast<uint4*>(at + r * 128) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(at + r * 128 + kHalfBytes) = make_uint4(0u, 0u, 0u, 0u);
  }
  if (found || rows < kTile) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return found;
}

// The values that clear_values took out of key tiles [j0, j1): bit l of up[x]
// (down[x]) is set if dim 4 l + x of a key that my row reads, one of [lo, hi), is
// infinite or not a number and not negative (not positive).  One warp, a lane a row.
template <bool kBF16>
__device__ __forceinline__ void find_cleared(const PrefillArgs& a, const Item& it, int j0, int j1, int lo, int hi,
                                             uint32_t (&up)[4], uint32_t (&down)[4]) {
  const int end = min(j1 * kTile, it.n);
#pragma unroll 1
  for (int key = j0 * kTile; key < end; ++key) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.v + (it.row0 + key) * a.v_stride + it.kv_head * kHeadDim) +
                          (threadIdx.x & 31));
    if (!__any_sync(0xffffffffu, (not_finite<kBF16>(w.x) | not_finite<kBF16>(w.y)) != 0u)) continue;
    const float2 f = unpack2<kBF16>(w.x), g = unpack2<kBF16>(w.y);
    const float v[4] = {f.x, f.y, g.x, g.y};
    const uint32_t mine = key >= lo && key < hi ? 0xffffffffu : 0u;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const bool bad = !(fabsf(v[x]) < CUDART_INF_F);
      up[x] |= __ballot_sync(0xffffffffu, bad && !(v[x] < 0.0f)) & mine;
      down[x] |= __ballot_sync(0xffffffffu, bad && !(v[x] > 0.0f)) & mine;
    }
  }
}

// An output row's dims that read such values: with its p above 0 an infinity or
// a NaN decides the sum whatever its factor.
template <bool kBF16>
__device__ __forceinline__ void add_cleared(uint16_t* row, const uint32_t (&up)[4], const uint32_t (&down)[4]) {
#pragma unroll 1
  for (uint32_t left = up[0] | up[1] | up[2] | up[3] | down[0] | down[1] | down[2] | down[3]; left != 0u; left &= left - 1u) {
    const int l = __ffs(left) - 1;
    uint2* at = reinterpret_cast<uint2*>(row) + l;
    const uint2 w = *at;
    const float2 f = unpack2<kBF16>(w.x), g = unpack2<kBF16>(w.y);
    float v[4] = {f.x, f.y, g.x, g.y};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if ((up[x] >> l) & 1u) v[x] += CUDART_INF_F;
      if ((down[x] >> l) & 1u) v[x] -= CUDART_INF_F;
    }
    *at = make_uint2(pack2<kBF16>(v[0], v[1]), pack2<kBF16>(v[2], v[3]));
  }
}

// The items of a CTA, found by one warp ahead of the others.  Prompt b has
// ceil(length / 256 * G) row tile pairs (one whose bounds are not ascending or
// not within the rows has none and is recorded); the items, in falling order of
// the pair's index, ties by prompt, then by kv head, are dealt out to the CTAs
// back and forth, so that each gets about the same sum.
struct Items {
  const PrefillArgs& a;
  const int lane, log_tokens;
  int row0, n, mine;  // prompt `lane`: first row, length, pairs (all that is needed up to 32 prompts)
  int total;          // pairs of all prompts
  int index;          // the pair index last found (at first: no prompt has so many pairs)
  int above, upto;    // pairs with a larger index; with that or a larger one
  int base, seen;     // prompts before `base`, a multiple of 32: `seen` have such a pair
  __device__ __forceinline__ int tiles(int s, int e) const {
    return s >= 0 && e >= s && e <= a.n_tokens ? (e - s + (1 << log_tokens) - 1) >> log_tokens : -1;
  }
  __device__ __forceinline__ int tiles(int b) const { return tiles(__ldg(a.cu_seqlens + b), __ldg(a.cu_seqlens + b + 1)); }
  // pairs with an index >= i
  __device__ __forceinline__ int count(int i) const {
    int c = max(mine - i, 0);
    for (int b = 32 + lane; b < a.batch; b += 32) c += max(tiles(b) - i, 0);
    return __reduce_add_sync(0xffffffffu, c);
  }
  __device__ __forceinline__ Items(const PrefillArgs& args, int log_t)
      : a(args), lane(threadIdx.x & 31), log_tokens(log_t), row0(0), n(0), mine(0) {
    if (lane < a.batch) {
      const int e = __ldg(a.cu_seqlens + lane + 1);
      row0 = __ldg(a.cu_seqlens + lane);
      n = e - row0;
      mine = tiles(row0, e);
    }
    bool bad = mine < 0;
    int most = mine, sum = max(mine, 0);
    for (int b = 32 + lane; b < a.batch; b += 32) {
      const int x = tiles(b);
      bad |= x < 0;
      most = max(most, x);
      sum += max(x, 0);
    }
    total = __reduce_add_sync(0xffffffffu, sum);
    index = max(__reduce_max_sync(0xffffffffu, most), 0);
    above = upto = base = seen = 0;
    if (bad && blockIdx.x == 0) record_status(a.status, KVQ_ERR_OUT_OF_RANGE);
  }
  // the item of rank `rank` among the pairs; false if there is none.  Ranks rise
  // from call to call, so the index only falls, and among one index's prompts
  // the walk goes on where it was.
  __device__ __forceinline__ bool find(int rank, Item* it) {
    if (rank >= upto) {
      if (rank >= total) return false;
      int lo = 0, hi = index, at_lo = total, at_hi = upto;  // at_lo = count(lo) > rank >= at_hi = count(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1, c = count(mid);
        if (c > rank) {
          lo = mid;
          at_lo = c;
        } else {
          hi = mid;
          at_hi = c;
        }
      }
      index = lo;
      above = at_hi;
      upto = at_lo;
      base = seen = 0;
    }
    for (; base < a.batch; base += 32) {
      const int b = base + lane, k = rank - above - seen;  // my place among the prompts from base on
      const uint32_t has = __ballot_sync(0xffffffffu, b < a.batch && (base == 0 ? mine : tiles(b)) > index);
      if (k >= __popc(has)) {
        seen += __popc(has);
        continue;
      }
      const bool me = ((has >> lane) & 1u) != 0 && __popc(has & ((1u << lane) - 1u)) == k;
      const int src = __ffs(__ballot_sync(0xffffffffu, me)) - 1, at = base + src;
      if (base == 0) {
        it->row0 = __shfl_sync(0xffffffffu, row0, src);
        it->n = __shfl_sync(0xffffffffu, n, src);
      } else {
        it->row0 = __ldg(a.cu_seqlens + at);
        it->n = __ldg(a.cu_seqlens + at + 1) - it->row0;
      }
      it->prefix = a.prefix_lens != nullptr ? min(__ldg(a.prefix_lens + at), it->n) : 0;
      it->t0 = index << log_tokens;
      return true;
    }
    return false;
  }
};

// A ring position and the parity of its present use.
template <int kN>
struct Ring {
  uint32_t i = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++i == kN) {
      i = 0;
      ph ^= 1u;
    }
  }
};

template <bool kBF16, int kCap, bool kBias>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  volatile int* abort = &sm.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == kLoadWarp) {
    if (lane < 4)
      asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &a.map_q : lane == 1 ? &a.map_k : lane == 2 ? &a.map_v : &a.map_out)
                   : "memory");
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&sm.kv_full[i], 1);
        mbar_init(&sm.kv_empty[i], 1);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.q_full[i], 1);
        mbar_init(&sm.q_empty[i], 1);
        mbar_init(&sm.s_full[i], 1);
        mbar_init(&sm.p_early[i], kSoftWarps / 2);
        mbar_init(&sm.p_full[i], kSoftWarps / 2);
        mbar_init(&sm.o_full[i], 1);
      }
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        mbar_init(&sm.item_full[i], 1);
        mbar_init(&sm.item_empty[i], kItemReaders);
      }
      mbar_init(&sm.fin, 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) sm.cleared[i] = 0u;
      sm.abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tbase = sm.tmem_base;
  const int log_g = a.log_group, log_tokens = 8 - log_g, tile_tokens = kTile >> log_g;
  bool bad = false;
  // the next item of a reader's ring; false behind the last one or after a wait that gave up
  auto next_item = [&](Ring<kItems>& r, Item* it) {
    if (!mbar_wait(&sm.item_full[r.i], r.ph, abort)) {
      bad = true;
      return false;
    }
    *it = sm.item[r.i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[r.i]);
    r.next();
    return it->n >= 0;
  };

  // registers: 3 x 168 a thread at launch, 72 + 2 x 216 from here
  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kItemWarp) {
      Items items(a, log_tokens);
      Ring<kItems> r;
      const uint32_t ctas = gridDim.x;
      for (uint32_t k = 0;; ++k) {
        const uint32_t n = k * ctas + (k & 1u ? ctas - 1u - blockIdx.x : blockIdx.x);
        Item it;
        it.kv_head = static_cast<int>(n % a.num_kv_heads);
        const bool live = items.find(static_cast<int>(n / a.num_kv_heads), &it);
        if (!live) it.n = -1;
        if (k >= kItems && !mbar_wait(&sm.item_empty[r.i], r.ph ^ 1u, abort)) {
          bad = true;
          break;
        }
        if (lane == 0) {
          sm.item[r.i] = it;
          mbar_arrive(&sm.item_full[r.i]);
        }
        __syncwarp();
        if (!live) break;
        r.next();
      }
    } else if (warp == kLoadWarp) {
      Ring<kItems> ri;
      Ring<kStages> rk;
      uint32_t copies = 0, nq[2] = {0, 0};
      Item it;
      while (!bad && next_item(ri, &it)) {
        const Walk w(it, a.window, tile_tokens);
        auto box_q = [&](int i) {
          if (nq[i] > 0 && !mbar_wait(&sm.q_empty[i], (nq[i] - 1) & 1u, abort)) {
            bad = true;
            return;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.q_full[i], kTileBytes);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              tma_load4(smem_u32(sm.q[i]) + hf * kHalfBytes, &a.map_q, 64 * hf, 0, it.kv_head, it.row0 + w.first[i],
                        &sm.q_full[i]);
          }
          __syncwarp();
          ++nq[i];
        };
        box_q(0);
        for (int x = 0; x < 2 * w.steps && !bad; ++x) {  // K and V of step x / 2
          if (copies >= kStages && !mbar_wait(&sm.kv_empty[rk.i], rk.ph ^ 1u, abort)) {
            bad = true;  // no copy is issued any more
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.kv_full[rk.i], kTileBytes);
            const CUtensorMap* map = x & 1 ? &a.map_v : &a.map_k;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              tma_load3(smem_u32(sm.kv[rk.i]) + hf * kHalfBytes, map, 64 * hf, it.kv_head,
                        it.row0 + (w.top - 1 - x / 2) * kTile, &sm.kv_full[rk.i]);
          }
          __syncwarp();
          ++copies;
          rk.next();
          if (x == 0 && w.two) box_q(1);
        }
      }
      // The copies still in flight (after a wait that gave up; else none) land
      // before the CTA gives up its shared memory: the last one into each
      // stage, newest first, and into each query tile.
#pragma unroll 1
      for (uint32_t x = 0; x < kStages && x < copies; ++x) {
        if (rk.i == 0) {
          rk.i = kStages;
          rk.ph ^= 1u;
        }
        --rk.i;
        if (!mbar_wait_slow(&sm.kv_full[rk.i], rk.ph, nullptr)) bad = true;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (nq[i] > 0 && !mbar_wait_slow(&sm.q_full[i], (nq[i] - 1) & 1u, nullptr)) bad = true;
    } else if (warp == kMmaWarp) {
      // descriptors move by 16 bytes a unit: 16 dims (Q, K) 2, 64 dims 1024,
      // 16 tokens of V 128, a tile 2048
      const uint64_t dq = sdesc(smem_u32(sm.q[0]), 16), dk = sdesc(smem_u32(sm.kv[0]), 16);
      const uint64_t dv = sdesc(smem_u32(sm.kv[0]), kHalfBytes);
      const uint32_t elected = elect_one();
      Ring<kItems> ri;
      Ring<kStages> rk;
      uint32_t pph = 0, qph = 0;  // bit i: parity of tile i's next P, next Q
      uint32_t number = 0;        // items
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!mbar_wait(bar, parity, abort)) bad = true;
      };
      Item it;
      while (!bad && next_item(ri, &it)) {
        const Walk w(it, a.window, tile_tokens);
        ++number;
        bool started[2] = {false, false};
        // S of tile i with the keys in `stage`, walked at step c
        auto product_s = [&](int i, uint32_t stage, int c) {
          const uint64_t x = dq + 2048u * i, y = dk + 2048u * stage;
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const uint32_t off = (s >> 2) * 1024 + (s & 3) * 2;
            mma_ss(elected, tbase + kColS + 128 * i, x + off, y + off, idesc<kBF16>(false), s > 0);
          }
          mma_commit(elected, &sm.s_full[i]);
          if (c + 1 >= w.steps || !w.active(i, c + 1)) mma_commit(elected, &sm.q_empty[i]);
        };
        wait(&sm.kv_full[rk.i], rk.ph);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 0 || w.two) {
            wait(&sm.q_full[i], (qph >> i) & 1u);
            qph ^= 1u << i;
          }
          tc_fence_after();
          if (w.active(i, 0)) product_s(i, rk.i, 0);
        }
        mma_commit(elected, &sm.kv_empty[rk.i]);
        rk.next();
#pragma unroll 1
        for (int c = 0; c < w.steps; ++c) {
          const uint32_t sv = rk.i;
          wait(&sm.kv_full[sv], rk.ph);
          rk.next();
          const int j = w.top - 1 - c;
          if (!w.whole(j)) {  // (P is not here yet)
            // the keys that some row does not read: from the first row's newest on, those
            // behind the last one's (zeroed unseen); at the window's older end any
            const int r0 = j < w.whole0 ? 0 : max(w.sp.hi(it.t0) - j * kTile, 0);
            if (clear_values<kBF16>(sm.kv[sv], r0, min(w.newest - j * kTile, kTile)) && lane == 0)
              sm.cleared[number & 3u] = number;
            __syncwarp();
          }
          const bool more = c + 1 < w.steps;
          const uint32_t sk = rk.i;
          if (more) wait(&sm.kv_full[sk], rk.ph);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (w.active(i, c)) {
              const uint64_t y = dv + 2048u * sv;
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                wait(hf == 0 ? &sm.p_early[i] : &sm.p_full[i], (pph >> i) & 1u);
                tc_fence_after();
#pragma unroll
                for (int s = hf == 0 ? 0 : 2 * kEarly; s < (hf == 0 ? 2 * kEarly : 8); ++s)
                  mma_ts(elected, tbase + kColO + 128 * i, tbase + kColS + 128 * i + 8 * s, y + 128 * s,
                         idesc<kBF16>(true), started[i] || s > 0);
              }
              if (!more || !w.active(i, c + 1)) mma_commit(elected, &sm.o_full[i]);
              pph ^= 1u << i;
              started[i] = true;
            }
            if (more && w.active(i, c + 1)) product_s(i, sk, c + 1);
          }
          mma_commit(elected, &sm.kv_empty[sv]);
          if (more) {
            mma_commit(elected, &sm.kv_empty[sk]);
            rk.next();
          }
        }
      }
      mma_commit(elected, &sm.fin);
      if (!mbar_wait_slow(&sm.fin, 0, nullptr)) bad = true;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int i = warp >> 2;
    const int r = tid & (kTile - 1);
    const uint32_t lanes = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t ts = lanes + kColS + 128 * i, to = lanes + kColO + 128 * i;
    uint32_t sph = 0, oph = 0, number = 0;
    Ring<kItems> ri;
    Item it;
    while (!bad && next_item(ri, &it)) {
      const Walk w(it, a.window, tile_tokens);
      ++number;
      if (i == 1 && !w.two) continue;
      const Span& sp = w.sp;
      const int first = it.t0 + i * tile_tokens, last = min(first + tile_tokens, it.n) - 1;
      const int klo = i == 0 ? w.klo[0] : w.klo[1], khi = i == 0 ? w.khi[0] : w.khi[1];
      const int t = first + (r >> log_g);
      const int head = (it.kv_head << log_g) + (r & ((1 << log_g) - 1));
      const bool valid = t < it.n;
      const int lo = sp.lo(t), hi = sp.hi(t);  // (a row behind the last token: whatever it computes is dropped)
      const float slope2 = kBias ? __ldg(a.alibi_slopes + head) * 1.4426950408889634f : 0.0f;
      const float scale = kCap || kBias ? 1.0f : a.scale_log2;  // what is left to multiply by in the exponent
      float m = -CUDART_INF_F;
      u64x l2[2] = {0ull, 0ull};  // the sum of p, in four parts
      bool started = false;
#pragma unroll 1
      for (int j = khi - 1; j >= klo; --j) {
        const int j0 = j * kTile;
        if (!mbar_wait(&sm.s_full[i], sph, abort)) bad = true;
        sph ^= 1u;
        tc_fence_after();
        float s[kTile];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld32(ts + 32 * x, s + 32 * x);
        tmem_wait_ld();
        // The keys that my row reads, a bit each, where a row of the tile does not read
        // all.  (Comparisons of each score with both ends take more code, of which the
        // loop has too much: 12 ragged prompts 80.4 us against 78.6.)
        const bool edge = j0 + kTile > sp.hi(first) || j0 < sp.lo(last);
        uint32_t reads[4];
        if (edge) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int from = min(max(lo - j0 - 32 * w, 0), 32), to = min(max(hi - j0 - 32 * w, 0), 32);
            reads[w] = static_cast<uint32_t>((1ull << to) - 1ull) & ~static_cast<uint32_t>((1ull << from) - 1ull);
          }
        }
        auto mask_with = [&](float x) {
#pragma unroll
          for (int e = 0; e < kTile; ++e) s[e] = (reads[e / 32] >> (e % 32)) & 1u ? s[e] : x;
        };
        if (kCap == 1) {
          if (edge) mask_with(0.0f);  // (for now: the others have no say in the cap's form)
          cap_scores(s, a, valid, edge);
        }
        if (kCap == 2) {
#pragma unroll
          for (int e = 0; e < kTile; ++e) s[e] = capped(s[e], a);
        }
        if (kBias) {
          const float d0 = static_cast<float>(j0 - t);
          if (sp.prefix <= first + 1) {  // no query reads a key behind it: linear
            const u64x k2 = twice(kCap ? 1.0f : a.scale_log2);
            const u64x sl = twice(slope2), b2 = twice(slope2 * d0);
#pragma unroll
            for (int e = 0; e < kTile; e += 2)
              upk2(fma2(pk2(s[e], s[e + 1]), k2, fma2(pk2(static_cast<float>(e), static_cast<float>(e + 1)), sl, b2)),
                   s[e], s[e + 1]);
          } else {
#pragma unroll
            for (int e = 0; e < kTile; ++e)
              s[e] = fmaf(-slope2, fabsf(d0 + static_cast<float>(e)), kCap ? s[e] : s[e] * a.scale_log2);
          }
        }
        if (edge) mask_with(-CUDART_INF_F);
        float mx4[4];  // four chains
#pragma unroll
        for (int x = 0; x < 4; ++x) mx4[x] = fmaxf(s[2 * x], s[2 * x + 1]);
#pragma unroll
        for (int e = 8; e < kTile; e += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x) mx4[x] = max3f(mx4[x], s[e + 2 * x], s[e + 2 * x + 1]);
        const float mx = fmaxf(max3f(mx4[0], mx4[1], mx4[2]), mx4[3]) * scale;
        const bool moves = mx > m + kLazy || (m == -CUDART_INF_F && mx > m);
        if (__any_sync(0xffffffffu, moves)) {
          const float mn = moves ? mx : m;
          const float alpha = moves ? ex2(m - mn) : 1.0f;
          if (started) {  // O is at rest: the product before S is complete
#pragma unroll 1
            for (int x = 0; x < 8; ++x) {
              float o[16];
              tmem_ld16(to + 16 * x, o);
              tmem_wait_ld();
              uint32_t v[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(o[e] * alpha);
              tmem_st16(to + 16 * x, v);
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) l2[x] = fma2(l2[x], pk2(alpha, alpha), 0ull);
          m = mn;
        }
        started = true;
        const float base = m == -CUDART_INF_F ? 0.0f : -m;
        const u64x scale2 = twice(scale), base2 = twice(base);
        // P of 32 keys
        auto exps = [&](int x, uint32_t (&v)[16]) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float p0, p1;
            upk2(fma2(pk2(s[32 * x + 2 * e], s[32 * x + 2 * e + 1]), scale2, base2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            l2[e & 1] = add2(l2[e & 1], pk2(p0, p1));
            v[e] = pack2<kBF16>(p0, p1);
          }
        };
        auto hand_over = [&](uint64_t* bar) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);
        };
        uint32_t v[16];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          exps(x, v);
          tmem_st16(ts + 16 * x, v);
          if (x == kEarly - 1) hand_over(&sm.p_early[i]);
        }
        hand_over(&sm.p_full[i]);
      }
      if (!mbar_wait(&sm.o_full[i], oph, abort)) bad = true;
      oph ^= 1u;
      tc_fence_after();
      float l, l1;
      upk2(add2(l2[0], l2[1]), l, l1);
      l += l1;
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      // 64 dims at a time: my row in 16 bits into the warp's staging rows,
      // 16-byte piece x of row r at x ^ (r % 8), the copies' 128-byte swizzle;
      // then one copy writes the warp's 32 rows, or, where some are behind the
      // last token, the warp does, four at a time.  (Plain stores of all rows
      // took 1300 clocks a half, the copy runs on its own.)
      uint8_t* stage = sm.out[warp];
      const int wfirst = first + (((warp & 3) * 32) >> log_g);  // the warp's first token
      const bool whole = wfirst + (32 >> log_g) <= it.n;
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        float o[kHalf];
#pragma unroll
        for (int x = 0; x < 2; ++x) tmem_ld32(to + kHalf * hf + 32 * x, o + 32 * x);
        tmem_wait_ld();
        copies_read();  // the staging rows are free
#pragma unroll
        for (int x = 0; x < kHalf / 8; ++x) {
          uint32_t v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            v[y] = pack2<kBF16>(o[8 * x + 2 * y] * inv, o[8 * x + 2 * y + 1] * inv);
          }
          *reinterpret_cast<uint4*>(stage + lane * kHeadDim + 16 * (x ^ (lane & 7))) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        if (whole) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) tma_store4(&a.map_out, smem_u32(stage), 64 * hf, 0, it.kv_head, it.row0 + wfirst);
        } else {
          __syncwarp();
#pragma unroll 1
          for (int x = 0; x < 8; ++x) {
            const int wr = 4 * x + (lane >> 3), tr = wfirst + (wr >> log_g);
            if (tr < it.n)
              reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(it.row0 + tr) * a.out_stride +
                                       ((it.kv_head << log_g) + (wr & ((1 << log_g) - 1))) * kHeadDim +
                                       kHalf * hf)[lane & 7] =
                  *reinterpret_cast<const uint4*>(stage + wr * kHeadDim + 16 * ((lane & 7) ^ (wr & 7)));
          }
          __syncwarp();
        }
      }
      // (Items are at most two ahead of the one whose output is written, so its
      // number stands.)
      if (__any_sync(0xffffffffu, *const_cast<volatile uint32_t*>(&sm.cleared[number & 3u]) == number)) {
        uint32_t up[4] = {0u, 0u, 0u, 0u}, down[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
        for (int x = 0; x < 2; ++x)  // the older end's tiles, the newer one's
          find_cleared<kBF16>(a, it, x == 0 ? klo : max(max(w.whole0, w.whole1), klo), x == 0 ? min(w.whole0, khi) : khi, lo,
                              hi, up, down);
        copies_done();
        if (valid) add_cleared<kBF16>(a.out + (it.row0 + t) * a.out_stride + head * kHeadDim, up, down);
      }
      tc_fence_before();  // O is read: orders the next item's first P, which lets the products write it again
    }
    copies_done();
  }
  if (bad) record_status(a.status, KVQ_ERR_DEVICE_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "n"(kTmemCols));
  pdl_trigger();  // this CTA holds no tensor memory any more (earlier, ragged prompts took 5% longer)
}

// ---- tensor maps ----------------------------------------------------------------

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}
// [tokens][heads][128] in 16 bits as `rank` dimensions: 128 dims, `inner` heads
// (rank 4: the heads of a group), heads / inner, tokens.  A box takes 64 dims,
// `inner` heads and `tokens` tokens.
bool make_map(CUtensorMap* map, const void* p, bool bf16, int rank, int inner, int heads, int64_t n, int64_t stride,
              int tokens) {
  const cuuint64_t row = kHeadDim * 2;
  cuuint64_t dims[4] = {kHeadDim, static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(heads / inner),
                        static_cast<cuuint64_t>(n)};
  cuuint64_t strides[3] = {row, row * inner, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(inner), 1, static_cast<cuuint32_t>(tokens)};
  const cuuint32_t unit[4] = {1, 1, 1, 1};
  if (rank == 3) {
    dims[1] = dims[2];
    dims[2] = dims[3];
    strides[0] = strides[1];
    strides[1] = strides[2];
    box[1] = 1;
    box[2] = box[3];
  }
  return encode_tiled()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                        const_cast<void*>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kBF16, int kCap, bool kBias>
cudaError_t launch_one(const PrefillArgs& a, cudaStream_t stream) {
  const cudaError_t e = ensure_smem_limit<prefill_kernel<kBF16, kCap, kBias>>(kSmemBytes);
  if (e != cudaSuccess) return e;
  // the most items that these rows can make, or a CTA per multiprocessor
  const int64_t items = ((static_cast<int64_t>(a.n_tokens) >> (8 - a.log_group)) + a.batch) * a.num_kv_heads;
  const int64_t ctas = std::min<int64_t>(items, device_sm_count());
  return launch_pdl(prefill_kernel<kBF16, kCap, kBias>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), kSmemBytes,
                    stream, a);
}
template <bool kBF16, int kCap>
cudaError_t launch_cap(const PrefillArgs& a, cudaStream_t stream) {
  return a.alibi_slopes != nullptr ? launch_one<kBF16, kCap, true>(a, stream) : launch_one<kBF16, kCap, false>(a, stream);
}
template <bool kBF16>
cudaError_t launch_type(const PrefillArgs& a, cudaStream_t stream) {
  if (a.softcap > kLargeCap) return launch_cap<kBF16, 2>(a, stream);
  return a.softcap > 0.0f ? launch_cap<kBF16, 1>(a, stream) : launch_cap<kBF16, 0>(a, stream);
}

}  // namespace

cudaError_t launch_prefill(PrefillArgs& a, cudaStream_t stream) {
  if (!encode_tiled()) return cudaErrorNotSupported;
  const int group = 1 << a.log_group;
  if (!make_map(&a.map_q, a.q, a.bf16, 4, group, a.num_kv_heads * group, a.n_tokens, a.q_stride, kTile / group) ||
      !make_map(&a.map_out, a.out, a.bf16, 4, group, a.num_kv_heads * group, a.n_tokens, a.out_stride, 32 / group) ||
      !make_map(&a.map_k, a.k, a.bf16, 3, 1, a.num_kv_heads, a.n_tokens, a.k_stride, kTile) ||
      !make_map(&a.map_v, a.v, a.bf16, 3, 1, a.num_kv_heads, a.n_tokens, a.v_stride, kTile))
    return cudaErrorInvalidValue;
  return a.bf16 ? launch_type<true>(a, stream) : launch_type<false>(a, stream);
}

}  // namespace kvq
