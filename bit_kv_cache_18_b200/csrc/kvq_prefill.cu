// kvq_prefill.cu -- attention of whole prompts over their own rows, on the
// fifth-generation tensor cores (tcgen05): the definition is in include/kvq.h.
//
// Rows.  The G query heads of a kv head share its keys and values, so the
// tile of a matrix product is (128 / G tokens) x (G heads): 128 rows, row r =
// token r / G, head r % G.  A CTA takes two such tiles, 256 / G tokens in a
// row, and walks the 128-token key tiles that either reads, from the newest
// to the oldest (with a distance bias the largest scores come first).  Packed
// this way the two tiles cover 32 tokens at G = 8, so little of the diagonal
// is computed for nothing, and a prompt of 20 tokens fills its tiles.
//
// Roles.  Warps 0-3 and 4-7 are the softmax of tile 0 and 1, a thread per row;
// warp 8 issues the products, warp 9 the copies (TMA, 128-byte swizzle; K and
// V tiles of 32 KB through one ring of five).  Tensor memory holds, per tile,
// the scores S (128 fp32 columns) and the output O (128 columns): all 512.
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
// fewer bits before the output's own: half a step, 2^-9 (bf16) or 2^-12
// (fp16) relative to p, of either sign, so it averages out over the keys.
//
// Masked places.  A masked score is replaced, not added to, so nothing that
// stands in a masked key reaches a row; a masked value is multiplied by p = 0,
// which only a NaN or an infinity survives.  A row that ends up not finite
// while its l is finite looks for one in the masked places of its tiles and,
// if there is one, is computed again without them (fix_row).
//
// Work.  The prompts' lengths are on the device, so the grid is the bound
// n / (256 / G) + batch per kv head, and each CTA finds its (prompt, tile)
// by its rank: items are ordered by falling tile index over all prompts, so
// the longest walks start first.
#include <cuda.h>
#include <math_constants.h>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kTile = 128;         // rows of a product, keys of a tile
constexpr int kStages = 5;         // K and V tiles in shared memory
constexpr int kTileBytes = kTile * kHeadDim * 2;
constexpr int kHalfBytes = kTileBytes / 2;  // 64 of the 128 dims: one swizzle width
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 per tile
constexpr float kLazy = 8.0f;      // log2 of the largest p
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // a device-side wait gives up after one second

struct __align__(1024) Smem {
  uint8_t q[2][kTileBytes];
  uint8_t kv[kStages][kTileBytes];
  uint64_t q_full[2];
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t s_full[2];  // S of the tile is written (and every product before it is complete)
  uint64_t p_full[2];  // P of the tile is written, O rescaled
  uint64_t o_full[2];  // O of the tile is final
  uint64_t fin;        // every product issued is complete
  uint32_t tmem_base;
  int abort;           // a wait ran out: every other wait gives up at once
  int seq, tile;       // this CTA's item
  int red[2][kThreads / 32];
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
__device__ __noinline__ bool mbar_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort) {
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
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

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
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %3, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(static_cast<uint32_t>(acc)), "r"(id)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %3, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(static_cast<uint32_t>(acc)), "r"(id)
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
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float* v) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
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

// cap tanh(s / cap) in base-2 units (cap_exp = 2 / (cap ln 2), cap2 = cap log2 e):
// tanh(x) = 1 - 2 / (e^2x + 1), an absolute error of about 2^-22 cap.
__device__ __forceinline__ float capped(float s, float cap_exp, float cap2) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(s * cap_exp) + 1.0f));
  return fmaf(-2.0f * cap2, r, cap2);
}

// The key interval [lo, hi) of the query at position t of a prompt of n tokens.
struct Span {
  int n, prefix, window;
  __device__ __forceinline__ int lo(int t) const { return window > 0 ? max(t - window + 1, 0) : 0; }
  __device__ __forceinline__ int hi(int t) const { return max(t + 1, prefix); }
};

// A row whose output is not finite though its l is: one warp looks for a value
// that is not finite among the masked keys [k0, k1) - [lo, hi) that the row's
// products read, and if there is one forms the output again over [lo, hi).
// True if it wrote the row.
template <bool kBF16>
__device__ __noinline__ bool fix_row(const PrefillArgs& a, int64_t row0, int t, int head, int kv_head, int k0, int k1,
                                     int lo, int hi, float slope2, float m, float l) {
  const int lane = threadIdx.x & 31;
  auto four = [&](const uint16_t* base, int64_t stride, int64_t r, int h) {
    const uint2 w = *reinterpret_cast<const uint2*>(base + r * stride + h * kHeadDim + 4 * lane);
    const float2 x = unpack2<kBF16>(w.x), y = unpack2<kBF16>(w.y);
    return make_float4(x.x, x.y, y.x, y.y);
  };
  bool found = false;
  for (int j = k0; j < k1 && !found; ++j) {
    if (j == lo) j = hi;
    if (j >= k1) break;
    const float4 v = four(a.v, a.v_stride, row0 + j, kv_head);
    found = __any_sync(0xffffffffu, !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w)));
  }
  if (!found) return false;
  const float4 q = four(a.q, a.q_stride, row0 + t, head);
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j = lo; j < hi; ++j) {
    const float4 k = four(a.k, a.k_stride, row0 + j, kv_head);
    float s = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, q.w * k.w)));
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    float y = a.softcap > 0.0f ? capped(s, a.softcap_exp, a.softcap) : s * a.scale_log2;
    y = fmaf(-slope2, fabsf(static_cast<float>(t - j)), y);
    const float p = ex2(y - m);
    const float4 v = four(a.v, a.v_stride, row0 + j, kv_head);
    o.x = fmaf(p, v.x, o.x);
    o.y = fmaf(p, v.y, o.y);
    o.z = fmaf(p, v.z, o.z);
    o.w = fmaf(p, v.w, o.w);
  }
  const float inv = 1.0f / l;
  *reinterpret_cast<uint2*>(a.out + (row0 + t) * a.out_stride + head * kHeadDim + 4 * lane) =
      make_uint2(pack2<kBF16>(o.x * inv, o.y * inv), pack2<kBF16>(o.z * inv, o.w * inv));
  return true;
}

// This CTA's item by its rank among the items in falling order of tile index
// (ties by prompt): sm.seq and sm.tile, or seq = -1.  Every thread calls.
// Prompt b has ceil(length / tokens) tiles; one whose bounds are not ascending
// or not within the rows has none and is recorded.
__device__ __forceinline__ void find_item(const PrefillArgs& a, Smem& sm, int rank, int tokens, int log_tokens) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
  auto tiles = [&](int b) {
    const int s = __ldg(a.cu_seqlens + b), e = __ldg(a.cu_seqlens + b + 1);
    return s >= 0 && e >= s && e <= a.n_tokens ? (e - s + tokens - 1) >> log_tokens : -1;
  };
  int step = 0;
  // items with a tile index >= i
  auto count = [&](int i) {
    int c = 0;
    for (int b = b0; b < b1; ++b) c += max(tiles(b) - i, 0);
    c = __reduce_add_sync(0xffffffffu, c);
    int* red = sm.red[step++ & 1];
    if (lane == 0) red[warp] = c;
    __syncthreads();
    c = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) c += red[w];
    return c;
  };
  if (blockIdx.x == 0)
    for (int b = b0; b < b1; ++b)
      if (tiles(b) < 0) record_status(a.status, KVQ_ERR_OUT_OF_RANGE);
  if (tid == 0) sm.seq = -1;
  if (rank >= count(0)) return;
  int lo = 0, hi = (a.n_tokens >> log_tokens) + 2;  // count(lo) > rank >= count(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (count(mid) > rank)
      lo = mid;
    else
      hi = mid;
  }
  const int k = rank - count(lo + 1);  // my place among the prompts with more than lo tiles
  int c = 0;
  for (int b = b0; b < b1; ++b) c += tiles(b) > lo ? 1 : 0;
  int inc = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  int* red = sm.red[step & 1];
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  int at = inc - c;
  for (int w = 0; w < warp; ++w) at += red[w];
  for (int b = b0; b < b1; ++b)
    if (tiles(b) > lo && at++ == k) {
      sm.seq = b;
      sm.tile = lo;
    }
}

template <bool kBF16, bool kCap, bool kBias>
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
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&sm.kv_full[i], 1);
        mbar_init(&sm.kv_empty[i], 1);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.q_full[i], 1);
        mbar_init(&sm.s_full[i], 1);
        mbar_init(&sm.p_full[i], kSoftWarps / 2);
        mbar_init(&sm.o_full[i], 1);
      }
      mbar_init(&sm.fin, 1);
      sm.abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
  }
  pdl_wait();
  const int log_g = a.log_group, log_tokens = 8 - log_g, tile_tokens = kTile >> log_g;
  const int kv_head = blockIdx.x % a.num_kv_heads;
  find_item(a, sm, blockIdx.x / a.num_kv_heads, 2 * tile_tokens, log_tokens);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  const int seq = sm.seq;
  bool bad = false;
  if (seq >= 0) {
    const int t0 = sm.tile << log_tokens;
    const int64_t row0 = __ldg(a.cu_seqlens + seq);
    Span sp;
    sp.n = __ldg(a.cu_seqlens + seq + 1) - static_cast<int>(row0);
    sp.window = a.window;
    sp.prefix = a.prefix_lens != nullptr ? min(__ldg(a.prefix_lens + seq), sp.n) : 0;
    // key tiles [klo, khi) of each row tile; the second may have no token
    const bool two = t0 + tile_tokens < sp.n;
    int klo[2], khi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int first = t0 + i * tile_tokens, last = min(first + tile_tokens, sp.n) - 1;
      klo[i] = sp.lo(first) / kTile;
      khi[i] = (sp.hi(last) + kTile - 1) / kTile;
      if (i == 1 && !two) khi[i] = klo[i] = klo[0];
    }
    const int top = max(khi[0], khi[1]), steps = top - klo[0];
    auto active = [&](int i, int c) { return top - 1 - c >= klo[i] && top - 1 - c < khi[i]; };

    if (warp == kLoadWarp) {
      auto box_q = [&](int i) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full[i], kTileBytes);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            tma_load4(smem_u32(sm.q[i]) + hf * kHalfBytes, &a.map_q, 64 * hf, 0, kv_head,
                      static_cast<int>(row0) + t0 + i * tile_tokens, &sm.q_full[i]);
        }
        __syncwarp();
      };
      int st = 0;
      uint32_t ph = 0;
      bool live = true;
      box_q(0);
      for (int x = 0; x < 2 * steps && live; ++x) {  // K and V of step x / 2
        if (x >= kStages && !mbar_wait(&sm.kv_empty[st], ph ^ 1u, abort)) {
          bad = true;
          live = false;  // no copy is issued any more
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.kv_full[st], kTileBytes);
          const CUtensorMap* map = x & 1 ? &a.map_v : &a.map_k;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            tma_load3(smem_u32(sm.kv[st]) + hf * kHalfBytes, map, 64 * hf, kv_head,
                      static_cast<int>(row0) + (top - 1 - x / 2) * kTile, &sm.kv_full[st]);
        }
        __syncwarp();
        if (x == 0 && two) box_q(1);
        if (++st == kStages) {
          st = 0;
          ph ^= 1u;
        }
        // after the last copy, or a wait that gave up: the copies still in
        // flight land before the CTA gives up its shared memory (below)
      }
      // the last copy into each stage, newest first
      for (int x = 0; x < kStages && x < 2 * steps; ++x) {
        if (--st < 0) {
          st = kStages - 1;
          ph ^= 1u;
        }
        if (!mbar_wait_slow(&sm.kv_full[st], ph, nullptr)) bad = true;
      }
      if (!mbar_wait_slow(&sm.q_full[0], 0, nullptr)) bad = true;
      if (two && !mbar_wait_slow(&sm.q_full[1], 0, nullptr)) bad = true;
    } else if (warp == kMmaWarp) {
      const uint32_t q0 = smem_u32(sm.q[0]), kv0 = smem_u32(sm.kv[0]);
      int st = 0;
      uint32_t ph = 0;
      uint32_t pph[2] = {0, 0};
      bool started[2] = {false, false};
      auto next = [&] {
        if (++st == kStages) {
          st = 0;
          ph ^= 1u;
        }
      };
      auto product_s = [&](int i, int stage) {
        if (lane == 0) {
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const uint32_t off = (s >> 2) * kHalfBytes + (s & 3) * 32;
            mma_ss(tbase + kColS + 128 * i, sdesc(q0 + i * kTileBytes + off, 16), sdesc(kv0 + stage * kTileBytes + off, 16),
                   idesc<kBF16>(false), s > 0);
          }
          mma_commit(&sm.s_full[i]);
        }
        __syncwarp();
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!mbar_wait(bar, parity, abort)) bad = true;
      };
      wait(&sm.q_full[0], 0);
      if (two) wait(&sm.q_full[1], 0);
      wait(&sm.kv_full[0], 0);
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (active(i, 0)) product_s(i, 0);
      if (lane == 0) mma_commit(&sm.kv_empty[0]);
      __syncwarp();
      next();
#pragma unroll 1
      for (int c = 0; c < steps; ++c) {
        const int sv = st;
        wait(&sm.kv_full[st], ph);
        next();
        const bool more = c + 1 < steps;
        const int sk = st;
        bool have_k = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (active(i, c)) {
            wait(&sm.p_full[i], pph[i]);
            pph[i] ^= 1u;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
              for (int s = 0; s < 8; ++s)
                mma_ts(tbase + kColO + 128 * i, tbase + kColS + 128 * i + 8 * s,
                       sdesc(kv0 + sv * kTileBytes + 2048 * s, kHalfBytes), idesc<kBF16>(true), started[i] || s > 0);
              if (!more || !active(i, c + 1)) mma_commit(&sm.o_full[i]);
            }
            __syncwarp();
            started[i] = true;
          }
          if (more && active(i, c + 1)) {
            if (!have_k) wait(&sm.kv_full[sk], ph);
            have_k = true;
            tc_fence_after();
            product_s(i, sk);
          }
        }
        if (lane == 0) {
          mma_commit(&sm.kv_empty[sv]);
          if (more) mma_commit(&sm.kv_empty[sk]);
        }
        __syncwarp();
        if (more) next();
      }
      if (lane == 0) mma_commit(&sm.fin);
      __syncwarp();
      if (!mbar_wait_slow(&sm.fin, 0, nullptr)) bad = true;
    } else if (warp < kSoftWarps && (warp < 4 || two)) {
      const int i = warp >> 2;
      const int r = tid & (kTile - 1);
      const int first = t0 + i * tile_tokens, last = min(first + tile_tokens, sp.n) - 1;
      const int t = first + (r >> log_g);
      const int head = (kv_head << log_g) + (r & ((1 << log_g) - 1));
      const bool valid = t < sp.n;
      const int lo = sp.lo(t), hi = sp.hi(t);  // (a row behind the last token: whatever it computes is dropped)
      const uint32_t lanes = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const uint32_t ts = lanes + kColS + 128 * i, to = lanes + kColO + 128 * i;
      const float slope2 = kBias ? __ldg(a.alibi_slopes + head) * 1.4426950408889634f : 0.0f;
      const float scale = kCap || kBias ? 1.0f : a.scale_log2;  // what is left to multiply by in the exponent
      float m = -CUDART_INF_F, l = 0.0f;
      bool started = false;
      uint32_t sph = 0;
#pragma unroll 1
      for (int c = 0; c < steps; ++c) {
        if (!active(i, c)) continue;
        const int j0 = (top - 1 - c) * kTile;
        if (!mbar_wait(&sm.s_full[i], sph, abort)) bad = true;
        sph ^= 1u;
        tc_fence_after();
        float s[kTile];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld32(ts + 32 * x, s + 32 * x);
        tmem_wait_ld();
        if (kCap) {
#pragma unroll
          for (int e = 0; e < kTile; ++e) s[e] = capped(s[e], a.softcap_exp, a.softcap);
        }
        if (kBias) {
          const float d0 = static_cast<float>(j0 - t);
#pragma unroll
          for (int e = 0; e < kTile; ++e)
            s[e] = fmaf(-slope2, fabsf(d0 + static_cast<float>(e)), kCap ? s[e] : s[e] * a.scale_log2);
        }
        if (j0 + kTile > sp.hi(first) || j0 < sp.lo(last)) {
          const int e0 = lo - j0, e1 = hi - j0;
#pragma unroll
          for (int e = 0; e < kTile; ++e) s[e] = e >= e0 && e < e1 ? s[e] : -CUDART_INF_F;
        }
        float mx = max3f(s[0], s[1], s[2]);
#pragma unroll
        for (int e = 3; e < kTile - 1; e += 2) mx = max3f(mx, s[e], s[e + 1]);
        mx = fmaxf(mx, s[kTile - 1]) * scale;
        const bool moves = mx > m + kLazy || (m == -CUDART_INF_F && mx > m);
        if (__any_sync(0xffffffffu, moves)) {
          const float mn = moves ? mx : m;
          const float alpha = moves ? ex2(m - mn) : 1.0f;
          if (started) {  // O is at rest: the product before S is complete
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              float o[32];
              tmem_ld32(to + 32 * x, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tmem_st32(to + 32 * x, o);
            }
          }
          l *= alpha;
          m = mn;
        }
        started = true;
        const float base = m == -CUDART_INF_F ? 0.0f : -m;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = ex2(fmaf(s[32 * x + 2 * e], scale, base));
            const float p1 = ex2(fmaf(s[32 * x + 2 * e + 1], scale, base));
            l += p0 + p1;
            w[e] = pack2<kBF16>(p0, p1);
          }
          tmem_st16(ts + 16 * x, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[i]);
      }
      if (!mbar_wait(&sm.o_full[i], 0, abort)) bad = true;
      tc_fence_after();
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      bool finite = true;
      uint16_t* dst = a.out + (row0 + t) * a.out_stride + head * kHeadDim;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float o[32];
        tmem_ld32(to + 32 * x, o);
        tmem_wait_ld();
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          finite = finite && isfinite(o[2 * e]) && isfinite(o[2 * e + 1]);
          w[e] = pack2<kBF16>(o[2 * e] * inv, o[2 * e + 1] * inv);
        }
        if (valid) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            reinterpret_cast<uint4*>(dst)[4 * x + e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        }
      }
      // rows that a masked value may have spoilt
      __syncwarp();
      uint32_t todo = __ballot_sync(0xffffffffu, valid && !finite && l > 0.0f && l < CUDART_INF_F);
      while (todo != 0u) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1u;
        const int ts_ = __shfl_sync(0xffffffffu, t, src), hs = __shfl_sync(0xffffffffu, head, src);
        const float sl = __shfl_sync(0xffffffffu, slope2, src), ms = __shfl_sync(0xffffffffu, m, src);
        const float ls = __shfl_sync(0xffffffffu, l, src);
        const int k1 = static_cast<int>(min(static_cast<int64_t>(khi[i]) * kTile, a.n_tokens - row0));
        fix_row<kBF16>(a, row0, ts_, hs, kv_head, klo[i] * kTile, k1, sp.lo(ts_), sp.hi(ts_), sl, ms, ls);
      }
    }
  }
  if (bad) record_status(a.status, KVQ_ERR_DEVICE_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "n"(kTmemCols));
  pdl_trigger();  // this CTA holds no tensor memory any more
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

template <bool kBF16, bool kCap, bool kBias>
cudaError_t launch_one(const PrefillArgs& a, cudaStream_t stream) {
  const cudaError_t e = ensure_smem_limit<prefill_kernel<kBF16, kCap, kBias>>(kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t items = (static_cast<int64_t>(a.n_tokens) >> (8 - a.log_group)) + a.batch;
  return launch_pdl(prefill_kernel<kBF16, kCap, kBias>, dim3(static_cast<unsigned>(items * a.num_kv_heads)),
                    dim3(kThreads), kSmemBytes, stream, a);
}
template <bool kBF16>
cudaError_t launch_type(const PrefillArgs& a, cudaStream_t stream) {
  const bool cap = a.softcap > 0.0f, bias = a.alibi_slopes != nullptr;
  if (cap) return bias ? launch_one<kBF16, true, true>(a, stream) : launch_one<kBF16, true, false>(a, stream);
  return bias ? launch_one<kBF16, false, true>(a, stream) : launch_one<kBF16, false, false>(a, stream);
}

}  // namespace

cudaError_t launch_prefill(PrefillArgs& a, cudaStream_t stream) {
  if (!encode_tiled()) return cudaErrorNotSupported;
  const int group = 1 << a.log_group;
  if (!make_map(&a.map_q, a.q, a.bf16, 4, group, a.num_kv_heads * group, a.n_tokens, a.q_stride, kTile / group) ||
      !make_map(&a.map_k, a.k, a.bf16, 3, 1, a.num_kv_heads, a.n_tokens, a.k_stride, kTile) ||
      !make_map(&a.map_v, a.v, a.bf16, 3, 1, a.num_kv_heads, a.n_tokens, a.v_stride, kTile))
    return cudaErrorInvalidValue;
  return a.bf16 ? launch_type<true>(a, stream) : launch_type<false>(a, stream);
}

}  // namespace kvq
