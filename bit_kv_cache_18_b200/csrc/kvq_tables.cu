// kvq_tables.cu -- the tables of a serving step, built on the GPU from the
// requests' lengths: which pool blocks each sequence takes or gives back,
// where its new tokens lie in the packed batch and in the pool.
//
// The pages leave the block manager to the engine around the backend ("Трюк
// Huawei с KV-кэшем" (beyondheadline.xyz), section "Заявка, которая ломает
// привычный компромисс": the cache blocks); the rules are those of
// include/kvq.h.  With have = ceil(len / 16), want = ceil(target / 16), a
// growing sequence needs want - have blocks and target - len tokens, a
// shrinking one returns have - want blocks.  Running sums over the batch give
// every sequence its place in the free list and in the packed batch, and
// every item (token, taken block, returned block) then finds its sequence by
// a binary search in the sums: all the work after the sums is flat, whatever
// the lengths.
//
// What bounds it: latency.  A decode step of 64 requests moves a few kilobytes
// and takes 3.6 us, 2048 requests with 131072 new tokens 10.6 us.  So the design
// is one launch: every CTA forms the (same) running sums for itself in shared
// memory rather than wait for another kernel or CTA, nothing that a CTA reads
// is written by another during the call (a new entry is read from the free
// list, not from the table), and the words that may alias inputs (the lengths
// and the free list's state) are written by the CTA that finishes last.
#include <climits>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

// Tokens a CTA takes before another one is launched: below it the launch of
// the second CTA and the ticket cost more than the loop.
constexpr int kTokensPerCta = 2048;
constexpr int kSmallThreads = 256, kLargeThreads = 1024;

// The CTAs of a call count themselves in state_out[2] by this step, so that what
// the word may hold, 0 .. CTAs - 1 steps, is told from anything else, a word
// that was never zeroed for one: a count that starts elsewhere would find its
// last CTA too early or never.
constexpr uint32_t kTicketStep = 0x9E3779B1u;
constexpr uint32_t inverse(uint32_t x) {  // modulo 2^32, by Newton's iteration (x odd)
  uint32_t y = x;
  for (int i = 0; i < 5; ++i) y *= 2u - x * y;
  return y;
}
static_assert(kTicketStep * inverse(kTicketStep) == 1u, "steps to a count");

struct Sums {
  long long need, tok, back;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) {
  return Sums{x.need + y.need, x.tok + y.tok, x.back + y.back};
}

// For each v: the last i in [0, n) with x[i] <= v (x ascending, x[0] = 0 <= v).
// The searches of a thread run side by side, so their reads overlap.
template <int kN>
__device__ __forceinline__ void find_seqs(const int* x, int n, const int (&v)[kN], int (&at)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) at[i] = 0;
  for (int step = 1 << (31 - __clz(n | 1)); step > 0; step >>= 1) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int to = at[i] + step;
      if (to < n && x[to] <= v[i]) at[i] = to;
    }
  }
}
// One search, by halves: one step fewer.
__device__ __forceinline__ int find_seq(const int* x, int n, int v) {
  int lo = 0, hi = n;  // x[lo] <= v < x[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (x[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// kLarge: the form for many requests and tokens.  A thread keeps what its first
// requests ask for (instead of reading the lengths anew in each pass), every
// warp scans the warps' sums (instead of adding them one after the other), and
// tokens are looked up two at a time.  2048 requests take 10.6 us so, 13.5 in
// the small form; 64 requests 4.1, and 3.6 in the small form, whose code is
// shorter.
template <bool kLarge>
__global__ void __launch_bounds__(kLarge ? kLargeThreads : kSmallThreads) tables_kernel(TablesArgs a) {
  constexpr int kKeep = kLarge ? 2 : 0;   // requests whose needs a thread keeps
  constexpr int kTokens = kLarge ? 2 : 1;  // tokens looked up at a time
  extern __shared__ int sums_smem[];
  int* tokx = sums_smem;          // [batch]: new tokens of the sequences before b
  int* needx = tokx + a.batch;    // [batch]: blocks taken by them
  int* backx = needx + a.batch;   // [batch]: blocks returned by them
  __shared__ long long warp_need[32], warp_tok[32], warp_back[32];
  __shared__ long long total_need, total_tok;
  __shared__ int first_refused, is_last, ticket_bad;
  const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) first_refused = INT_MAX;
  pdl_wait();
  pdl_trigger();
  const uint32_t ticket =
      kLarge && gridDim.x > 1 && tid == 0 ? __ldcg(reinterpret_cast<const uint32_t*>(a.state_out + 2)) : 0u;
  int head = a.state_in[0], count = a.state_in[1];
  const bool bad_state = head < 0 || head >= a.capacity || count < 0 || count > a.capacity;
  if (bad_state) {
    if (tid == 0 && blockIdx.x == 0) record_status(a.status, KVQ_ERR_OUT_OF_RANGE);
    head = count = 0;
  }
  const long long longest = static_cast<long long>(a.max_blocks) * kBlockSize;

  // What sequence b asks for.  A length outside [0, longest] leaves the
  // sequence as it was.
  auto asks = [&](int b, bool* ok) {
    const int len = a.lens[b], target = a.target[b];
    *ok = len >= 0 && len <= longest && target >= 0 && target <= longest;
    Sums s{0, 0, 0};
    if (*ok) {
      const int have = (len + kBlockSize - 1) / kBlockSize, want = (target + kBlockSize - 1) / kBlockSize;
      if (target > len) {
        s.need = want - have;
        s.tok = target - len;
      } else if (!bad_state) {
        s.back = have - want;
      }
    }
    return s;
  };

  // running sums: thread t takes sequences [b0, b1)
  const int per = (a.batch + nthr - 1) / nthr;
  const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
  Sums keep[kKeep > 0 ? kKeep : 1];
  bool out_of_range = false;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    bool ok = true;
    keep[i] = b0 + i < b1 ? asks(b0 + i, &ok) : Sums{0, 0, 0};
    out_of_range |= !ok;
  }
  // f(b, what it asks for) for my sequences in order
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (b0 + i < b1) f(b0 + i, keep[i]);
    for (int b = b0 + kKeep; b < b1; ++b) {
      bool ok;
      f(b, asks(b, &ok));
      out_of_range |= !ok;
    }
  };
  Sums mine{0, 0, 0};
  each([&](int, const Sums& s) { mine = mine + s; });
  if (out_of_range && blockIdx.x == 0) record_status(a.status, KVQ_ERR_OUT_OF_RANGE);
  auto warp_scan = [&](Sums v) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums up{__shfl_up_sync(0xffffffffu, v.need, o), __shfl_up_sync(0xffffffffu, v.tok, o),
                    __shfl_up_sync(0xffffffffu, v.back, o)};
      if (lane >= o) v = v + up;
    }
    return v;
  };
  auto from_lane = [&](const Sums& v, int src) {
    return Sums{__shfl_sync(0xffffffffu, v.need, src), __shfl_sync(0xffffffffu, v.tok, src),
                __shfl_sync(0xffffffffu, v.back, src)};
  };
  // (Looked at only now, so that its way from memory costs nothing.)  A bad one is
  // the same for every CTA: then none counts itself, and every sequence is refused.
  if (kLarge && tid == 0) {
    ticket_bad = ticket * inverse(kTicketStep) >= gridDim.x;
    if (ticket_bad) {
      first_refused = 0;
      if (blockIdx.x == 0) record_status(a.status, KVQ_ERR_OUT_OF_RANGE);
    }
  }
  const Sums inc = warp_scan(mine);
  if (lane == 31) {
    warp_need[warp] = inc.need;
    warp_tok[warp] = inc.tok;
    warp_back[warp] = inc.back;
  }
  __syncthreads();
  // the sums before my warp and in all
  Sums to_warp{0, 0, 0}, all{0, 0, 0};
  if (!kLarge) {
    for (int w = 0; w < nthr / 32; ++w) {
      if (w == warp) to_warp = all;
      all = all + Sums{warp_need[w], warp_tok[w], warp_back[w]};
    }
  } else {
    const Sums own{warp_need[lane], warp_tok[lane], warp_back[lane]};  // (32 warps)
    const Sums upto = warp_scan(own);
    all = from_lane(upto, 31);
    to_warp = from_lane(upto, warp == 0 ? 31 : warp - 1);
    if (warp == 0) to_warp = Sums{0, 0, 0};
  }
  const Sums before{to_warp.need + inc.need - mine.need, to_warp.tok + inc.tok - mine.tok,
                    to_warp.back + inc.back - mine.back};

  // A growing sequence is served while the blocks and the packed batch last;
  // the running sums only rise, so everything behind the first refusal that
  // grows is refused too.
  Sums run = before;
  bool stop = false;
  each([&](int b, const Sums& s) {
    if (!stop && s.tok > 0 && (run.need + s.need > count || run.tok + s.tok > a.max_tokens)) {
      atomicMin(&first_refused, b);
      stop = true;
    }
    run = run + s;
  });
  if (tid == 0) {
    total_need = all.need;
    total_tok = all.tok;
  }
  __syncthreads();
  const int refused = first_refused;
  const bool bad_ticket = kLarge && ticket_bad != 0;
  if (refused >= b0 && refused < b1) {
    run = before;
    bool ok;
    for (int b = b0; b < refused; ++b) run = run + asks(b, &ok);
    total_need = run.need;
    total_tok = run.tok;
    if (blockIdx.x == 0)
      record_status(a.status, run.need + asks(refused, &ok).need > count ? KVQ_ERR_POOL_EXHAUSTED
                                                                         : KVQ_ERR_OUT_OF_RANGE);
  }
  if (refused != INT_MAX) __syncthreads();  // (the same for every thread)
  const long long need = total_need, tok = total_tok;
  run = before;
  each([&](int b, const Sums& s) {
    needx[b] = static_cast<int>(min(run.need, need));
    tokx[b] = static_cast<int>(min(run.tok, tok));
    backx[b] = static_cast<int>(min(run.back, static_cast<long long>(INT_MAX)));
    if (blockIdx.x == 0) a.cu_seqlens[b] = tokx[b];
    run = run + s;
  });
  if (blockIdx.x == 0 && tid == 0) a.cu_seqlens[a.batch] = static_cast<int>(tok);
  // returned blocks that fit the ring (all, unless the caller's counts are off)
  const int back = bad_ticket ? 0 : static_cast<int>(min(all.back, static_cast<long long>(a.capacity - count)));
  if (back < all.back && blockIdx.x == 0 && tid == 0) record_status(a.status, KVQ_ERR_OUT_OF_RANGE);
  __syncthreads();

  const int g0 = blockIdx.x * nthr + tid, gstride = gridDim.x * nthr;
  auto ring_at = [&](long long i) {  // i-th entry from the head, i < 2 capacity
    long long p = head + i;
    if (p >= a.capacity) p -= a.capacity;
    return a.ring + p;
  };
  // new tokens: position, sequence, slot; -1 behind the last one.
  for (int64_t n0 = g0; n0 < a.max_tokens; n0 += kTokens * static_cast<int64_t>(gstride)) {
    int v[kTokens], b[kTokens];
#pragma unroll
    for (int x = 0; x < kTokens; ++x)
      v[x] = static_cast<int>(min(n0 + x * static_cast<int64_t>(gstride), static_cast<int64_t>(INT_MAX)));
    if (v[0] < tok) {
      if (kTokens == 1)
        b[0] = find_seq(tokx, a.batch, v[0]);
      else
        find_seqs(tokx, a.batch, v, b);
    }
    int pos[kTokens], p[kTokens];
#pragma unroll
    for (int x = 0; x < kTokens; ++x) {
      pos[x] = p[x] = -1;
      if (v[x] < tok) {
        const int len = a.lens[b[x]];
        pos[x] = len + v[x] - tokx[b[x]];
        const int e = pos[x] / kBlockSize, have = (len + kBlockSize - 1) / kBlockSize;
        p[x] = e < have ? a.table[static_cast<int64_t>(b[x]) * a.max_blocks + e] : *ring_at(needx[b[x]] + e - have);
      }
    }
#pragma unroll
    for (int x = 0; x < kTokens; ++x) {
      if (v[x] >= a.max_tokens) break;
      int slot = -1;
      if (pos[x] >= 0) {
        if (p[x] >= 0 && p[x] < INT_MAX / kBlockSize)
          slot = p[x] * kBlockSize + pos[x] % kBlockSize;
        else
          record_status(a.status, KVQ_ERR_OUT_OF_RANGE);
      }
      a.positions[v[x]] = pos[x];
      a.seq_ids[v[x]] = pos[x] >= 0 ? b[x] : -1;
      a.slots[v[x]] = slot;
    }
  }
  // taken blocks: from the head of the ring into the rows
  for (int64_t i = g0; i < need; i += gstride) {
    const int b = find_seq(needx, a.batch, static_cast<int>(i));
    const int have = (a.lens[b] + kBlockSize - 1) / kBlockSize;
    a.table[static_cast<int64_t>(b) * a.max_blocks + have + static_cast<int>(i) - needx[b]] = *ring_at(i);
  }
  // returned blocks: from the rows to the tail of the ring (entries that no
  // sequence takes in this call: the free ones end before them)
  for (int64_t i = g0; i < back; i += gstride) {
    const int b = find_seq(backx, a.batch, static_cast<int>(i));
    const int want = (a.target[b] + kBlockSize - 1) / kBlockSize;
    *ring_at(static_cast<long long>(count) + i) =
        a.table[static_cast<int64_t>(b) * a.max_blocks + want + static_cast<int>(i) - backx[b]];
  }

  // The last CTA writes what may alias an input: every CTA has read it by then.
  __syncthreads();
  if (bad_ticket) {
    if (blockIdx.x == 0) {
      for (int b = tid; b < a.batch; b += nthr) a.lens_out[b] = a.lens[b];
      if (tid == 0) {
        const int h = a.state_in[0], c = a.state_in[1];
        a.state_out[0] = h;
        a.state_out[1] = c;
      }
    }
    return;
  }
  if (gridDim.x > 1) {
    if (tid == 0) {
      __threadfence();
      is_last = atomicAdd(reinterpret_cast<uint32_t*>(a.state_out + 2), kTicketStep) == (gridDim.x - 1) * kTicketStep;
      __threadfence();
    }
    __syncthreads();
    if (!is_last) return;
  }
  for (int b = tid; b < a.batch; b += nthr) {
    bool ok;
    const Sums s = asks(b, &ok);
    const bool kept = !ok || (s.tok > 0 && b >= refused) || (bad_state && s.tok == 0);
    a.lens_out[b] = kept ? a.lens[b] : a.target[b];
  }
  if (tid == 0) {
    if (bad_state) {  // the caller's words as they are
      const int h = a.state_in[0], c = a.state_in[1];
      a.state_out[0] = h;
      a.state_out[1] = c;
    } else {
      long long h = head + need;
      if (h >= a.capacity) h -= a.capacity;
      a.state_out[0] = static_cast<int>(h);
      a.state_out[1] = static_cast<int>(count - need + back);
    }
    a.state_out[2] = 0;
  }
}

}  // namespace

cudaError_t launch_tables(const TablesArgs& a, cudaStream_t stream) {
  const int bytes = 3 * a.batch * static_cast<int>(sizeof(int));
  const int64_t items = static_cast<int64_t>(a.max_tokens) + a.batch;
  if (items <= kSmallThreads) return launch_pdl(tables_kernel<false>, dim3(1), dim3(kSmallThreads), bytes, stream, a);
  const cudaError_t e = ensure_smem_limit<tables_kernel<true>>(3 * kMaxTableBatch * static_cast<int>(sizeof(int)));
  if (e != cudaSuccess) return e;
  int64_t ctas = (items + kTokensPerCta - 1) / kTokensPerCta;
  if (ctas > device_sm_count()) ctas = device_sm_count();
  return launch_pdl(tables_kernel<true>, dim3(static_cast<unsigned>(ctas)), dim3(kLargeThreads), bytes, stream, a);
}

}  // namespace kvq
