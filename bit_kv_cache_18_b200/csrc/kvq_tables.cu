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
// and takes 3.5 us, 2048 requests with 131072 new tokens 13.5 us.  So the design
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

struct Sums {
  long long need, tok, back;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) {
  return Sums{x.need + y.need, x.tok + y.tok, x.back + y.back};
}

// The last i in [0, n) with x[i] <= v (x ascending, x[0] = 0 <= v).
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

__global__ void __launch_bounds__(1024) tables_kernel(TablesArgs a) {
  extern __shared__ int sums_smem[];
  int* tokx = sums_smem;          // [batch]: new tokens of the sequences before b
  int* needx = tokx + a.batch;    // [batch]: blocks taken by them
  int* backx = needx + a.batch;   // [batch]: blocks returned by them
  __shared__ Sums warp_sum[32];
  __shared__ long long total_need, total_tok;
  __shared__ int first_refused, is_last;
  const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) first_refused = INT_MAX;
  pdl_wait();
  pdl_trigger();
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
  Sums mine{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    bool ok;
    mine = mine + asks(b, &ok);
    if (!ok && blockIdx.x == 0) record_status(a.status, KVQ_ERR_OUT_OF_RANGE);
  }
  Sums inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums up{__shfl_up_sync(0xffffffffu, inc.need, o), __shfl_up_sync(0xffffffffu, inc.tok, o),
                  __shfl_up_sync(0xffffffffu, inc.back, o)};
    if (lane >= o) inc = inc + up;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  Sums before{0, 0, 0}, all{0, 0, 0};
  for (int w = 0; w < nthr / 32; ++w) {
    if (w == warp) before = all;
    all = all + warp_sum[w];
  }
  before = before + Sums{inc.need - mine.need, inc.tok - mine.tok, inc.back - mine.back};

  // A growing sequence is served while the blocks and the packed batch last;
  // the running sums only rise, so everything behind the first refusal that
  // grows is refused too.
  Sums run = before;
  for (int b = b0; b < b1; ++b) {
    bool ok;
    const Sums s = asks(b, &ok);
    if (s.tok > 0 && (run.need + s.need > count || run.tok + s.tok > a.max_tokens)) {
      atomicMin(&first_refused, b);
      break;
    }
    run = run + s;
  }
  if (tid == 0) {
    total_need = all.need;
    total_tok = all.tok;
  }
  __syncthreads();
  const int refused = first_refused;
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
  __syncthreads();
  const long long need = total_need, tok = total_tok;
  run = before;
  for (int b = b0; b < b1; ++b) {
    bool ok;
    needx[b] = static_cast<int>(min(run.need, need));
    tokx[b] = static_cast<int>(min(run.tok, tok));
    backx[b] = static_cast<int>(min(run.back, static_cast<long long>(INT_MAX)));
    if (blockIdx.x == 0) a.cu_seqlens[b] = tokx[b];
    run = run + asks(b, &ok);
  }
  if (blockIdx.x == 0 && tid == 0) a.cu_seqlens[a.batch] = static_cast<int>(tok);
  // returned blocks that fit the ring (all, unless the caller's counts are off)
  const int back = static_cast<int>(min(all.back, static_cast<long long>(a.capacity - count)));
  if (back < all.back && blockIdx.x == 0 && tid == 0) record_status(a.status, KVQ_ERR_OUT_OF_RANGE);
  __syncthreads();

  const int g0 = blockIdx.x * nthr + tid, gstride = gridDim.x * nthr;
  auto ring_at = [&](long long i) {  // i-th entry from the head, i < 2 capacity
    long long p = head + i;
    if (p >= a.capacity) p -= a.capacity;
    return a.ring + p;
  };
  // new tokens: position, sequence, slot; -1 behind the last one
  for (int64_t n = g0; n < a.max_tokens; n += gstride) {
    int pos = -1, b = -1, slot = -1;
    if (n < tok) {
      b = find_seq(tokx, a.batch, static_cast<int>(n));
      const int len = a.lens[b];
      pos = len + static_cast<int>(n) - tokx[b];
      const int e = pos / kBlockSize, have = (len + kBlockSize - 1) / kBlockSize;
      const int p = e < have ? a.table[static_cast<int64_t>(b) * a.max_blocks + e] : *ring_at(needx[b] + e - have);
      if (p >= 0 && p < INT_MAX / kBlockSize)
        slot = p * kBlockSize + pos % kBlockSize;
      else
        record_status(a.status, KVQ_ERR_OUT_OF_RANGE);
    }
    a.positions[n] = pos;
    a.seq_ids[n] = b;
    a.slots[n] = slot;
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
  if (gridDim.x > 1) {
    if (tid == 0) {
      __threadfence();
      is_last = atomicAdd(a.state_out + 2, 1) == static_cast<int>(gridDim.x) - 1;
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
  const cudaError_t e = ensure_smem_limit<tables_kernel>(3 * kMaxTableBatch * static_cast<int>(sizeof(int)));
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(a.max_tokens) + a.batch;
  int64_t ctas = (items + kTokensPerCta - 1) / kTokensPerCta;
  if (ctas > device_sm_count()) ctas = device_sm_count();
  if (ctas < 1) ctas = 1;
  const int threads = items <= 256 ? 256 : 1024;
  return launch_pdl(tables_kernel, dim3(static_cast<unsigned>(ctas)), dim3(threads), bytes, stream, a);
}

}  // namespace kvq
