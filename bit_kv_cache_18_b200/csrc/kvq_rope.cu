// kvq_rope.cu -- rotary positions of a step's queries and keys, one launch.
//
// Pair i of a head vector, (a, b) = (x_2i, x_2i+1) interleaved or
// (x_i, x_i+rd/2) in the half layout, becomes
//   m (a cos t - b sin t, b cos t + a sin t),  t = 2 pi f_i position,
// f_i in turns per position; the dims behind rotary_dim stay as they are.
//
// Angles.  f_i is a 64-bit fixed-point fraction of a turn, so position x f_i
// modulo one turn is the wrapped 64-bit integer product: off by the table's last
// place times the position, 2^-33 of a turn at the furthest (a 32-bit float
// product is off by 0.06 radians at position 2^20).  The upper 32 bits, as a
// signed number of half turns, round to fp32 once (2^-26 of a turn) and go to
// sincospif; the arithmetic on the values is fp32, rounded once to the output
// type.
//
// What bounds it: HBM, every row is read and written once; 65536 tokens of 64 +
// 8 heads (2.4 GB) take 369 us, 6.55 TB/s, the measured copy rate.  Eight
// threads take a row, 16 elements each as two 16-byte pieces (both members of
// eight pairs in either layout, so a row may be rotated in place), and keep
// their eight cosines and sines in registers for all the rows of the token
// that the CTA gives them; a thread's first two rows are on their way while it
// forms them, and four loads are in flight after that.
#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kRowThreads = 8;   // threads per 128-element row
constexpr int kRopeThreads = 192;  // at most: small CTAs, many to a multiprocessor (65536 x 72 rows: 369 us, 256 threads 391, 320 430)

template <bool kBF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (kBF16) return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
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

template <bool kBF16, bool kInterleaved>
__device__ __forceinline__ void rotate(uint4& u, uint4& v, const float (&cs)[8], const float (&sn)[8]) {
  uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  if (kInterleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // word j holds pair j
      const float2 x = unpack2<kBF16>(w[j]);
      w[j] = pack2<kBF16>(fmaf(x.x, cs[j], -x.y * sn[j]), fmaf(x.y, cs[j], x.x * sn[j]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // word j and word 4 + j hold pairs 2j and 2j + 1
      const float2 x = unpack2<kBF16>(w[j]), y = unpack2<kBF16>(w[4 + j]);
      w[j] = pack2<kBF16>(fmaf(x.x, cs[2 * j], -y.x * sn[2 * j]), fmaf(x.y, cs[2 * j + 1], -y.y * sn[2 * j + 1]));
      w[4 + j] = pack2<kBF16>(fmaf(y.x, cs[2 * j], x.x * sn[2 * j]), fmaf(y.y, cs[2 * j + 1], x.y * sn[2 * j + 1]));
    }
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
  v = make_uint4(w[4], w[5], w[6], w[7]);
}

template <bool kBF16, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
  const int64_t n = blockIdx.x;
  const int c = threadIdx.x % kRowThreads;  // pairs 8c .. 8c+7, or 16 plain elements
  const int r0 = threadIdx.x / kRowThreads, rstep = blockDim.x / kRowThreads;
  const int half = a.rotary_dim / 2;
  const bool rotates = 8 * c < half;
  pdl_wait();
  pdl_trigger();
  const int pos = a.positions[n];
  if (pos < 0) return;  // a padding row
  // offsets (16-byte pieces) of my two pieces in a row
  const int p0 = rotates && !kInterleaved ? c : 2 * c;
  const int p1 = rotates && !kInterleaved ? half / 8 + c : 2 * c + 1;
  const int rows = a.num_q_heads + a.num_k_heads;
  auto source = [&](int r) {
    return reinterpret_cast<const uint4*>(r < a.num_q_heads ? a.q + n * a.q_stride + r * kHeadDim
                                                            : a.k + n * a.k_stride + (r - a.num_q_heads) * kHeadDim);
  };
  auto target = [&](int r) {
    return reinterpret_cast<uint4*>(r < a.num_q_heads ? a.q_out + n * a.q_out_stride + r * kHeadDim
                                                      : a.k_out + n * a.k_out_stride + (r - a.num_q_heads) * kHeadDim);
  };
  // two rows at a time, the first two on their way while the angles are formed
  uint4 u[2], v[2];
  auto load = [&](int r) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (r + x * rstep < rows) {
        u[x] = source(r + x * rstep)[p0];
        v[x] = source(r + x * rstep)[p1];
      }
  };
  load(r0);
  float cs[8], sn[8];
  if (rotates) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t phase = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * __ldg(a.turns + 8 * c + j);
      const float x = __int2float_rn(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31: half turns
      sincospif(x, &sn[j], &cs[j]);
      cs[j] *= a.magnitude;
      sn[j] *= a.magnitude;
    }
  }
  for (int r = r0; r < rows; r += 2 * rstep) {
    if (r != r0) load(r);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (r + x * rstep >= rows) break;
      uint4* d4 = target(r + x * rstep);
      if (rotates)
        rotate<kBF16, kInterleaved>(u[x], v[x], cs, sn);
      else if (d4 == source(r + x * rstep))
        continue;
      d4[p0] = u[x];
      d4[p1] = v[x];
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  const int rows = a.num_q_heads + a.num_k_heads;
  // as few passes over a token's rows as kRopeThreads threads allow, evenly filled
  const int want = rows * kRowThreads, passes = (want + kRopeThreads - 1) / kRopeThreads;
  const int threads = ((want + passes - 1) / passes + 31) / 32 * 32;
  const dim3 grid(static_cast<unsigned>(a.n_tokens)), block(threads);
  if (a.bf16)
    return a.interleaved ? launch_pdl(rope_kernel<true, true>, grid, block, 0, stream, a)
                         : launch_pdl(rope_kernel<true, false>, grid, block, 0, stream, a);
  return a.interleaved ? launch_pdl(rope_kernel<false, true>, grid, block, 0, stream, a)
                       : launch_pdl(rope_kernel<false, false>, grid, block, 0, stream, a);
}

}  // namespace kvq
