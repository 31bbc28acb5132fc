// Log probabilities of given tokens, entropy and the most likely tokens of rows of logits (sm_103a):
//   lse = log sum_t e^x_t,   logprob = x_token - lse,   entropy = lse - sum_t p_t x_t.
#include "lq_seq.cuh"

namespace lqi {

namespace {

constexpr int kNT = 256;

// Floats as unsigned numbers in the same order (-0 counts as +0), and an element's place in its row's order: larger
// logits first, then lower indices.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(float x, int64_t t) {
  return ((uint64_t)ordered(x) << 32) | (0xffffffffu - (uint32_t)t);
}

// What a thread, warp or CTA knows of its elements: sum e^(x - ref) and sum e^(x - ref) (x - ref).
struct Sum {
  float ref, s, e;
};

__device__ __forceinline__ Sum join(Sum a, Sum b) {
  if (!(b.ref <= a.ref)) {  // (a NaN goes on)
    const Sum t = a;
    a = b;
    b = t;
  }
  if (b.ref == -INFINITY) return a;
  const float d = __fsub_rn(b.ref, a.ref), f = ex2_approx(__fmul_rn(d, kLog2E));
  a.s = __fmaf_rn(f, b.s, a.s);
  // (beyond fp32's range of exponents nothing of b is left, and f d would not be a number)
  a.e = __fmaf_rn(f, __fmaf_rn(fmaxf(d, -1e30f), b.s, b.e), a.e);
  return a;
}

// One CTA a row, which it reads 1 + n_top times.
template <typename T>
__global__ void __launch_bounds__(kNT) k_logprob(LogprobParams p) {
  __shared__ Sum part[kNT / 32];
  __shared__ uint64_t best[kNT / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x;
  const T* x = static_cast<const T*>(p.logits) + r * p.row_stride;
  Sum m = {-INFINITY, 0.0f, 0.0f};
  for (int64_t t = tid; t < p.vocab; t += kNT) m = join(m, {to_f(x[t]), 1.0f, 0.0f});
  for (int o = 16; o; o >>= 1)
    m = join(m, {__shfl_xor_sync(0xffffffffu, m.ref, o), __shfl_xor_sync(0xffffffffu, m.s, o),
                 __shfl_xor_sync(0xffffffffu, m.e, o)});
  if (lane == 0) part[warp] = m;
  __syncthreads();
  m = part[0];
  for (int w = 1; w < kNT / 32; ++w) m = join(m, part[w]);
  const bool fine = m.ref > -INFINITY && m.ref < INFINITY && m.s < INFINITY;
  const float ls = logf(m.s);
  if (tid == 0) {
    if (p.logprob) {
      const int32_t t = p.tokens[r];
      float v = t < 0 ? 0.0f : NAN;
      if (t >= 0 && t < p.vocab && fine) v = __fsub_rn(__fsub_rn(to_f(x[t]), m.ref), ls);
      p.logprob[r] = v;
    }
    if (p.entropy) p.entropy[r] = fine ? __fsub_rn(ls, __fdiv_rn(m.e, m.s)) : NAN;
  }
  uint64_t last = ~0ull;
  for (int k = 0; k < p.n_top; ++k) {
    uint64_t b = 0;
    for (int64_t t = tid; t < p.vocab; t += kNT) {
      const uint64_t key = key_of(to_f(x[t]), t);
      if (key < last && key > b) b = key;
    }
    for (int o = 16; o; o >>= 1) {
      const uint64_t y = __shfl_xor_sync(0xffffffffu, b, o);
      b = y > b ? y : b;
    }
    __syncthreads();
    if (lane == 0) best[warp] = b;
    __syncthreads();
    for (int w = 0; w < kNT / 32; ++w) b = best[w] > b ? best[w] : b;
    last = b;
    if (tid == 0) {
      const int64_t t = 0xffffffffu - (uint32_t)b;
      p.top_token[r * p.n_top + k] = fine ? (int32_t)t : -1;
      p.top_logprob[r * p.n_top + k] = fine ? __fsub_rn(__fsub_rn(to_f(x[t]), m.ref), ls) : NAN;
    }
  }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams& p, cudaStream_t st) {
  const unsigned grid = (unsigned)p.rows;
  if (p.dtype == LQ_F32) k_logprob<float><<<grid, kNT, 0, st>>>(p);
  else if (p.dtype == LQ_BF16) k_logprob<__nv_bfloat16><<<grid, kNT, 0, st>>>(p);
  else k_logprob<__half><<<grid, kNT, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace lqi
