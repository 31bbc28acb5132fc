// Selective state space scan (sm_103a), over packed prompts and for single tokens: for every channel and state
//   h <- exp(d A) h + d x B,   y = (sum_n C h + D x) silu(z).
#include "lq_seq.cuh"

namespace lqi {

namespace {

constexpr int kNT = 128;

template <typename T, int N>
__device__ __forceinline__ void token(const SsmParams& p, int64_t t, int c, int g, const float (&A)[N], float bias,
                                      float D, float (&h)[N]) {
  const float v = __fadd_rn(to_f(static_cast<const T*>(p.dt)[t * p.sdt + c]), bias);
  const float d = p.softplus ? softplus(v) : v;
  const float x = to_f(static_cast<const T*>(p.x)[t * p.sx + c]), dx = __fmul_rn(d, x);
  const T* B = static_cast<const T*>(p.B) + t * p.sb + (int64_t)g * p.n_state;
  const T* C = static_cast<const T*>(p.C) + t * p.sc + (int64_t)g * p.n_state;
  float y = 0.0f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (n >= p.n_state) break;
    h[n] = __fmaf_rn(ex2_approx(__fmul_rn(d, A[n])), h[n], __fmul_rn(dx, to_f(B[n])));
    y = __fmaf_rn(to_f(C[n]), h[n], y);
  }
  y = __fmaf_rn(D, x, y);
  if (p.z) y = __fmul_rn(y, silu(to_f(static_cast<const T*>(p.z)[t * p.sz + c])));
  static_cast<T*>(p.y)[t * p.sy + c] = from_f<T>(y);
}

// One thread: all states of a channel, a sequence's tokens one after the other.
template <typename T, int N>
__global__ void __launch_bounds__(kNT) k_ssm(SsmParams p, int blocks, int step) {
  const int64_t b = blockIdx.x / (unsigned)blocks;
  const int c = (int)(blockIdx.x % (unsigned)blocks) * kNT + threadIdx.x;
  if (c >= p.channels) return;
  int64_t begin = b, len = 1;
  if (!step) bounds(p, b, begin, len);
  const int g = c / p.per_group;
  const float* S0 = step ? p.S : p.S0;
  const int64_t at = (b * p.channels + c) * p.n_state;
  float A[N], h[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    A[n] = h[n] = 0.0f;
    if (n < p.n_state) {
      A[n] = __fmul_rn(p.A[(int64_t)c * p.n_state + n], kLog2E);
      if (S0) h[n] = S0[at + n];
    }
  }
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, D = p.D ? p.D[c] : 0.0f;
  for (int64_t t = begin; t < begin + len; ++t) token<T, N>(p, t, c, g, A, bias, D, h);
  if (!p.S) return;
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (n < p.n_state) p.S[at + n] = h[n];
}

template <typename T>
cudaError_t launch(const SsmParams& p, int step, cudaStream_t st) {
  const int blocks = (p.channels + kNT - 1) / kNT;
  const unsigned grid = (unsigned)(p.n_seqs * blocks);
  if (p.n_state <= 16) k_ssm<T, 16><<<grid, kNT, 0, st>>>(p, blocks, step);
  else k_ssm<T, 64><<<grid, kNT, 0, st>>>(p, blocks, step);
  return cudaGetLastError();
}

cudaError_t launch_any(const SsmParams& p, int step, cudaStream_t st) {
  if (p.dtype == LQ_F32) return launch<float>(p, step, st);
  if (p.dtype == LQ_BF16) return launch<__nv_bfloat16>(p, step, st);
  return launch<__half>(p, step, st);
}

}  // namespace

int64_t ssm_blocks(const lq_ssm_config* c) { return (c->channels + kNT - 1) / kNT; }

void ssm_plan(const lq_ssm_config*, int64_t n_seqs, int64_t, int64_t, int64_t* seg, int64_t* slots) {
  *seg = 0;
  *slots = n_seqs;
}

int64_t ssm_most_slots(const lq_ssm_config*, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_ssm_prefill(const SsmParams& p, cudaStream_t st) { return launch_any(p, 0, st); }
cudaError_t launch_ssm_step(const SsmParams& p, cudaStream_t st) { return launch_any(p, 1, st); }

}  // namespace lqi
