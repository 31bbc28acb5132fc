// Selective state space scan (sm_103a): how prompts are divided, and the kernel for single tokens.
#include "lq_ssm.cuh"

namespace lqi {

namespace {

// --------------------------------------------------------------------------------------------
// Single tokens.
template <typename T, int N>
__device__ __forceinline__ void token(const SsmParams& p, int64_t t, int c, int g, const float (&A)[N], float bias,
                                      float D, float (&h)[N]) {
  const float d = p.softplus ? step_of<T, true>(static_cast<const T*>(p.dt)[t * p.sdt + c], bias)
                             : step_of<T, false>(static_cast<const T*>(p.dt)[t * p.sdt + c], bias);
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

template <typename T, int N>
__global__ void __launch_bounds__(kNT) k_ssm_step(SsmParams p, int blocks) {
  const int64_t b = blockIdx.x / (unsigned)blocks;
  const int c = (int)(blockIdx.x % (unsigned)blocks) * kNT + threadIdx.x;
  if (c >= p.channels) return;
  const int64_t at = (b * p.channels + c) * p.n_state;
  float A[N], h[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    A[n] = h[n] = 0.0f;
    if (n < p.n_state) {
      A[n] = __fmul_rn(p.A[(int64_t)c * p.n_state + n], kLog2E);
      h[n] = p.S[at + n];
    }
  }
  token<T, N>(p, b, c, c / p.per_group, A, p.dt_bias ? p.dt_bias[c] : 0.0f, p.D ? p.D[c] : 0.0f, h);
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (n < p.n_state) p.S[at + n] = h[n];
}

template <typename T>
cudaError_t launch_token(const SsmParams& p, cudaStream_t st) {
  const int blocks = (p.channels + kNT - 1) / kNT;
  const unsigned grid = (unsigned)(p.n_seqs * blocks);
  if (p.n_state <= 16) k_ssm_step<T, 16><<<grid, kNT, 0, st>>>(p, blocks);
  else k_ssm_step<T, 64><<<grid, kNT, 0, st>>>(p, blocks);
  return cudaGetLastError();
}

// --------------------------------------------------------------------------------------------
// Prompts: how many states a thread holds, and whether sequences are split.
struct Shape {
  int spt, lpc;  // states a thread, lanes a channel
};

// What a token costs: ns of an SM with nothing else to do, and ns each of many CTAs on it. Measured with 8 to 64 states, bf16 and
// fp32: 106 to 136 and 98 to 110 with 16 states a thread, 69 to 112 and 50 to 63 with 8, 50 to 71 and 33 to 36 with 4.
struct Cost {
  double alone, many;
};
Cost cost_of(int spt) { return spt == 16 ? Cost{125, 99} : spt == 8 ? Cost{100, 54} : Cost{56, 33}; }

int padded(int n_state) { return n_state <= 8 ? 8 : n_state <= 16 ? 16 : n_state <= 32 ? 32 : 64; }
int most_states(int n_state) { return padded(n_state) < 16 ? padded(n_state) : 16; }

constexpr int64_t kSms = 152, kLeastSeg = 64;  // (tokens of a segment)
// CTAs that fit on the GPU at a time, by the kernels' registers
int64_t ctas_of(Shape s) {
  return kSms * (s.spt == 16 ? (s.lpc > 1 ? 2 : 4) : s.spt == 8 ? (s.lpc == 1 ? 5 : s.lpc == 8 ? 2 : 4) : s.lpc == 4 ? 3 : 4);
}

int64_t blocks_of(const lq_ssm_config* c, Shape s) {
  return (int64_t)c->groups * ssm_group_blocks(c->channels / c->groups, s.lpc);
}

// Segments that fill the GPU once; of each split sequence one is left out of either pass.
int64_t segment(int64_t n_tokens, int64_t ctas, int64_t blocks) {
  const int64_t n = ctas / blocks + 1, s = ((n_tokens + n - 1) / n + 15) / 16 * 16;
  return s < kLeastSeg ? kLeastSeg : s;
}

}  // namespace

// Of the shapes and of whole and split sequences what should take the least time. Whole sequences take as long as the
// longest one alone or as all tokens of all CTAs together, and some of the other as well; split ones 1.55 times the latter
// (the first pass has no outputs) or two segments one after the other, and 8 us for two more launches. Measured against the other
// choices: one sequence of 16,384 tokens x 4,096 channels of 16 states 490 us split with 16 states a thread, 833 whole with
// four; 16 ragged ones of up to 1,500 150 and 129; one of 300 x 2,048 channels 33 and 19.
void ssm_plan(const lq_ssm_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len, SsmPlan* plan) {
  const int64_t longest = max_len > 0 && max_len < n_tokens ? max_len : n_tokens;
  double best = 0;
  for (int spt = most_states(c->n_state); spt >= 4; spt /= 2) {
    const Shape s = {spt, padded(c->n_state) / spt};
    if (s.lpc > 8) break;
    const Cost cost = cost_of(spt);
    const int64_t blocks = blocks_of(c, s), seg = segment(n_tokens, ctas_of(s), blocks);
    const double alone = cost.alone * (double)longest, all = cost.many * (double)n_tokens * (double)blocks / kSms;
    const double whole = (alone > all ? alone + 0.3 * all : all + 0.3 * alone) + 3000;
    if (best == 0 || whole < best) {
      best = whole;
      *plan = {s.spt, s.lpc, 0, n_seqs, blocks};
    }
    if (longest < 3 * seg) continue;
    const double two = 2 * cost.alone * (double)seg, both = 1.55 * all;
    const double split = (two > both ? two : both) + 11000 + 60.0 * (double)(longest / seg);
    if (split < best) {
      best = split;
      *plan = {s.spt, s.lpc, seg, n_tokens / seg + n_seqs, blocks};
    }
  }
}

// A segment has at least kLeastSeg tokens, and there are no more than segment() makes of a call.
int64_t ssm_most_slots(const lq_ssm_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len) {
  const int64_t longest = max_len > 0 && max_len < n_tokens ? max_len : n_tokens;
  if (longest < 3 * kLeastSeg) return 0;
  int64_t most = 0;
  for (int spt = most_states(c->n_state); spt >= 4; spt /= 2) {
    const Shape s = {spt, padded(c->n_state) / spt};
    if (s.lpc > 8) break;
    const int64_t n = ctas_of(s) / blocks_of(c, s) + 1;
    if (n >= 3 && n > most) most = n;
  }
  const int64_t n = n_tokens / kLeastSeg;
  return most ? (n < most ? n : most) + n_seqs : 0;
}

cudaError_t launch_ssm_prefill(const SsmParams& p, cudaStream_t st) {
  if (p.dtype == LQ_F32) return launch_ssm_prefill_f32(p, st);
  if (p.dtype == LQ_BF16) return launch_ssm_prefill_bf16(p, st);
  return launch_ssm_prefill_f16(p, st);
}

cudaError_t launch_ssm_step(const SsmParams& p, cudaStream_t st) {
  if (p.dtype == LQ_F32) return launch_token<float>(p, st);
  if (p.dtype == LQ_BF16) return launch_token<__nv_bfloat16>(p, st);
  return launch_token<__half>(p, st);
}

}  // namespace lqi
