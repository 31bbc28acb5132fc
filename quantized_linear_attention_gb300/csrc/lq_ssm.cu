// Selective state space scan (sm_103a): how prompts are divided, and the kernel for single tokens.
#include "lq_ssm.cuh"

namespace lqi {

namespace {

// --------------------------------------------------------------------------------------------
// Single tokens.
// Bound by memory: a state is read and written, 8 bytes for about six operations. A lane holds four neighbouring states of a
// channel (V4: by 16 bytes), LPC lanes a channel; a CTA takes one block of channels and K sequences after K others, whose
// loads are all begun before the first is used, so that A is read once for all of them. (512 sequences x 4,096 channels of 16
// states, bf16, three batches of states in turn: 63 us with K = 2 and 32 warps an SM, 67% of the copy bandwidth; 66 with 3, 70 with
// 1 and 48 warps, 77 with 4 and 24 warps; 71 with loads and stores marked as streaming.)
template <typename T, int LPC, bool V4, int K>
__device__ __forceinline__ void tokens(const SsmParams& p, int64_t b, int c, int g, bool live, const float (&A)[4],
                                       float bias, float D) {
  const int part = threadIdx.x % LPC, n0 = 4 * part;
  const int64_t row = (int64_t)p.channels * p.n_state;
  float* const S = p.S + b * row + (int64_t)c * p.n_state + n0;
  const T* const Bp = static_cast<const T*>(p.B) + b * p.sb + (int64_t)g * p.n_state + n0;
  const T* const Cp = static_cast<const T*>(p.C) + b * p.sc + (int64_t)g * p.n_state + n0;
  const bool in = n0 < p.n_state;
  float h[K][4], B[K][4], C[K][4];
  T dt[K], x[K], z[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    dt[k] = static_cast<const T*>(p.dt)[(b + k) * p.sdt + c];
    x[k] = static_cast<const T*>(p.x)[(b + k) * p.sx + c];
    z[k] = p.z ? static_cast<const T*>(p.z)[(b + k) * p.sz + c] : x[k];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[k][e] = B[k][e] = C[k][e] = 0.0f;
    if (V4) {
      if (in) {
        const float4 v = *reinterpret_cast<const float4*>(S + k * row);
        h[k][0] = v.x, h[k][1] = v.y, h[k][2] = v.z, h[k][3] = v.w;
        ld4(Bp + k * p.sb, B[k]);
        ld4(Cp + k * p.sc, C[k]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (n0 + e < p.n_state) {
          h[k][e] = S[k * row + e];
          B[k][e] = to_f(Bp[k * p.sb + e]);
          C[k][e] = to_f(Cp[k * p.sc + e]);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float d = p.softplus ? step_of<T, true>(dt[k], bias) : step_of<T, false>(dt[k], bias);
    const float xv = to_f(x[k]), dx = __fmul_rn(d, xv);
    float y = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[k][e] = __fmaf_rn(ex2_approx(__fmul_rn(d, A[e])), h[k][e], __fmul_rn(dx, B[k][e]));
      y = __fmaf_rn(C[k][e], h[k][e], y);
    }
    if (V4 && in && live) {
      *reinterpret_cast<float4*>(S + k * row) = make_float4(h[k][0], h[k][1], h[k][2], h[k][3]);
    } else if (!V4 && live) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n0 + e < p.n_state) S[k * row + e] = h[k][e];
    }
#pragma unroll
    for (int s = 1; s < LPC; s <<= 1) y = __fadd_rn(y, __shfl_xor_sync(0xffffffffu, y, s));
    if (p.D) y = __fmaf_rn(D, xv, y);
    if (p.z) y = __fmul_rn(y, silu<T>(to_f(z[k])));
    if (part == 0 && live) static_cast<T*>(p.y)[(b + k) * p.sy + c] = from_f<T>(y);
  }
}

// Neighbouring lanes hold neighbouring parts of a channel, so that eight lanes' states are 128 bytes in a row.
template <typename T, int LPC, bool V4>
__global__ void __launch_bounds__(kNT, 8) k_ssm_step(SsmParams p, int blocks, int seqs) {
  constexpr int K = 2;
  const int part = threadIdx.x % LPC;
  const int at = (int)(blockIdx.x % (unsigned)blocks) * (kNT / LPC) + threadIdx.x / LPC;
  const bool live = at < p.channels;
  const int c = live ? at : 0;
  float A[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int n = 4 * part + e;
    A[e] = n < p.n_state ? __fmul_rn(p.A[(int64_t)c * p.n_state + n], kLog2E) : 0.0f;
  }
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, D = p.D ? p.D[c] : 0.0f;
  const int g = c / p.per_group;
  int64_t b = (int64_t)(blockIdx.x / (unsigned)blocks) * seqs;
  const int64_t end = min(b + seqs, p.n_seqs);
  for (; b + K <= end; b += K) tokens<T, LPC, V4, K>(p, b, c, g, live, A, bias, D);
  for (; b < end; ++b) tokens<T, LPC, V4, 1>(p, b, c, g, live, A, bias, D);
}

template <typename T, int LPC, bool V4>
cudaError_t launch_lanes(const SsmParams& p, cudaStream_t st) {
  const int blocks = (int)(((int64_t)p.channels * LPC + kNT - 1) / kNT);
  // one sequence a CTA until they fill the GPU twice over, then up to eight
  int seqs = 1;
  while (seqs < 8 && p.n_seqs * blocks >= (int64_t)seqs * 2 * 152 * 16) seqs *= 2;
  const unsigned grid = (unsigned)((p.n_seqs + seqs - 1) / seqs * blocks);
  k_ssm_step<T, LPC, V4><<<grid, kNT, 0, st>>>(p, blocks, seqs);
  return cudaGetLastError();
}

template <typename T, bool V4>
cudaError_t launch_step(const SsmParams& p, cudaStream_t st) {
  if (p.n_state <= 4) return launch_lanes<T, 1, V4>(p, st);
  if (p.n_state <= 8) return launch_lanes<T, 2, V4>(p, st);
  if (p.n_state <= 16) return launch_lanes<T, 4, V4>(p, st);
  if (p.n_state <= 32) return launch_lanes<T, 8, V4>(p, st);
  return launch_lanes<T, 16, V4>(p, st);
}

template <typename T>
cudaError_t launch_token(const SsmParams& p, cudaStream_t st) {
  const uint64_t four = (uint64_t)p.B | (uint64_t)p.C | (uint64_t)(p.sb | p.sc) * sizeof(T);
  const bool v4 = p.n_state % 4 == 0 && (uint64_t)p.S % 16 == 0 && four % (4 * sizeof(T)) == 0;
  return v4 ? launch_step<T, true>(p, st) : launch_step<T, false>(p, st);
}

// --------------------------------------------------------------------------------------------
// Prompts: how many states a thread holds, and whether sequences are split.
struct Shape {
  int spt, lpc;  // states a thread, lanes a channel
};

// What a token costs: ns of an SM with nothing else to do, and ns each of many CTAs on it. Measured with 8 to 64 states, bf16 and
// fp32: 106 to 136 and 98 to 110 with 16 states a thread, 97 to 112 and 50 to 63 with 8 (eight lanes a channel: 69 and 56),
// 50 to 71 and 33 to 36 with 4 (eight lanes: 61 to 63 alone, 78 and 94 where some SMs have two CTAs).
struct Cost {
  double alone, many;
};
Cost cost_of(Shape s) {
  if (s.spt == 16) return {125, 99};
  if (s.spt == 8) return {s.lpc == 8 ? 72.0 : 102.0, 54};
  return {s.lpc == 4 ? 52.0 : s.lpc == 8 ? 70.0 : 65.0, 34};
}

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
// longest one alone or as all tokens of all CTAs together, and some of the other as well; split ones two segments one after
// the other and most of 1.55 times all tokens (the first pass has no outputs), and 16 us for two more launches. Measured against the other
// choices: one sequence of 16,384 tokens x 4,096 channels of 16 states 496 us split with 16 states a thread, 833 whole with
// four; 16 ragged ones of up to 1,500 150 and 131; one of 300 x 2,048 channels 33 and 19.
void ssm_plan(const lq_ssm_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len, SsmPlan* plan) {
  const int64_t longest = max_len > 0 && max_len < n_tokens ? max_len : n_tokens;
  double best = 0;
  for (int spt = most_states(c->n_state); spt >= 4; spt /= 2) {
    const Shape s = {spt, padded(c->n_state) / spt};
    if (s.lpc > 8) break;
    const Cost cost = cost_of(s);
    const int64_t blocks = blocks_of(c, s), seg = segment(n_tokens, ctas_of(s), blocks);
    const double alone = cost.alone * (double)longest, all = cost.many * (double)n_tokens * (double)blocks / kSms;
    const double whole = (alone > all ? alone + 0.3 * all : all + 0.3 * alone) + 3000;
    if (best == 0 || whole < best) {
      best = whole;
      *plan = {s.spt, s.lpc, 0, n_seqs, blocks};
    }
    if (longest < 3 * seg) continue;
    const double two = 2 * cost.alone * (double)seg, both = 1.55 * all;
    const double split = two + 0.6 * both + 16000 + 60.0 * (double)(longest / seg);
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
