// Short causal convolution of every channel (sm_103a), over packed prompts and for single tokens:
//   y[t][c] = act(bias[c] + sum_j weight[c][j] x[t - (W-1) + j][c]).
// Bound by memory: 2 (1 + e) bytes in and out and W fmas an element.
#include "lq_seq.cuh"

namespace lqi {

namespace {

constexpr int kNT = 128;

// One thread: a channel's tokens of one tile, the last W - 1 inputs in registers.
template <typename T, int W>
__global__ void __launch_bounds__(kNT) k_conv(ConvParams p, int blocks) {
  const int64_t slot = blockIdx.x / (unsigned)blocks;
  const Piece pc = find_slot<kNT>(p, slot);
  const int c = (int)(blockIdx.x % (unsigned)blocks) * kNT + threadIdx.x;
  if (pc.b < 0 || c >= p.channels) return;
  const int64_t C = p.channels;
  const T* x = static_cast<const T*>(p.x) + c;
  T* y = static_cast<T*>(p.y) + c;
  const T* S0 = p.S0 ? static_cast<const T*>(p.S0) + pc.b * (W - 1) * C + c : nullptr;
  float w[W], in[W];
#pragma unroll
  for (int j = 0; j < W; ++j) w[j] = p.weight[(int64_t)c * W + j];
  const float bias = p.bias ? p.bias[c] : 0.0f;
  const int64_t at = pc.i * p.seg;  // the tile's first token within its sequence
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {  // the inputs before it
    const int64_t t = at - (W - 1) + j;
    in[j] = t >= 0 ? to_f(x[(pc.begin - (W - 1) + j) * p.sx]) : (S0 ? to_f(S0[(t + W - 1) * C]) : 0.0f);
  }
  if (p.S && pc.i == 0) {
    // The sequence's first tile also leaves its last inputs: S may be S0, which no other CTA touches.
    int64_t begin, len;
    bounds(p, pc.b, begin, len);
    T last[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t t = len - (W - 1) + j;
      last[j] = t >= 0 ? x[(begin + t) * p.sx] : (S0 ? S0[(t + W - 1) * C] : from_f<T>(0.0f));
    }
    T* S = static_cast<T*>(p.S) + pc.b * (W - 1) * C + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) S[j * C] = last[j];
  }
  for (int64_t t = pc.begin; t < pc.begin + pc.len; ++t) {
    in[W - 1] = to_f(x[t * p.sx]);
    float s = bias;
#pragma unroll
    for (int j = 0; j < W; ++j) s = __fmaf_rn(w[j], in[j], s);
    y[t * p.sy] = from_f<T>(p.silu ? silu(s) : s);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) in[j] = in[j + 1];
  }
}

template <typename T, int W>
__global__ void __launch_bounds__(kNT) k_conv_step(ConvParams p, int blocks) {
  const int64_t b = blockIdx.x / (unsigned)blocks;
  const int c = (int)(blockIdx.x % (unsigned)blocks) * kNT + threadIdx.x;
  if (c >= p.channels) return;
  const int64_t C = p.channels;
  T* S = static_cast<T*>(p.S) + b * (W - 1) * C + c;
  T in[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) in[j] = S[j * C];
  in[W - 1] = static_cast<const T*>(p.x)[b * p.sx + c];
  float s = p.bias ? p.bias[c] : 0.0f;
#pragma unroll
  for (int j = 0; j < W; ++j) s = __fmaf_rn(p.weight[(int64_t)c * W + j], to_f(in[j]), s);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) S[j * C] = in[j + 1];
  static_cast<T*>(p.y)[b * p.sy + c] = from_f<T>(p.silu ? silu(s) : s);
}

template <typename T>
cudaError_t launch(const ConvParams& p, bool step, cudaStream_t st) {
  const int blocks = (p.channels + kNT - 1) / kNT;
  const unsigned grid = (unsigned)((step ? p.n_seqs : p.slots) * blocks);
  switch (p.width) {
    case 2: step ? k_conv_step<T, 2><<<grid, kNT, 0, st>>>(p, blocks) : k_conv<T, 2><<<grid, kNT, 0, st>>>(p, blocks); break;
    case 3: step ? k_conv_step<T, 3><<<grid, kNT, 0, st>>>(p, blocks) : k_conv<T, 3><<<grid, kNT, 0, st>>>(p, blocks); break;
    default: step ? k_conv_step<T, 4><<<grid, kNT, 0, st>>>(p, blocks) : k_conv<T, 4><<<grid, kNT, 0, st>>>(p, blocks); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_any(const ConvParams& p, bool step, cudaStream_t st) {
  if (p.dtype == LQ_F32) return launch<float>(p, step, st);
  if (p.dtype == LQ_BF16) return launch<__nv_bfloat16>(p, step, st);
  return launch<__half>(p, step, st);
}

}  // namespace

void conv_plan(ConvParams& p) {
  p.seg = 32;
  p.slots = p.n_tokens / p.seg + p.n_seqs;
}

cudaError_t launch_conv_prefill(const ConvParams& p, cudaStream_t st) { return launch_any(p, false, st); }
cudaError_t launch_conv_step(const ConvParams& p, cudaStream_t st) { return launch_any(p, true, st); }

}  // namespace lqi
