// Short causal convolution of every channel (sm_103a), over packed prompts and for single tokens:
//   y[t][c] = act(bias[c] + sum_j weight[c][j] x[t - (W-1) + j][c]).
// Bound by memory: an element is read and written once, for W fmas and a silu. A thread has V neighbouring channels, 8 bytes
// of a prompt's token or 16 of a single one (one channel where arrays or strides are not aligned to 16 bytes), in packed pairs,
// and their weights in registers.
#include <type_traits>

#include "lq_device.cuh"
#include "lq_seq.cuh"

namespace lqi {

namespace {

constexpr int kNT = 128;

// V neighbouring channels as they lie in memory (one, or 8 or 16 bytes of them, kept as words), and as floats in pairs (where V
// is 1 the other half of the only pair is 0).
template <typename T, int V>
struct Raw {
  using Word = typename std::conditional<V == 1, T, typename std::conditional<V * sizeof(T) == 16, uint4, uint2>::type>::type;
  Word v;
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load(const T* p) {
  return {*reinterpret_cast<const typename Raw<T, V>::Word*>(p)};
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const Raw<T, V>& r) {
  *reinterpret_cast<typename Raw<T, V>::Word*>(p) = r.v;
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> nothing() {
  Raw<T, V> r;
  memset(&r, 0, sizeof r);
  return r;
}

template <int V>
constexpr int kPairs = (V + 1) / 2;

template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, f32x2 (&f)[kPairs<V>]) {
  T t[V];
  memcpy(t, &r, sizeof t);
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) f[i] = f2_pack(to_f(t[2 * i]), 2 * i + 1 < V ? to_f(t[(2 * i + 1) % V]) : 0.0f);
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> pack(const f32x2 (&f)[kPairs<V>]) {
  T t[V];
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) {
    float a, b;
    f2_unpack(f[i], a, b);
    t[2 * i] = from_f<T>(a);
    if (2 * i + 1 < V) t[(2 * i + 1) % V] = from_f<T>(b);
  }
  Raw<T, V> r;
  memcpy(&r, t, sizeof t);
  return r;
}

// A thread's weights, by tap, and bias.
template <int W, int V>
struct Taps {
  f32x2 w[W][kPairs<V>], bias[kPairs<V>];
  __device__ __forceinline__ void read(const ConvParams& p, int c) {
    float a[2 * kPairs<V>][W] = {}, b[2 * kPairs<V>] = {};
    const float* const src = p.weight + (int64_t)c * W;
    if (V > 1 && W == 4) {  // (aligned to 16 bytes: the rule for V)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(src) + i);
        a[i][0] = q.x, a[i][1 % W] = q.y, a[i][2 % W] = q.z, a[i][3 % W] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) a[i][j] = src[i * W + j];
    }
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = p.bias[c + i];
    }
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
      bias[i] = f2_pack(b[2 * i], b[2 * i + 1]);
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = f2_pack(a[2 * i][j], a[2 * i + 1][j]);
    }
  }
  // The output of the inputs in[0] (oldest) .. in[W - 1].
  template <typename T>
  __device__ __forceinline__ Raw<T, V> out(const f32x2 (&in)[W][kPairs<V>], int act) const {
    f32x2 s[kPairs<V>];
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
      s[i] = bias[i];
#pragma unroll
      for (int j = 0; j < W; ++j) s[i] = f2_fma(w[j][i], in[j][i], s[i]);
      if (act) s[i] = silu2<T>(s[i]);
    }
    return pack<T, V>(s);
  }
};

// One thread: V channels' tokens of one tile, the last W - 1 inputs in registers, the next eight tokens on
// their way.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kNT) k_conv(ConvParams p, int blocks) {
  constexpr int U = 8, P = kPairs<V>;
  const int64_t slot = blockIdx.x / (unsigned)blocks;
  const Piece pc = find_slot<kNT>(p, slot);
  const int c = ((int)(blockIdx.x % (unsigned)blocks) * kNT + threadIdx.x) * V;
  if (pc.b < 0 || c >= p.channels) return;
  const int64_t C = p.channels;
  const T* const x = static_cast<const T*>(p.x) + c;
  const T* const S0 = p.S0 ? static_cast<const T*>(p.S0) + pc.b * (W - 1) * C + c : nullptr;
  const int64_t at = pc.i * p.seg;  // the tile's first token within its sequence
  // input t of the sequence, from -(W - 1) on
  auto input = [&](int64_t begin, int64_t t) {
    if (t >= 0) return load<T, V>(x + (begin + t) * p.sx);
    return S0 ? load<T, V>(S0 + (t + W - 1) * C) : nothing<T, V>();
  };
  const int n = (int)pc.len;
  const T* from = x + pc.begin * p.sx;
  T* to = static_cast<T*>(p.y) + c + pc.begin * p.sy;
  Raw<T, V> first[W - 1], r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) r[u] = u < n ? load<T, V>(from + u * p.sx) : nothing<T, V>();
#pragma unroll
  for (int j = 0; j < W - 1; ++j) first[j] = input(pc.begin - at, at - (W - 1) + j);
  from += U * p.sx;
  Taps<W, V> taps;
  taps.read(p, c);
  if (p.S && pc.i == 0) {
    // The sequence's first tile also leaves its last inputs: S may be S0, which no other CTA touches.
    int64_t begin, len;
    bounds(p, pc.b, begin, len);
    Raw<T, V> last[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) last[j] = input(begin, len - (W - 1) + j);
    T* const S = static_cast<T*>(p.S) + pc.b * (W - 1) * C + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store<T, V>(S + j * C, last[j]);
  }
  f32x2 in[W][P];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) unpack<T, V>(first[j], in[j]);
  for (int t0 = 0; t0 < n; t0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t0 + u >= n) break;
      unpack<T, V>(r[u], in[W - 1]);
      if (t0 + u + U < n) r[u] = load<T, V>(from);
      from += p.sx;
      store<T, V>(to, taps.template out<T>(in, p.silu));
      to += p.sy;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) in[j][i] = in[j + 1][i];
    }
  }
}

// Single tokens: V channels of `seqs` sequences one after the other, two at a time (their weights are read once). 512 sequences x
// 8,192 channels, bf16: 13 us out of L2 (67 MB, three quarters of the copy bandwidth's rate), 16.5 with states in turn.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kNT) k_conv_step(ConvParams p, int blocks, int seqs) {
  constexpr int P = kPairs<V>, K = 2;
  const int c = ((int)(blockIdx.x % (unsigned)blocks) * kNT + threadIdx.x) * V;
  if (c >= p.channels) return;
  const int64_t C = p.channels, b0 = (int64_t)(blockIdx.x / (unsigned)blocks) * seqs, end = min(b0 + seqs, p.n_seqs);
  Taps<W, V> taps;
  taps.read(p, c);
  for (int64_t b = b0; b < end; b += K) {
    Raw<T, V> r[K][W];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (b + k >= end) break;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) r[k][j] = load<T, V>(static_cast<const T*>(p.S) + ((b + k) * (W - 1) + j) * C + c);
      r[k][W - 1] = load<T, V>(static_cast<const T*>(p.x) + (b + k) * p.sx + c);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (b + k >= end) break;
      f32x2 in[W][P];
#pragma unroll
      for (int j = 0; j < W; ++j) unpack<T, V>(r[k][j], in[j]);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) store<T, V>(static_cast<T*>(p.S) + ((b + k) * (W - 1) + j) * C + c, r[k][j + 1]);
      store<T, V>(static_cast<T*>(p.y) + (b + k) * p.sy + c, taps.template out<T>(in, p.silu));
    }
  }
}

// Bytes of a token that a thread of a prompt has: 16 take 128 registers and more, which leaves 12 warps an SM (4,132 tokens of
// 16 sequences x 8,192 channels, bf16: 29.9 us, 68% of the copy bandwidth; 33.0 with 16 bytes).
constexpr int kPrompt = 8;

template <typename T, int W, int V>
cudaError_t launch_prompts(const ConvParams& p, cudaStream_t st) {
  const int blocks = (p.channels + kNT * V - 1) / (kNT * V);
  k_conv<T, W, V><<<(unsigned)(p.slots * blocks), kNT, 0, st>>>(p, blocks);
  return cudaGetLastError();
}

template <typename T, int W, int V>
cudaError_t launch_tokens(const ConvParams& p, cudaStream_t st) {
  const int blocks = (p.channels + kNT * V - 1) / (kNT * V);
  int seqs = 1;  // one a CTA until they fill the GPU twice over, then up to eight
  while (seqs < 8 && p.n_seqs * blocks >= (int64_t)seqs * 2 * 152 * 4) seqs *= 2;
  k_conv_step<T, W, V><<<(unsigned)((p.n_seqs + seqs - 1) / seqs * blocks), kNT, 0, st>>>(p, blocks, seqs);
  return cudaGetLastError();
}

template <typename T, int W>
cudaError_t launch_width(const ConvParams& p, bool step, bool vec, cudaStream_t st) {
  if (step) return vec ? launch_tokens<T, W, 16 / (int)sizeof(T)>(p, st) : launch_tokens<T, W, 1>(p, st);
  return vec ? launch_prompts<T, W, kPrompt / (int)sizeof(T)>(p, st) : launch_prompts<T, W, 1>(p, st);
}

int wide(const ConvParams& p) {  // channels of 16 bytes, or 1
  const uint64_t e = p.dtype == LQ_F32 ? 4 : 2;
  const uint64_t at = (uint64_t)p.x | (uint64_t)p.y | (uint64_t)p.S0 | (uint64_t)p.S | (uint64_t)p.weight;
  return (at | (uint64_t)(p.sx | p.sy | p.channels) * e) % 16 == 0 ? (int)(16 / e) : 1;
}

template <typename T>
cudaError_t launch(const ConvParams& p, bool step, cudaStream_t st) {
  const bool vec = wide(p) > 1;
  if (p.width == 2) return launch_width<T, 2>(p, step, vec, st);
  if (p.width == 3) return launch_width<T, 3>(p, step, vec, st);
  return launch_width<T, 4>(p, step, vec, st);
}

cudaError_t launch_any(const ConvParams& p, bool step, cudaStream_t st) {
  if (p.dtype == LQ_F32) return launch<float>(p, step, st);
  if (p.dtype == LQ_BF16) return launch<__nv_bfloat16>(p, step, st);
  return launch<__half>(p, step, st);
}

}  // namespace

// Tiles of 64 tokens, or of fewer down to 8 where those would not fill the GPU.
void conv_plan(ConvParams& p) {
  const int v = wide(p) > 1 ? wide(p) * kPrompt / 16 : 1;
  const int64_t blocks = (p.channels + kNT * v - 1) / (kNT * v);
  p.seg = 64;
  while (p.seg > 8 && p.n_tokens / p.seg * blocks < 152 * 12) p.seg /= 2;
  p.slots = p.n_tokens / p.seg + p.n_seqs;
}

cudaError_t launch_conv_prefill(const ConvParams& p, cudaStream_t st) { return launch_any(p, false, st); }
cudaError_t launch_conv_step(const ConvParams& p, cudaStream_t st) { return launch_any(p, true, st); }

}  // namespace lqi
