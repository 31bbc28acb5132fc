// Short causal convolution of every channel (sm_103a), over packed prompts and for single tokens:
//   y[t][c] = act(bias[c] + sum_j weight[c][j] x[t - (W-1) + j][c]).
// Bound by memory: an element is read and written once, for W fmas and a silu. A thread has V neighbouring channels, 16 bytes
// of a token (one where arrays or strides are not aligned to that), in packed pairs, and their weights in registers.
#include "lq_device.cuh"
#include "lq_seq.cuh"

namespace lqi {

namespace {

constexpr int kNT = 128;

// V neighbouring channels as they lie in memory, and as floats in pairs (the last one's other half is 0 where V is 1).
template <typename T, int V>
struct Raw {
  uint4 v;
};
template <typename T>
struct Raw<T, 1> {
  T v;
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load(const T* p) {
  Raw<T, V> r;
  if constexpr (V == 1) r.v = *p;
  else r.v = *reinterpret_cast<const uint4*>(p);
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const Raw<T, V>& r) {
  if constexpr (V == 1) *p = r.v;
  else *reinterpret_cast<uint4*>(p) = r.v;
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> nothing() {
  Raw<T, V> r;
  if constexpr (V == 1) r.v = from_f<T>(0.0f);
  else r.v = make_uint4(0, 0, 0, 0);
  return r;
}

template <int V>
constexpr int kPairs = (V + 1) / 2;

template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, f32x2 (&f)[kPairs<V>]) {
  if constexpr (V == 1) {
    f[0] = f2_pack(to_f(r.v), 0.0f);
  } else {
    T t[V];
    memcpy(t, &r.v, 16);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[i] = f2_pack(to_f(t[2 * i]), to_f(t[2 * i + 1]));
  }
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> pack(const f32x2 (&f)[kPairs<V>]) {
  Raw<T, V> r;
  T t[2 * kPairs<V>];
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) {
    float a, b;
    f2_unpack(f[i], a, b);
    t[2 * i] = from_f<T>(a);
    t[2 * i + 1] = from_f<T>(b);
  }
  if constexpr (V == 1) r.v = t[0];
  else memcpy(&r.v, t, 16);
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
      if (act) s[i] = silu2(s[i]);
    }
    return pack<T, V>(s);
  }
};

// One thread: V channels' tokens of one tile, the last W - 1 inputs in registers, eight tokens' loads at a time.
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
  Raw<T, V> first[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) first[j] = input(pc.begin - at, at - (W - 1) + j);
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
  const T* from = x + pc.begin * p.sx;
  T* to = static_cast<T*>(p.y) + c + pc.begin * p.sy;
  const int n = (int)pc.len;
  for (int t0 = 0; t0 < n; t0 += U) {
    Raw<T, V> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = t0 + u < n ? load<T, V>(from + u * p.sx) : nothing<T, V>();
    from += U * p.sx;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t0 + u >= n) break;
      unpack<T, V>(r[u], in[W - 1]);
      store<T, V>(to, taps.template out<T>(in, p.silu));
      to += p.sy;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) in[j][i] = in[j + 1][i];
    }
  }
}

// Single tokens: V channels of `seqs` sequences one after the other, two at a time (their weights are read once).
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

template <typename T, int W, int V>
cudaError_t launch_taps(const ConvParams& p, bool step, cudaStream_t st) {
  const int blocks = (p.channels + kNT * V - 1) / (kNT * V);
  if (!step) {
    k_conv<T, W, V><<<(unsigned)(p.slots * blocks), kNT, 0, st>>>(p, blocks);
  } else {
    int seqs = 1;  // one a CTA until they fill the GPU twice over, then up to eight
    while (seqs < 8 && p.n_seqs * blocks >= (int64_t)seqs * 2 * 152 * 4) seqs *= 2;
    k_conv_step<T, W, V><<<(unsigned)((p.n_seqs + seqs - 1) / seqs * blocks), kNT, 0, st>>>(p, blocks, seqs);
  }
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_width(const ConvParams& p, bool step, cudaStream_t st) {
  if (p.width == 2) return launch_taps<T, 2, V>(p, step, st);
  if (p.width == 3) return launch_taps<T, 3, V>(p, step, st);
  return launch_taps<T, 4, V>(p, step, st);
}

int wide(const ConvParams& p) {  // channels of 16 bytes, or 1
  const uint64_t e = p.dtype == LQ_F32 ? 4 : 2;
  const uint64_t at = (uint64_t)p.x | (uint64_t)p.y | (uint64_t)p.S0 | (uint64_t)p.S | (uint64_t)p.weight;
  return (at | (uint64_t)(p.sx | p.sy | p.channels) * e) % 16 == 0 ? (int)(16 / e) : 1;
}

template <typename T>
cudaError_t launch(const ConvParams& p, bool step, cudaStream_t st) {
  return wide(p) > 1 ? launch_width<T, 16 / sizeof(T)>(p, step, st) : launch_width<T, 1>(p, step, st);
}

cudaError_t launch_any(const ConvParams& p, bool step, cudaStream_t st) {
  if (p.dtype == LQ_F32) return launch<float>(p, step, st);
  if (p.dtype == LQ_BF16) return launch<__nv_bfloat16>(p, step, st);
  return launch<__half>(p, step, st);
}

}  // namespace

// Tiles of 64 tokens, or of fewer down to 8 where those would not fill the GPU.
void conv_plan(ConvParams& p) {
  const int64_t blocks = (p.channels + kNT * wide(p) - 1) / (kNT * wide(p));
  p.seg = 64;
  while (p.seg > 8 && p.n_tokens / p.seg * blocks < 152 * 6) p.seg /= 2;
  p.slots = p.n_tokens / p.seg + p.n_seqs;
}

cudaError_t launch_conv_prefill(const ConvParams& p, cudaStream_t st) { return launch_any(p, false, st); }
cudaError_t launch_conv_step(const ConvParams& p, cudaStream_t st) { return launch_any(p, true, st); }

}  // namespace lqi
