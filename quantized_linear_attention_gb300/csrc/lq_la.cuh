// What the kernels of linear attention with a decay per head share (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lq_internal.h"

namespace lqi {

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// One rounding, to nearest even, of an fp32 sum to the type of the tokens.
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

// Four consecutive channels as floats.
__device__ __forceinline__ void ld4(const float* p, float d[4]) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  d[0] = x.x, d[1] = x.y, d[2] = x.z, d[3] = x.w;
}
template <typename T>
__device__ __forceinline__ void ld4(const T* p, float d[4]) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  T t[4];
  static_assert(sizeof(T) == 2, "16-bit tokens");
  memcpy(t, &x, 8);
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = to_f(t[e]);
}

// The bounds of sequence b; one whose bounds are not 0 <= begin <= end <= n_tokens,
// or that is longer than a stated max_len, counts as empty.
template <typename P>
__device__ __forceinline__ void bounds(const P& p, int64_t b, int64_t& begin, int64_t& len) {
  begin = 0;
  int64_t end = p.n_tokens;
  if (p.cu) {
    begin = p.cu[b];
    end = p.cu[b + 1];
  }
  len = end - begin;
  if (begin < 0 || end > p.n_tokens || len < 0 || (p.max_len > 0 && len > p.max_len)) begin = len = 0;
}

// The part of a sequence that a CTA takes.
struct Piece {
  int64_t b;      // sequence (-1: none)
  int64_t begin;  // first token
  int64_t len;
  int64_t i, n;   // segment i of the sequence's n
};

// Slot -> segment. Sequence b has max(1, ceil(len / seg)) slots, one after the
// other; a warp counts them 32 sequences at a time. All lanes get the result.
__device__ __forceinline__ Piece find_piece(const LaParams& p, int64_t slot) {
  Piece r;
  r.b = -1;
  r.begin = r.len = r.i = 0;
  r.n = 1;
  if (p.seg == 0) {
    r.b = slot;
    bounds(p, slot, r.begin, r.len);
    return r;
  }
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int64_t b0 = 0; b0 < p.n_seqs; b0 += 32) {
    const int64_t b = b0 + lane;
    int64_t begin = 0, len = 0, n = 0;
    if (b < p.n_seqs) {
      bounds(p, b, begin, len);
      n = len > p.seg ? (len + p.seg - 1) / p.seg : 1;
    }
    int64_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, slot < before + sum);
    if (hit) {
      const int l = __ffs((int)hit) - 1;
      const int64_t i = slot - before - (sum - n);
      r.b = b0 + l;
      r.i = __shfl_sync(0xffffffffu, i, l);
      r.n = __shfl_sync(0xffffffffu, n, l);
      r.begin = __shfl_sync(0xffffffffu, begin, l) + r.i * p.seg;
      const int64_t left = __shfl_sync(0xffffffffu, len, l) - r.i * p.seg;
      r.len = left < p.seg ? left : p.seg;
      return r;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return r;
}

// A product of two numbers in two parts each (high + low), to about 2^-45.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  const float p = __fmul_rn(a.x, b.x);
  const float e = __fmaf_rn(a.y, b.x, __fmaf_rn(a.x, b.y, __fmaf_rn(a.x, b.x, -p)));
  const float h = __fadd_rn(p, e);
  return make_float2(h, __fsub_rn(e, __fsub_rn(h, p)));
}

__device__ __forceinline__ float2 in_two(double x) {
  const float hi = (float)x;
  return make_float2(hi, (float)(x - (double)hi));
}

// The state before a piece: S0 (NULL: zero), or where a sequence is split what k_la_scan left in the piece's slot.
__device__ __forceinline__ const float* start_state(const LaParams& p, const Piece& pc, int64_t slot, int h) {
  if (pc.n > 1) return p.ws_state + (slot * p.heads + h) * (kD * kD);
  return p.S0 ? p.S0 + (pc.b * p.heads + h) * (kD * kD) : nullptr;
}

// Split sequences in which a state between the segments is not finite: where a segment's decays multiply to infinity (a
// zero state stays zero under them) or a state is infinite (under the second part of a product it is NaN), the sum over
// segments is not the recurrence any more. k_la_scan notes them, and the second pass takes such a sequence's head token by
// token in its first segment's CTA. The note is where the last segment's product would be, which nothing needs; slots
// past the workspace (sequences that overlap, against the rules) have none.
__device__ __forceinline__ float2* serial_note(const LaParams& p, const Piece& pc, int64_t slot, int h) {
  const int64_t last = slot - pc.i + pc.n - 1;
  return pc.n > 1 && last < p.slots ? p.ws_decay + last * p.heads + h : nullptr;
}

// A piece again token by token, exactly as the recurrence is written: the first NT threads of the CTA (all of it come here), four
// lanes to a row, 32 columns each, TOK tokens staged at a time in sm, (3 kD + 1) TOK floats. `from` NULL: from zero.
// OUT: with outputs. decay, if not NULL, gets the product of the decays. For pieces in which a faster form's own
// intermediate values have left fp32's range, or may have: 0.8 to 0.9 us a token (20,000 tokens of one head: 16 ms bf16,
// 18 ms fp32), bound by a token's latency through shared memory and two barriers for each TOK.
template <typename T, bool OUT, int NT, int TOK>
__device__ __noinline__ void redo(const LaParams& p, int64_t begin, int64_t len, int h, const float* from, float* sm,
                                  float* S_out, float2* decay) {
  const int tid = threadIdx.x, part = tid & 3, kh = h / p.group;
  float(*sk)[kD] = reinterpret_cast<float(*)[kD]>(sm);
  float(*sq)[kD] = sk + TOK;
  float(*sv)[kD] = sq + TOK;
  float* sa = reinterpret_cast<float*>(sv + TOK);
  const T* q = static_cast<const T*>(p.q) + kh * kD;
  const T* k = static_cast<const T*>(p.k) + kh * kD;
  const T* v = static_cast<const T*>(p.v) + h * kD;
  T* o = static_cast<T*>(p.o) + h * kD;
  double prod = 1.0;
  for (int row = tid >> 2; row < kD + (tid >> 2); row += NT / 4) {  // (as many rounds for every thread)
    float S[8][4];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      S[c][0] = S[c][1] = S[c][2] = S[c][3] = 0.f;
      if (from && tid < NT) ld4(from + row * kD + 4 * (4 * c + part), S[c]);
    }
    prod = 1.0;
    for (int64_t t0 = 0; t0 < len; t0 += TOK) {
      const int n = (int)min((int64_t)TOK, len - t0);
      __syncthreads();
      for (int x = tid; x < 32 * n; x += NT) {
        if (tid >= NT) break;
        const int t = x >> 5, c = 4 * (x & 31);
        const int64_t at = begin + t0 + t;
        ld4(k + at * p.sk + c, &sk[t][c]);
        if (OUT) ld4(q + at * p.sq + c, &sq[t][c]);
        ld4(v + at * p.sv + c, &sv[t][c]);
        if (c == 0) sa[t] = p.alpha[at * p.sa + h];
      }
      __syncthreads();
      if (tid < NT) {
        for (int t = 0; t < n; ++t) {
          const float a = sa[t], vv = sv[t][row];
          prod *= (double)a;
          float acc = 0.f;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float kk[4], qq[4] = {0.f, 0.f, 0.f, 0.f};
            ld4(&sk[t][4 * (4 * c + part)], kk);
            if (OUT) ld4(&sq[t][4 * (4 * c + part)], qq);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              S[c][e] = __fmaf_rn(vv, kk[e], __fmul_rn(a, S[c][e]));
              if (OUT) acc = __fmaf_rn(S[c][e], qq[e], acc);
            }
          }
          if (OUT) {
            acc += __shfl_xor_sync(0xffffffffu, acc, 1);
            acc += __shfl_xor_sync(0xffffffffu, acc, 2);
            if (part == 0) o[(begin + t0 + t) * p.so + row] = from_f<T>(acc);
          }
        }
      }
    }
    if (S_out && tid < NT) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<float4*>(S_out + row * kD + 4 * (4 * c + part)) =
            make_float4(S[c][0], S[c][1], S[c][2], S[c][3]);
    }
  }
  if (decay && tid == 0) *decay = in_two(prod);
}

cudaError_t launch_la_chunk_bf16(const LaParams& p, cudaStream_t st);

// The kernels of a split prompt are launched one upon the other: a kernel is set up while the one before still
// runs (each lets its successor in as soon as all its CTAs have begun) and waits for that one's end
// (cudaGridDependencySynchronize) before it reads what it left.
template <typename... A>
inline cudaError_t launch_upon(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Split sequences: the states before the segments, from what the first pass left in the workspace.
cudaError_t launch_la_scan(const LaParams& p, cudaStream_t st);
// Split sequences whose last states replace S0: other segments may not have read it yet, so the second pass leaves
// them in the workspace and launch_la_unstage copies them.
inline bool la_staged(const LaParams& p) { return p.seg && p.S && p.S == p.S0; }
cudaError_t launch_la_unstage(const LaParams& p, cudaStream_t st);

}  // namespace lqi
