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
__device__ __forceinline__ void bounds(const LaParams& p, int64_t b, int64_t& begin, int64_t& len) {
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
