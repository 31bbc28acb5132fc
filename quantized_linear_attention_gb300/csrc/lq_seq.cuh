// Packed sequences cut into slots, and the elementwise functions of the state space layers (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "lq_device.cuh"
#include "lq_internal.h"
#include "lq_la.cuh"

namespace lqi {

constexpr float kLog2E = 1.44269504088896340736f;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Larger of two; a NaN comes through.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// e^x for x from -128 to 88: 2^h with h = x log2 e as it is rounded, times 1 + c for what that left out, c = x - h ln 2 (Cody
// and Waite's reduction; c is at most 2^-18). So the error hardly grows with x, where that of 2^h alone does (2^-19 at -30,
// 2^-18 at -86): ex2.approx's 2^-22, a rounding, and 0.05 |x| 2^-24 for the constant. Below -87.3 the result is 0.
constexpr float kLn2 = 0.693147180559945309417f;
__device__ __forceinline__ float exp_near(float x) {
  const float h = __fmul_rn(x, kLog2E), e = ex2_approx(h);
  return __fmaf_rn(e, __fmaf_rn(h, -kLn2, x), e);
}
__device__ __forceinline__ f32x2 exp_near2(f32x2 x) {
  const f32x2 h = f2_mul(x, f2_dup(kLog2E)), c = f2_fma(h, f2_dup(-kLn2), x);
  float a, b;
  f2_unpack(h, a, b);
  const f32x2 e = f2_pack(ex2_approx(a), ex2_approx(b));
  return f2_fma(e, c, e);
}

// x / (1 + e^-x); 0 where 1 + e^-x passes 2^126. For fp32 outputs to (9 + 0.05 |x|) 2^-24 of itself (2^-21.3 at most
// measured); for 16-bit ones, whose rounding is 2^-12 or 2^-9, with 2^h alone: to (9 + 1.3 |x|) 2^-24. The single and the
// paired form round alike.
template <typename T>
__device__ __forceinline__ float silu(float x) {
  const float e = sizeof(T) == 4 ? exp_near(fmaxf(fminf(-x, 88.0f), -128.0f)) : ex2_approx(__fmul_rn(x, -kLog2E));
  return __fmul_rn(x, rcp_approx(__fadd_rn(1.0f, e)));
}
template <typename T>
__device__ __forceinline__ f32x2 silu2(f32x2 x) {
  float a, b;
  f32x2 e;
  if (sizeof(T) == 4) {
    f2_unpack(x, a, b);
    e = exp_near2(f2_pack(fmaxf(fminf(-a, 88.0f), -128.0f), fmaxf(fminf(-b, 88.0f), -128.0f)));
  } else {
    f2_unpack(f2_mul(x, f2_dup(-kLog2E)), a, b);
    e = f2_pack(ex2_approx(a), ex2_approx(b));
  }
  f2_unpack(f2_add(e, f2_dup(1.0f)), a, b);
  return f2_mul(x, f2_pack(rcp_approx(a), rcp_approx(b)));
}

// log(1 + e^v) = max(v, 0) + log(1 + e) with e = e^-|v| <= 1, and log(1 + e) = 2 artanh(s) with s = e / (2 + e) <= 1/3: an
// odd function of s, here s times a polynomial of degree 4 in s^2, fitted by exchange to 2e-8 of it (the power series takes
// two terms more). So small steps keep their relative accuracy, as the logarithm of a rounded 1 + e would not: they are
// good to (12 + 0.05 |v|) 2^-24 (2^-21.4 at most measured), for tokens of any type, since states are fp32. (The reduction in
// exp_near costs a scan of 16,384 x 4,096 x 16 in bf16 1.6%.) The single and the paired form round alike.
constexpr float kArtanh8 = 0.296150803565979f, kArtanh6 = 0.27632495760917664f, kArtanh4 = 0.4004742205142975f,
                kArtanh2 = 0.6666590571403503f;
__device__ __forceinline__ float softplus(float v) {
  const float e = exp_near(max_nan(-fabsf(v), -128.0f));  // (a NaN comes through s)
  const float s = __fmul_rn(e, rcp_approx(__fadd_rn(2.0f, e))), q = __fmul_rn(s, s);
  const float r = __fmaf_rn(__fmaf_rn(__fmaf_rn(kArtanh8, q, kArtanh6), q, kArtanh4), q, kArtanh2);
  return __fmaf_rn(__fmaf_rn(r, q, 2.0f), s, fmaxf(v, 0.0f));
}
__device__ __forceinline__ f32x2 softplus2(f32x2 v) {
  float a, b, c, d;
  f2_unpack(v, a, b);
  const f32x2 e = exp_near2(f2_pack(max_nan(-fabsf(a), -128.0f), max_nan(-fabsf(b), -128.0f)));
  f2_unpack(f2_add(e, f2_dup(2.0f)), c, d);
  const f32x2 s = f2_mul(e, f2_pack(rcp_approx(c), rcp_approx(d))), q = f2_mul(s, s);
  const f32x2 r = f2_fma(f2_fma(f2_fma(f2_dup(kArtanh8), q, f2_dup(kArtanh6)), q, f2_dup(kArtanh4)), q, f2_dup(kArtanh2));
  return f2_fma(f2_fma(r, q, f2_dup(2.0f)), s, f2_pack(fmaxf(a, 0.0f), fmaxf(b, 0.0f)));
}

// Copies 16 bytes into shared memory without holding the thread up; the first `bytes` are read, the rest is zero.
__device__ __forceinline__ void copy_ahead(void* to, const void* from, int bytes) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Slot -> piece of a sequence, for a whole CTA of NT threads (all of them come here and get the same). Sequence b has
// max(1, ceil(len / seg)) slots, one after the other (one each where seg is 0); NT sequences are counted at a time.
template <int NT, typename P>
__device__ __forceinline__ Piece find_slot(const P& p, int64_t slot) {
  Piece r;
  r.b = -1;
  r.begin = r.len = r.i = 0;
  r.n = 1;
  if (p.seg == 0 || !p.cu) {
    if (p.seg == 0 ? slot < p.n_seqs : true) {
      int64_t begin, len;
      r.b = p.seg == 0 ? slot : 0;
      bounds(p, r.b, begin, len);
      r.begin = begin;
      r.len = len;
      if (p.seg) {
        r.n = len > p.seg ? (len + p.seg - 1) / p.seg : 1;
        r.i = slot;
        if (slot >= r.n) r.b = -1;
        r.begin = begin + slot * p.seg;
        r.len = min(p.seg, len - slot * p.seg);
      }
    }
    return r;
  }
  constexpr int NW = NT / 32;
  __shared__ int64_t wsum[NW];
  __shared__ Piece found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) found = r;
  int64_t before = 0;
  for (int64_t b0 = 0; b0 < p.n_seqs; b0 += NT) {
    const int64_t b = b0 + tid;
    int64_t begin = 0, len = 0;
    int64_t n = 0;
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
    __syncthreads();
    if (lane == 31) wsum[warp] = sum;
    __syncthreads();
    int64_t mine = before, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) mine += wsum[w];
      total += wsum[w];
    }
    const int64_t i = slot - (mine + sum - n);
    if (n && i >= 0 && i < n) {
      found.b = b;
      found.i = i;
      found.n = n;
      found.begin = begin + i * p.seg;
      found.len = min(p.seg, len - i * p.seg);
    }
    before += total;
    if (before > slot) break;  // (the same for all threads)
  }
  __syncthreads();
  return found;
}

// The first slot of sequence b, counted by a whole CTA of NT threads (all get it).
template <int NT, typename P>
__device__ __forceinline__ int64_t first_slot(const P& p, int64_t b) {
  __shared__ int64_t part[NT / 32];
  int64_t n = 0;
  for (int64_t x = threadIdx.x; x < b; x += NT) {
    int64_t begin, len;
    bounds(p, x, begin, len);
    n += len > p.seg ? (len + p.seg - 1) / p.seg : 1;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) n += part[w];
  return n;
}

}  // namespace lqi
