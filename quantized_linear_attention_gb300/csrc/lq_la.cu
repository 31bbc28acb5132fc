// Linear attention with a decay for each head (sm_103a):
//   S_t = alpha_t S_{t-1} + v_t k_t^T,   o_t = S_t q_t
// on fp32 states of 128 x 128, over prompts and for single tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lq_internal.h"
#include "lq_la.cuh"

namespace lqi {

namespace {

// --------------------------------------------------------------------------------------------
// Prompts, token by token: one CTA of 128 threads per (sequence, head, 32 value
// rows); four lanes hold a row, 32 columns each (float4 groups p, p + 4, ... so
// that the four lanes read 64 consecutive bytes of a staged key).
constexpr int kRecTok = 16;  // tokens staged at a time

template <typename T>
__global__ void __launch_bounds__(128) k_la_recurrent(LaParams p) {
  __shared__ __align__(16) float sk[kRecTok][kD], sq[kRecTok][kD];
  __shared__ float sv[kRecTok][32], sa[kRecTok];
  const int tid = threadIdx.x, part = tid & 3, row = tid >> 2;
  const int slab = blockIdx.x & 3, h = (blockIdx.x >> 2) % p.heads, kh = h / p.group;
  const int64_t b = (blockIdx.x >> 2) / p.heads;
  int64_t begin, len;
  bounds(p, b, begin, len);
  const T* q = static_cast<const T*>(p.q) + kh * kD;
  const T* k = static_cast<const T*>(p.k) + kh * kD;
  const T* v = static_cast<const T*>(p.v) + h * kD + slab * 32;
  T* o = static_cast<T*>(p.o) + h * kD + slab * 32;
  const int64_t sbase = ((b * p.heads + h) * kD + slab * 32 + row) * kD;
  float S[8][4];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    if (p.S0) ld4(p.S0 + sbase + 4 * (4 * c + part), S[c]);
    else S[c][0] = S[c][1] = S[c][2] = S[c][3] = 0.f;
  }
  for (int64_t t0 = 0; t0 < len; t0 += kRecTok) {
    const int n = (int)min((int64_t)kRecTok, len - t0);
    __syncthreads();
    for (int e = tid; e < n * 32; e += 128) {
      const int t = e >> 5, c = 4 * (e & 31);
      const int64_t at = begin + t0 + t;
      ld4(k + at * p.sk + c, &sk[t][c]);
      ld4(q + at * p.sq + c, &sq[t][c]);
      sv[t][e & 31] = to_f(v[at * p.sv + (e & 31)]);
    }
    if (tid < n) sa[tid] = p.alpha[(begin + t0 + tid) * p.sa + h];
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float a = sa[t], vv = sv[t][row];
      float acc = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float kk[4], qq[4];
        ld4(&sk[t][4 * (4 * c + part)], kk);
        ld4(&sq[t][4 * (4 * c + part)], qq);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          S[c][e] = __fmaf_rn(vv, kk[e], __fmul_rn(a, S[c][e]));
          acc = __fmaf_rn(S[c][e], qq[e], acc);
        }
      }
      acc += __shfl_xor_sync(0xffffffffu, acc, 1);
      acc += __shfl_xor_sync(0xffffffffu, acc, 2);
      if (part == 0) o[(begin + t0 + t) * p.so + row] = from_f<T>(acc);
    }
  }
  if (p.S) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<float4*>(p.S + sbase + 4 * (4 * c + part)) = make_float4(S[c][0], S[c][1], S[c][2], S[c][3]);
  }
}

// --------------------------------------------------------------------------------------------
// One token for each sequence: every state is read once and written once, 131,072
// of the 132 KB a head-state takes, so HBM bounds it. 256 threads; eight lanes hold
// a row, 16 columns each (a warp instruction reads four rows x 128 consecutive
// bytes); keys and queries come straight from global memory, each lane its own 16
// channels, so nothing waits on a barrier. P CTAs share a head-state.
template <typename T, int P>
__global__ void __launch_bounds__(256) k_la_step(LaParams p) {
  constexpr int NR = 4 / P;  // row groups of a thread
  const int tid = threadIdx.x, w = tid >> 5, r = (tid & 31) >> 3, qq = tid & 7;
  const int64_t s = blockIdx.x / P;
  const int row0 = (int)(blockIdx.x % P) * (kD / P) + 4 * w + r;
  const int h = (int)(s % p.heads), kh = h / p.group;
  const int64_t b = s / p.heads;
  float* S = p.S + (s * kD + row0) * kD + 4 * qq;
  float4 x[NR][4];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) x[i][c] = __ldcs(reinterpret_cast<const float4*>(S + i * 32 * kD + 32 * c));
  float kk[4][4], qv[4][4];
  const T* k = static_cast<const T*>(p.k) + b * p.sk + kh * kD + 4 * qq;
  const T* q = static_cast<const T*>(p.q) + b * p.sq + kh * kD + 4 * qq;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    ld4(k + 32 * c, kk[c]);
    ld4(q + 32 * c, qv[c]);
  }
  const float a = p.alpha[b * p.sa + h];
  const T* v = static_cast<const T*>(p.v) + b * p.sv + h * kD + row0;
  T* o = static_cast<T*>(p.o) + b * p.so + h * kD + row0;
  float vv[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) vv[i] = to_f(v[32 * i]);
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    float acc = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float y[4] = {x[i][c].x, x[i][c].y, x[i][c].z, x[i][c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] = __fmaf_rn(vv[i], kk[c][e], __fmul_rn(a, y[e]));
        acc = __fmaf_rn(y[e], qv[c][e], acc);
      }
      __stcs(reinterpret_cast<float4*>(S + i * 32 * kD + 32 * c), make_float4(y[0], y[1], y[2], y[3]));
    }
    acc += __shfl_xor_sync(0xffffffffu, acc, 1);
    acc += __shfl_xor_sync(0xffffffffu, acc, 2);
    acc += __shfl_xor_sync(0xffffffffu, acc, 4);
    if (qq == 0) o[32 * i] = from_f<T>(acc);
  }
}

template <typename T>
cudaError_t prefill(const LaParams& p, cudaStream_t st) {
  k_la_recurrent<T><<<(unsigned)(p.n_seqs * p.heads * 4), 128, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t step(const LaParams& p, cudaStream_t st) {
  const int64_t n = p.n_seqs * p.heads;
  // Few head-states: four CTAs share one, so that the loads spread over the SMs.
  if (n < 2 * 152) k_la_step<T, 4><<<(unsigned)(4 * n), 256, 0, st>>>(p);
  else k_la_step<T, 1><<<(unsigned)n, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

void la_plan(const lq_la_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len, int64_t* seg, int64_t* slots) {
  *seg = *slots = 0;
  if (c->dtype != LQ_BF16) return;
  const int64_t longest = max_len > 0 && max_len < n_tokens ? max_len : n_tokens;
  const int64_t share = n_tokens * c->heads / 152;  // head-tokens of an SM
  // Splitting reads k and v twice (1.5 times the bytes), so it pays where the longest
  // sequence alone takes longer than that: 1.6 shares.
  if (5 * longest <= 8 * share || longest <= 1024) return;
  // Two rounds of CTAs, less the last piece of each head, which is shorter: a piece costs about as much again as
  // six chunks (32,768 tokens x 32 heads: four rounds 437 us, three 417, two 381).
  const int64_t pieces = c->heads < 152 ? 304 - c->heads : 152;
  *seg = (n_tokens * c->heads / pieces + 127) / 128 * 128;
  if (*seg < 512) *seg = 512;
  *slots = n_tokens / *seg + n_seqs;
}

cudaError_t launch_la_prefill(const LaParams& p, cudaStream_t st) {
  if (p.dtype == LQ_BF16) return launch_la_chunk_bf16(p, st);
  if (p.dtype == LQ_F16) return prefill<__half>(p, st);
  return prefill<float>(p, st);
}

cudaError_t launch_la_step(const LaParams& p, cudaStream_t st) {
  if (p.dtype == LQ_BF16) return step<__nv_bfloat16>(p, st);
  if (p.dtype == LQ_F16) return step<__half>(p, st);
  return step<float>(p, st);
}

}  // namespace lqi
