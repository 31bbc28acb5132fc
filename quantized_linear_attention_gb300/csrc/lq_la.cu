// Linear attention with a decay for each head (sm_103a):
//   S_t = alpha_t S_{t-1} + v_t k_t^T,   o_t = S_t q_t
// on fp32 states of 128 x 128, over prompts and for single tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lq_device.cuh"
#include "lq_internal.h"
#include "lq_la.cuh"

namespace lqi {

namespace {

// --------------------------------------------------------------------------------------------
// Prompts of fp32 and fp16 tokens, token by token in fp32: bound by the FMA units, 32,768
// FMAs a token and head (256 cycles of an SM). One CTA of 256 threads per piece of a sequence and head; four
// lanes hold two rows of the state, 32 columns each (float4 groups part, part + 4, ..: the four lanes read 64
// consecutive bytes of a staged key), in packed pairs.
//
// The decay would take a third multiplication per entry. It is kept apart instead: S = A s with one number A
// for the whole state, s += (v / A) k^T, o = A (s q). Every 16 tokens A goes back into s, in two parts (rounded
// to one it would be off in the same direction again and again), and so it does before a token at which it
// would leave 2^-12 .. 2^12 (a decay of zero among them) or is not a number.
constexpr int kRecTok = 16;  // tokens staged at a time

struct RecTok {
  float hi, lo;  // what s is multiplied by before this token's update, where `now` is set
  float inv, a;  // 1 / A and A after this token's decay
  int now;
};

template <typename T, bool OUT>
__global__ void __launch_bounds__(256, 2) k_la_recurrent(LaParams p) {
  __shared__ __align__(16) float sk[kRecTok][kD], sq[OUT ? kRecTok : 1][kD], sv[kRecTok][kD];
  __shared__ RecTok tok[kRecTok + 1];
  __shared__ Piece spc;
  const int tid = threadIdx.x, part = tid & 3, row = tid >> 2;  // and row + 64
  const int h = (int)(blockIdx.x % (unsigned)p.heads), kh = h / p.group;
  const int64_t slot = blockIdx.x / (unsigned)p.heads;
  if (tid < 32) {
    const Piece f = find_piece(p, slot);
    if (tid == 0) spc = f;
  }
  __syncthreads();
  const Piece pc = spc;
  if (pc.b < 0 || (!OUT && pc.i == pc.n - 1)) return;
  float* S_out = OUT ? (pc.i == pc.n - 1 && p.S ? p.S + (pc.b * p.heads + h) * (kD * kD) : nullptr)
                     : p.ws_state + (slot * p.heads + h) * (kD * kD);
  const T* q = static_cast<const T*>(p.q) + kh * kD;
  const T* k = static_cast<const T*>(p.k) + kh * kD;
  const T* v = static_cast<const T*>(p.v) + h * kD;
  T* o = static_cast<T*>(p.o) + h * kD;

  f32x2 S[2][8][2];  // row + 64 x, columns 16 c + 4 part .. + 3
  const float* from = OUT ? start_state(p, pc, slot, h) : nullptr;
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (from) y = *reinterpret_cast<const float4*>(from + (row + 64 * x) * kD + 16 * c + 4 * part);
      S[x][c][0] = f2_pack(y.x, y.y);
      S[x][c][1] = f2_pack(y.z, y.w);
    }

  // Tokens of a block: thread tid takes channels 4 (tid & 31) .. of tokens tid / 32 and tid / 32 + 8.
  float ld[2][3][4], la = 1.f;
  const int nb = (int)((pc.len + kRecTok - 1) / kRecTok);
  auto fetch = [&](int b) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int64_t t = (int64_t)b * kRecTok + (tid >> 5) + 8 * x;
      if (t < pc.len) {
        const int64_t at = pc.begin + t;
        const int c = 4 * (tid & 31);
        if (OUT) ld4(q + at * p.sq + c, ld[x][0]);
        ld4(k + at * p.sk + c, ld[x][1]);
        ld4(v + at * p.sv + c, ld[x][2]);
      }
    }
    const int64_t t = (int64_t)b * kRecTok + tid;
    if (tid < kRecTok) la = t < pc.len ? p.alpha[(pc.begin + t) * p.sa + h] : 1.f;
  };
  double prod = 1.0;
  auto stage = [&]() {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int t = (tid >> 5) + 8 * x, c = 4 * (tid & 31);
      if (OUT) *reinterpret_cast<float4*>(&sq[OUT ? t : 0][c]) = make_float4(ld[x][0][0], ld[x][0][1], ld[x][0][2], ld[x][0][3]);
      *reinterpret_cast<float4*>(&sk[t][c]) = make_float4(ld[x][1][0], ld[x][1][1], ld[x][1][2], ld[x][1][3]);
      *reinterpret_cast<float4*>(&sv[t][c]) = make_float4(ld[x][2][0], ld[x][2][1], ld[x][2][2], ld[x][2][3]);
    }
    if (tid < 32) {  // A from token to token, in two parts
      const float one = tid < kRecTok ? la : 1.f;
      float2 a = make_float2(one, 0.f);
#pragma unroll
      for (int d = 1; d < kRecTok; d <<= 1) {
        const float2 y = make_float2(__shfl_up_sync(0xffffffffu, a.x, d), __shfl_up_sync(0xffffffffu, a.y, d));
        if (tid >= d && tid < kRecTok) a = mul2(a, y);
      }
      const float g = fabsf(a.x);
      if (__all_sync(0xffffffffu, tid >= kRecTok || (g > 2.44140625e-4f && g < 4096.f))) {
        if (tid < kRecTok) tok[tid] = RecTok{1.f, 0.f, __fdiv_rn(1.f, a.x), a.x, 0};
        if (tid == kRecTok - 1) tok[kRecTok] = RecTok{a.x, a.y, 1.f, 1.f, 1};
      } else {
        float2 A = make_float2(1.f, 0.f);
        for (int t = 0; t < kRecTok; ++t) {
          const float x = __shfl_sync(0xffffffffu, one, t);
          float2 f = x == x && fabsf(x) < INFINITY ? mul2(A, make_float2(x, 0.f)) : make_float2(x, 0.f);
          const float m = fabsf(f.x);
          const bool now = !(m > 2.44140625e-4f && m < 4096.f);
          A = now ? make_float2(1.f, 0.f) : f;
          if (tid == 0) tok[t] = RecTok{f.x, f.y, __fdiv_rn(1.f, A.x), A.x, now};
        }
        if (tid == 0) tok[kRecTok] = RecTok{A.x, A.y, 1.f, 1.f, 1};
      }
      if (!OUT) {
        for (int t = 0; t < kRecTok; ++t) prod *= (double)__shfl_sync(0xffffffffu, one, t);
      }
    }
  };
  auto scale = [&](float hi, float lo) {
    const f32x2 h2 = f2_dup(hi), l2 = f2_dup(lo);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) S[x][c][e] = f2_fma(S[x][c][e], h2, f2_mul(S[x][c][e], l2));
  };
  if (nb) fetch(0);
  for (int b = 0; b < nb; ++b) {
    const int n = (int)min((int64_t)kRecTok, pc.len - (int64_t)b * kRecTok);
    stage();
    __syncthreads();
    if (b + 1 < nb) fetch(b + 1);
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
      const RecTok k0 = tok[t];
      if (k0.now) scale(k0.hi, k0.lo);
      const f32x2 v0 = f2_dup(__fmul_rn(sv[t][row], k0.inv)), v1 = f2_dup(__fmul_rn(sv[t][row + 64], k0.inv));
      f32x2 a0 = 0ull, a1 = 0ull, b0 = 0ull, b1 = 0ull;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const ulonglong2 kk = *reinterpret_cast<const ulonglong2*>(&sk[t][16 * c + 4 * part]);
        S[0][c][0] = f2_fma(v0, kk.x, S[0][c][0]);
        S[0][c][1] = f2_fma(v0, kk.y, S[0][c][1]);
        S[1][c][0] = f2_fma(v1, kk.x, S[1][c][0]);
        S[1][c][1] = f2_fma(v1, kk.y, S[1][c][1]);
        if (OUT) {
          const ulonglong2 qq = *reinterpret_cast<const ulonglong2*>(&sq[OUT ? t : 0][16 * c + 4 * part]);
          a0 = f2_fma(S[0][c][0], qq.x, a0);
          a1 = f2_fma(S[0][c][1], qq.y, a1);
          b0 = f2_fma(S[1][c][0], qq.x, b0);
          b1 = f2_fma(S[1][c][1], qq.y, b1);
        }
      }
      if (OUT) {
        float x0, x1, y0, y1;
        f2_unpack(f2_add(a0, a1), x0, x1);
        f2_unpack(f2_add(b0, b1), y0, y1);
        // lanes 0, 1 of the four end with row's sum, lanes 2, 3 with row + 64's
        const bool up = part & 2;
        const float mine = up ? __fadd_rn(y0, y1) : __fadd_rn(x0, x1);
        const float other = up ? __fadd_rn(x0, x1) : __fadd_rn(y0, y1);
        float r = __fadd_rn(mine, __shfl_xor_sync(0xffffffffu, other, 2));
        r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 1));
        if (!(part & 1))
          o[(pc.begin + (int64_t)b * kRecTok + t) * p.so + row + 64 * (part >> 1)] = from_f<T>(__fmul_rn(r, k0.a));
      }
    }
    const RecTok k0 = tok[kRecTok];
    scale(k0.hi, k0.lo);
    __syncthreads();
  }
  if (S_out) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float4 y;
        f2_unpack(S[x][c][0], y.x, y.y);
        f2_unpack(S[x][c][1], y.z, y.w);
        *reinterpret_cast<float4*>(S_out + (row + 64 * x) * kD + 16 * c + 4 * part) = y;
      }
  }
  if (!OUT && tid == 0) p.ws_decay[slot * p.heads + h] = prod;
}

// Between the passes: each segment's growth becomes the state before it, S_{i+1} = decay_i S_i + growth_i from S0 on.
// One thread per four entries; the segments of a sequence are read a few ahead.
__global__ void __launch_bounds__(256) k_la_scan(LaParams p) {
  __shared__ int64_t sfirst, sn;
  const int h = blockIdx.y;
  const int64_t b = blockIdx.z;
  if (threadIdx.x < 32) {
    int64_t first = 0, n = 1, begin, len;
    for (int64_t x = threadIdx.x; x < b; x += 32) {
      bounds(p, x, begin, len);
      first += len > p.seg ? (len + p.seg - 1) / p.seg : 1;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) first += __shfl_xor_sync(0xffffffffu, first, o);
    bounds(p, b, begin, len);
    if (len > p.seg) n = (len + p.seg - 1) / p.seg;
    if (threadIdx.x == 0) sfirst = first, sn = n;
  }
  __syncthreads();
  const int64_t first = sfirst, n = sn;
  if (n == 1 || first + n > p.slots) return;
  const int at = 4 * (blockIdx.x * 256 + threadIdx.x);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.S0) ld4(p.S0 + (b * p.heads + h) * (kD * kD) + at, s);
  float* w = p.ws_state + (first * p.heads + h) * (kD * kD) + at;
  const int64_t pitch = (int64_t)p.heads * (kD * kD);
  constexpr int kAhead = 8;
  for (int64_t i = 0; i < n; i += kAhead) {
    float u[kAhead][4];
    double d[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x)
      if (i + x < n - 1) {
        ld4(w + (i + x) * pitch, u[x]);
        d[x] = p.ws_decay[(first + i + x) * p.heads + h];
      }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      if (i + x < n) *reinterpret_cast<float4*>(w + (i + x) * pitch) = make_float4(s[0], s[1], s[2], s[3]);
      if (i + x < n - 1) {
        const float hi = (float)d[x], lo = (float)(d[x] - (double)hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = __fmaf_rn(s[e], hi, __fmaf_rn(s[e], lo, u[x][e]));
      }
    }
  }
}

// The states of split sequences that were staged in the workspace (last states that replace S0 in place).
__global__ void k_copy_states(LaParams p, const float* from) {
  const int64_t n = p.n_seqs * p.heads * (int64_t)(kD * kD / 4);
  for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < n; x += (int64_t)gridDim.x * blockDim.x)
    reinterpret_cast<float4*>(p.S)[x] = reinterpret_cast<const float4*>(from)[x];
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
cudaError_t prefill(const LaParams& p0, cudaStream_t st) {
  LaParams p = p0;
  const unsigned grid = (unsigned)((p.seg ? p.slots : p.n_seqs) * p.heads);
  cudaError_t e;
  if (p.seg) {
    k_la_recurrent<T, false><<<grid, 256, 0, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess || (e = launch_la_scan(p, st)) != cudaSuccess) return e;
  }
  if (la_staged(p)) p.S = p.ws_last;
  k_la_recurrent<T, true><<<grid, 256, 0, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return la_staged(p0) ? launch_la_unstage(p0, st) : cudaSuccess;
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

cudaError_t launch_la_scan(const LaParams& p, cudaStream_t st) {
  k_la_scan<<<dim3(kD * kD / 1024, (unsigned)p.heads, (unsigned)p.n_seqs), 256, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_la_unstage(const LaParams& p, cudaStream_t st) {
  k_copy_states<<<608, 256, 0, st>>>(p, p.ws_last);
  return cudaGetLastError();
}

void la_plan(const lq_la_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len, int64_t* seg, int64_t* slots) {
  *seg = *slots = 0;
  const int64_t longest = max_len > 0 && max_len < n_tokens ? max_len : n_tokens;
  const int64_t work = n_tokens * c->heads;  // head-tokens
  if (c->dtype == LQ_BF16) {
    // Splitting reads k and v twice (1.5 times the bytes), so it pays where the longest
    // sequence alone takes longer than that: 1.6 times an SM's share.
    if (5 * longest <= 8 * (work / 152) || longest <= 1024) return;
    // Two rounds of CTAs, less the last piece of each head, which is shorter: a piece costs about as much again as
    // six chunks (32,768 tokens x 32 heads: four rounds 437 us, three 417, two 381).
    const int64_t pieces = c->heads < 152 ? 304 - c->heads : 152;
    *seg = (work / pieces + 127) / 128 * 128;
    if (*seg < 512) *seg = 512;
  } else {
    // Two CTAs to an SM; the first pass costs half of the second.
    if (5 * longest <= 8 * (work / 304) || longest <= 256) return;
    *seg = (work / 304 + 15) / 16 * 16;
    if (*seg < 128) *seg = 128;
  }
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
