// Linear attention with a decay for each head (sm_103a):
//   S_t = alpha_t S_{t-1} + v_t k_t^T,   o_t = S_t q_t
// on fp32 states of 128 x 128, over prompts and for single tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "lq_device.cuh"
#include "lq_internal.h"
#include "lq_la.cuh"

namespace lqi {

namespace {

// --------------------------------------------------------------------------------------------
// Prompts of fp32 and fp16 tokens, token by token in fp32: bound by the FMA units, 32,768
// FMAs a token and head (256 cycles of an SM). One CTA of 256 threads per piece of a sequence and head; a thread
// holds 8 x 8 entries of the state in packed pairs: 32 cycles of shared memory a warp and token (two rows of 32 took
// 73, more than the FMAs). Values are staged divided by A, and with
// outputs twice over, so that they load as pairs: copying each into a pair took the FMA pipe. (Without outputs that
// would be more shared memory than the FMAs cover.)
//
// The decay would take a third multiplication per entry. It is kept apart instead: S = A s with one number A
// for the whole state, s += (v / A) k^T, o = A (s q). Every 8 tokens A goes back into s, in two parts (rounded
// to one it would be off in the same direction again and again), and so it does before a token at which it
// would leave 2^-12 .. 2^12 (a decay of zero among them) or is not a number. So s and v / A may pass fp32's largest number
// where S and v do not, and an infinity in s becomes NaN by the second part of A: where the state or an output comes
// out not finite, the CTA takes its tokens again as the recurrence is written (redo).
//
// 2,764 fp32 tokens of 4 sequences x 16 heads: 172 us, 54 in the first pass and 117 in the second. The packed FMAs
// alone are 60 of those 117; with 16 warps to an SM the shuffles' and shared memory's latencies are not all covered.
constexpr int kRecTok = 8;  // tokens staged at a time
// Prompts of bf16 tokens up to this length go token by token too. Replayed from a graph with 4 head-sequences: 5.3 us for
// 3 tokens, 7.9 for 8, 9.9 for 12, against 9.9 for a chunk; with 2,048: 39 us + 3 to 5 a token against 136.
constexpr int kShort = 12;

struct RecTok {
  float hi, lo;  // what s is multiplied by before this token's update, where `now` is set
  float inv, a;  // 1 / A and A after this token's decay
  int now;
};

template <typename T, bool OUT>
__global__ void __launch_bounds__(256, 2) k_la_recurrent(LaParams p) {
  using Val = typename std::conditional<OUT, f32x2, float>::type;
  constexpr int kQ = OUT ? kRecTok : 1, kBufK = 2 * kRecTok * kD * 4, kBufQ = OUT ? 2 * kQ * kD * 4 : 0;
  __shared__ __align__(16) char buf[kBufK + kBufQ + 2 * kRecTok * kD * sizeof(Val)];
  static_assert(sizeof(buf) >= (3 * kD + 1) * kRecTok * 4, "redo's tokens");
  float(*const sk)[kRecTok][kD] = reinterpret_cast<float(*)[kRecTok][kD]>(buf);
  float(*const sq)[kQ][kD] = reinterpret_cast<float(*)[kQ][kD]>(buf + kBufK);
  Val(*const sv)[kRecTok][kD] = reinterpret_cast<Val(*)[kRecTok][kD]>(buf + kBufK + kBufQ);
  __shared__ RecTok tok[4][kRecTok + 1];
  __shared__ bool even[4];  // no token of the block needs A put back before it
  __shared__ float2 sprod[8];
  __shared__ Piece spc;
  __shared__ int again;
  cudaTriggerProgrammaticLaunchCompletion();
  const int tid = threadIdx.x, tx = tid & 15, row = 8 * (tid >> 4), warp = tid >> 5, lane = tid & 31;
  const int h = (int)(blockIdx.x % (unsigned)p.heads), kh = h / p.group;
  const int64_t slot = blockIdx.x / (unsigned)p.heads;
  if (tid < 32) {
    const Piece f = find_piece(p, slot);
    if (tid == 0) spc = f, again = 0;
  }
  __syncthreads();
  const Piece pc = spc;
  if (pc.b < 0 || (!OUT && pc.i == pc.n - 1)) return;
  float2* const serial = serial_note(p, pc, slot, h);
  if (!OUT && pc.i == 0 && tid == 0 && serial) *serial = make_float2(0.f, 0.f);
  float* S_out = OUT ? (pc.i == pc.n - 1 && p.S ? p.S + (pc.b * p.heads + h) * (kD * kD) : nullptr)
                     : p.ws_state + (slot * p.heads + h) * (kD * kD);
  const T* q = static_cast<const T*>(p.q) + kh * kD;
  const T* k = static_cast<const T*>(p.k) + kh * kD;
  const T* v = static_cast<const T*>(p.v) + h * kD;
  T* o = static_cast<T*>(p.o) + h * kD;

  if (OUT && p.seg) cudaGridDependencySynchronize();
  f32x2 S[8][4];  // row + x, columns 4 tx .. + 3 (pairs 0, 1) and 64 + 4 tx .. + 3 (pairs 2, 3)
  const float* from = OUT ? start_state(p, pc, slot, h) : nullptr;
#pragma unroll
  for (int x = 0; x < 8; ++x)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (from) y = *reinterpret_cast<const float4*>(from + (row + x) * kD + 64 * c + 4 * tx);
      S[x][2 * c] = f2_pack(y.x, y.y);
      S[x][2 * c + 1] = f2_pack(y.z, y.w);
    }

  if (OUT && serial && serial->x != 0.f) {
    if (pc.i) return;
    int64_t begin, len;
    bounds(p, pc.b, begin, len);
    const int64_t at = (pc.b * p.heads + h) * (kD * kD);
    redo<T, true, 256, kRecTok>(p, begin, len, h, p.S0 ? p.S0 + at : nullptr, reinterpret_cast<float*>(buf),
                                p.S ? p.S + at : nullptr, nullptr);
    return;
  }

  // Tokens of a block: warp w takes token w of each, a lane four channels.
  float ld[3][4];
  const int nb = (int)((pc.len + kRecTok - 1) / kRecTok);
  auto fetch = [&](int b) {
    const int64_t t = (int64_t)b * kRecTok + warp, at = pc.begin + t;
    if (t < pc.len) {
      if (OUT) ld4(q + at * p.sq + 4 * lane, ld[0]);
      ld4(k + at * p.sk + 4 * lane, ld[1]);
      ld4(v + at * p.sv + 4 * lane, ld[2]);
    }
  };
  auto stage = [&](int b) {
    const int s = b & 1;
    const float inv = tok[b & 3][warp].inv;
    if (OUT) *reinterpret_cast<float4*>(&sq[s][OUT ? warp : 0][4 * lane]) = make_float4(ld[0][0], ld[0][1], ld[0][2], ld[0][3]);
    *reinterpret_cast<float4*>(&sk[s][warp][4 * lane]) = make_float4(ld[1][0], ld[1][1], ld[1][2], ld[1][3]);
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __fmul_rn(ld[2][e], inv);
    if (OUT) {
      *reinterpret_cast<float4*>(&sv[s][warp][4 * lane]) = make_float4(x[0], x[0], x[1], x[1]);
      *reinterpret_cast<float4*>(&sv[s][warp][4 * lane + 2]) = make_float4(x[2], x[2], x[3], x[3]);
    } else {
      *reinterpret_cast<float4*>(&sv[s][warp][4 * lane]) = make_float4(x[0], x[1], x[2], x[3]);
    }
  };
  // A from token to token of block b, in two parts: warp b mod 8, which has had the block's decays since its last turn.
  float2 prod = make_float2(1.f, 0.f);
  auto decays = [&](int b) {
    const int64_t t = (int64_t)b * kRecTok + lane;
    return lane < kRecTok && t < pc.len ? p.alpha[(pc.begin + t) * p.sa + h] : 1.f;
  };
  float la = decays(warp);
  auto prepare = [&](int b) {
    const int s = b & 3;
    const float one = la;
    la = decays(b + 8);
    float2 a = make_float2(one, 0.f);
#pragma unroll
    for (int d = 1; d < kRecTok; d <<= 1) {
      const float2 y = make_float2(__shfl_up_sync(0xffffffffu, a.x, d), __shfl_up_sync(0xffffffffu, a.y, d));
      if (lane >= d) a = mul2(a, y);
    }
    const float g = fabsf(a.x);
    if (__all_sync(0xffffffffu, lane >= kRecTok || (g > 2.44140625e-4f && g < 4096.f))) {
      if (lane < kRecTok) tok[s][lane] = RecTok{1.f, 0.f, __fdiv_rn(1.f, a.x), a.x, 0};
      if (lane == kRecTok - 1) tok[s][kRecTok] = RecTok{a.x, a.y, 1.f, 1.f, 1};
      if (lane == 0) even[s] = true;
    } else {
      float2 A = make_float2(1.f, 0.f);
      for (int t = 0; t < kRecTok; ++t) {
        const float x = __shfl_sync(0xffffffffu, one, t);
        const float2 f = fabsf(x) < INFINITY ? mul2(A, make_float2(x, 0.f)) : make_float2(x, 0.f);
        const float m = fabsf(f.x);
        const bool now = !(m > 2.44140625e-4f && m < 4096.f);
        A = now ? make_float2(1.f, 0.f) : f;
        if (lane == 0) tok[s][t] = RecTok{f.x, f.y, __fdiv_rn(1.f, A.x), A.x, now};
      }
      if (lane == 0) tok[s][kRecTok] = RecTok{A.x, A.y, 1.f, 1.f, 1}, even[s] = false;
    }
    if (!OUT)
      prod = mul2(prod, make_float2(__shfl_sync(0xffffffffu, a.x, kRecTok - 1), __shfl_sync(0xffffffffu, a.y, kRecTok - 1)));
  };
  auto scale = [&](float hi, float lo) {
    const f32x2 h2 = f2_dup(hi), l2 = f2_dup(lo);
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[x][c] = f2_fma(S[x][c], h2, f2_mul(S[x][c], l2));
  };
  T* out = o + pc.begin * p.so + row + (tx >> 1);
  float odd = 0.f;  // NaN once an output is not finite
  auto token = [&](int s, int t, float A) {
    const ulonglong2 k0 = *reinterpret_cast<const ulonglong2*>(&sk[s][t][4 * tx]);
    const ulonglong2 k1 = *reinterpret_cast<const ulonglong2*>(&sk[s][t][64 + 4 * tx]);
#pragma unroll
    for (int x = 0; x < 8; x += 2) {
      ulonglong2 v;
      if (OUT) {
        v = *reinterpret_cast<const ulonglong2*>(&sv[s][t][row + x]);
      } else {
        const float2 y = *reinterpret_cast<const float2*>(&sv[s][t][row + x]);
        v = make_ulonglong2(f2_dup(y.x), f2_dup(y.y));
      }
      S[x][0] = f2_fma(v.x, k0.x, S[x][0]);
      S[x][1] = f2_fma(v.x, k0.y, S[x][1]);
      S[x][2] = f2_fma(v.x, k1.x, S[x][2]);
      S[x][3] = f2_fma(v.x, k1.y, S[x][3]);
      S[x + 1][0] = f2_fma(v.y, k0.x, S[x + 1][0]);
      S[x + 1][1] = f2_fma(v.y, k0.y, S[x + 1][1]);
      S[x + 1][2] = f2_fma(v.y, k1.x, S[x + 1][2]);
      S[x + 1][3] = f2_fma(v.y, k1.y, S[x + 1][3]);
    }
    if (OUT) {
      const ulonglong2 q0 = *reinterpret_cast<const ulonglong2*>(&sq[s][OUT ? t : 0][4 * tx]);
      const ulonglong2 q1 = *reinterpret_cast<const ulonglong2*>(&sq[s][OUT ? t : 0][64 + 4 * tx]);
      float r[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        float lo, hi;
        f2_unpack(f2_fma(S[x][3], q1.y, f2_fma(S[x][2], q1.x, f2_fma(S[x][1], q0.y, f2_mul(S[x][0], q0.x)))), lo, hi);
        r[x] = __fadd_rn(lo, hi);
      }
      // sums over the 16 lanes of a row group, half of the rows changing hands at each step: lane tx ends with
      // row tx / 2
#pragma unroll
      for (int w = 4; w; w >>= 1) {
        const bool up = tx & (2 * w);
#pragma unroll
        for (int x = 0; x < w; ++x) {
          const float keep = up ? r[w + x] : r[x], send = up ? r[x] : r[w + x];
          r[x] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, 2 * w));
        }
      }
      r[0] = __fadd_rn(r[0], __shfl_xor_sync(0xffffffffu, r[0], 1));
      r[0] = __fmul_rn(r[0], A);
      odd = __fmaf_rn(r[0], 0.f, odd);
      if (!(tx & 1)) *out = from_f<T>(r[0]);
      out += p.so;
    }
  };
  if (nb) {
    fetch(0);
    if (warp < min(2, nb)) prepare(warp);
  }
  __syncthreads();
  for (int b = 0; b < nb; ++b) {
    const int s = b & 1, n = (int)min((int64_t)kRecTok, pc.len - (int64_t)b * kRecTok);
    const RecTok* tk = tok[b & 3];
    stage(b);
    __syncthreads();  // (whoever is here is through with block b - 1, so its buffers may be written after this)
    if (b + 1 < nb) fetch(b + 1);
    if (b + 2 < nb && warp == ((b + 2) & 7)) prepare(b + 2);
    if (n == kRecTok && even[b & 3]) {
#pragma unroll 2
      for (int t = 0; t < kRecTok; ++t) token(s, t, tk[t].a);
    } else {
#pragma unroll 1
      for (int t = 0; t < n; ++t) {
        if (tk[t].now) scale(tk[t].hi, tk[t].lo);
        token(s, t, tk[t].a);
      }
    }
    scale(tk[kRecTok].hi, tk[kRecTok].lo);
  }
  f32x2 sum = f2_pack(odd, 0.f);  // (an entry that is not finite never comes back)
#pragma unroll
  for (int x = 0; x < 8; ++x)
#pragma unroll
    for (int c = 0; c < 4; ++c) sum = f2_fma(S[x][c], 0ull, sum);
  float s0, s1;
  f2_unpack(sum, s0, s1);
  if (s0 != 0.f || s1 != 0.f) again = 1;
  __syncthreads();
  if (again) {
    redo<T, OUT, 256, kRecTok>(p, spc.begin, spc.len, h, OUT ? start_state(p, spc, slot, h) : nullptr,
                               reinterpret_cast<float*>(buf), S_out, nullptr);
  } else if (S_out) {
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float4 y;
        f2_unpack(S[x][2 * c], y.x, y.y);
        f2_unpack(S[x][2 * c + 1], y.z, y.w);
        *reinterpret_cast<float4*>(S_out + (row + x) * kD + 64 * c + 4 * tx) = y;
      }
  }
  if (!OUT) {
    if (lane == 0) sprod[warp] = prod;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < 8; ++w) prod = mul2(prod, sprod[w]);
      p.ws_decay[slot * p.heads + h] = prod;
    }
  }
}

// Between the passes: each segment's growth becomes the state before it, S_{i+1} = decay_i S_i + growth_i from S0 on.
// One thread per four entries; the segments of a sequence are read a few ahead.
__device__ __forceinline__ void scan_sequence(const LaParams& p, int64_t b, int h) {
  int64_t begin, len;
  bounds(p, b, begin, len);
  if (len <= p.seg) return;  // (most sequences of a batch)
  __shared__ int64_t sfirst;
  __syncthreads();
  if (threadIdx.x < 32) {
    int64_t first = 0, b1, l1;
    for (int64_t x = threadIdx.x; x < b; x += 32) {
      bounds(p, x, b1, l1);
      first += l1 > p.seg ? (l1 + p.seg - 1) / p.seg : 1;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) first += __shfl_xor_sync(0xffffffffu, first, o);
    if (threadIdx.x == 0) sfirst = first;
  }
  __syncthreads();
  const int64_t first = sfirst, n = (len + p.seg - 1) / p.seg;
  if (first + n > p.slots) return;
  cudaGridDependencySynchronize();
  const int at = 4 * (blockIdx.x * 256 + threadIdx.x);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.S0) ld4(p.S0 + (b * p.heads + h) * (kD * kD) + at, s);
  float* w = p.ws_state + (first * p.heads + h) * (kD * kD) + at;
  const int64_t pitch = (int64_t)p.heads * (kD * kD);
  constexpr int kAhead = 4;
  for (int64_t i = 0; i < n; i += kAhead) {
    float u[kAhead][4];
    float2 d[kAhead];
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
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = __fmaf_rn(s[e], d[x].x, __fmaf_rn(s[e], d[x].y, u[x][e]));
      }
    }
  }
  // (a state that is not finite, S0 among them, never comes back: the last one tells)
  const float odd = __fmaf_rn(s[0], 0.f, __fmaf_rn(s[1], 0.f, __fmaf_rn(s[2], 0.f, s[3] * 0.f)));
  if (odd != 0.f) p.ws_decay[(first + n - 1) * p.heads + h] = make_float2(1.f, 0.f);
}

__global__ void __launch_bounds__(256, 5) k_la_scan(LaParams p) {
  cudaTriggerProgrammaticLaunchCompletion();
  // Where no sequence is split, one CTA still waits for the first pass: the kernel after this one, and what the
  // caller does next in the stream, count on that pass' end when this grid has ended.
  if (blockIdx.x + blockIdx.y + blockIdx.z == 0) cudaGridDependencySynchronize();
  for (int64_t b = blockIdx.z; b < p.n_seqs; b += gridDim.z) scan_sequence(p, b, blockIdx.y);
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
// channels, so nothing waits on a barrier. P CTAs share a head-state. 16,384 states of
// bf16 tokens: 324 us for 2.16 GB, 98% of the copy bandwidth; 32 states 2 us replayed from a graph (11 to 14 a call,
// which is the host's time).
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
  if (p.seg) {
    e = launch_upon(k_la_recurrent<T, true>, dim3(grid), 256, 0, st, p);
  } else {
    k_la_recurrent<T, true><<<grid, 256, 0, st>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return la_staged(p0) ? launch_la_unstage(p0, st) : cudaSuccess;
}

template <typename T>
cudaError_t step(const LaParams& p, cudaStream_t st) {
  const int64_t n = p.n_seqs * p.heads;
  // Few head-states: four CTAs share one, so that the loads spread over the SMs (replayed from a graph, 8 and 32
  // head-states 2.1 us against 3.1; 128 3.1 either way; 256 4.9 against 4.6, 512 7.7 either way).
  if (n < 128) k_la_step<T, 4><<<(unsigned)(4 * n), 256, 0, st>>>(p);
  else k_la_step<T, 1><<<(unsigned)n, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_scan(const LaParams& p, cudaStream_t st) {
  const unsigned z = (unsigned)(p.n_seqs < 65535 ? p.n_seqs : 65535);
  return launch_upon(k_la_scan, dim3(kD * kD / 1024, (unsigned)p.heads, z), 256, 0, st, p);
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
    // Two CTAs to an SM; the first pass costs half of the second. Sequences past 2,048 tokens are split in any case,
    // into segments of 1,024 at most: every token rounds the state once, and after 16,000 of them in a row that
    // was 2e-6 of it (sums over segments and then over the segments' sums: 5e-7).
    if (longest <= 2048 && (5 * longest <= 8 * (work / 304) || longest <= 256)) return;
    *seg = (work / 304 + 15) / 16 * 16;
    if (*seg < 128) *seg = 128;
    if (*seg > 1024) *seg = 1024;
  }
  *slots = n_tokens / *seg + n_seqs;
}

// A call with fewer tokens may be split where a larger one is not, and its segments are rounded, so this is not la_plan's
// answer for the largest. With W CTAs' shares (152 or 304) a call of n tokens is split only if 5 min(longest, n) > 8 (n heads / W),
// the quotient rounded down: where any n is, one of the shortest or (past 2,048) the longest is. A segment of g tokens
// has n < (g + 1) pieces / heads, so n / g < pieces / heads (1 + 1 / g), but for the longest segments, of 1,024.
int64_t la_most_slots(const lq_la_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len) {
  const int64_t longest = max_len > 0 && max_len < n_tokens ? max_len : n_tokens, h = c->heads;
  const bool bf16 = c->dtype == LQ_BF16;
  const int64_t share = bf16 ? 152 : 304, least = bf16 ? 1025 : 257;
  if (longest < least || ((8 * h - 5 * share) * least >= 8 * share && (bf16 || longest <= 2048))) return 0;
  const int64_t pieces = !bf16 ? 304 : h < 152 ? 304 - h : 152, g = bf16 ? 512 : 128;
  int64_t n = pieces * (g + 1) / (h * g);
  if (n > n_tokens / g) n = n_tokens / g;
  if (!bf16 && n < n_tokens / 1024) n = n_tokens / 1024;
  return n + n_seqs;
}

cudaError_t launch_la_prefill(const LaParams& p, cudaStream_t st) {
  const int64_t longest = p.max_len > 0 && p.max_len < p.n_tokens ? p.max_len : p.n_tokens;
  if (p.dtype == LQ_BF16) return longest <= kShort ? prefill<__nv_bfloat16>(p, st) : launch_la_chunk_bf16(p, st);
  if (p.dtype == LQ_F16) return prefill<__half>(p, st);
  return prefill<float>(p, st);
}

cudaError_t launch_la_step(const LaParams& p, cudaStream_t st) {
  if (p.dtype == LQ_BF16) return step<__nv_bfloat16>(p, st);
  if (p.dtype == LQ_F16) return step<__half>(p, st);
  return step<float>(p, st);
}

}  // namespace lqi
