// The selection of beam search (sm_103a): for each request the n_best of
//   scores[b] + logits[b][t] - log sum_t' exp(logits[b][t'])
// over its beams b and tokens t, equal scores to the lowest b * vocab + t.
//
// Two kernels. k_beam_scan reads the logits once, the only large traffic (HBM
// bounds it): a CTA holds one slice of one row in registers, sums its
// exponentials and keeps its n_best largest logits. Inside a row the order of the
// scores is the order of the logits, so no score is needed there. k_beam_pick
// joins a request's slices: log-sum-exps and scores in 64 bits, because the
// order of nearly equal candidates of different beams hangs on their rows' sums.
//
// The sum of a slice: with m = ceil(max * log2 e), a whole number, each term is
// 2^(x log2 e - m), its exponent formed by two fmas from a two-part log2 e (one
// rounding, relative to the exponent itself), and the slices' sums join by exact
// powers of two. Rows with equal contents sum in the same order whatever their
// place in memory, so equal hypotheses tie exactly.
//
// The n_best of a slice without a sort: 64 groups of four threads give their
// maxima; at least n_best elements are not below the n_best-th largest of those
// (each of the n_best groups has one), so the few elements at or above it are
// collected and ranked by counting. At 16,384 elements and n_best = 16 they are
// about 18. Where ties make them more than the list holds, a bisection over
// (value, index) finds the exact n_best-th key.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "lq_internal.h"

namespace lqi {

namespace {

constexpr int kNT = 256;
constexpr double kLn2 = 0.693147180559945309417;
constexpr int kList = 512;   // candidates a slice collects before ranking
constexpr int kPick = 2048;  // candidates a request collects before ranking

struct Cand {
  float x;
  int32_t t;
};

// Workspace, per (row, slice): the sum (64 bits), what it is relative to, the number of candidates, the candidates.
constexpr int32_t kByTop = INT32_MAX;
struct Ws {
  double* sum;
  int32_t* exp2;  // the sum stands for sum * 2^exp2, or where this is kByTop
  float* top;     // for sum * e^top
  int32_t* n;
  Cand* cand;
};

__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

__host__ __device__ inline Ws carve(void* ws, int64_t lists) {
  char* c = static_cast<char*>(ws);
  Ws w;
  w.sum = reinterpret_cast<double*>(c);
  c += up256(8 * lists);
  w.exp2 = reinterpret_cast<int32_t*>(c);
  c += up256(4 * lists);
  w.top = reinterpret_cast<float*>(c);
  c += up256(4 * lists);
  w.n = reinterpret_cast<int32_t*>(c);
  c += up256(4 * lists);
  w.cand = reinterpret_cast<Cand*>(c);
  return w;
}

// Floats as unsigned numbers in the same order; -0 counts as +0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u ^ ((u >> 63) ? 0xffffffffffffffffull : 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered(uint64_t u) {
  return __longlong_as_double((long long)(u ^ ((u >> 63) ? 0x8000000000000000ull : 0xffffffffffffffffull)));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ float get(const uint32_t* w, int i) { return __uint_as_float(w[i]); }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr uint32_t kNegInf = 0xff80u;
  static __device__ __forceinline__ float get(const uint32_t* w, int i) {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
  }
};
template <>
struct Elem<__half> {
  static constexpr uint32_t kNegInf = 0xfc00u;
  static __device__ __forceinline__ float get(const uint32_t* w, int i) {
    const uint16_t u = (uint16_t)((i & 1) ? (w[i >> 1] >> 16) : (w[i >> 1] & 0xffffu));
    return __half2float(__ushort_as_half(u));
  }
};

// W words (of 32 bits) of a row held by a thread, VE elements to a load. Element i
// of the thread is element ((i / VE) * 256 + tid) * VE + i % VE of the slice.
template <typename T, int VE, int W>
__global__ void __launch_bounds__(kNT, 4) k_beam_scan(BeamParams p) {
  constexpr int EPW = 4 / (int)sizeof(T), E = W * EPW;  // elements per word, per thread
  __shared__ float gmax[64];
  __shared__ double wsum[8];
  __shared__ uint64_t list[kList];
  __shared__ float sT;
  __shared__ int cnt;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / p.splits;
  const int64_t base = (int64_t)(blockIdx.x % p.splits) * (kNT * E);
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride + base;
  const int64_t left = p.vocab - base;  // elements from the slice's first on
  if (tid == 0) cnt = 0;

  uint32_t w[W];
  auto word_of = [&](int i) -> uint32_t {  // one element's bits, -inf past the end
    const int64_t e = ((int64_t)(i / VE) * kNT + tid) * VE + i % VE;
    if (e >= left) return Elem<T>::kNegInf;
    if (sizeof(T) == 4) return reinterpret_cast<const uint32_t*>(x)[e];
    return reinterpret_cast<const uint16_t*>(x)[e];
  };
  constexpr int WPV = VE / EPW;  // words per load (0: less than a word)
#pragma unroll
  for (int j = 0; j < (WPV ? W / (WPV ? WPV : 1) : 0); ++j) {
    const int64_t e0 = ((int64_t)j * kNT + tid) * VE;
    if (e0 + VE <= left) {
      if (WPV == 4) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(x + e0));
        w[j * 4] = v.x, w[j * 4 + 1] = v.y, w[j * 4 + 2] = v.z, w[j * 4 + 3] = v.w;
      } else {
        w[j] = __ldcs(reinterpret_cast<const uint32_t*>(x + e0));
      }
    } else {
#pragma unroll
      for (int c = 0; c < WPV; ++c) {
        const int i = (j * WPV + c) * EPW;
        w[j * WPV + c] = EPW == 1 ? word_of(i) : (word_of(i) | (word_of(i + 1) << 16));
      }
    }
  }
  if (WPV == 0) {
#pragma unroll
    for (int c = 0; c < W; ++c) w[c] = word_of(2 * c) | (word_of(2 * c + 1) << 16);
  }

  float mx = -INFINITY;  // (fmaxf passes NaN over: the sum meets it)
#pragma unroll
  for (int i = 0; i < E; ++i) mx = fmaxf(mx, Elem<T>::get(w, i));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  if ((tid & 3) == 0) gmax[tid >> 2] = mx;
  __syncthreads();
  float top = fmaxf(gmax[lane], gmax[lane + 32]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  {  // four threads rank one group's maximum among the 64; equal ones in the order of the groups
    const int g = tid >> 2;
    const float mine = gmax[g];
    int rank = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int u = (tid & 3) * 16 + j;
      const float y = gmax[u];
      rank += (y > mine || (y == mine && u < g)) ? 1 : 0;
    }
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    if ((tid & 3) == 0 && rank == p.n_best - 1) sT = mine;
  }
  __syncthreads();
  const float T0 = sT;
  // A whole exponent of two not below the largest term's; nothing finite in the slice: any will do.
  constexpr float kL2Ehi = 1.44269502162933349609375f, kL2Elo = 1.92596299e-8f;  // log2 e in two parts
  // Past 2^20 the exponents' own rounding would show: then relative to the largest logit itself.
  const bool byTop = top < INFINITY && top > -INFINITY && fabsf(top) > 1048576.0f;
  const float m = (!byTop && fabsf(top) < INFINITY) ? ceilf(__fmul_rn(top, kL2Ehi)) : 0.0f;
  const float less = byTop ? top : 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float v = Elem<T>::get(w, i);
    const float d = __fsub_rn(v, less);  // (v itself, exactly, in the usual case; -inf stays -inf)
    sum = __fadd_rn(sum, ex2(__fmaf_rn(d, kL2Elo, __fmaf_rn(d, kL2Ehi, -m))));
    if (v >= T0 && v > -INFINITY) {
      const int at = atomicAdd(&cnt, 1);
      const int64_t e = ((int64_t)(i / VE) * kNT + tid) * VE + i % VE;
      if (at < kList) list[at] = ((uint64_t)ordered(v) << 32) | (0xffffffffu - (uint32_t)(base + e));
    }
  }
  double s = (double)sum;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) wsum[warp] = s;
  __syncthreads();
  int n = cnt;
  if (n > kList) {
    // Too many at or above the group threshold: the largest key with at least n_best keys not below it, bit by bit.
    __shared__ int above;
    uint64_t key = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t want = key | (1ull << bit);
      int c = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float v = Elem<T>::get(w, i);
        const int64_t e = ((int64_t)(i / VE) * kNT + tid) * VE + i % VE;
        const uint64_t u = ((uint64_t)ordered(v) << 32) | (0xffffffffu - (uint32_t)(base + e));
        c += (v > -INFINITY && u >= want) ? 1 : 0;
      }
      c = __reduce_add_sync(0xffffffffu, c);
      if (tid == 0) above = 0;
      __syncthreads();
      if (lane == 0) atomicAdd(&above, c);
      __syncthreads();
      if (above >= p.n_best) key = want;
      __syncthreads();
    }
    if (tid == 0) cnt = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float v = Elem<T>::get(w, i);
      const int64_t e = ((int64_t)(i / VE) * kNT + tid) * VE + i % VE;
      const uint64_t u = ((uint64_t)ordered(v) << 32) | (0xffffffffu - (uint32_t)(base + e));
      if (v > -INFINITY && u >= key) {
        const int at = atomicAdd(&cnt, 1);
        if (at < kList) list[at] = u;
      }
    }
    __syncthreads();
    n = min(cnt, kList);
  }
  const Ws ws = carve(p.ws, p.batch * p.beams * p.splits);
  const int64_t l = blockIdx.x;
  for (int c = tid; c < n; c += kNT) {
    const uint64_t mine = list[c];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += list[j] > mine ? 1 : 0;
    if (rank < p.n_best)
      ws.cand[l * p.n_best + rank] = Cand{unordered((uint32_t)(mine >> 32)), (int32_t)(0xffffffffu - (uint32_t)mine)};
  }
  if (tid == 0) {
    double t = wsum[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) t += wsum[j];
    ws.sum[l] = t;
    ws.exp2[l] = byTop ? kByTop : (int32_t)m;
    ws.top[l] = top;
    ws.n[l] = min(n, p.n_best);
  }
}

// A score's place in the order: larger keys first, then lower flat indices.
__device__ __forceinline__ bool before(uint64_t s1, uint32_t f1, uint64_t s2, uint32_t f2) {
  return s1 > s2 || (s1 == s2 && f1 < f2);
}

template <typename T>
__device__ __forceinline__ bool is_masked(const BeamParams& p, int64_t row, int64_t t) {
  const T x = static_cast<const T*>(p.logits)[row * p.row_stride + t];
  return (float)x == -INFINITY;
}

// One CTA per request.
template <typename T>
__global__ void __launch_bounds__(kNT) k_beam_pick(BeamParams p) {
  extern __shared__ __align__(16) unsigned char dyn[];
  uint64_t* ks = reinterpret_cast<uint64_t*>(dyn);
  uint32_t* kf = reinterpret_cast<uint32_t*>(dyn + 8 * kPick);
  __shared__ double sum[kMaxBeams], sco[kMaxBeams];  // log-sum-exps (NaN: a dead hypothesis) and scores
  __shared__ uint64_t hs[kNT], sT;
  __shared__ uint32_t hf[kNT];
  __shared__ int cnt, total;
  const int tid = threadIdx.x, M = p.n_best;
  const int64_t r = blockIdx.x;
  const Ws ws = carve(p.ws, p.batch * p.beams * p.splits);
  const int64_t l0 = r * p.beams * p.splits;  // the request's first list
  const int64_t NL = (int64_t)p.beams * p.splits;
  if (tid == 0) cnt = total = 0, sT = 0;
  if (tid < p.beams) {
    const int64_t l = l0 + (int64_t)tid * p.splits;
    int e = INT32_MIN;
    for (int j = 0; j < p.splits; ++j)
      if (ws.sum[l + j] != 0.0) e = max(e, ws.exp2[l + j]);
    double s = 0.0, lse;
    if (e != kByTop) {
      for (int j = 0; j < p.splits; ++j)
        if (ws.sum[l + j] != 0.0) s += ldexp(ws.sum[l + j], max(ws.exp2[l + j] - e, -4000));
      lse = log(s) + (double)e * kLn2;
    } else {
      auto ref = [&](int64_t i) { return ws.exp2[i] == kByTop ? (double)ws.top[i] : ws.exp2[i] * kLn2; };
      double most = -INFINITY;
      for (int j = 0; j < p.splits; ++j)
        if (ws.sum[l + j] != 0.0) most = fmax(most, ref(l + j));
      for (int j = 0; j < p.splits; ++j)
        if (ws.sum[l + j] != 0.0) s += ws.sum[l + j] * exp(ref(l + j) - most);
      lse = log(s) + most;
    }
    const double sc = (double)p.scores[r * p.beams + tid];
    sum[tid] = (isfinite(lse) && isfinite(sc)) ? lse : (double)NAN;
    sco[tid] = sc;
  }
  __syncthreads();
  auto entry = [&](int64_t l, int j, uint64_t& s, uint32_t& f) -> bool {  // candidate j of list l
    if (j >= ws.n[l0 + l]) return false;
    const int b = (int)(l / p.splits);
    if (isnan(sum[b])) return false;
    const Cand c = ws.cand[(l0 + l) * M + j];
    s = ordered(sco[b] + ((double)c.x - sum[b]));
    f = (uint32_t)((int64_t)b * p.vocab + c.t);
    return true;
  };
  // A threshold with at least M candidates not below it: the M-th largest of the
  // threads' best among the lists' first candidates (first few, where there are
  // fewer lists than M).
  const int first = (int)((M + NL - 1) / NL);
  uint64_t s, bs = 0;
  uint32_t f, bf = 0xffffffffu;
  int live = 0;
  for (int64_t e = tid; e < NL * first; e += kNT)
    if (entry(e / first, (int)(e % first), s, f) && before(s, f, bs, bf)) bs = s, bf = f;
  for (int64_t l = tid; l < NL; l += kNT)
    if (!isnan(sum[l / p.splits])) live += min(ws.n[l0 + l], M);
  hs[tid] = bs;
  hf[tid] = bf;
  atomicAdd(&total, min(live, 1 << 20));
  __syncthreads();
  if (bs) {
    int rank = 0;
    for (int j = 0; j < kNT; ++j) rank += before(hs[j], hf[j], bs, bf) ? 1 : 0;
    if (rank == M - 1) sT = bs;
  }
  __syncthreads();
  const int take = min(total, M);
  const uint64_t T0 = sT;  // 0: fewer than M threads have a candidate, so all are taken
  for (int64_t e = tid; e < NL * M; e += kNT)
    if (entry(e / M, (int)(e % M), s, f) && s >= T0) {
      const int at = atomicAdd(&cnt, 1);
      if (at < kPick) ks[at] = s, kf[at] = f;
    }
  __syncthreads();
  float* os = p.out_scores + r * M;
  int32_t* op = p.out_parent + r * M;
  int32_t* ot = p.out_token + r * M;
  auto put = [&](int at, double score, uint32_t flat) {
    os[at] = (float)score;
    op[at] = (int32_t)(flat / (uint64_t)p.vocab);
    ot[at] = (int32_t)(flat % (uint64_t)p.vocab);
  };
  if (cnt <= kPick) {
    const int n = cnt;
    for (int c = tid; c < n; c += kNT) {
      const uint64_t ms = ks[c];
      const uint32_t mf = kf[c];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += before(ks[j], kf[j], ms, mf) ? 1 : 0;
      if (rank < M) put(rank, unordered(ms), mf);
    }
  } else {
    // More at the threshold than the list holds: one after the other, the best of those after the last one.
    uint64_t ls = 0xffffffffffffffffull;
    uint32_t lf = 0;
    bool any = false;
    for (int i = 0; i < take; ++i) {
      bs = 0, bf = 0xffffffffu;
      for (int64_t e = tid; e < NL * M; e += kNT)
        if (entry(e / M, (int)(e % M), s, f) && (!any || before(ls, lf, s, f)) && before(s, f, bs, bf)) bs = s, bf = f;
      __syncthreads();
      hs[tid] = bs;
      hf[tid] = bf;
      __syncthreads();
      ls = 0, lf = 0xffffffffu;
      for (int j = 0; j < kNT; ++j)
        if (before(hs[j], hf[j], ls, lf)) ls = hs[j], lf = hf[j];
      any = true;
      if (tid == 0) put(i, unordered(ls), lf);
    }
  }
  // Fewer finite candidates than n_best: tokens that score -inf, in the order of their index.
  if (take < M && tid < 32) {
    int at = take;
    for (int b = 0; b < p.beams && at < M; ++b) {
      const bool dead = isnan(sum[b]);
      for (int64_t t0 = 0; t0 < p.vocab && at < M; t0 += 32) {
        const int64_t t = t0 + tid;
        const bool yes = t < p.vocab && (dead || is_masked<T>(p, r * p.beams + b, t));
        const unsigned all = __ballot_sync(0xffffffffu, yes);
        const int mine = at + __popc(all & ((1u << tid) - 1u));
        if (yes && mine < M) put(mine, -INFINITY, (uint32_t)((int64_t)b * p.vocab + t));
        at += __popc(all);
      }
    }
  }
}

template <typename T, int VE>
cudaError_t scan(const BeamParams& p, cudaStream_t st) {
  const unsigned grid = (unsigned)(p.batch * p.beams * p.splits);
  k_beam_scan<T, VE, 32><<<grid, kNT, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t select(const BeamParams& p, cudaStream_t st) {
  // The widest load that every row's alignment allows (equal rows must sum in the same order, so all rows load alike).
  const uintptr_t a = (uintptr_t)p.logits | (uintptr_t)(p.row_stride * (int64_t)sizeof(T));
  cudaError_t e;
  if (a % 16 == 0) e = scan<T, 16 / (int)sizeof(T)>(p, st);
  else e = scan<T, 1>(p, st);
  if (e != cudaSuccess) return e;
  constexpr int smem = 12 * kPick;
  k_beam_pick<T><<<(unsigned)p.batch, kNT, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Elements of a slice: 32 words of 256 threads.
int beam_splits(int dtype, int64_t vocab) {
  const int64_t n = (int64_t)kNT * 32 * (dtype == LQ_F32 ? 1 : 2);
  return (int)((vocab + n - 1) / n);
}

// Enough for any type: as many slices as fp32 logits take.
size_t beam_workspace(int64_t batch, int beams, int64_t vocab, int n_best) {
  const int64_t lists = batch * beams * beam_splits(LQ_F32, vocab);
  return up256(8 * lists) + 3 * up256(4 * lists) + up256(sizeof(Cand) * lists * n_best);
}

cudaError_t launch_beam_select(const BeamParams& p, cudaStream_t st) {
  if (p.dtype == LQ_BF16) return select<__nv_bfloat16>(p, st);
  if (p.dtype == LQ_F16) return select<__half>(p, st);
  return select<float>(p, st);
}

}  // namespace lqi
