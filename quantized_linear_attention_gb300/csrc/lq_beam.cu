// The selection of beam search (sm_103a): for each request the n_best of
//   scores[b] + logits[b][t] - log sum_t' exp(logits[b][t'])
// over its beams b and tokens t, equal scores to the lowest b * vocab + t.
//
// Two kernels. k_beam_scan reads the logits once, the only large
// traffic: a CTA holds one slice of one row in registers, sums its
// exponentials and keeps its n_best largest logits. Inside a row the order of the
// scores is the order of the logits, so no score is needed there. k_beam_pick
// joins a request's slices: log-sum-exps and scores in 64 bits, because the
// order of nearly equal candidates of different beams hangs on their rows' sums. The scan's sums are good to
// 3e-6 at worst (1e-8 to 1e-7 as a rule); where two candidates of different beams among the n_best lie closer than
// that leaves certain, their rows' sums are taken again, to 1e-10, and the choice is made anew.
//
// The sum of a slice: with m = ceil(max * log2 e), a whole number, each term is
// 2^(x log2 e - m), its exponent formed by two fmas from a two-part log2 e (two
// roundings, relative to the exponent itself). Threads' sums join as whole numbers of
// 2^-40 and slices by shifts: exact, and 64-bit floating point is slow here. A slice's sum stays below
// 2^55, but a row of 2^24 terms of 1 passes 2^64: slices join in two words, their upper and lower 32 bits.
// Rows with equal contents sum in the same order whatever their place in memory, so equal hypotheses tie exactly.
//
// The n_best of a slice without a sort: 64 groups of four threads give their
// maxima; at least n_best elements are not below the n_best-th largest of those
// (each of the n_best groups has one), so the few elements at or above it are
// collected and ranked by counting. At 16,384 elements and n_best = 16 they are
// about 18. Where ties make them more than the list holds, a bisection over
// (value, index) finds the exact n_best-th key.
//
// Measured at 64 x 8 x 131,071 bf16: 52 us, the scan 38 (134 MB, 52% of the copy
// bandwidth), the choice about 13. The scan is bound by instructions: 62% of the issue
// slots at half of the warps, the exponentials' unit alone 16 us (without them 42 us in
// all). Smaller slices were slower, 64 us, by what every slice does once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "lq_device.cuh"
#include "lq_internal.h"

namespace lqi {

namespace {

constexpr int kNT = 256;
constexpr int kWords = 32;   // words of a slice in a thread's registers
constexpr double kLn2 = 0.693147180559945309417;
constexpr float kL2Ehi = 1.44269502162933349609375f, kL2Elo = 1.92596299e-8f;  // log2 e in two parts
constexpr int kList = 512;   // candidates a slice collects before ranking
constexpr int kFours = 256;  // groups of four words with one among them
constexpr int kPick = 2048;  // candidates a request collects before ranking

struct Cand {
  float x;
  int32_t t;
};

// Workspace, per (row, slice): the sum of its exponentials in whole numbers of 2^-40 (kNotFinite where it is not
// finite), what it is relative to, and n_best candidates (x = -inf: none).
constexpr int32_t kByTop = INT32_MAX;
constexpr uint64_t kNotFinite = ~0ull;
struct Ws {
  uint64_t* sum;
  int32_t* exp2;  // the sum stands for sum * 2^exp2, or where this is kByTop
  float* top;     // for sum * e^top
  Cand* cand;
};

__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

__host__ __device__ inline Ws carve(void* ws, int64_t lists) {
  char* c = static_cast<char*>(ws);
  Ws w;
  w.sum = reinterpret_cast<uint64_t*>(c);
  c += up256(8 * lists);
  w.exp2 = reinterpret_cast<int32_t*>(c);
  c += up256(4 * lists);
  w.top = reinterpret_cast<float*>(c);
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
// An element's place in its row's order: larger logits first, then lower indices.
__device__ __forceinline__ uint64_t key_of(float x, int64_t t) {
  return ((uint64_t)ordered(x) << 32) | (0xffffffffu - (uint32_t)t);
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

// The larger of two words' elements, each by itself; a NaN gives way to a number (the sum meets it).
template <typename T>
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t max_words<float>(uint32_t a, uint32_t b) {
  return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}
template <>
__device__ __forceinline__ uint32_t max_words<__nv_bfloat16>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <>
__device__ __forceinline__ uint32_t max_words<__half>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A slice of a row: 32 words (of 32 bits) to a thread, VE elements to a load. Element i of
// thread t is element ((i / VE) * 256 + t) * VE + i % VE of the slice. (Slices a quarter the
// size were no faster even for four rows, and 12.1 -> 15.9 us for 256 rows of 32,000.)
// Loads of single 16-bit elements need more registers than four CTAs on an SM leave: three
// take 80 us at 64 x 8 x 131,071, four 94 (spills), two 91.
template <typename T, int VE>
__global__ void __launch_bounds__(kNT, VE == 1 && sizeof(T) == 2 ? 3 : 4) k_beam_scan(BeamParams p) {
  constexpr int W = kWords;
  constexpr int EPW = 4 / (int)sizeof(T), E = W * EPW;  // elements per word, per thread
  __shared__ float gmax[64];
  __shared__ uint64_t wsum[8];
  __shared__ int bad;
  __shared__ uint64_t list[kList];
  __shared__ uint4 fourw[kFours];
  __shared__ uint16_t fours[kFours];
  __shared__ float sT;
  __shared__ int cnt, nfour;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / (unsigned)p.splits;
  const int64_t base = (int64_t)(blockIdx.x % (unsigned)p.splits) * (kNT * E);
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride + base;
  const int left = (int)min(p.vocab - base, (int64_t)(kNT * E));  // elements of the slice
  if (tid == 0) cnt = nfour = bad = 0;
  cudaTriggerProgrammaticLaunchCompletion();  // k_beam_pick may be set up; it waits for this grid's end

  uint32_t w[W];
  auto at = [&](int i) { return ((i / VE) * kNT + tid) * VE + i % VE; };
  auto bits_of = [&](int i) -> uint32_t {  // one element's bits, -inf past the end
    const int e = at(i);
    if (e >= left) return Elem<T>::kNegInf;
    if (sizeof(T) == 4) return reinterpret_cast<const uint32_t*>(x)[e];
    return reinterpret_cast<const uint16_t*>(x)[e];
  };
  constexpr int WPV = VE / EPW;  // words per load (0: less than a word)
  if (WPV > 0) {
#pragma unroll
    for (int j = 0; j < W / (WPV ? WPV : 1); ++j) {
      const int e0 = (j * kNT + tid) * VE;
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
          w[j * WPV + c] = EPW == 1 ? bits_of(i) : (bits_of(i) | (bits_of(i + 1) << 16));
        }
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < W; ++c) w[c] = bits_of(2 * c) | (bits_of(2 * c + 1) << 16);
  }

  uint32_t mw = w[0];
#pragma unroll
  for (int c = 1; c < W; ++c) mw = max_words<T>(mw, w[c]);
  float mx = Elem<T>::get(&mw, 0);
  if (EPW == 2) mx = fmaxf(mx, Elem<T>::get(&mw, EPW - 1));
  if (!(mx >= -INFINITY)) mx = -INFINITY;  // (all NaN)
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
  // A whole exponent of two not below the largest term's; nothing finite in the slice: any will do.
  // Past 2^20 the exponents' own rounding would show: then relative to the largest logit itself.
  const bool byTop = top < INFINITY && top > -INFINITY && fabsf(top) > 1048576.0f;
  const float m = (!byTop && fabsf(top) < INFINITY) ? ceilf(__fmul_rn(top, kL2Ehi)) : 0.0f;
  float sum = 0.0f;
  if (!byTop) {
    f32x2 s2[2] = {0ull, 0ull};
    const f32x2 hi2 = f2_dup(kL2Ehi), lo2 = f2_dup(kL2Elo), m2 = f2_dup(-m);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const f32x2 v = f2_pack(Elem<T>::get(w, i), Elem<T>::get(w, i + 1));
      // (-inf: the first fma is -inf and the second keeps it)
      float t0, t1;
      f2_unpack(f2_fma(v, lo2, f2_fma(v, hi2, m2)), t0, t1);
      s2[(i >> 1) & 1] = f2_add(s2[(i >> 1) & 1], f2_pack(ex2(t0), ex2(t1)));
    }
    float t0, t1;
    f2_unpack(f2_add(s2[0], s2[1]), t0, t1);
    sum = __fadd_rn(t0, t1);
  } else {
#pragma unroll 1
    for (int i = 0; i < E; ++i) {
      if (at(i) >= left) continue;
      const float d = __fsub_rn((float)x[at(i)], top);
      sum = __fadd_rn(sum, ex2(__fmaf_rn(d, kL2Elo, __fmul_rn(d, kL2Ehi))));
    }
  }
  __syncthreads();
  // The few elements at or above the threshold, read again (they are in cache).
  const float T0 = sT;
  // Four words at a time; those with a hit are listed, and looked through by all threads together.
  constexpr int G = 4 * EPW;
#pragma unroll
  for (int j = 0; j < W / 4; ++j) {
    const uint32_t g = max_words<T>(max_words<T>(w[4 * j], w[4 * j + 1]), max_words<T>(w[4 * j + 2], w[4 * j + 3]));
    const float v = fmaxf(Elem<T>::get(&g, 0), Elem<T>::get(&g, EPW - 1));
    if (v >= T0 && v > -INFINITY) {
      const int f = atomicAdd(&nfour, 1);
      if (f < kFours) {
        fours[f] = (uint16_t)(j * kNT + tid);
        fourw[f] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      }
    }
  }
  uint64_t s = __float2ull_rn(__fmul_rn(sum, 1099511627776.f));  // (a thread has at most 64 terms of at most 1)
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) wsum[warp] = s;
  if (!(sum < 1e30f)) bad = 1;
  __syncthreads();
  for (int h = tid; h < min(nfour, kFours) * G; h += kNT) {
    const int f = fours[h / G], i = f / kNT * G + h % G;  // element i of thread f % kNT
    const int e = ((i / VE) * kNT + f % kNT) * VE + i % VE;
    const float v = (float)reinterpret_cast<const T*>(fourw)[h];
    if (v >= T0 && v > -INFINITY) {
      const int at1 = atomicAdd(&cnt, 1);
      if (at1 < kList) list[at1] = key_of(v, base + e);
    }
  }
  __syncthreads();
  int n = cnt;
  if (n > kList || nfour > kFours) {
    // Too many at or above the group threshold: the largest key with at least n_best keys not below it, bit by bit.
    __shared__ int above;
    uint64_t key = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t want = key | (1ull << bit);
      int c = 0;
      for (int i = 0; i < E; ++i) {
        const int e = at(i);
        const float v = e < left ? (float)x[e] : -INFINITY;
        c += (v > -INFINITY && key_of(v, base + e) >= want) ? 1 : 0;
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
    for (int i = 0; i < E; ++i) {
      const int e = at(i);
      const float v = e < left ? (float)x[e] : -INFINITY;
      if (v > -INFINITY && key_of(v, base + e) >= key) {
        const int at1 = atomicAdd(&cnt, 1);
        if (at1 < kList) list[at1] = key_of(v, base + e);
      }
    }
    __syncthreads();
    n = min(cnt, kList);
  }
  const Ws ws = carve(p.ws, p.batch * p.beams * p.splits);
  const int64_t l = blockIdx.x;
  Cand* out = ws.cand + l * p.n_best;
  for (int c = tid; c < n; c += kNT) {
    const uint64_t mine = list[c];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += list[j] > mine ? 1 : 0;
    if (rank < p.n_best) out[rank] = Cand{unordered((uint32_t)(mine >> 32)), (int32_t)(0xffffffffu - (uint32_t)mine)};
  }
  for (int c = n + tid; c < p.n_best; c += kNT) out[c] = Cand{-INFINITY, 0};
  if (tid == 0) {
    uint64_t t = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) t += wsum[j];
    ws.sum[l] = bad ? kNotFinite : t;
    ws.exp2[l] = byTop ? kByTop : (int32_t)m;
    ws.top[l] = top;
  }
}

// A score's place in the order: larger keys first, then lower flat indices.
__device__ __forceinline__ bool before(uint64_t s1, uint32_t f1, uint64_t s2, uint32_t f2) {
  return s1 > s2 || (s1 == s2 && f1 < f2);
}

// log of a positive finite s to about 1e-13 with few 64-bit steps (64-bit arithmetic is slow here, and the sums are
// good to 1e-10 at best): s = 2^k m, m in [0.703, 1.406); with r near 1/m from a table of 32, log m = log(1 + u) - log r,
// u = r m - 1, |u| < 0.017, by its series (table-driven, after P. Tang, "Table-driven implementation of the logarithm
// function", 1990).
__constant__ double kLog[32][2] = {
    {1.4003, -0.33668649937959438},
    {1.3585, -0.3063811498842654},
    {1.3192, -0.27702549226325202},
    {1.2820, -0.24842135849847832},
    {1.2469, -0.22066047102040334},
    {1.2136, -0.19359114905218544},
    {1.1821, -0.16729251777419415},
    {1.1522, -0.1416731583161456},
    {1.1237, -0.11662681193171956},
    {1.0967, -0.092305670784026142},
    {1.0708, -0.068406032664060368},
    {1.0462, -0.045164551954373661},
    {1.0227, -0.022446188829829995},
    {1.0002, -0.00019998000266624471},
    {0.9787, 0.021530118550363214},
    {0.9581, 0.042803122325309445},
    {0.9384, 0.063578981642871332},
    {0.9194, 0.084033995610009446},
    {0.9012, 0.10402807042404769},
    {0.8837, 0.12363764045817827},
    {0.8669, 0.14283164910754234},
    {0.8507, 0.16169573900029838},
    {0.8351, 0.18020380082295337},
    {0.8200, 0.19845093872383832},
    {0.8055, 0.216292076365108},
    {0.7915, 0.23382539966107024},
    {0.7780, 0.25102875480374542},
    {0.7649, 0.26801017265431665},
    {0.7522, 0.28475303294590104},
    {0.7400, 0.30110509278392161},
    {0.7282, 0.31717954324080405},
    {0.7167, 0.3330979359822635}};
__device__ __forceinline__ double log_of(double s) {
  if (!(s > 0.0 && s < INFINITY)) return log(s);
  int hi = __double2hiint(s), k = (hi >> 20) - 1023;
  double m = __hiloint2double((hi & 0xfffff) | (1023 << 20), __double2loint(s));  // [1, 2)
  if (m >= 1.40625) m *= 0.5, ++k;
  const int i = min(31, (int)(((float)m - 0.703125f) * (32.0f / 0.703125f)));
  const double u = fma(m, kLog[i][0], -1.0);
  double t = fma(u, -1.0 / 6.0, 1.0 / 5.0);
  t = fma(u, t, -1.0 / 4.0);
  t = fma(u, t, 1.0 / 3.0);
  t = fma(u, t, -0.5);
  return fma((double)k, kLn2, kLog[i][1] + fma(u * u, t, u));
}

// How far a row's sum may be off, relative to it: 2^-22 for each term's ex2, two roundings of 2^-24 |t| for its exponent
// t (over a row's terms, as they weigh, |t| is at most log2 vocab + 1), 18 roundings in a thread's sum, and a last one
// for what whole numbers of 2^-40 leave off. Relative to the largest logit: three roundings of t, 66 in the sum.
__device__ __forceinline__ float sum_bound(int64_t vocab, bool byTop) {
  const float bits = (float)(65 - __clzll(vocab));
  return 5.9604645e-8f * (byTop ? 71.f + 2.08f * bits : 23.f + 1.39f * bits);
}

// The log-sum-exp of a row to 1e-10, by all threads of the CTA, for rows whose order the scan's sums leave open. In pairs
// of 32-bit numbers throughout: d = x - top with its rounding; d = k ln2 / 64 + h + l, k whole, |h| < 0.0055 (reduction in
// two parts, after W. Cody and W. Waite, 1980); e^d = 2^(k / 64) (1 + h + (l + h^2 / 2 + h^3 / 6 + h^4 / 24)), the power
// from a table in two parts; sums by the two-sum of D. Knuth. 26 instructions a term: 131,071 terms take 50 us.
template <typename T>
__device__ __noinline__ double row_lse(const BeamParams& p, const float* tops, const T* x, unsigned char* dyn) {
  float2* table = reinterpret_cast<float2*>(dyn);
  float* wtop = reinterpret_cast<float*>(dyn + 512);
  double* wsum = reinterpret_cast<double*>(dyn + 576);
  const int tid = threadIdx.x;
  float top = -INFINITY;
  for (int j = tid; j < p.splits; j += kNT) top = fmaxf(top, tops[j]);
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) wtop[tid >> 5] = top;
  if (tid < 64) {
    const double t = exp2(tid / 64.0);
    table[tid] = make_float2((float)t, (float)(t - (double)(float)t));
  }
  __syncthreads();
  for (int w = 0; w < kNT / 32; ++w) top = fmaxf(top, wtop[w]);
  const f32x2 t2 = f2_dup(top), per = f2_dup(92.3324826f), magic = f2_dup(12582912.f);
  const f32x2 c1 = f2_dup(-0x1.63p-7f), c2 = f2_dup(0x1.bd0106p-19f);  // -ln2 / 64 in two parts, the first of 9 bits
  f32x2 S = 0ull, C = 0ull;
  auto add = [&](float x0, float x1) {
    const bool on0 = __fsub_rn(x0, top) > -87.f, on1 = __fsub_rn(x1, top) > -87.f;  // the rest is below 2^-125
    const f32x2 v = f2_pack(on0 ? x0 : top, on1 ? x1 : top);
    const f32x2 d = f2_sub(v, t2), y = f2_sub(d, v);
    const f32x2 e = f2_sub(f2_sub(v, f2_sub(d, y)), f2_add(t2, y));  // d + e = x - top
    const f32x2 kf = f2_fma(d, per, magic), k = f2_sub(kf, magic);
    const f32x2 r = f2_fma(k, c1, d), rl = f2_fma(k, c2, e);
    const f32x2 h = f2_add(r, rl), z = f2_sub(h, r), l = f2_add(f2_sub(r, f2_sub(h, z)), f2_sub(rl, z));
    f32x2 q = f2_fma(h, f2_fma(h, f2_dup(1.f / 24.f), f2_dup(1.f / 6.f)), f2_dup(0.5f));
    q = f2_fma(f2_mul(h, h), q, l);
    const int i0 = (int)((uint32_t)kf - 0x4b400000u), i1 = (int)((uint32_t)(kf >> 32) - 0x4b400000u);
    const float2 u0 = table[i0 & 63], u1 = table[i1 & 63];
    const f32x2 th = f2_pack(u0.x, u1.x), tl = f2_pack(u0.y, u1.y);
    const f32x2 scale = f2_bits(on0 ? (uint32_t)((i0 >> 6) + 127) << 23 : 0u, on1 ? (uint32_t)((i1 >> 6) + 127) << 23 : 0u);
    f32x2 a = f2_fma(th, h, th);
    f32x2 b = f2_add(f2_fma(th, h, f2_sub(th, a)), f2_fma(th, q, f2_fma(tl, h, tl)));
    a = f2_mul(a, scale), b = f2_mul(b, scale);  // (exact)
    const f32x2 s1 = f2_add(S, a), w = f2_sub(s1, S);
    C = f2_add(C, f2_add(f2_add(f2_sub(S, f2_sub(s1, w)), f2_sub(a, w)), b));
    S = s1;
  };
  int64_t i = tid;
#pragma unroll 1
  for (; i + 7 * kNT < p.vocab; i += 8 * kNT) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)x[i + j * kNT];
#pragma unroll
    for (int j = 0; j < 8; j += 2) add(v[j], v[j + 1]);
  }
#pragma unroll 1
  for (; i < p.vocab; i += kNT) add((float)x[i], -INFINITY);
  float s0, s1, e0, e1;
  f2_unpack(S, s0, s1);
  f2_unpack(C, e0, e1);
  double sum = ((double)s0 + (double)s1) + ((double)e0 + (double)e1);
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((tid & 31) == 0) wsum[tid >> 5] = sum;
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < kNT / 32; ++w) sum += wsum[w];
  __syncthreads();
  return (double)top + log_of(sum);
}

// What the choice knows of a request's hypotheses.
struct Rows {
  double lse[kMaxBeams], score[kMaxBeams];  // log-sum-exps, scores so far
  uint64_t up[kMaxBeams], low[kMaxBeams];   // sums in units of 2^-40, 2^32 up + low (0 also where one is not finite),
  double ref[kMaxBeams];                    // and what they are relative to: an exponent of two, or (byTop) a logit
  double open;                              // how far apart the scores of two beams' candidates have to be
  float cut[kMaxBeams];
  bool alive[kMaxBeams], byTop[kMaxBeams];
  uint32_t settled, which;  // beams whose sums were taken again, and are to be
};

// Where candidates of different beams lie closer than `open` among the M best of n (more than kPick: anywhere), their
// rows' sums are taken again. False if none is.
template <typename T>
__device__ __noinline__ bool take_again(const BeamParams& p, int64_t r, int n, Rows& rows, const float* tops,
                                        unsigned char* dyn) {
  const uint64_t* ks = reinterpret_cast<const uint64_t*>(dyn);
  const uint32_t* kf = reinterpret_cast<const uint32_t*>(dyn + 8 * kPick);
  const int tid = threadIdx.x;
  if (tid == 0) rows.which = 0;
  __syncthreads();
  // Sums that agree in every bit are equal rows', whose errors are equal too.
  auto both = [&](int b1, int b2) -> uint32_t {
    const uint32_t open = ~rows.settled & (1u << b1 | 1u << b2);
    if (b1 == b2 || !rows.alive[b1] || !rows.alive[b2]) return 0;
    return (open >> b1 & open >> b2 & 1) && rows.up[b1] == rows.up[b2] && rows.low[b1] == rows.low[b2] &&
                   rows.ref[b1] == rows.ref[b2]
               ? 0
               : open;
  };
  uint32_t which = 0;
  if (n <= kPick) {
#pragma unroll 1
    for (int c = tid; c < n; c += kNT) {
      const uint64_t ms = ks[c], low = ordered(unordered(ms) - rows.open), span = ordered(unordered(ms) + rows.open) - low;
      const uint32_t mf = kf[c], V = (uint32_t)p.vocab, b = mf / V;
      int rank = 0;
      uint32_t near = 0;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        rank += before(ks[j], kf[j], ms, mf) ? 1 : 0;
        if (ks[j] - low <= span && kf[j] - b * V >= V) near |= both(b, kf[j] / V);
      }
      if (rank < p.n_best) which |= near;
    }
  } else if (tid < p.beams) {
    for (int b = 0; b < p.beams; ++b) which |= both(tid, b);
  }
  if (which) atomicOr(&rows.which, which);
  __syncthreads();
  which = rows.which;
#pragma unroll 1
  for (int b = 0; b < p.beams; ++b)
    if (which >> b & 1) {
      const T* x = static_cast<const T*>(p.logits) + (r * p.beams + b) * p.row_stride;
      const double lse = row_lse<T>(p, tops + b * p.splits, x, dyn);
      if (tid == 0) rows.lse[b] = lse, rows.settled |= 1u << b;
    }
  return which != 0;
}

template <typename T>
__device__ __forceinline__ bool is_masked(const BeamParams& p, int64_t row, int64_t t) {
  const T x = static_cast<const T*>(p.logits)[row * p.row_stride + t];
  return (float)x == -INFINITY;
}

// One CTA per request. It runs once through little data, so it is bound by latencies, those of its own
// instructions' fetches among them: loops stay rolled.
template <typename T>
__global__ void __launch_bounds__(kNT) k_beam_pick(const __grid_constant__ BeamParams p) {
  extern __shared__ __align__(16) unsigned char dyn[];
  uint64_t* ks = reinterpret_cast<uint64_t*>(dyn);
  uint32_t* kf = reinterpret_cast<uint32_t*>(dyn + 8 * kPick);
  Cand* sc = reinterpret_cast<Cand*>(dyn + 12 * kPick);  // the first kPick candidates
  __shared__ Rows rows;
  __shared__ uint64_t hs[kNT], sT;
  __shared__ uint32_t hf[kNT];
  __shared__ int cnt;
  const int tid = threadIdx.x, lane = tid & 31, M = p.n_best;
  const int64_t r = blockIdx.x;
  const int NL = p.beams * p.splits, NC = NL * M;  // (below 2^25: a slice has 8,192 tokens at least)
  const float mine = tid < p.beams ? p.scores[r * p.beams + tid] : 0.f;
  if (tid == 0) cnt = 0, sT = 0, rows.settled = 0;
  cudaGridDependencySynchronize();
  const Ws ws = carve(p.ws, p.batch * p.beams * p.splits);
  const int64_t l0 = r * NL;  // the request's first list
  const Cand* gc = ws.cand + l0 * M;
#pragma unroll 2
  for (int e = tid; e < min(NC, kPick); e += kNT) sc[e] = gc[e];
  // A warp joins a hypothesis' slices by shifts; the logarithms are then taken side by side in one warp.
  for (int b = tid >> 5; b < p.beams; b += kNT / 32) {
    const int64_t l = l0 + b * p.splits;
    int e = INT32_MIN;
    bool nf = false;
    for (int j = lane; j < p.splits; j += 32) {
      const uint64_t x = ws.sum[l + j];
      if (x) e = max(e, ws.exp2[l + j]);
      nf |= x == kNotFinite;
    }
    e = __reduce_max_sync(0xffffffffu, e);
    uint64_t up = 0, low = 0;  // 2^18 slices at most: neither sum passes 2^50
    auto join = [&](uint64_t x) { up += x >> 32, low += x & 0xffffffffu; };
    double base = 0.0;
    if (e != kByTop) {
      for (int j = lane; j < p.splits; j += 32) {
        const uint64_t x = ws.sum[l + j];
        if (x && e - ws.exp2[l + j] < 64) join(x >> (e - ws.exp2[l + j]));
      }
    } else {  // logits past 2^20
      auto at = [&](int64_t i) { return ws.exp2[i] == kByTop ? (double)ws.top[i] : ws.exp2[i] * kLn2; };
      base = -INFINITY;
      for (int j = 0; j < p.splits; ++j)
        if (ws.sum[l + j]) base = fmax(base, at(l + j));
      for (int j = lane; j < p.splits; j += 32)
        if (ws.sum[l + j]) join((uint64_t)((double)ws.sum[l + j] * exp(at(l + j) - base)));
    }
    for (int o = 16; o; o >>= 1) {
      up += __shfl_xor_sync(0xffffffffu, up, o);
      low += __shfl_xor_sync(0xffffffffu, low, o);
    }
    nf = __any_sync(0xffffffffu, nf);
    if (lane == 0) {
      rows.up[b] = nf ? 0 : up;
      rows.low[b] = nf ? 0 : low;
      rows.ref[b] = e == kByTop ? base : (double)e;
      rows.byTop[b] = e == kByTop;
    }
  }
  __syncthreads();
  if (tid < 32) {
    const bool mineTop = tid < p.beams && rows.byTop[tid], byTop = __any_sync(0xffffffffu, mineTop);
    if (tid < p.beams) {
      const double sum = fma((double)rows.up[tid], 0x1p-8, (double)rows.low[tid] * 0x1p-40);
      const double x = log_of(sum);  // (of zero: -inf)
      rows.lse[tid] = x + (mineTop ? rows.ref[tid] : rows.ref[tid] * kLn2);
      rows.score[tid] = (double)mine;
      rows.alive[tid] = isfinite(mine) && sum != 0.0;
    }
    if (tid == 0) rows.open = p.beams > 1 ? 2.0 * (double)sum_bound(p.vocab, byTop) : 0.0;
  }
  __syncthreads();
  auto look = [&](int e, uint64_t& s, uint32_t& f) -> bool {  // candidate e % M of list e / M
    const Cand c = e < kPick ? sc[e] : gc[e];
    const int b = e / (M * p.splits);
    if (!(c.x > -INFINITY) || !rows.alive[b] || c.x < rows.cut[b]) return false;
    s = ordered(rows.score[b] + ((double)c.x - rows.lse[b]));
    f = (uint32_t)((int64_t)b * p.vocab + c.t);
    return true;
  };
  const int first = (M + NL - 1) / NL;
  uint64_t s, bs;
  uint32_t f, bf;
  int take;
  float* os = p.out_scores + r * M;
  int32_t* op = p.out_parent + r * M;
  int32_t* ot = p.out_token + r * M;
  auto put = [&](int at, double score, uint32_t b, uint32_t flat) {  // (beams x vocab < 2^31)
    os[at] = (float)score;
    op[at] = (int32_t)b;
    ot[at] = (int32_t)(flat - b * (uint32_t)p.vocab);
  };
#pragma unroll 1
  for (;;) {  // once, but where sums are taken again
    if (tid < p.beams) rows.cut[tid] = -INFINITY;
    __syncthreads();
    // A threshold with at least M candidates not below it: the M-th largest of the
    // threads' best among the lists' first candidates (first few, where there are
    // fewer lists than M).
    bs = 0, bf = 0xffffffffu;
#pragma unroll 1
    for (int h = tid; h < NL * first; h += kNT)
      if (look(h / first * M + h % first, s, f) && before(s, f, bs, bf)) bs = s, bf = f;
    hs[tid] = bs;
    hf[tid] = bf;
    __syncthreads();
    if (bs) {
      const int n = min(kNT, NL * first);
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank += before(hs[j], hf[j], bs, bf) ? 1 : 0;
      // Those within `open` below it may yet come before it.
      if (rank == M - 1) sT = ordered(unordered(bs) - rows.open);
    }
    __syncthreads();
    const uint64_t T0 = sT;  // 0: fewer than M threads have a candidate, so all are taken
    // Per hypothesis the logit that the threshold stands for, rounded down past every rounding of a score: most
    // candidates are told by it without 64-bit arithmetic.
    if (tid < p.beams && T0 && rows.alive[tid]) {
      const double t = unordered(T0), slack = 4e-15 * (fabs(t) + fabs(rows.score[tid]) + fabs(rows.lse[tid]));
      rows.cut[tid] = __double2float_rd((t - rows.score[tid]) + rows.lse[tid] - slack);
    }
    __syncthreads();
#pragma unroll 1
    for (int e = tid; e < NC; e += kNT)
      if (look(e, s, f) && s >= T0) {
        const int at = atomicAdd(&cnt, 1);
        if (at < kPick) ks[at] = s, kf[at] = f;
      }
    __syncthreads();
    const int n = cnt;
    take = min(n, M);
    // In their order, a step from one beam's to another's within `open` says that there may be a closer look to take.
    bool close = n > kNT;
    if (n <= kPick) {
      for (int c = tid; c < n; c += kNT) {
        const uint64_t ms = ks[c];
        const uint32_t mf = kf[c];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += before(ks[j], kf[j], ms, mf) ? 1 : 0;
        const double score = unordered(ms);
        const uint32_t b = mf / (uint32_t)p.vocab;
        if (rank < M) put(rank, score, b, mf);
        if (rank < kNT) hs[rank] = ms, hf[rank] = b;
      }
      __syncthreads();
      if (tid + 1 < min(n, kNT) && hf[tid] != hf[tid + 1])
        close = unordered(hs[tid]) - unordered(hs[tid + 1]) <= rows.open;
    }
    if (!__syncthreads_or(close) || !take_again<T>(p, r, n, rows, ws.top + l0, dyn)) break;
    __syncthreads();
    if (tid == 0) cnt = 0, sT = 0;
  }
  if (cnt > kPick) {
    // More at the threshold than the list holds: one after the other, the best of those after the last one.
    uint64_t ls = 0xffffffffffffffffull;
    uint32_t lf = 0;
    bool any = false;
    for (int i = 0; i < take; ++i) {
      bs = 0, bf = 0xffffffffu;
      for (int e = tid; e < NC; e += kNT)
        if (look(e, s, f) && (!any || before(ls, lf, s, f)) && before(s, f, bs, bf)) bs = s, bf = f;
      __syncthreads();
      hs[tid] = bs;
      hf[tid] = bf;
      __syncthreads();
      ls = 0, lf = 0xffffffffu;
      for (int j = 0; j < kNT; ++j)
        if (before(hs[j], hf[j], ls, lf)) ls = hs[j], lf = hf[j];
      any = true;
      if (tid == 0) put(i, unordered(ls), lf / (uint32_t)p.vocab, lf);
    }
  }
  // Fewer finite candidates than n_best: tokens that score -inf, in the order of their index.
  if (take < M && tid < 32) {
    int at = take;
    for (int b = 0; b < p.beams && at < M; ++b) {
      const bool dead = !rows.alive[b];
      for (int64_t t0 = 0; t0 < p.vocab && at < M; t0 += 32) {
        const int64_t t = t0 + tid;
        const bool yes = t < p.vocab && (dead || is_masked<T>(p, r * p.beams + b, t));
        const unsigned all = __ballot_sync(0xffffffffu, yes);
        const int mine = at + __popc(all & ((1u << tid) - 1u));
        if (yes && mine < M) put(mine, -INFINITY, b, (uint32_t)((int64_t)b * p.vocab + t));
        at += __popc(all);
      }
    }
  }
}

template <typename T, int VE>
cudaError_t scan(const BeamParams& p, cudaStream_t st) {
  const unsigned grid = (unsigned)(p.batch * p.beams * p.splits);
  k_beam_scan<T, VE><<<grid, kNT, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t select(const BeamParams& p, cudaStream_t st) {
  // The widest load that every row's alignment allows (equal rows must sum in the same order, so all rows load alike).
  // bf16, 64 x 8 rows with no gap between them: 45 us for 131,072 by 16 bytes, 50 for 131,070 by 4, 79 for 131,071 by 2.
  const uintptr_t a = (uintptr_t)p.logits | (uintptr_t)(p.row_stride * (int64_t)sizeof(T));
  cudaError_t e;
  if (a % 16 == 0) e = scan<T, 16 / (int)sizeof(T)>(p, st);
  else if (a % 4 == 0) e = scan<T, 4 / (int)sizeof(T)>(p, st);
  else e = scan<T, 1>(p, st);
  if (e != cudaSuccess) return e;
  // k_beam_pick is set up while the scan runs and waits for its end itself.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.batch);
  cfg.blockDim = dim3(kNT);
  cfg.dynamicSmemBytes = 20 * kPick;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_beam_pick<T>, p);
}

}  // namespace

int beam_splits(int dtype, int64_t vocab) {
  const int64_t n = (int64_t)kNT * kWords * (dtype == LQ_F32 ? 1 : 2);
  return (int)((vocab + n - 1) / n);
}

// Enough for any type: fp32 has the most slices.
size_t beam_workspace(int64_t batch, int beams, int64_t vocab, int n_best) {
  const int64_t lists = batch * beams * beam_splits(LQ_F32, vocab);
  return up256(8 * lists) + 2 * up256(4 * lists) + up256(sizeof(Cand) * lists * n_best);
}

cudaError_t launch_beam_select(const BeamParams& p, cudaStream_t st) {
  if (p.dtype == LQ_BF16) return select<__nv_bfloat16>(p, st);
  if (p.dtype == LQ_F16) return select<__half>(p, st);
  return select<float>(p, st);
}

}  // namespace lqi
