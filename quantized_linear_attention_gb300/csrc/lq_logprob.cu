// Log probabilities of given tokens, entropy and the most likely tokens of rows of logits (sm_103a):
//   lse = log sum_t e^x_t,   logprob = x_token - lse,   entropy = lse - sum_t p_t x_t.
//
// One kernel, bound by memory: the logits are read once. A cluster of 1 to 8 CTAs has a row, each a slice of it, and joins
// its parts through distributed shared memory. A thread keeps the largest logit it has met and, relative to that, the sum of
// the exponentials and the sum of the exponentials times their exponents; 32 elements at a time are compared with
// the largest, so the sums are rescaled by one rare branch.
//
// The n_top largest without a sort: after the first tile, and whenever eight times as many have gone by, the CTA looks at the
// maxima of 8 or 64 groups of its threads: at least n_top elements are not below the n_top-th largest of those. Elements at or
// above that bound are collected as they go by, a few times n_top in all; those that still are when the slice is through
// are ranked by counting. Where rising or very many equal logits make them more than the list holds, the slice is read
// again: a bisection over the values finds one that few enough are not below, or, where equal ones are too many, the exact
// n_top-th value, of which those with the lowest indices are taken in order.
//
// Measured: 4,096 rows of 50,257 bf16 82 us (74% of the copy bandwidth), bound by instructions: about six an element, and what a
// row costs once, a sixth of it; 128 rows of 131,071 fp32 with 20 alternatives 25 us (39%), the barriers of a slice's few
// tiles; one row of 32,000 7 us of latency.
#include <cooperative_groups.h>

#include <type_traits>

#include "lq_device.cuh"
#include "lq_seq.cuh"

namespace lqi {

namespace {

namespace cg = cooperative_groups;

constexpr int kNT = 256;
constexpr int kLoads = 4;     // 16-byte loads in flight
constexpr int kList = 1024;   // elements collected
constexpr int kRank = 512;    // of which at most so many are ranked
constexpr int kFew = 64;      // ranked without another look at the bound
constexpr int kMaxCluster = 8;

// Floats as unsigned numbers in the same order; -0 counts as +0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
// An element's place in its row's order: larger logits first, then lower indices. 0 is no element's.
__device__ __forceinline__ uint64_t key_of(float x, int64_t t) {
  return ((uint64_t)ordered(x) << 32) | (0xffffffffu - (uint32_t)t);
}
__device__ __forceinline__ float value_of(uint64_t key) { return unordered((uint32_t)(key >> 32)); }
__device__ __forceinline__ int32_t index_of(uint64_t key) { return (int32_t)(0xffffffffu - (uint32_t)key); }

// What a thread, warp or CTA knows of its elements: the largest, sum 2^u and sum 2^u u with u = (x - ref) log2 e.
struct Sum {
  float ref, s, e;
};

__device__ __forceinline__ Sum join(Sum a, Sum b) {
  if (b.ref > a.ref || b.ref != b.ref) {  // (a NaN goes on)
    const Sum t = a;
    a = b;
    b = t;
  }
  if (b.ref == -INFINITY) return a;
  const float u = __fmul_rn(__fsub_rn(b.ref, a.ref), kLog2E), f = ex2_approx(u);
  a.s = __fmaf_rn(f, b.s, a.s);
  // (u = -inf: nothing of b is left, and f u would not be a number)
  a.e = __fmaf_rn(f, __fmaf_rn(fmaxf(u, -1e30f), b.s, b.e), a.e);
  return a;
}

template <typename T>
struct Vec {
  static constexpr int N = 16 / (int)sizeof(T);
  T v[N];
};

// Largest of four or eight elements; a NaN comes through.
__device__ __forceinline__ float largest(const uint4& w, float) {
  return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)), max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
}
__device__ __forceinline__ float largest(const uint4& w, __nv_bfloat16) {
  uint32_t a, b;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
  return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
}
__device__ __forceinline__ float largest(const uint4& w, __half) {
  uint32_t a, b;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
  __half2 h;
  memcpy(&h, &a, 4);
  return max_nan(__low2float(h), __high2float(h));
}
__device__ __forceinline__ void floats4(const uint4& w, f32x2 (&f)[2], float) {
  f[0] = f2_bits(w.x, w.y);
  f[1] = f2_bits(w.z, w.w);
}
__device__ __forceinline__ void floats4(const uint4& w, f32x2 (&f)[4], __nv_bfloat16) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_bits(a[i] << 16, a[i] & 0xffff0000u);
}
__device__ __forceinline__ void floats4(const uint4& w, f32x2 (&f)[4], __half) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 h;
    memcpy(&h, &a[i], 4);
    f[i] = f2_pack(__low2float(h), __high2float(h));
  }
}
template <typename T>
__device__ __forceinline__ uint4 all_masked();
template <>
__device__ __forceinline__ uint4 all_masked<float>() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
template <>
__device__ __forceinline__ uint4 all_masked<__nv_bfloat16>() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
template <>
__device__ __forceinline__ uint4 all_masked<__half>() { return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u); }

struct Shared {
  uint64_t list[kList];
  uint64_t best[32];  // kMaxTop of this CTA's elements in order, 0 past the last
  float groups[64];
  Sum part[kNT / 32], all;
  float refs[kNT / 32];
  int warp_count[kNT / 32];
  float bound;
  int count, kept;
};
static_assert(kMaxTop <= 32 && kRank * 2 <= kList, "one warp joins the lists");

// Adds (c)(all threads of the CTA come here) and gives every thread the sum.
__device__ __forceinline__ int count_all(Shared& sm, int c) {
  c = __reduce_add_sync(0xffffffffu, c);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm.warp_count[threadIdx.x >> 5] = c;
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int w = 0; w < kNT / 32; ++w) n += sm.warp_count[w];
  return n;
}

// The k-th largest of the maxima of groups of threads (-inf if fewer have any): a warp each for k up to 8, else four threads.
__device__ __forceinline__ float new_bound(Shared& sm, float mine, int k) {
  const int tid = threadIdx.x;
  if (!(mine >= -INFINITY)) mine = -INFINITY;  // (a row with a NaN has no answer: any bound will do)
  mine = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, 1));
  mine = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, 2));
  if (k <= kNT / 32) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) mine = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, o));
    __syncthreads();
    if ((tid & 31) == 0) sm.groups[tid >> 5] = mine;
    __syncthreads();
    const float me = sm.groups[tid & 7];
    int rank = 0;
#pragma unroll
    for (int j = 0; j < kNT / 32; ++j) {
      const float y = sm.groups[j];
      rank += (y > me || (y == me && j < (tid & 7))) ? 1 : 0;
    }
    const unsigned at = __ballot_sync(0xffffffffu, rank == k - 1);
    return __shfl_sync(0xffffffffu, me, __ffs((int)at) - 1);
  }
  __syncthreads();
  if ((tid & 3) == 0) sm.groups[tid >> 2] = mine;
  __syncthreads();
  int rank = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int u = (tid & 3) * 16 + j;
    const float y = sm.groups[u];
    rank += (y > mine || (y == mine && u < (tid >> 2))) ? 1 : 0;
  }
  rank += __shfl_xor_sync(0xffffffffu, rank, 1);
  rank += __shfl_xor_sync(0xffffffffu, rank, 2);
  if ((tid & 3) == 0 && rank == k - 1) sm.bound = mine;
  __syncthreads();
  return sm.bound;
}

// The first `want` elements, in the order of their index, of the n from x on that are equal to `at`: their keys go to
// list[from ..]. `base`: x's index in the row. All threads of the CTA come here.
template <typename T>
__device__ __noinline__ void take_equal(Shared& sm, const T* x, int64_t n, int64_t base, uint32_t at, int from, int want) {
  const int tid = threadIdx.x;
  for (int64_t t0 = 0; want > 0 && t0 < n; t0 += kNT) {
    const bool hit = t0 + tid < n && ordered(to_f(x[t0 + tid])) == at;
    const unsigned m = __ballot_sync(0xffffffffu, hit);
    __syncthreads();
    if ((tid & 31) == 0) sm.warp_count[tid >> 5] = __popc(m);
    __syncthreads();
    int before = __popc(m & ((1u << (tid & 31)) - 1)), all = 0;
    for (int w = 0; w < kNT / 32; ++w) {
      if (w < (tid >> 5)) before += sm.warp_count[w];
      all += sm.warp_count[w];
    }
    if (hit && before < want) sm.list[from + before] = key_of(unordered(at), base + t0 + tid);
    from += min(all, want);
    want -= min(all, want);
  }
  __syncthreads();
}

// The slice again, for one whose list ran over: leaves at most kRank keys in list, the n_top largest of the slice's
// elements above -inf among them. Returns how many.
template <typename T>
__device__ __noinline__ int take_again(Shared& sm, const T* x, int64_t n, int64_t base, int k, float bound, float top) {
  const int tid = threadIdx.x;
  const uint32_t none = ordered(-INFINITY);
  // the largest value that at least k elements are not below, or one below it that at most kRank are not below
  uint32_t lo = max(ordered(bound), none + 1), hi = ordered(top);
  int above;
  auto count = [&](uint32_t v) {
    int c = 0;
    for (int64_t t = tid; t < n; t += kNT) c += ordered(to_f(x[t])) >= v ? 1 : 0;
    return count_all(sm, c);
  };
  above = count(lo);
  while (above > kRank && lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const int c = count(mid);
    if (c >= k) {
      lo = mid;
      above = c;
    } else {
      hi = mid - 1;
    }
  }
  // too many: they are equal ones for the most part, fewer than k are larger
  const bool equal = above > kRank;
  __syncthreads();
  if (tid == 0) sm.count = 0;
  __syncthreads();
  for (int64_t t = tid; t < n; t += kNT) {
    const float v = to_f(x[t]);
    if (equal ? ordered(v) > lo : ordered(v) >= lo) {
      const int i = atomicAdd(&sm.count, 1);
      if (i < kRank) sm.list[i] = key_of(v, base + t);
    }
  }
  __syncthreads();
  const int c = min(sm.count, kRank);
  if (!equal) return c;
  take_equal(sm, x, n, base, lo, c, k - c);
  return min(k, kRank);
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kNT) k_logprob(LogprobParams p, int cluster) {
  constexpr int N = Vec<T>::N, P = N / 2;
  __shared__ Shared sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)cluster);
  const int64_t r = blockIdx.x / (unsigned)cluster;
  const T* const x = static_cast<const T*>(p.logits) + r * p.row_stride;
  // the row: up to N - 1 elements before the first 16 bytes, whole vectors, up to N - 1 after; this CTA's vectors
  const int64_t head = min(p.vocab, (int64_t)(((16 - ((uintptr_t)x & 15)) & 15) / sizeof(T)));
  const int64_t vecs = (p.vocab - head) / N, tail = p.vocab - head - vecs * N;
  const int64_t v0 = vecs * rank / cluster, v1 = vecs * (rank + 1) / cluster;
  const uint4* const body = reinterpret_cast<const uint4*>(x + head);
  // the slice in elements, for what reads it again
  const int64_t e0 = rank == 0 ? 0 : head + v0 * N, e1 = rank == cluster - 1 ? p.vocab : head + v1 * N;
  if (TOP && tid == 0) {
    sm.bound = -INFINITY;
    sm.count = sm.kept = 0;
  }
  Sum m = {-INFINITY, 0.0f, 0.0f};
  f32x2 s2 = 0ull, e2 = 0ull;
  float top = -INFINITY, bound = -INFINITY;  // largest so far; what is collected

  // The elements at either end, one to a thread
  float edge = -INFINITY;
  int64_t edge_at = 0;
  if (rank == 0 && tid < head) {
    edge_at = tid;
    edge = to_f(x[edge_at]);
  } else if (rank == cluster - 1 && tid >= 32 && tid < 32 + tail) {
    edge_at = head + vecs * N + tid - 32;
    edge = to_f(x[edge_at]);
  }

  int64_t next = 1, tile = 0;  // tiles before the bound is looked at again
  // J vectors of every thread, kNT apart; WHOLE: all of them are the slice's.
  auto take = [&](int64_t v, auto count, auto whole) {
    constexpr int J = decltype(count)::value;
    constexpr bool WHOLE = decltype(whole)::value;
    uint4 w[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t at = v + j * kNT + tid;
      w[j] = WHOLE || at < v1 ? __ldcs(body + at) : all_masked<T>();
    }
    float big[J], now;
#pragma unroll
    for (int j = 0; j < J; ++j) big[j] = largest(w[j], T());
    now = big[0];
#pragma unroll
    for (int j = 1; j < J; ++j) now = max_nan(now, big[j]);
    if (!(now <= m.ref)) {  // a new largest (or a NaN, which stays)
      if (m.ref > -INFINITY) {
        const float u = __fmul_rn(__fsub_rn(m.ref, now), kLog2E);
        const f32x2 f = f2_dup(ex2_approx(u));
        e2 = f2_mul(f, f2_fma(f2_dup(fmaxf(u, -1e30f)), s2, e2));
        s2 = f2_mul(f, s2);
      } else if (m.ref != m.ref) {
        now = m.ref;
      }
      m.ref = now;
    }
    if (m.ref > -INFINITY || m.ref != m.ref) {
      const f32x2 ref2 = f2_dup(-m.ref), l2 = f2_dup(kLog2E);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        f32x2 f[P];
        floats4(w[j], f, T());
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float a, b;
          f2_unpack(f2_mul(f2_add(f[i], ref2), l2), a, b);
          // (far below the largest nothing is left; and 2^-inf (-inf) would not be a number)
          a = max_nan(a, -1e4f);
          b = max_nan(b, -1e4f);
          const f32x2 u = f2_pack(a, b), q = f2_pack(ex2_approx(a), ex2_approx(b));
          s2 = f2_add(s2, q);
          e2 = f2_fma(q, u, e2);
        }
      }
    }
    if (TOP) {
      top = fmaxf(top, now);
      if (++tile == next) {
        next *= 8;
        bound = new_bound(sm, fmaxf(top, edge), p.n_top);
      }
      if (now >= bound && now > -INFINITY) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (!(big[j] >= bound)) continue;
          const T* const el = reinterpret_cast<const T*>(&w[j]);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float xv = to_f(el[i]);
            if (xv >= bound && xv > -INFINITY) {
              const int c = atomicAdd(&sm.count, 1);
              if (c < kList) sm.list[c] = key_of(xv, head + (v + j * kNT + tid) * N + i);
            }
          }
        }
      }
    }
  };
  int64_t v = v0;
  for (; v + kLoads * kNT <= v1; v += kLoads * kNT) take(v, std::integral_constant<int, kLoads>(), std::true_type());
  for (; v < v1; v += kNT) take(v, std::integral_constant<int, 1>(), std::false_type());

  // The CTA's largest, and the threads' sums relative to it
  if (!(edge <= -INFINITY)) {
    float a, b;
    f2_unpack(s2, a, b);
    m.s = __fadd_rn(a, b);
    f2_unpack(e2, a, b);
    m.e = __fadd_rn(a, b);
    m = join(m, {edge, 1.0f, 0.0f});
    s2 = f2_pack(m.s, 0.0f);
    e2 = f2_pack(m.e, 0.0f);
  }
  float all = m.ref;
#pragma unroll
  for (int o = 16; o; o >>= 1) all = max_nan(all, __shfl_xor_sync(0xffffffffu, all, o));
  if (lane == 0) sm.refs[warp] = all;
  if (TOP) top = fmaxf(top, edge);
  __syncthreads();
  if (TOP && edge >= bound && edge > -INFINITY) {
    const int c = atomicAdd(&sm.count, 1);
    if (c < kList) sm.list[c] = key_of(edge, edge_at);
  }
#pragma unroll
  for (int w = 0; w < kNT / 32; ++w) all = max_nan(all, sm.refs[w]);
  {
    float a, b, s, e;
    f2_unpack(s2, a, b);
    s = __fadd_rn(a, b);
    f2_unpack(e2, a, b);
    e = __fadd_rn(a, b);
    if (m.ref == -INFINITY) {
      s = e = 0.0f;  // (nothing met; a NaN is in the reference)
    } else {
      const float u = __fmul_rn(__fsub_rn(m.ref, all), kLog2E), f = ex2_approx(u);
      e = __fmul_rn(f, __fmaf_rn(fmaxf(u, -1e30f), s, e));
      s = __fmul_rn(f, s);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
      e = __fadd_rn(e, __shfl_xor_sync(0xffffffffu, e, o));
    }
    if (lane == 0) sm.part[warp] = {all, s, e};
  }
  __syncthreads();
  if (tid == 0) {
    m = sm.part[0];
#pragma unroll
    for (int w = 1; w < kNT / 32; ++w) {
      m.s = __fadd_rn(m.s, sm.part[w].s);
      m.e = __fadd_rn(m.e, sm.part[w].e);
    }
    sm.all = m;
  }

  if (TOP) {
    // The elements collected are ranked by counting: where they are many, those that are not below a last bound.
    int n = sm.count;
    if (n > kFew) {
      const bool over = n > kList;
      bound = new_bound(sm, top, p.n_top);
      if (!over) {
        uint64_t mine[kList / kNT];
#pragma unroll
        for (int i = 0; i < kList / kNT; ++i) {
          const int at = i * kNT + tid;
          mine[i] = at < n ? sm.list[at] : 0;
          if (mine[i] && value_of(mine[i]) < bound) mine[i] = 0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kList / kNT; ++i)
          if (mine[i]) sm.list[atomicAdd(&sm.kept, 1)] = mine[i];
        __syncthreads();
        n = sm.kept;
      }
      if (over || n > kRank) n = take_again(sm, x + e0, e1 - e0, e0, p.n_top, bound, all);
    }
    if (tid < 32) sm.best[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kNT) {
      const uint64_t key = sm.list[i];
      int above = 0;
      for (int j = 0; j < n; ++j) above += sm.list[j] > key ? 1 : 0;
      if (above < p.n_top) sm.best[above] = key;
    }
  }
  if (cluster > 1) {
    cg::this_cluster().sync();
  } else {
    __syncthreads();
  }
  if (rank == 0) {
    m = sm.all;
    if (tid < 32 && cluster > 1) {
      cg::cluster_group cl = cg::this_cluster();
      m = {-INFINITY, 0.0f, 0.0f};
      if (lane < cluster) m = *cl.map_shared_rank(&sm.all, lane);
#pragma unroll
      for (int o = 16; o; o >>= 1)  // (every lane needs it)
        m = join(m, {__shfl_xor_sync(0xffffffffu, m.ref, o), __shfl_xor_sync(0xffffffffu, m.s, o),
                     __shfl_xor_sync(0xffffffffu, m.e, o)});
    }
    if (tid < 32) {
      const bool fine = m.ref > -INFINITY && m.ref < INFINITY && m.s < INFINITY;
      const float ls = logf(m.s);
      if (lane == 0) {
        if (p.logprob) {
          const int32_t t = p.tokens[r];
          float v = t < 0 ? 0.0f : NAN;
          if (t >= 0 && t < p.vocab && fine) v = __fsub_rn(__fsub_rn(to_f(x[t]), m.ref), ls);
          p.logprob[r] = v;
        }
        if (p.entropy) p.entropy[r] = fine ? __fsub_rn(ls, __fmul_rn(__fdiv_rn(m.e, m.s), kLn2)) : NAN;
      }
      if (TOP) {
        // The CTAs' lists, each in order: lane i has the first of CTA i's that is not taken.
        const uint64_t* from = sm.best;
        if (cluster > 1) from = cg::this_cluster().map_shared_rank(sm.best, min(lane, cluster - 1));
        int at = 0, k = 0;
        uint64_t mine = lane < cluster ? from[0] : 0, taken = 0;
        for (; k < p.n_top; ++k) {
          const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32));
          const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
          const uint64_t key = ((uint64_t)hi << 32) | lo;
          if (key == 0) break;
          if (mine == key) {
            ++at;
            mine = at < p.n_top ? from[at] : 0;
          }
          if (lane == k) taken = key;
        }
        if (lane < k) {
          p.top_token[r * p.n_top + lane] = fine ? index_of(taken) : -1;
          p.top_logprob[r * p.n_top + lane] = fine ? __fsub_rn(__fsub_rn(value_of(taken), m.ref), ls) : NAN;
        }
        if (lane == 0) sm.kept = fine ? k : -1;
      }
    }
    if (TOP) {
      __syncthreads();
      // Fewer tokens than n_top are allowed: masked ones follow, in the order of their index.
      const int k = sm.kept;
      __syncthreads();
      if (k >= 0 && k < p.n_top) take_equal(sm, x, p.vocab, 0, ordered(-INFINITY), 0, p.n_top - k);
      for (int i = max(k, 0) + tid; i < p.n_top; i += kNT) {
        p.top_token[r * p.n_top + i] = k < 0 ? -1 : index_of(sm.list[i - k]);
        p.top_logprob[r * p.n_top + i] = k < 0 ? NAN : -INFINITY;
      }
    }
  }
  if (cluster > 1) cg::this_cluster().sync();  // the others' shared memory is read until here
}

// CTAs for a row: enough for two an SM, as long as a slice has a few KB (128 rows of 131,071 fp32: 25 us with 4
// CTAs a row, 31 with 8).
int cluster_of(const LogprobParams& p) {
  const int64_t bytes = p.vocab * (p.dtype == LQ_F32 ? 4 : 2);
  int c = 1;
  while (c < kMaxCluster && p.rows * c < 2 * 152 && bytes / (2 * c) >= 4096) c *= 2;
  return c;
}

template <typename T, bool TOP>
cudaError_t launch_rows(const LogprobParams& p, cudaStream_t st) {
  const int c = cluster_of(p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * c));
  cfg.blockDim = dim3(kNT);
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)c;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_logprob<T, TOP>, p, c);
}

template <typename T>
cudaError_t launch(const LogprobParams& p, cudaStream_t st) {
  return p.n_top ? launch_rows<T, true>(p, st) : launch_rows<T, false>(p, st);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams& p, cudaStream_t st) {
  if (p.dtype == LQ_F32) return launch<float>(p, st);
  if (p.dtype == LQ_BF16) return launch<__nv_bfloat16>(p, st);
  return launch<__half>(p, st);
}

}  // namespace lqi
