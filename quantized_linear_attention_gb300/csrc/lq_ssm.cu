// Selective state space scan (sm_103a), over packed prompts and for single tokens: for every channel and state
//   h <- exp(d A) h + d x B,   y = (sum_n C h + D x) silu(z).
#include "lq_device.cuh"
#include "lq_seq.cuh"

namespace lqi {

namespace {

// --------------------------------------------------------------------------------------------
// Prompts. A thread holds SPT states of a channel (LPC lanes of a warp share one channel) and takes the tokens of a piece
// one after the other: per state and token a multiplication and an exponential for the decay, a multiplication and an fma for
// the state and an fma for y, in packed pairs of states. B and C are the same for all channels of a group: 16 tokens of them
// at a time lie in shared memory as floats, read by broadcast; x, dt and z come straight into registers, 8 tokens ahead.
//
// A sequence that would leave most of the GPU idle is split into segments (ssm_plan). The first pass takes
// every segment but the last from a zero state (the first from its true one, with its outputs) and leaves its last state and
// the sum of its d; since the decays of a segment multiply to exp(A sum d), k_ssm_join finds the state before each segment,
// and the second pass takes the segments from there. What that sum over segments does not give as the recurrence does (a
// positive A or a negative d, where it may overflow though the recurrence does not, infinities, values near fp32's largest
// number) k_ssm_join takes token by token.
constexpr int kNT = 128;
constexpr int kTile = 16;   // tokens of B and C in shared memory at a time, double-buffered
constexpr int kAhead = 8;   // tokens whose x, dt and z are in flight

// A token's step d.
template <typename T>
__device__ __forceinline__ float step_of(T dt, float bias, int plus) {
  const float v = __fadd_rn(to_f(dt), bias);
  return plus ? softplus(v) : v;
}

template <typename T, int SPT, int LPC, bool OUT, bool Z>
__device__ __forceinline__ void scan_piece(const SsmParams& p, const Piece& pc, int c, int g, bool live, const float* from,
                                           float* to, float* step_sum, float (*sB)[kTile][SPT * LPC],
                                           float (*sC)[kTile][SPT * LPC], float* smax) {
  constexpr int NP = SPT * LPC, CW = 32 / LPC, PER = kTile * NP / kNT, H = SPT / 2;
  const int tid = threadIdx.x, part = (tid & 31) / CW, n0 = part * SPT;
  const int len = (int)pc.len;
  const T* x = static_cast<const T*>(p.x) + pc.begin * p.sx + c;
  const T* dt = static_cast<const T*>(p.dt) + pc.begin * p.sdt + c;
  const T* z = Z ? static_cast<const T*>(p.z) + pc.begin * p.sz + c : nullptr;
  T* y = static_cast<T*>(p.y) + pc.begin * p.sy + c;
  const T* B = static_cast<const T*>(p.B) + pc.begin * p.sb + (int64_t)g * p.n_state;
  const T* C = static_cast<const T*>(p.C) + pc.begin * p.sc + (int64_t)g * p.n_state;
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, D = p.D ? p.D[c] : 0.0f;
  const T zero = from_f<T>(0.0f);

  f32x2 A[H], h[H];
#pragma unroll
  for (int j = 0; j < H; ++j) {
    float a[2], s[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int n = n0 + 2 * j + e;
      const bool in = n < p.n_state;
      a[e] = in ? __fmul_rn(p.A[(int64_t)c * p.n_state + n], kLog2E) : 0.0f;
      s[e] = in && from ? from[n] : 0.0f;
    }
    A[j] = f2_pack(a[0], a[1]);
    h[j] = f2_pack(s[0], s[1]);
  }

  // B and C of a tile: element i * kNT + tid of [token][state], into registers and from there into shared memory
  T rb[PER], rc[PER];
  float bmax = 0.0f;
  auto load_bc = [&](int t0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = i * kNT + tid, t = t0 + at / NP, n = at % NP;
      const bool in = t < len && n < p.n_state;
      rb[i] = in ? B[t * p.sb + n] : zero;
      if (OUT) rc[i] = in ? C[t * p.sc + n] : zero;
    }
  };
  auto put_bc = [&](int buf) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = i * kNT + tid;
      const float b = to_f(rb[i]);
      (&sB[buf][0][0])[at] = b;
      if (OUT) (&sC[buf][0][0])[at] = to_f(rc[i]);
      else bmax = fmaxf(bmax, fabsf(b));
    }
  };
  T rx[kAhead], rd[kAhead], rz[kAhead];
  auto load_x = [&](int u, int t) {
    const bool in = t < len;
    rx[u] = in ? x[t * p.sx] : zero;
    rd[u] = in ? dt[t * p.sdt] : zero;
    if (OUT && Z) rz[u] = in ? z[t * p.sz] : zero;
  };
  load_bc(0);
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load_x(u, u);
  put_bc(0);
  __syncthreads();

  float dsum = 0.0f, dmin = 0.0f, ax = 0.0f;
  for (int t0 = 0, buf = 0; t0 < len; t0 += kTile, buf ^= 1) {
    load_bc(t0 + kTile);
    float dpart = 0.0f;
    auto token = [&](int u, int tt) {
      const int t = t0 + tt;
      const float xv = to_f(rx[u]), d = step_of(rd[u], bias, p.softplus), zv = OUT && Z ? to_f(rz[u]) : 0.0f;
      load_x(u, t + kAhead);
      const float dx = __fmul_rn(d, xv);
      const f32x2 d2 = f2_dup(d), dx2 = f2_dup(dx);
      f32x2 acc[2] = {0ull, 0ull};
      const ulonglong2* b2 = reinterpret_cast<const ulonglong2*>(&sB[buf][tt][n0]);
      const ulonglong2* c2 = reinterpret_cast<const ulonglong2*>(&sC[buf][tt][n0]);
#pragma unroll
      for (int j = 0; j < H; j += 2) {
        const ulonglong2 b = b2[j / 2];
        float e0, e1, e2, e3;
        f2_unpack(f2_mul(d2, A[j]), e0, e1);
        f2_unpack(f2_mul(d2, A[j + 1]), e2, e3);
        h[j] = f2_fma(f2_pack(ex2_approx(e0), ex2_approx(e1)), h[j], f2_mul(dx2, b.x));
        h[j + 1] = f2_fma(f2_pack(ex2_approx(e2), ex2_approx(e3)), h[j + 1], f2_mul(dx2, b.y));
        if (OUT) {
          const ulonglong2 cc = c2[j / 2];
          acc[0] = f2_fma(h[j], cc.x, acc[0]);
          acc[1] = f2_fma(h[j + 1], cc.y, acc[1]);
        }
      }
      if (OUT) {
        float y0, y1;
        f2_unpack(f2_add(acc[0], acc[1]), y0, y1);
        float o = __fadd_rn(y0, y1);
#pragma unroll
        for (int s = CW; s < 32; s <<= 1) o = __fadd_rn(o, __shfl_xor_sync(0xffffffffu, o, s));
        o = __fmaf_rn(D, xv, o);
        if (Z) o = __fmul_rn(o, silu(zv));
        if (live && part == 0) y[t * p.sy] = from_f<T>(o);
      } else {
        dpart = __fadd_rn(dpart, d);
        dmin = d >= dmin ? dmin : (d < dmin ? d : -1.0f);  // (a NaN counts as negative)
        ax = __fadd_rn(ax, fabsf(dx));
      }
    };
#pragma unroll 1
    for (int t8 = 0; t8 < kTile; t8 += kAhead) {
      if (t0 + t8 + kAhead <= len) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) token(u, t8 + u);
      } else {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (t0 + t8 + u < len) token(u, t8 + u);
      }
    }
    if (!OUT) dsum = __fadd_rn(dsum, dpart);
    put_bc(buf ^ 1);
    __syncthreads();
  }

  if (to && live) {
#pragma unroll
    for (int j = 0; j < H; ++j) {
      float s[2];
      f2_unpack(h[j], s[0], s[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (n0 + 2 * j + e < p.n_state) to[n0 + 2 * j + e] = s[e];
    }
  }
  if (!OUT) {
    // The sum of d, or NaN where the join cannot go by it: a negative d, or values that may have passed 1e30 on the way
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) bmax = fmaxf(bmax, __shfl_xor_sync(0xffffffffu, bmax, s));
    if ((tid & 31) == 0) smax[tid >> 5] = bmax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kNT / 32; ++w) bmax = fmaxf(bmax, smax[w]);
    const bool sure = dmin >= 0.0f && dsum < 1e30f && __fmul_rn(ax, bmax) < 1e30f;
    if (live && part == 0) *step_sum = sure ? dsum : NAN;
  }
}

// Blocks of channels never cross a group: block i is channels i % per of group i / per.
template <typename T, int SPT, int LPC, bool Z>
__global__ void __launch_bounds__(kNT) k_ssm(SsmParams p, int blocks, int per, int second) {
  constexpr int CH = kNT / LPC, CW = 32 / LPC;
  __shared__ __align__(16) float sB[2][kTile][SPT * LPC], sC[2][kTile][SPT * LPC];
  __shared__ float smax[kNT / 32];
  if (!second) cudaTriggerProgrammaticLaunchCompletion();  // k_ssm_join may be set up; it waits for this grid's end
  const int64_t slot = blockIdx.x / (unsigned)blocks;
  const int blk = (int)(blockIdx.x % (unsigned)blocks), g = blk / per;
  const int in_group = (blk % per) * CH + (threadIdx.x >> 5) * CW + (threadIdx.x & 31) % CW;
  const bool live = in_group < p.per_group;
  const int c = g * p.per_group + (live ? in_group : 0);
  const Piece pc = find_slot<kNT>(p, slot);
  if (second) cudaGridDependencySynchronize();
  if (pc.b < 0 || (second ? pc.i == 0 : pc.i > 0 && pc.i == pc.n - 1)) return;
  float* const S = p.S ? p.S + (pc.b * p.channels + c) * p.n_state : nullptr;
  float* const ws = p.seg ? p.ws_state + (slot * p.channels + c) * p.n_state : nullptr;
  const bool last = pc.i == pc.n - 1;
  if (!second && pc.i > 0) {
    scan_piece<T, SPT, LPC, false, Z>(p, pc, c, g, live, nullptr, ws, p.ws_step + slot * p.channels + c, sB, sC, smax);
  } else {
    const float* from = second ? ws : p.S0 ? p.S0 + (pc.b * p.channels + c) * p.n_state : nullptr;
    scan_piece<T, SPT, LPC, true, Z>(p, pc, c, g, live, from, last ? S : ws, nullptr, sB, sC, smax);
  }
}

// One state through a segment as the recurrence is written.
template <typename T>
__device__ __noinline__ float walk(const SsmParams& p, int64_t begin, int64_t at, float h) {
  const int64_t c = at / p.n_state, n = at % p.n_state, g = c / p.per_group;
  const float A2 = __fmul_rn(p.A[at], kLog2E), bias = p.dt_bias ? p.dt_bias[c] : 0.0f;
  for (int64_t t = begin; t < begin + p.seg; ++t) {
    const float d = step_of(static_cast<const T*>(p.dt)[t * p.sdt + c], bias, p.softplus);
    const float dx = __fmul_rn(d, to_f(static_cast<const T*>(p.x)[t * p.sx + c]));
    const float B = to_f(static_cast<const T*>(p.B)[t * p.sb + g * p.n_state + n]);
    h = __fmaf_rn(ex2_approx(__fmul_rn(d, A2)), h, __fmul_rn(dx, B));
  }
  return h;
}

// Split sequences: one thread a state, from segment to segment. ws_state holds what the first pass left, the first segment's
// last state and what each other one adds; afterwards the state before each segment but the first.
template <typename T>
__global__ void __launch_bounds__(256) k_ssm_join(SsmParams p, int blocks) {
  constexpr int U = 8;  // segments read at a time
  cudaTriggerProgrammaticLaunchCompletion();
  const int64_t slot = blockIdx.x / (unsigned)blocks;
  const int64_t row = (int64_t)p.channels * p.n_state;
  const int64_t at = (int64_t)(blockIdx.x % (unsigned)blocks) * 256 + threadIdx.x;
  const Piece pc = find_slot<256>(p, slot);
  cudaGridDependencySynchronize();
  if (pc.b < 0 || pc.i > 0 || pc.n == 1 || at >= row) return;
  const int64_t c = at / p.n_state, segs = min(pc.n, p.slots - slot);
  float* ws = p.ws_state + slot * row + at;
  const float* step = p.ws_step + slot * p.channels + c;
  const float A = p.A[at], A2 = __fmul_rn(A, kLog2E);
  const bool falls = A <= 0.0f && A > -1e30f;
  float h = ws[0];
  for (int64_t i0 = 1; i0 < segs; i0 += U) {
    float add[U], sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      add[u] = sum[u] = 0.0f;
      if (i0 + u < segs - 1) {
        add[u] = ws[(i0 + u) * row];
        sum[u] = step[(i0 + u) * p.channels];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u;
      if (i >= segs) break;
      ws[i * row] = h;
      if (i == segs - 1) break;
      if (falls && sum[u] == sum[u] && fabsf(h) < 1e30f) {
        h = __fmaf_rn(ex2_approx(__fmul_rn(sum[u], A2)), h, add[u]);
      } else {
        h = walk<T>(p, pc.begin + i * p.seg, at, h);
      }
    }
  }
}

struct Shape {
  int spt, lpc;
};

// States a thread, lanes a channel.
__host__ inline Shape shape_of(int n_state) {
  if (n_state <= 8) return {8, 1};
  if (n_state <= 16) return {16, 1};
  if (n_state <= 32) return {16, 2};
  return {16, 4};
}

__host__ inline int blocks_of_group(int per_group, int n_state) {
  const int ch = kNT / shape_of(n_state).lpc;
  return (per_group + ch - 1) / ch;
}

template <typename T, int SPT, int LPC, bool Z>
cudaError_t launch_shape(const SsmParams& p, cudaStream_t st) {
  const int per = blocks_of_group(p.per_group, p.n_state), blocks = per * p.groups;
  const unsigned grid = (unsigned)(p.slots * blocks);
  k_ssm<T, SPT, LPC, Z><<<grid, kNT, 0, st>>>(p, blocks, per, 0);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.seg) return e;
  const int jb = (int)(((int64_t)p.channels * p.n_state + 255) / 256);
  e = launch_upon(k_ssm_join<T>, dim3((unsigned)(p.slots * jb)), 256, 0, st, p, jb);
  if (e != cudaSuccess) return e;
  return launch_upon(k_ssm<T, SPT, LPC, Z>, dim3(grid), kNT, 0, st, p, blocks, per, 1);
}

template <typename T, bool Z>
cudaError_t launch_states(const SsmParams& p, cudaStream_t st) {
  if (p.n_state <= 8) return launch_shape<T, 8, 1, Z>(p, st);
  if (p.n_state <= 16) return launch_shape<T, 16, 1, Z>(p, st);
  if (p.n_state <= 32) return launch_shape<T, 16, 2, Z>(p, st);
  return launch_shape<T, 16, 4, Z>(p, st);
}

template <typename T>
cudaError_t launch(const SsmParams& p, cudaStream_t st) {
  return p.z ? launch_states<T, true>(p, st) : launch_states<T, false>(p, st);
}

// --------------------------------------------------------------------------------------------
// Single tokens.
template <typename T, int N>
__device__ __forceinline__ void token(const SsmParams& p, int64_t t, int c, int g, const float (&A)[N], float bias,
                                      float D, float (&h)[N]) {
  const float d = step_of(static_cast<const T*>(p.dt)[t * p.sdt + c], bias, p.softplus);
  const float x = to_f(static_cast<const T*>(p.x)[t * p.sx + c]), dx = __fmul_rn(d, x);
  const T* B = static_cast<const T*>(p.B) + t * p.sb + (int64_t)g * p.n_state;
  const T* C = static_cast<const T*>(p.C) + t * p.sc + (int64_t)g * p.n_state;
  float y = 0.0f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (n >= p.n_state) break;
    h[n] = __fmaf_rn(ex2_approx(__fmul_rn(d, A[n])), h[n], __fmul_rn(dx, to_f(B[n])));
    y = __fmaf_rn(to_f(C[n]), h[n], y);
  }
  y = __fmaf_rn(D, x, y);
  if (p.z) y = __fmul_rn(y, silu(to_f(static_cast<const T*>(p.z)[t * p.sz + c])));
  static_cast<T*>(p.y)[t * p.sy + c] = from_f<T>(y);
}

template <typename T, int N>
__global__ void __launch_bounds__(kNT) k_ssm_step(SsmParams p, int blocks) {
  const int64_t b = blockIdx.x / (unsigned)blocks;
  const int c = (int)(blockIdx.x % (unsigned)blocks) * kNT + threadIdx.x;
  if (c >= p.channels) return;
  const int64_t at = (b * p.channels + c) * p.n_state;
  float A[N], h[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    A[n] = h[n] = 0.0f;
    if (n < p.n_state) {
      A[n] = __fmul_rn(p.A[(int64_t)c * p.n_state + n], kLog2E);
      h[n] = p.S[at + n];
    }
  }
  token<T, N>(p, b, c, c / p.per_group, A, p.dt_bias ? p.dt_bias[c] : 0.0f, p.D ? p.D[c] : 0.0f, h);
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (n < p.n_state) p.S[at + n] = h[n];
}

template <typename T>
cudaError_t launch_token(const SsmParams& p, cudaStream_t st) {
  const int blocks = (p.channels + kNT - 1) / kNT;
  const unsigned grid = (unsigned)(p.n_seqs * blocks);
  if (p.n_state <= 16) k_ssm_step<T, 16><<<grid, kNT, 0, st>>>(p, blocks);
  else k_ssm_step<T, 64><<<grid, kNT, 0, st>>>(p, blocks);
  return cudaGetLastError();
}

// CTAs that a split call should come to, and the least tokens of a segment.
constexpr int64_t kSplitCtas = 152 * 5, kLeastSeg = 64;

}  // namespace

int64_t ssm_blocks(const lq_ssm_config* c) {
  return (int64_t)c->groups * blocks_of_group(c->channels / c->groups, c->n_state);
}

// Whole sequences take as long as the longest one alone, about 140 cycles a token, or as all tokens together, about 95 a
// token and CTA on each of 152 SMs; split, 1.8 times the latter, two segments one after the other, and two launches.
void ssm_plan(const lq_ssm_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len, int64_t* seg, int64_t* slots) {
  *seg = 0;
  *slots = n_seqs;
  const int64_t blocks = ssm_blocks(c), longest = max_len > 0 && max_len < n_tokens ? max_len : n_tokens;
  const int64_t work = n_tokens * blocks;
  int64_t s = ((work + kSplitCtas - 1) / kSplitCtas + kTile - 1) / kTile * kTile;
  s = s < kLeastSeg ? kLeastSeg : s;
  if (longest < 3 * s) return;
  const double all = 95.0 / 152 * (double)work, whole = 140.0 * (double)longest;
  if ((all > whole ? all : whole) <= 1.8 * all + 280.0 * (double)s + 8000.0) return;
  *seg = s;
  *slots = n_tokens / s + n_seqs;
}

// A segment has at least kLeastSeg tokens and at least a kSplitCtas-th of the call's work.
int64_t ssm_most_slots(const lq_ssm_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len) {
  const int64_t longest = max_len > 0 && max_len < n_tokens ? max_len : n_tokens;
  if (longest < 3 * kLeastSeg) return 0;
  const int64_t a = n_tokens / kLeastSeg, b = kSplitCtas / ssm_blocks(c);
  return a < 3 || b < 3 ? 0 : (a < b ? a : b) + n_seqs;
}

cudaError_t launch_ssm_prefill(const SsmParams& p, cudaStream_t st) {
  if (p.dtype == LQ_F32) return launch<float>(p, st);
  if (p.dtype == LQ_BF16) return launch<__nv_bfloat16>(p, st);
  return launch<__half>(p, st);
}

cudaError_t launch_ssm_step(const SsmParams& p, cudaStream_t st) {
  if (p.dtype == LQ_F32) return launch_token<float>(p, st);
  if (p.dtype == LQ_BF16) return launch_token<__nv_bfloat16>(p, st);
  return launch_token<__half>(p, st);
}

}  // namespace lqi
