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
template <typename T>
constexpr int kTile = 32 / (int)sizeof(T);  // tokens in shared memory at a time
constexpr int kUnroll = 8;

// A token's step d.
template <typename T, bool PLUS>
__device__ __forceinline__ float step_of(T dt, float bias) {
  const float v = __fadd_rn(to_f(dt), bias);
  return PLUS ? softplus(v) : v;
}

template <typename T, int SPT, int LPC>
struct Smem {
  static constexpr int CH = kNT / LPC, NP = SPT * LPC, TT = kTile<T>;
  T x[2][TT][CH], dt[2][TT][CH], z[2][TT][CH], y[TT][CH];
  float B[2][TT][NP], C[2][TT][NP];
  float max[kNT / 32];
};

// Which channels a CTA has: CH of them from c0 on, of which `left` belong to its group.
struct Channels {
  int c0, left, g;
};

// One array's rows of tokens t0 .. t0 + TT - 1 (those below len) into shared memory. VEC: by 16 bytes, not waited for.
template <typename T, int CH, int TT, bool VEC>
__device__ __forceinline__ void stage(T (*to)[CH], const T* from, int64_t stride, int t0, int len, int left) {
  constexpr int E = VEC ? 16 / (int)sizeof(T) : 1, Q = CH / E;
#pragma unroll
  for (int i = 0; i < (TT * Q + kNT - 1) / kNT; ++i) {
    const int at = i * kNT + threadIdx.x, t = at / Q, c = at % Q * E;
    if (TT * Q % kNT && t >= TT) break;
    const int n = t0 + t < len ? min(max(left - c, 0), E) : 0;
    if (VEC) copy16(&to[t][c], n ? from + (int64_t)(t0 + t) * stride + c : from, n * (int)sizeof(T));
    else if (n) to[t][c] = from[(int64_t)(t0 + t) * stride + c];
  }
}

template <typename T, int CH, int TT, bool VEC>
__device__ __forceinline__ void unstage(const T (*from)[CH], T* to, int64_t stride, int t0, int len, int left) {
  constexpr int E = VEC ? 16 / (int)sizeof(T) : 1, Q = CH / E;
#pragma unroll
  for (int i = 0; i < (TT * Q + kNT - 1) / kNT; ++i) {
    const int at = i * kNT + threadIdx.x, t = at / Q, c = at % Q * E;
    if (TT * Q % kNT && t >= TT) break;
    if (t0 + t >= len || c >= left) continue;
    T* const y = to + (int64_t)(t0 + t) * stride + c;
    if (VEC && c + E <= left) *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(&from[t][c]);
    else
      for (int e = 0; e < E && c + e < left; ++e) y[e] = from[t][c + e];
  }
}

template <typename T, int SPT, int LPC, bool PLUS, bool VEC, bool OUT>
__device__ __forceinline__ void scan_piece(const SsmParams& p, const Piece& pc, const Channels& ch, const float* from,
                                           float* to, float* step_sum, Smem<T, SPT, LPC>& sm) {
  constexpr int NP = SPT * LPC, CW = 32 / LPC, CH = kNT / LPC, TT = kTile<T>, PER = (TT * NP + kNT - 1) / kNT, H = SPT / 2;
  const int tid = threadIdx.x, part = (tid & 31) / CW, n0 = part * SPT, col = (tid >> 5) * CW + (tid & 31) % CW;
  const int len = (int)pc.len;
  const bool live = col < ch.left, gate = p.z != nullptr;
  const int c = ch.c0 + (live ? col : 0);
  const T* x = static_cast<const T*>(p.x) + pc.begin * p.sx + ch.c0;
  const T* dt = static_cast<const T*>(p.dt) + pc.begin * p.sdt + ch.c0;
  const T* z = gate ? static_cast<const T*>(p.z) + pc.begin * p.sz + ch.c0 : nullptr;
  T* y = static_cast<T*>(p.y) + pc.begin * p.sy + ch.c0;
  const T* B = static_cast<const T*>(p.B) + pc.begin * p.sb + (int64_t)ch.g * p.n_state;
  const T* C = static_cast<const T*>(p.C) + pc.begin * p.sc + (int64_t)ch.g * p.n_state;
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, D = p.D ? p.D[c] : 0.0f;
  const T zero = from_f<T>(0.0f);

  // B and C of a tile: element i * kNT + tid of [token][state], into registers and from there into shared memory
  T rb[PER], rc[PER];
  float bmax = 0.0f;
  auto load_bc = [&](int t0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = i * kNT + tid, t = t0 + at / NP, n = at % NP;
      const bool in = at < TT * NP && t < len && n < p.n_state;
      rb[i] = in ? B[t * p.sb + n] : zero;
      if (OUT) rc[i] = in ? C[t * p.sc + n] : zero;
    }
  };
  auto put_bc = [&](int buf) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = i * kNT + tid;
      if (TT * NP % kNT && at >= TT * NP) break;
      const float b = to_f(rb[i]);
      (&sm.B[buf][0][0])[at] = b;
      if (OUT) (&sm.C[buf][0][0])[at] = to_f(rc[i]);
      else bmax = fmaxf(bmax, fabsf(b));
    }
  };
  auto stage_x = [&](int t0, int buf) {
    stage<T, CH, TT, VEC>(sm.x[buf], x, p.sx, t0, len, ch.left);
    stage<T, CH, TT, VEC>(sm.dt[buf], dt, p.sdt, t0, len, ch.left);
    if (OUT && gate) stage<T, CH, TT, VEC>(sm.z[buf], z, p.sz, t0, len, ch.left);
    if (VEC) copy_commit();
  };
  load_bc(0);
  if (len > 0) stage_x(0, 0);

  f32x2 A[H], h[H];
#pragma unroll
  for (int j = 0; j < H; ++j) {
    float a[2], s[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int n = n0 + 2 * j + e;
      const bool in = n < p.n_state;
      a[e] = in ? __fmul_rn(p.A[(int64_t)c * p.n_state + n], kLog2E) : 0.0f;
      s[e] = in && from ? from[(int64_t)c * p.n_state + n] : 0.0f;
    }
    A[j] = f2_pack(a[0], a[1]);
    h[j] = f2_pack(s[0], s[1]);
  }
  put_bc(0);

  float dsum = 0.0f, dmin = 0.0f, ax = 0.0f;
  for (int t0 = 0, buf = 0; t0 < len; t0 += TT, buf ^= 1) {
    const bool more = t0 + TT < len;
    if (more) {
      load_bc(t0 + TT);
      stage_x(t0 + TT, buf ^ 1);
      if (VEC) copy_wait<1>();
    } else if (VEC) {
      copy_wait<0>();
    }
    __syncthreads();
    float dpart = 0.0f;
    auto token = [&](int t) {
      const float xv = to_f(sm.x[buf][t][col]), d = step_of<T, PLUS>(sm.dt[buf][t][col], bias), dx = __fmul_rn(d, xv);
      const f32x2 d2 = f2_dup(d), dx2 = f2_dup(dx);
      f32x2 acc[2] = {0ull, 0ull};
      const ulonglong2* b2 = reinterpret_cast<const ulonglong2*>(&sm.B[buf][t][n0]);
      const ulonglong2* c2 = reinterpret_cast<const ulonglong2*>(&sm.C[buf][t][n0]);
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
        const float gated = __fmul_rn(o, silu(to_f(sm.z[buf][t][col])));
        if (part == 0) sm.y[t][col] = from_f<T>(gate ? gated : o);
      } else {
        dpart = __fadd_rn(dpart, d);
        dmin = d >= dmin ? dmin : (d < dmin ? d : -1.0f);  // (a NaN counts as negative)
        ax = __fadd_rn(ax, fabsf(dx));
      }
    };
#pragma unroll 1
    for (int t8 = 0; t8 < TT; t8 += kUnroll) {
      if (t0 + t8 + kUnroll <= len) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) token(t8 + u);
      } else {
#pragma unroll 1
        for (int u = t8; t0 + u < len; ++u) token(u);
        break;
      }
    }
    if (!OUT) dsum = __fadd_rn(dsum, dpart);
    if (more) put_bc(buf ^ 1);
    __syncthreads();
    if (OUT) unstage<T, CH, TT, VEC>(sm.y, y, p.sy, t0, len, ch.left);
  }

  if (to && live) {
#pragma unroll
    for (int j = 0; j < H; ++j) {
      float s[2];
      f2_unpack(h[j], s[0], s[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (n0 + 2 * j + e < p.n_state) to[(int64_t)c * p.n_state + n0 + 2 * j + e] = s[e];
    }
  }
  if (!OUT) {
    // The sum of d, or NaN where the join cannot go by it: a negative d, or values that may have passed 1e30 on the way
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) bmax = fmaxf(bmax, __shfl_xor_sync(0xffffffffu, bmax, s));
    if ((tid & 31) == 0) sm.max[tid >> 5] = bmax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kNT / 32; ++w) bmax = fmaxf(bmax, sm.max[w]);
    const bool sure = dmin >= 0.0f && dsum < 1e30f && __fmul_rn(ax, bmax) < 1e30f;
    if (live && part == 0) step_sum[c] = sure ? dsum : NAN;
  }
}

// Blocks of channels never cross a group: block i is channels i % per of group i / per.
template <typename T, int SPT, int LPC, bool PLUS, bool VEC>
__global__ void __launch_bounds__(kNT) k_ssm(SsmParams p, int blocks, int per, int second) {
  extern __shared__ __align__(16) char smem[];
  Smem<T, SPT, LPC>& sm = *reinterpret_cast<Smem<T, SPT, LPC>*>(smem);
  if (!second) cudaTriggerProgrammaticLaunchCompletion();  // k_ssm_join may be set up; it waits for this grid's end
  const int64_t slot = blockIdx.x / (unsigned)blocks;
  const int blk = (int)(blockIdx.x % (unsigned)blocks), in_group = (blk % per) * (kNT / LPC);
  const Channels ch = {blk / per * p.per_group + in_group, p.per_group - in_group, blk / per};
  const Piece pc = find_slot<kNT>(p, slot);
  if (second) cudaGridDependencySynchronize();
  if (pc.b < 0 || (second ? pc.i == 0 : pc.i > 0 && pc.i == pc.n - 1)) return;
  const int64_t row = (int64_t)p.channels * p.n_state;
  float* const ws = p.seg ? p.ws_state + slot * row : nullptr;
  if (!second && pc.i > 0) {
    scan_piece<T, SPT, LPC, PLUS, VEC, false>(p, pc, ch, nullptr, ws, p.ws_step + slot * p.channels, sm);
  } else {
    float* const S = p.S ? p.S + pc.b * row : nullptr;
    const float* const from = second ? ws : p.S0 ? p.S0 + pc.b * row : nullptr;
    scan_piece<T, SPT, LPC, PLUS, VEC, true>(p, pc, ch, from, pc.i == pc.n - 1 ? S : ws, nullptr, sm);
  }
}

// One state through a segment as the recurrence is written.
template <typename T, bool PLUS>
__device__ __noinline__ float walk(const SsmParams& p, int64_t begin, int64_t at, float h) {
  const int64_t c = at / p.n_state, n = at % p.n_state, g = c / p.per_group;
  const float A2 = __fmul_rn(p.A[at], kLog2E), bias = p.dt_bias ? p.dt_bias[c] : 0.0f;
  for (int64_t t = begin; t < begin + p.seg; ++t) {
    const float d = step_of<T, PLUS>(static_cast<const T*>(p.dt)[t * p.sdt + c], bias);
    const float dx = __fmul_rn(d, to_f(static_cast<const T*>(p.x)[t * p.sx + c]));
    const float B = to_f(static_cast<const T*>(p.B)[t * p.sb + g * p.n_state + n]);
    h = __fmaf_rn(ex2_approx(__fmul_rn(d, A2)), h, __fmul_rn(dx, B));
  }
  return h;
}

// Split sequences: one thread a state, from segment to segment. ws_state holds what the first pass left, the first segment's
// last state and what each other one adds; afterwards the state before each segment but the first.
template <typename T, bool PLUS>
__global__ void __launch_bounds__(256, 4) k_ssm_join(SsmParams p, int blocks) {
  constexpr int U = 8;  // segments read at a time
  cudaTriggerProgrammaticLaunchCompletion();
  const int64_t b = blockIdx.x / (unsigned)blocks, row = (int64_t)p.channels * p.n_state;
  const int64_t at = (int64_t)(blockIdx.x % (unsigned)blocks) * 256 + threadIdx.x;
  Piece pc;
  bounds(p, b, pc.begin, pc.len);
  pc.n = pc.len > p.seg ? (pc.len + p.seg - 1) / p.seg : 1;
  if (pc.n == 1) return;
  const int64_t slot = first_slot<256>(p, b);
  cudaGridDependencySynchronize();
  if (at >= row) return;
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
        h = walk<T, PLUS>(p, pc.begin + i * p.seg, at, h);
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

template <typename T, int SPT, int LPC, bool PLUS, bool VEC>
cudaError_t launch_shape(const SsmParams& p, cudaStream_t st) {
  const int per = blocks_of_group(p.per_group, p.n_state), blocks = per * p.groups;
  const unsigned grid = (unsigned)(p.slots * blocks);
  auto* const kernel = k_ssm<T, SPT, LPC, PLUS, VEC>;
  constexpr int smem = (int)sizeof(Smem<T, SPT, LPC>);
  cudaError_t e = set_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kNT, smem, st>>>(p, blocks, per, 0);
  e = cudaGetLastError();
  if (e != cudaSuccess || !p.seg) return e;
  const int jb = (int)(((int64_t)p.channels * p.n_state + 255) / 256);
  e = launch_upon(k_ssm_join<T, PLUS>, dim3((unsigned)(p.n_seqs * jb)), 256, 0, st, p, jb);
  if (e != cudaSuccess) return e;
  return launch_upon(kernel, dim3(grid), kNT, smem, st, p, blocks, per, 1);
}

template <typename T, bool PLUS, bool VEC>
cudaError_t launch_states(const SsmParams& p, cudaStream_t st) {
  if (p.n_state <= 8) return launch_shape<T, 8, 1, PLUS, VEC>(p, st);
  if (p.n_state <= 16) return launch_shape<T, 16, 1, PLUS, VEC>(p, st);
  if (p.n_state <= 32) return launch_shape<T, 16, 2, PLUS, VEC>(p, st);
  return launch_shape<T, 16, 4, PLUS, VEC>(p, st);
}

// Whether every token's channels, and every group's, start on 16 bytes.
bool by_16_bytes(const SsmParams& p) {
  const int64_t e = p.dtype == LQ_F32 ? 4 : 2;
  uint64_t bits = (uint64_t)p.x | (uint64_t)p.dt | (uint64_t)p.z | (uint64_t)p.y;
  bits |= (uint64_t)((p.sx | p.sdt | p.sy | (p.z ? p.sz : 0)) * e);
  if (p.groups > 1) bits |= (uint64_t)(p.per_group * e);
  return bits % 16 == 0;
}

template <typename T>
cudaError_t launch(const SsmParams& p, cudaStream_t st) {
  if (by_16_bytes(p)) return p.softplus ? launch_states<T, true, true>(p, st) : launch_states<T, false, true>(p, st);
  return p.softplus ? launch_states<T, true, false>(p, st) : launch_states<T, false, false>(p, st);
}

// --------------------------------------------------------------------------------------------
// Single tokens.
template <typename T, int N>
__device__ __forceinline__ void token(const SsmParams& p, int64_t t, int c, int g, const float (&A)[N], float bias,
                                      float D, float (&h)[N]) {
  const float d = p.softplus ? step_of<T, true>(static_cast<const T*>(p.dt)[t * p.sdt + c], bias)
                             : step_of<T, false>(static_cast<const T*>(p.dt)[t * p.sdt + c], bias);
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

// CTAs that a split call should come to, as many as 152 SMs hold at a time, and the least tokens of a segment.
int64_t split_ctas(int n_state) { return 152 * (n_state <= 8 ? 8 : n_state <= 16 ? 6 : 5); }
constexpr int64_t kLeastSeg = 64;

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
  const int64_t ctas = split_ctas(c->n_state);
  int64_t s = ((work + ctas - 1) / ctas + 15) / 16 * 16;
  s = s < kLeastSeg ? kLeastSeg : s;
  if (longest < 3 * s) return;
  const double all = 95.0 / 152 * (double)work, whole = 140.0 * (double)longest;
  if ((all > whole ? all : whole) <= 1.8 * all + 280.0 * (double)s + 8000.0) return;
  *seg = s;
  *slots = n_tokens / s + n_seqs;
}

// A segment has at least kLeastSeg tokens and at least a split_ctas-th of the call's work.
int64_t ssm_most_slots(const lq_ssm_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len) {
  const int64_t longest = max_len > 0 && max_len < n_tokens ? max_len : n_tokens;
  if (longest < 3 * kLeastSeg) return 0;
  const int64_t a = n_tokens / kLeastSeg, b = split_ctas(c->n_state) / ssm_blocks(c);
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
