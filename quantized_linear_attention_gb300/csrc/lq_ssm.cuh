// Selective state space scan over packed prompts (sm_103a): for every channel and state
//   h <- exp(d A) h + d x B,   y = (sum_n C h + D x) silu(z).
#pragma once

#include <type_traits>

#include "lq_device.cuh"
#include "lq_seq.cuh"

namespace lqi {

// Blocks of channels of a group.
__host__ __device__ inline int ssm_group_blocks(int per_group, int lpc) {
  return (int)(((int64_t)per_group * lpc + 127) / 128);
}

cudaError_t launch_ssm_prefill_f32(const SsmParams& p, cudaStream_t st);
cudaError_t launch_ssm_prefill_bf16(const SsmParams& p, cudaStream_t st);
cudaError_t launch_ssm_prefill_f16(const SsmParams& p, cudaStream_t st);

namespace {

// --------------------------------------------------------------------------------------------
// Prompts. A thread holds SPT states of a channel (LPC lanes of a warp share one channel) and takes the tokens of a piece
// one after the other: per state and token a multiplication and an exponential for the decay, a multiplication and an fma for
// the state and an fma for y, in packed pairs of states. x, dt and z come into shared memory a tile ahead by asynchronous
// copies, y goes out from there by 16 bytes; B and C, the same for all channels of a group, lie there as floats.
//
// What bounds it: 11 operands from the register file for each state and token, whose two banks give two a cycle: 105 cycles
// of an SM's quarter for 512 states and a token, measured on these operations alone (their FMAs and their exponentials take
// 64 each). Steps, gates and copies come on top: 1,024 tokens x 65,536 channels of 16 states (bf16) take 340 us, 187 cycles. With
// so few channels that an SM has one CTA the waits count instead: 136 ns a token with 16 states a thread, 52 with four
// and 32 tokens begun together, which is a third slower where there are many.
//
// A decay is ex2.approx of d times A log2 e: off by (4 + 2.3 |d A|) 2^-24 of itself, for ex2 and for three roundings of the
// exponent. What those leave out could be put back as in exp_near, for the unrounded A in as many registers again and two more
// packed fmas to every five operations of a pair of states, where register operands are what bounds the kernel. Measured
// after 8,192 tokens against 64 bits (fp32, no softplus; relative L2 of the states, d around 0.1, 0.01, 0.001): 5e-7, 1.2e-6,
// 1.2e-6 split and 6e-7, 2.8e-6, 1.2e-5 whole, where an fp32 exp of a rounded d A gives 2e-7, 3.9e-6, 2.8e-5: twice to three
// times its error where memories are short, less where they are long.
//
// A sequence that would leave most of the GPU idle is split into segments (ssm_plan). The first pass takes
// every segment but the last from a zero state (the first from its true one, with its outputs) and leaves its last state and
// the sum of its d; since the decays of a segment multiply to exp(A sum d), k_ssm_join finds the state before each segment,
// and the second pass takes the segments from there. What that sum over segments does not give as the recurrence does (a
// positive A or a negative d, where it may overflow though the recurrence does not, infinities, values near fp32's largest
// number) k_ssm_join takes token by token. 16,384 tokens x 4,096 channels of 16 states (bf16) take 496 us: two fifths the first
// pass, the rest the second, which a single pass that leaves three quarters of the GPU idle cannot match (833).
constexpr int kNT = 128;
// Tokens begun together, and in shared memory at a time. More of them hide more of each other's waits (one CTA an SM: 136 ->
// 52 ns a token with four states a thread and 32 tokens), as far as the registers go. (Four states and eight lanes: 61 to 63 ns
// in bf16 and fp32 with 16 tokens; 52 and 74 with 32, 56 and 53 with 64, but short calls then wait for a larger first tile.)
template <typename T, int SPT, int LPC>
constexpr int kGroup = SPT == 4 ? (LPC == 8 ? 16 : 8 * LPC) : SPT == 8 ? (LPC == 1 ? 8 : LPC == 8 ? 32 : 16) : LPC > 1 ? 32 : sizeof(T) == 4 ? 16 : 8;
template <typename T, int SPT, int LPC>
constexpr int kTile = kGroup<T, SPT, LPC> < 32 / (int)sizeof(T) ? 32 / (int)sizeof(T) : kGroup<T, SPT, LPC>;

// A token's step d.
template <typename T, bool PLUS>
__device__ __forceinline__ float step_of(T dt, float bias) {
  const float v = __fadd_rn(to_f(dt), bias);
  return PLUS ? softplus(v) : v;
}

template <typename T, int SPT, int LPC>
struct Smem {
  static constexpr int CH = kNT / LPC, NP = SPT * LPC, TT = kTile<T, SPT, LPC>;
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
    if (VEC) copy_ahead(&to[t][c], n ? from + (int64_t)(t0 + t) * stride + c : from, n * (int)sizeof(T));
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
  constexpr int NP = SPT * LPC, CW = 32 / LPC, CH = kNT / LPC, TT = kTile<T, SPT, LPC>, kUnroll = kGroup<T, SPT, LPC>, PER = (TT * NP + kNT - 1) / kNT, H = SPT / 2;
  const int tid = threadIdx.x, part = (tid & 31) / CW, n0 = part * SPT, col = (tid >> 5) * CW + (tid & 31) % CW;
  const int len = (int)pc.len;
  const bool live = col < ch.left, gate = p.z != nullptr, skip = p.D != nullptr;
  const int c = ch.c0 + (live ? col : 0);
  const T* x = static_cast<const T*>(p.x) + pc.begin * p.sx + ch.c0;
  const T* dt = static_cast<const T*>(p.dt) + pc.begin * p.sdt + ch.c0;
  const T* z = gate ? static_cast<const T*>(p.z) + pc.begin * p.sz + ch.c0 : nullptr;
  T* y = static_cast<T*>(p.y) + pc.begin * p.sy + ch.c0;
  const T* B = static_cast<const T*>(p.B) + pc.begin * p.sb + (int64_t)ch.g * p.n_state;
  const T* C = static_cast<const T*>(p.C) + pc.begin * p.sc + (int64_t)ch.g * p.n_state;
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, D = skip ? p.D[c] : 0.0f;
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
    // A group of kUnroll tokens: all steps d first, two tokens to a packed pair, then the recurrence, then the gates; shared
    // memory is read before it is written, so that the compiler may begin the whole group at once. Lanes that share a channel
    // make the steps and gates of OWN tokens each and pass them on. CHECK: some of the group are past the end.
    constexpr int OWN = kUnroll / LPC;
    static_assert(OWN % 2 == 0 && TT % kUnroll == 0, "tokens go in pairs, tiles in whole groups");
    auto group = [&](int tg, auto check) {
      constexpr bool CHECK = decltype(check)::value;
      const int n = min(kUnroll, len - t0 - tg);
      float d[OWN], dx[OWN];
#pragma unroll
      for (int u = 0; u < OWN; u += 2) {
        const int t = tg + part * OWN + u;
        float v[2], xv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v[e] = __fadd_rn(to_f(sm.dt[buf][t + e][col]), bias);
          xv[e] = to_f(sm.x[buf][t + e][col]);
        }
        f32x2 d2 = f2_pack(v[0], v[1]);
        if (PLUS) d2 = softplus2(d2);
        f2_unpack(d2, d[u], d[u + 1]);
        f2_unpack(f2_mul(d2, f2_pack(xv[0], xv[1])), dx[u], dx[u + 1]);
      }
      float o[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (CHECK && u >= n) break;
        const int t = tg + u;
        float du = d[u % OWN], dxu = dx[u % OWN];
        if (LPC > 1) {
          const int lane = u / OWN * CW + (tid & 31) % CW;
          du = __shfl_sync(0xffffffffu, du, lane);
          dxu = __shfl_sync(0xffffffffu, dxu, lane);
        }
        const f32x2 d2 = f2_dup(du), dx2 = f2_dup(dxu);
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
          o[u] = __fadd_rn(y0, y1);
#pragma unroll
          for (int s = CW; s < 32; s <<= 1) o[u] = __fadd_rn(o[u], __shfl_xor_sync(0xffffffffu, o[u], s));
        } else {
          dpart = __fadd_rn(dpart, du);
          dmin = du >= dmin ? dmin : (du < dmin ? du : -1.0f);  // (a NaN counts as negative)
          ax = __fadd_rn(ax, fabsf(dxu));
        }
      }
      if (OUT) {
        float r[OWN];
#pragma unroll
        for (int u = 0; u < OWN; u += 2) {
          float v[2], zv[2], xv[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = tg + part * OWN + u + e;
            v[e] = o[u + e];
#pragma unroll
            for (int q = 1; q < LPC; ++q) v[e] = part == q ? o[q * OWN + u + e] : v[e];
            xv[e] = to_f(sm.x[buf][t][col]);
            zv[e] = to_f(sm.z[buf][t][col]);
          }
          f32x2 g = f2_pack(v[0], v[1]);
          if (skip) g = f2_fma(f2_dup(D), f2_pack(xv[0], xv[1]), g);
          if (gate) g = f2_mul(g, silu2<T>(f2_pack(zv[0], zv[1])));
          f2_unpack(g, r[u], r[u + 1]);
        }
#pragma unroll
        for (int u = 0; u < OWN; ++u) sm.y[tg + part * OWN + u][col] = from_f<T>(r[u]);  // (past the end nobody reads it)
      }
    };
#pragma unroll 1
    for (int tg = 0; tg < TT; tg += kUnroll) {
      if (t0 + tg + kUnroll <= len) {
        group(tg, std::false_type());
      } else {
        if (t0 + tg < len) group(tg, std::true_type());
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
  // Where no sequence is longer than a segment every CTA leaves below. One waits for the first pass all the same: the second
  // pass, and what the caller does next in the stream, count on that pass' end when this grid has ended.
  if (blockIdx.x == 0) cudaGridDependencySynchronize();
  const int64_t b = blockIdx.x / (unsigned)blocks, row = (int64_t)p.channels * p.n_state;
  const int64_t at = (int64_t)(blockIdx.x % (unsigned)blocks) * 256 + threadIdx.x;
  Piece pc;
  bounds(p, b, pc.begin, pc.len);
  pc.n = pc.len > p.seg ? (pc.len + p.seg - 1) / p.seg : 1;
  if (pc.n == 1) return;
  const int64_t slot = first_slot<256>(p, b);
  cudaGridDependencySynchronize();
  if (at >= row || slot >= p.slots) return;  // (no such slots where sequences do not overlap)
  const int64_t c = at / p.n_state, segs = min(pc.n, p.slots - slot);
  float* ws = p.ws_state + slot * row + at;
  const float* step = p.ws_step + slot * p.channels + c;
  const float A = p.A[at], A2 = __fmul_rn(A, kLog2E);
  const bool falls = A <= 0.0f && A > -1e30f;
  float h = ws[0];
  int64_t i = 1;
  auto goes = [&](float sum) { return falls && sum == sum && fabsf(h) < 1e30f; };
  for (bool fine = true; fine && i < segs; i += fine ? U : 0) {
    float add[U], sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      add[u] = sum[u] = 0.0f;
      if (i + u < segs - 1) {
        add[u] = ws[(i + u) * row];
        sum[u] = step[(i + u) * p.channels];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!fine || i + u >= segs) continue;
      ws[(i + u) * row] = h;
      if (i + u == segs - 1) continue;
      if (goes(sum[u])) {
        h = __fmaf_rn(ex2_approx(__fmul_rn(sum[u], A2)), h, add[u]);
      } else {
        fine = false;
        i += u;
      }
    }
  }
  // from the first segment on that its sum does not tell of
  for (; i < segs; ++i) {
    const float add = ws[i * row];
    ws[i * row] = h;
    if (i == segs - 1) break;
    const float sum = step[i * p.channels];
    h = goes(sum) ? __fmaf_rn(ex2_approx(__fmul_rn(sum, A2)), h, add) : walk<T, PLUS>(p, pc.begin + i * p.seg, at, h);
  }
}

template <typename T, int SPT, int LPC, bool PLUS, bool VEC>
cudaError_t launch_shape(const SsmParams& p, cudaStream_t st) {
  const int per = ssm_group_blocks(p.per_group, LPC), blocks = per * p.groups;
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
  switch (p.spt * 16 + p.lpc) {
    case 8 * 16 + 1: return launch_shape<T, 8, 1, PLUS, VEC>(p, st);
    case 4 * 16 + 2: return launch_shape<T, 4, 2, PLUS, VEC>(p, st);
    case 16 * 16 + 1: return launch_shape<T, 16, 1, PLUS, VEC>(p, st);
    case 8 * 16 + 2: return launch_shape<T, 8, 2, PLUS, VEC>(p, st);
    case 4 * 16 + 4: return launch_shape<T, 4, 4, PLUS, VEC>(p, st);
    case 16 * 16 + 2: return launch_shape<T, 16, 2, PLUS, VEC>(p, st);
    case 8 * 16 + 4: return launch_shape<T, 8, 4, PLUS, VEC>(p, st);
    case 4 * 16 + 8: return launch_shape<T, 4, 8, PLUS, VEC>(p, st);
    case 16 * 16 + 4: return launch_shape<T, 16, 4, PLUS, VEC>(p, st);
    case 8 * 16 + 8: return launch_shape<T, 8, 8, PLUS, VEC>(p, st);
    default: return cudaErrorInvalidConfiguration;  // (ssm_plan's loop has no other shape)
  }
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

}  // namespace

}  // namespace lqi
