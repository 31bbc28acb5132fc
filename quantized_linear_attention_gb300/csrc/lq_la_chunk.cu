// Linear attention with a decay per head over prompts of bf16 tokens, in chunks of
// 128 on the tensor cores (sm_103a, tcgen05).
//
// With G_i the sum of log2 alpha over tokens 0..i of a chunk and S the state before it,
//   o_i = 2^{G_i} S q_i + sum_{j <= i} 2^{G_i - G_j} (q_i . k_j) v_j
//   S  <- 2^{G_127} S + sum_j 2^{G_127 - G_j} v_j k_j^T.
// One CTA takes a head of a sequence (or of a segment of one) from its first
// chunk to its last; the state never leaves the SM. Four products per chunk, all
// 128 x 128 x 128 with fp32 accumulators in TMEM:
//   P  = Q K^T       both operands from shared memory
//   O  = Q S^T       S rounded to bf16 in shared memory: only o needs this product,
//                    and o is rounded to bf16 itself
//   O += P V         P (weighted, masked, rounded to bf16) from TMEM
//   U  = (wV)^T K    the state's growth. wV is an fp32 number; it goes in as three
//                    bf16 parts that hold all its 24 bits, so the state keeps fp32's
//                    accuracy (two parts, 16 bits, were not enough: 2.8e-6).
// S itself stays in fp32 registers: S <- gamma S + U in one rounding to nearest
// per step, with gamma in two parts, because a rounded gamma would be off in the
// same direction chunk after chunk. Sums of logarithms are whole numbers of 2^-40.
//
// Warps: 0-7 weigh P, scale O and write o (A); 8-15 keep the state and make
// the parts of wV (B); 16-17 copy tiles (even and odd chunks); 18 sums the
// logarithms; 19 issues the products. They meet at mbarriers only. Every wait is
// bounded; one that gives up ends the CTA's work, and the outputs become NaN.
//
// A masked product cannot hold back 0 x inf: where a chunk's values are not all
// finite, or a decay is not in [0, 1], the CTA takes its tokens again one by one
// (redo), exactly as the recurrence is written.
#include "lq_device.cuh"
#include "lq_la.cuh"

namespace lqi {

namespace {

constexpr int kC = 128;  // tokens per chunk
constexpr int kThreadsLa = 640;
constexpr uint32_t kTile = 32768;             // 128 x 128 bf16: two halves of 64 channels, 128-byte rows, swizzled
constexpr uint32_t kStage = 3 * kTile;        // Q, K, V
constexpr uint32_t kS16 = 2 * kStage;         // the state in bf16
constexpr uint32_t kSums = kS16 + kTile;      // G[2][128], w[2][128]
constexpr uint32_t kMisc = kSums + 2048;      // gammas, barriers
constexpr uint32_t kSmem = kMisc + 512;
static_assert(kSmem <= 232448, "shared memory of a CTA");
// TMEM columns
constexpr uint32_t kU = 0, kP = 128, kO = 256, kV3 = 384;  // kV3: two buffers of 3 parts x 16 columns (32 tokens)

struct Misc {
  float2 gamma[4];
  uint64_t full[2], empty[2], sums[2], qk, qs, pv, pvok, ofree, sready, vfull[2], vfree[2], drain;
  uint32_t tmem;
  int abort, flag;
  double prod;
  int64_t piece[5];
};
static_assert(sizeof(Misc) <= 512, "misc");

__device__ __forceinline__ uint64_t desc_k(uint32_t a) {  // rows of the operand are rows of the tile
  return (uint64_t)((a & 0x3ffff) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t a) {  // rows of the operand are channels of the tile
  return (uint64_t)((a & 0x3ffff) >> 4) | (1024ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// fp32 accumulators, bf16 operands, M = N = 128; B by channels or by rows
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (16u << 17) | (8u << 24);
constexpr uint32_t kIdescMn = kIdesc | (1u << 16);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tm_ld32(uint32_t a, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}
__device__ __forceinline__ void tm_st32(uint32_t a, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits for phase `parity`; false once this or any other wait of the CTA has given up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(abort)) return false;
    if (globaltimer_ns() - t0 > 2000000000ull) {
      *reinterpret_cast<volatile int*>(abort) = 1;
      return false;
    }
  }
}

// The same for a whole warp: all lanes go on or none does.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* abort) {
  return __all_sync(0xffffffffu, wait(bar, parity, abort));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {  // to nearest
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

using bf16 = __nv_bfloat16;

// The state before segment i, columns [c0, c0 + 16) of row `row`: S0 (or zero), then what segments 0..i-1 added.
__device__ __forceinline__ void start_state(const LaParams& p, const Piece& pc, int64_t slot, int h, int row, int c0,
                                            float s[16]) {
  if (p.S0) {
    const float* a = p.S0 + (((pc.b * p.heads + h) * kD) + row) * kD + c0;
#pragma unroll
    for (int e = 0; e < 16; e += 4) ld4(a + e, s + e);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = 0.f;
  }
  for (int64_t r = slot - pc.i; r < slot; ++r) {
    const double d = p.ws_decay[r * p.heads + h];
    const float hi = (float)d, lo = (float)(d - (double)hi);
    const float* a = p.ws_state + (((r * p.heads + h) * kD) + row) * kD + c0;
    float u[16];
#pragma unroll
    for (int e = 0; e < 16; e += 4) ld4(a + e, u + e);
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = __fmaf_rn(s[e], hi, __fmaf_rn(s[e], lo, u[e]));
  }
}

// Token by token: 512 threads, four lanes to a row, 32 columns each (as k_la_recurrent).
// OUT: from the segment's start, with outputs; else from zero, the segment's own sum.
template <bool OUT>
__device__ __noinline__ void redo(const LaParams& p, const Piece& pc, int64_t slot, int h, float* sm, float* S_out,
                                  double* decay) {
  const int tid = threadIdx.x, part = tid & 3, row = tid >> 2, kh = h / p.group;
  float(*sk)[kD] = reinterpret_cast<float(*)[kD]>(sm);
  float(*sq)[kD] = sk + 16;
  float(*sv)[kD] = sq + 16;
  float* sa = reinterpret_cast<float*>(sv + 16);
  const bf16* q = static_cast<const bf16*>(p.q) + kh * kD;
  const bf16* k = static_cast<const bf16*>(p.k) + kh * kD;
  const bf16* v = static_cast<const bf16*>(p.v) + h * kD;
  bf16* o = static_cast<bf16*>(p.o) + h * kD;
  float S[8][4];
  double prod = 1.0;
  if (tid < 512) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int col = 4 * (4 * c + part);
      S[c][0] = S[c][1] = S[c][2] = S[c][3] = 0.f;
      if (!OUT) continue;
      if (p.S0) ld4(p.S0 + (((pc.b * p.heads + h) * kD) + row) * kD + col, S[c]);
      for (int64_t r = slot - pc.i; r < slot; ++r) {
        const double d = p.ws_decay[r * p.heads + h];
        const float hi = (float)d, lo = (float)(d - (double)hi);
        float u[4];
        ld4(p.ws_state + (((r * p.heads + h) * kD) + row) * kD + col, u);
#pragma unroll
        for (int e = 0; e < 4; ++e) S[c][e] = __fmaf_rn(S[c][e], hi, __fmaf_rn(S[c][e], lo, u[e]));
      }
    }
  }
  for (int64_t t0 = 0; t0 < pc.len; t0 += 16) {
    const int n = (int)min((int64_t)16, pc.len - t0);
    __syncthreads();
    if (tid < 512 && (tid >> 5) < n) {
      const int t = tid >> 5, c = 4 * (tid & 31);
      const int64_t at = pc.begin + t0 + t;
      ld4(k + at * p.sk + c, &sk[t][c]);
      if (OUT) ld4(q + at * p.sq + c, &sq[t][c]);
      ld4(v + at * p.sv + c, &sv[t][c]);
      if (c == 0) sa[t] = p.alpha[at * p.sa + h];
    }
    __syncthreads();
    if (tid < 512) {
      for (int t = 0; t < n; ++t) {
        const float a = sa[t], vv = sv[t][row];
        prod *= (double)a;
        float acc = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float kk[4], qq[4] = {0.f, 0.f, 0.f, 0.f};
          ld4(&sk[t][4 * (4 * c + part)], kk);
          if (OUT) ld4(&sq[t][4 * (4 * c + part)], qq);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            S[c][e] = __fmaf_rn(vv, kk[e], __fmul_rn(a, S[c][e]));
            if (OUT) acc = __fmaf_rn(S[c][e], qq[e], acc);
          }
        }
        if (OUT) {
          acc += __shfl_xor_sync(0xffffffffu, acc, 1);
          acc += __shfl_xor_sync(0xffffffffu, acc, 2);
          if (part == 0) o[(pc.begin + t0 + t) * p.so + row] = __float2bfloat16_rn(acc);
        }
      }
    }
  }
  if (S_out && tid < 512) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<float4*>(S_out + row * kD + 4 * (4 * c + part)) =
          make_float4(S[c][0], S[c][1], S[c][2], S[c][3]);
  }
  if (decay && tid == 0) *decay = prod;
}

// OUT: outputs and last states. Otherwise the first pass over split sequences: what a segment adds to the state.
template <bool OUT>
__global__ void __launch_bounds__(kThreadsLa, 1) k_la_chunk(LaParams p) {
  extern __shared__ __align__(1024) char la_smem[];
  Misc& ms = *reinterpret_cast<Misc*>(la_smem + kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = (int)(blockIdx.x % (unsigned)p.heads), kh = h / p.group;
  const int64_t slot = blockIdx.x / (unsigned)p.heads;
  if (warp == 0) {
    const Piece f = find_piece(p, slot);
    if (lane == 0) ms.piece[0] = f.b, ms.piece[1] = f.begin, ms.piece[2] = f.len, ms.piece[3] = f.i, ms.piece[4] = f.n;
  }
  __syncthreads();
  Piece pc;
  pc.b = ms.piece[0], pc.begin = ms.piece[1], pc.len = ms.piece[2], pc.i = ms.piece[3], pc.n = ms.piece[4];
  if (pc.b < 0 || (!OUT && pc.i == pc.n - 1)) return;
  const bool last = pc.i == pc.n - 1;
  // Where the state after the piece goes.
  float* S_out = OUT ? (last && p.S ? p.S + (pc.b * p.heads + h) * (kD * kD) : nullptr)
                     : p.ws_state + (slot * p.heads + h) * (kD * kD);
  const int nc = (int)((pc.len + kC - 1) / kC);

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ms.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.full[i], 32);
      mbar_init(&ms.empty[i], 1);
      mbar_init(&ms.sums[i], 32);
      mbar_init(&ms.vfull[i], 256);
      mbar_init(&ms.vfree[i], 1);
    }
    mbar_init(&ms.qk, 1);
    mbar_init(&ms.qs, 1);
    mbar_init(&ms.pv, 1);
    mbar_init(&ms.pvok, 256);
    mbar_init(&ms.ofree, 256);
    mbar_init(&ms.sready, 256);
    mbar_init(&ms.drain, 1);
    ms.abort = ms.flag = 0;
    ms.prod = 1.0;
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = ms.tmem, sb = smem_u32(la_smem);
  float* sG = reinterpret_cast<float*>(la_smem + kSums);
  float* sw = sG + 2 * kC;
  int* ab = &ms.abort;
  float S[64];  // warps 8-15: row 32 (warp & 3) + lane, columns 64 (warp >= 12) ..

  if (warp < 8) {
    if (OUT) {
      // A: row i = 32 (warp & 3) + lane of the chunk, columns 64 half .. 64 half + 63
      const int quad = warp & 3, half = warp >> 2, i = 32 * quad + lane;
      const uint32_t tl = tm + ((uint32_t)(32 * quad) << 16);
      bf16* o = static_cast<bf16*>(p.o) + h * kD + 64 * half;
      for (int c = 0; c < nc; ++c) {
        const float* G = sG + (c & 1) * kC;
        if (!wait_warp(&ms.sums[c & 1], (c >> 1) & 1, ab)) break;
        const float gi = G[i];
        const float ei = ex2(gi);
        if (!wait_warp(&ms.qk, c & 1, ab)) break;
        tc_after();
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {  // 32 columns j at a time
          const int j0 = 64 * half + 32 * blk;
          uint32_t w[16];
          if (j0 > 32 * quad + 31) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = 0u;
          } else {
            uint32_t x[32];
            tm_ld32(tl + kP + j0, x);
            wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 g = *reinterpret_cast<const float4*>(G + j0 + e);
              const float gj[4] = {g.x, g.y, g.z, g.w};
              float y[4];
#pragma unroll
              for (int f = 0; f < 4; ++f)
                y[f] = j0 + e + f <= i ? __fmul_rn(__uint_as_float(x[e + f]), ex2(__fsub_rn(gi, gj[f]))) : 0.f;
              w[e / 2] = pack_bf16(y[0], y[1]);
              w[e / 2 + 1] = pack_bf16(y[2], y[3]);
            }
          }
          // P's tokens 64 half .. sit in columns 64 half .. of its own accumulator: a warp overwrites what it has read
          tm_st16(tl + kP + 64 * half + 16 * blk, w);
        }
        if (!wait_warp(&ms.qs, c & 1, ab)) break;
        tc_after();
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          uint32_t x[32];
          tm_ld32(tl + kO + 64 * half + 32 * blk, x);
          wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__fmul_rn(ei, __uint_as_float(x[e])));
          tm_st32(tl + kO + 64 * half + 32 * blk, x);
        }
        wait_st();
        tc_before();
        arrive(&ms.pvok);
        if (!wait_warp(&ms.pv, c & 1, ab)) break;
        tc_after();
        uint32_t y[32];
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          uint32_t x[32];
          tm_ld32(tl + kO + 64 * half + 32 * blk, x);
          wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            y[16 * blk + e] = pack_bf16(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
        }
        tc_before();
        arrive(&ms.ofree);
        const int64_t t = (int64_t)c * kC + i;
        if (t < pc.len) {
          uint4* dst = reinterpret_cast<uint4*>(o + (pc.begin + t) * p.so);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
        }
      }
    }
  } else if (warp < 16) {
    // B
    const int quad = warp & 3, half = (warp - 8) >> 2, row = 32 * quad + lane;
    const uint32_t tl = tm + ((uint32_t)(32 * quad) << 16);
#pragma unroll
    for (int blk = 0; blk < 4; ++blk) {
      if (OUT) start_state(p, pc, slot, h, row, 64 * half + 16 * blk, &S[16 * blk]);
      else
#pragma unroll
        for (int e = 0; e < 16; ++e) S[16 * blk + e] = 0.f;
    }
    bool ok = true, odd = false;
    for (int c = 0; c <= nc; ++c) {
      if (!(ok = wait_warp(&ms.sums[c & 1], (c >> 1) & 1, ab))) break;
      if (c) {  // S <- gamma S + U
        if (!(ok = wait_warp(&ms.empty[(c - 1) & 1], ((c - 1) >> 1) & 1, ab))) break;
        tc_after();
        const float2 g = ms.gamma[(c - 1) & 3];
#pragma unroll
        for (int blk = 0; blk < 4; ++blk) {
          uint32_t u[16];
          tm_ld16(tl + kU + 64 * half + 16 * blk, u);
          wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float& s = S[16 * blk + e];
            s = __fmaf_rn(s, g.x, __fmaf_rn(s, g.y, __uint_as_float(u[e])));
          }
        }
        tc_before();
      }
      if (c == nc) break;
      if (OUT) {
        char* s16 = la_smem + kS16 + half * 16384 + row * 128;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint4 x;
          x.x = pack_bf16(S[8 * e], S[8 * e + 1]);
          x.y = pack_bf16(S[8 * e + 2], S[8 * e + 3]);
          x.z = pack_bf16(S[8 * e + 4], S[8 * e + 5]);
          x.w = pack_bf16(S[8 * e + 6], S[8 * e + 7]);
          *reinterpret_cast<uint4*>(s16 + ((e ^ (row & 7)) << 4)) = x;
        }
        fence_proxy_async();
        arrive(&ms.sready);
      }
      if (!(ok = wait_warp(&ms.full[c & 1], (c >> 1) & 1, ab))) break;
      const char* V = la_smem + (c & 1) * kStage + 2 * kTile + (row >> 6) * 16384 + (row & 7) * 2;
      const int chunk16 = (row & 63) >> 3;
      const float* w = sw + (c & 1) * kC;
#pragma unroll 1
      for (int qt = 0; qt < 4; ++qt) {  // 32 tokens; this warp's 16 of them
        const int buf = qt & 1, use = 2 * c + (qt >> 1);
        if (use && !(ok = wait_warp(&ms.vfree[buf], (use - 1) & 1, ab))) break;
        tc_after();
        uint32_t p0[8], p1[8], p2[8];
        const int j0 = 32 * qt + 16 * half;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float r[2];
          uint32_t a[2], b[2], d[2];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int j = j0 + 2 * e + f;
            const uint32_t bits = *reinterpret_cast<const uint16_t*>(V + j * 128 + ((chunk16 ^ (j & 7)) << 4));
            odd |= (bits & 0x7f80u) == 0x7f80u;
            const float x = __fmul_rn(__uint_as_float(bits << 16), w[j]);
            // the top 8 bits, the next 8, the last 8: each difference is exact
            a[f] = __float_as_uint(x) & 0xffff0000u;
            r[f] = __fsub_rn(x, __uint_as_float(a[f]));
            b[f] = __float_as_uint(r[f]) & 0xffff0000u;
            d[f] = __float_as_uint(__fsub_rn(r[f], __uint_as_float(b[f])));
          }
          p0[e] = __byte_perm(a[0], a[1], 0x7632);
          p1[e] = __byte_perm(b[0], b[1], 0x7632);
          p2[e] = __byte_perm(d[0], d[1], 0x7632);
        }
        const uint32_t at = tl + kV3 + 48 * buf + 8 * half;
        tm_st8(at, p0);
        tm_st8(at + 16, p1);
        tm_st8(at + 32, p2);
        wait_st();
        tc_before();
        arrive(&ms.vfull[buf]);
      }
      if (!ok) break;
    }
    if (odd) ms.flag = 1;
  } else if (warp < 18) {
    // Copies: tokens past the end are zeros.
    const bf16* src[3] = {static_cast<const bf16*>(p.q) + kh * kD, static_cast<const bf16*>(p.k) + kh * kD,
                          static_cast<const bf16*>(p.v) + h * kD};
    const int64_t st[3] = {p.sq, p.sk, p.sv};
    for (int c = warp - 16; c < nc; c += 2) {
      if (c >= 2 && !wait_warp(&ms.empty[c & 1], ((c - 2) >> 1) & 1, ab)) break;
      const int64_t t0 = pc.begin + (int64_t)c * kC;
      const int n = (int)min((int64_t)kC, pc.len - (int64_t)c * kC);
      const int ch = lane & 15;
#pragma unroll
      for (int x = OUT ? 0 : 1; x < 3; ++x) {
        const uint32_t dst = sb + (c & 1) * kStage + x * kTile + (ch >> 3) * 16384;
        const bf16* from = src[x] + t0 * st[x] + 8 * ch;
#pragma unroll 8
        for (int r = lane >> 4; r < kC; r += 2)
          cp16(dst + r * 128 + (((ch & 7) ^ (r & 7)) << 4), r < n ? from + r * st[x] : from, r < n);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async();
      arrive(&ms.full[c & 1]);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 18) {
    // Sums of log2 alpha in whole numbers of 2^-40, four tokens to a lane. A decay of
    // zero counts 2^-200: any weight across it is below fp32's smallest number.
    double prod = 1.0;
    bool odd = false;
    for (int c = 0; c <= nc; ++c) {
      if (c >= 2 && !wait_warp(&ms.empty[c & 1], ((c - 2) >> 1) & 1, ab)) break;
      if (c == nc) {
        arrive(&ms.sums[c & 1]);
        break;
      }
      long long g[4], run = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t t = (int64_t)c * kC + 4 * lane + e;
        float l = 0.f;
        if (t < pc.len) {
          const float a = p.alpha[(pc.begin + t) * p.sa + h];
          if (!(a >= 0.f && a <= 1.f)) odd = true;
          l = a > 0.f ? fmaxf(log2f(a), -200.f) : -200.f;
        }
        run += __float2ll_rn(__fmul_rn(l, 1099511627776.f));
        g[e] = run;
      }
      long long sum = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      const long long end = __shfl_sync(0xffffffffu, sum, 31);
      float G[4], w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] += sum - run;
        G[e] = __fmul_rn(__ll2float_rn(g[e]), 9.094947017729282e-13f);
        w[e] = exp2f(__fmul_rn(__ll2float_rn(end - g[e]), 9.094947017729282e-13f));
      }
      *reinterpret_cast<float4*>(sG + (c & 1) * kC + 4 * lane) = make_float4(G[0], G[1], G[2], G[3]);
      *reinterpret_cast<float4*>(sw + (c & 1) * kC + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
      arrive(&ms.sums[c & 1]);
      // gamma is wanted one chunk later
      const double gm = exp2((double)end * 9.094947017729282e-13);
      prod *= gm;
      if (lane == 0) {
        const float hi = (float)gm;
        ms.gamma[c & 3] = make_float2(hi, (float)(gm - (double)hi));
      }
      __syncwarp();
    }
    if (odd) ms.flag = 1;
    if (lane == 0) ms.prod = prod;
  } else if (lane == 0) {
    // The products.
    for (int c = 0; c < nc; ++c) {
      const uint32_t Q = sb + (c & 1) * kStage, K = Q + kTile, V = K + kTile, S16 = sb + kS16;
      if (!wait(&ms.full[c & 1], (c >> 1) & 1, ab)) break;
      tc_after();
      if (OUT) {
        for (int s = 0; s < 8; ++s) {
          const uint32_t off = (s >> 2) * 16384 + (s & 3) * 32;
          mma_ss(tm + kP, desc_k(Q + off), desc_k(K + off), kIdesc, s > 0);
        }
        commit(&ms.qk);
        if (!wait(&ms.sready, c & 1, ab)) break;
        if (c && !wait(&ms.ofree, (c - 1) & 1, ab)) break;
        tc_after();
        for (int s = 0; s < 8; ++s) {
          const uint32_t off = (s >> 2) * 16384 + (s & 3) * 32;
          mma_ss(tm + kO, desc_k(Q + off), desc_k(S16 + off), kIdesc, s > 0);
        }
        commit(&ms.qs);
      }
      bool ok = true;
      for (int qt = 0; qt < 4; ++qt) {
        const int buf = qt & 1, use = 2 * c + (qt >> 1);
        if (OUT && qt == 2) {
          if (!(ok = wait(&ms.pvok, c & 1, ab))) break;
          tc_after();
          for (int s = 0; s < 8; ++s)
            mma_ts(tm + kO, tm + kP + 64 * (s >> 2) + 8 * (s & 3), desc_mn(V + s * 2048), kIdescMn, true);
          commit(&ms.pv);
        }
        if (!(ok = wait(&ms.vfull[buf], use & 1, ab))) break;
        tc_after();
        for (int part = 2; part >= 0; --part)  // the small parts first
          for (int s = 0; s < 2; ++s)
            mma_ts(tm + kU, tm + kV3 + 48 * buf + 16 * part + 8 * s, desc_mn(K + (2 * qt + s) * 2048), kIdescMn,
                   !(qt == 0 && part == 2 && s == 0));
        commit(&ms.vfree[buf]);
      }
      if (!ok) break;
      commit(&ms.empty[c & 1]);
    }
    // nothing may be in flight when TMEM is given back
    commit(&ms.drain);
    int ignored = 0;
    wait(&ms.drain, 0, &ignored);
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  if (ms.abort) {  // a wait gave up: make that visible
    const bf16 bad = __float2bfloat16_rn(__int_as_float(0x7fc00000));
    if (OUT)
      for (int64_t x = tid; x < pc.len * kD; x += kThreadsLa)
        static_cast<bf16*>(p.o)[(pc.begin + x / kD) * p.so + h * kD + x % kD] = bad;
    if (S_out)
      for (int x = tid; x < kD * kD; x += kThreadsLa) S_out[x] = __int_as_float(0x7fc00000);
    if (!OUT && tid == 0) p.ws_decay[slot * p.heads + h] = 1.0;
    return;
  }
  if (ms.flag) {
    redo<OUT>(p, pc, slot, h, reinterpret_cast<float*>(la_smem), S_out,
              OUT ? nullptr : p.ws_decay + slot * p.heads + h);
    return;
  }
  if (warp >= 8 && warp < 16 && S_out) {
    float* dst = S_out + (32 * (warp & 3) + lane) * kD + 64 * ((warp - 8) >> 2);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      *reinterpret_cast<float4*>(dst + 4 * e) = make_float4(S[4 * e], S[4 * e + 1], S[4 * e + 2], S[4 * e + 3]);
  }
  if (!OUT && tid == 0) p.ws_decay[slot * p.heads + h] = ms.prod;
}

// The states of split sequences that were staged in the workspace (last states that replace S0 in place).
__global__ void k_copy_states(LaParams p, const float* from) {
  const int64_t n = p.n_seqs * p.heads * (int64_t)(kD * kD / 4);
  for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < n; x += (int64_t)gridDim.x * blockDim.x)
    reinterpret_cast<float4*>(p.S)[x] = reinterpret_cast<const float4*>(from)[x];
}

}  // namespace

cudaError_t launch_la_chunk_bf16(const LaParams& p0, cudaStream_t st) {
  LaParams p = p0;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(k_la_chunk<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess)
    return e;
  const int64_t slots = p.seg ? p.slots : p.n_seqs;
  const unsigned grid = (unsigned)(slots * p.heads);
  const bool staged = p.seg && p.S && p.S == p.S0;
  if (p.seg) {
    e = cudaFuncSetAttribute(k_la_chunk<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    k_la_chunk<false><<<grid, kThreadsLa, kSmem, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (staged) p.S = p.ws_last;
  }
  k_la_chunk<true><<<grid, kThreadsLa, kSmem, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (staged) {
    p.S = p0.S;
    k_copy_states<<<608, 256, 0, st>>>(p, p.ws_last);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace lqi
