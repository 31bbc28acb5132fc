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
//                    and o is rounded to bf16 itself (in two parts where a chunk is all)
//   O += P V         P (weighted, masked, rounded to bf16 alike) from TMEM
//   U  = (wV)^T K    the state's growth. wV is an fp32 number; it goes in as three
//                    bf16 parts that hold all its 24 bits, so the state keeps fp32's
//                    accuracy (two parts, 16 bits, round to 2.8e-6 of it).
// S itself stays in fp32 registers: S <- gamma S + U in one rounding to nearest
// per step, with gamma in two parts, because a rounded gamma would be off in the
// same direction chunk after chunk. Sums of logarithms are whole numbers of 2^-40.
//
// Warps: 0-7 weigh P, scale O and write o (A); 8-15 keep the state (B); 16-23 make the
// parts of wV (C); 24 copies tiles in and out (TMA); 25 and 26 sum the logarithms (even
// and odd chunks); 27 issues the products. They meet at mbarriers only. Every wait is
// bounded; one that gives up ends the CTA's work, and the outputs become NaN. What a
// chunk waits for is the chain U -> S -> bf16 copy of S -> products -> U; the rest is
// placed beside it: the first half of wV before the state is there, S q between the
// halves, P v and the next chunk's scores while the state is brought up to date.
//
// A barrier's phases are told apart by one bit, so whoever waits for a phase must do so before
// the phase after the next can end: every wait below comes before an arrival of
// the same warp that this next phase needs. (Slow loads bring a mistake in this to light.)
//
// What bounds it, at 32,768 tokens x 32 heads: 332 us, 110 in the first pass and 217 in
// the second, 1.9 and 3.5 us a chunk of an SM. Of these the tensor cores take 0.8 and
// 1.6, HBM at its full rate would take 1.5 and 2.9. The chain's hand-overs make up the rest;
// taking out the exponentials, the loads of V or the stores, one at a time,
// changes less than 6%. (The tensors' bytes once: 159 us; the split reads k and v twice.)
//
// A masked product cannot hold back 0 x inf, and S q and q k may pass fp32's largest number before their
// decays bring them down: where the state comes out not finite (any value or key that is not makes it so),
// or an output does, or a decay is not in [0, 1], the CTA takes its tokens again one by one (redo), exactly as
// the recurrence is written.
#include <cuda.h>

#include "lq_device.cuh"
#include "lq_la.cuh"

namespace lqi {

namespace {

constexpr int kC = 128;  // tokens per chunk
constexpr int kThreadsLa = 896;
// Registers of a thread: 72 at launch (64,512 in all), then 64, 96, 64 and 48 for A, B, C and the rest (63,488).
// An increase waits until the registers are there, and nothing bounds that wait: all but B give theirs up first
// thing and take them back only after B has (roles_done), so each increase finds what it needs.
constexpr int kRegs = 72, kRegsA = 64, kRegsB = 96, kRegsC = 64, kRegsRest = 48;
// (without outputs A's warps work as C's)
static_assert(256 * ((kRegsA > kRegsC ? kRegsA : kRegsC) + kRegsB + kRegsC) + 128 * kRegsRest <= kThreadsLa * kRegs,
              "the roles' registers come out of those of the launch");
constexpr uint32_t kTile = 32768;             // 128 x 128 bf16: two halves of 64 channels, 128-byte rows, swizzled
constexpr uint32_t kS16 = 6 * kTile;          // the state in bf16
constexpr uint32_t kSums = kS16 + kTile;      // G[2][128], w[2][128]
constexpr uint32_t kMisc = kSums + 2048;      // gammas, barriers
constexpr uint32_t kSmem = kMisc + 512;
static_assert(kSmem <= 232448, "shared memory of a CTA");
// The stages of tiles below kS16: two of Q, K, V with outputs, else three of K, V (with two, the next chunk but one
// was asked for too late: 2.2 us a chunk of 64 KB).
template <bool OUT>
struct Tiles {
  static constexpr int kN = OUT ? 2 : 3;
  static constexpr uint32_t kK = OUT ? kTile : 0, kV = kK + kTile, kStage = kV + kTile;
  static __device__ __forceinline__ int at(int c) { return c % kN; }
  static __device__ __forceinline__ uint32_t phase(int c) { return (uint32_t)(c / kN) & 1u; }
  static __device__ __forceinline__ uint32_t offset(int c) { return (uint32_t)at(c) * kStage; }
};
// TMEM columns. With outputs: U, P, O and two buffers for a quarter of wV (3 parts x 16 columns). Without: U twice, so
// that its products run ahead of the state, and a buffer for each quarter.
constexpr uint32_t kU = 0, kP = 128, kO = 256;
template <bool OUT>
constexpr uint32_t kV3 = OUT ? 384 : 256;

// Whether a wait of the CTA has given up, and after how long one does.
struct Halt {
  int abort;
  uint64_t limit_ns;
};

struct Misc {
  float2 gamma[4];
  // barriers; of a chunk unless it says otherwise
  uint64_t land[3], full[3];    // tiles of the last, ragged chunk have landed; tiles are ready
  uint64_t empty[3];            // everything that reads the tiles is done
  uint64_t sums[2];             // G, w and gamma are there
  uint64_t qk, qs, pv;          // products done: P; S q in O; P v added to O
  uint64_t pvok, ofree;         // P and the scaled O are in TMEM; O has been read
  uint64_t oready[2];           // o is in Q's tile
  uint64_t uread[2], sready;    // U has been read; the bf16 copy of S is in place
  uint64_t grown[2];            // U is complete
  uint64_t vfull[4], vfree[4];  // of a quarter's buffer: parts are in TMEM; products have read them
  uint64_t drain;               // all products are done
  uint32_t tmem;
  int flag, serial;
  Halt halt;
  double prod[2];
  int64_t piece[5];
};
static_assert(sizeof(Misc) <= 512, "misc");

// Shared-memory operands: 128-byte rows, swizzled; the low word has the address, the high word
// the 1,024 bytes between groups of eight rows. Rows of the operand are rows of the tile (kByRow) or its
// channels, 64 of them to a half tile (kByChannel).
constexpr uint32_t kByRow = 1u << 16, kByChannel = 1024u << 16;
__device__ __forceinline__ uint64_t desc(uint32_t lo) {
  return (uint64_t)lo | ((uint64_t)(64u | (1u << 14) | (2u << 29)) << 32);
}
// fp32 accumulators, bf16 operands, M = N = 128; B by rows or by channels
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (16u << 17) | (8u << 24);
constexpr uint32_t kIdescMn = kIdesc | (1u << 16);

// The products are issued by one thread, chosen by elect.sync, with warp-uniform operands: from a thread chosen by its
// lane number the same instructions took 220 cycles each to issue (64 to run).
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(desc(a)), "l"(desc(b)), "r"(id), "n"(ACC ? 1 : 0)
      : "memory");
}
template <bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(desc(b)), "r"(id), "n"(ACC ? 1 : 0)
      : "memory");
}
// d = a b^T, both 128 x 128 by rows: eight steps of 16 channels
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t b) {
  mma_ss<false>(d, a, b, kIdesc);
#pragma unroll
  for (int s = 1; s < 8; ++s)
    mma_ss<true>(d, a + (s >> 2) * 1024 + (s & 3) * 2, b + (s >> 2) * 1024 + (s & 3) * 2, kIdesc);
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

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// All warps, each at the end of its role.
__device__ __forceinline__ void roles_done() {
  __syncwarp();
  asm volatile("bar.sync 2, %0;" ::"n"(kThreadsLa) : "memory");
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits for phase `parity`; false once this or any other wait of the CTA has given up. The clock is read only after
// a good many tries (a try waits by itself for a while): reading it first held up every wait.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Halt* halt) {
#pragma unroll 1
  for (int i = 0; i < 4096; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&halt->abort)) return false;
    if (globaltimer_ns() - t0 > halt->limit_ns) {
      *reinterpret_cast<volatile int*>(&halt->abort) = 1;
      return false;
    }
  }
}

// The same for a whole warp: all lanes go on or none does.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Halt* halt) {
  return __all_sync(0xffffffffu, wait(bar, parity, halt));
}

// 128 tokens x 64 channels into half a tile; tokens past the tensor's end are zeros. x is a multiple of 64.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int x, int t, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(dst),
      "l"(map), "r"(x), "r"(t), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int t, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
               "r"(t), "r"(src)
               : "memory");
}

__device__ __forceinline__ void ld_32bytes(const float* p, f32x2& a, f32x2& b, f32x2& c, f32x2& d) {
  asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];" : "=l"(a), "=l"(b), "=l"(c), "=l"(d) : "l"(p) : "memory");
}
__device__ __forceinline__ void st_32bytes(float* p, f32x2 a, f32x2 b, f32x2 c, f32x2 d) {
  asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(a), "l"(b), "l"(c), "l"(d) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {  // to nearest
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t bf16_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

using bf16 = __nv_bfloat16;
using PFN_encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A's first step: the scores of row i, columns 64 half .. + 63, weighted, masked and rounded to bf16 as an A operand; TWO:
// what the rounding took off as well (see the products). Loops are kept rolled here and below: five roles run at once,
// and with everything unrolled the warps waited for instructions more than for data.
template <bool TWO>
__device__ __forceinline__ void weigh_scores(uint32_t tl, const float* G, float gi, int i, int quad, int half) {
#pragma unroll 1
  for (int j0 = 64 * half; j0 < 64 * half + 64; j0 += 16) {
    uint32_t w[8], w2[8];
    if (j0 > 32 * quad + 31) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = w2[e] = 0u;
    } else {
      uint32_t x[16];
      tm_ld16(tl + kP + j0, x);
      wait_ld();
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 g = *reinterpret_cast<const float4*>(G + j0 + e);
        const float gj[4] = {g.x, g.y, g.z, g.w};
        float y[4];
#pragma unroll
        for (int f = 0; f < 4; ++f)
          y[f] = j0 + e + f <= i ? __fmul_rn(__uint_as_float(x[e + f]), ex2(__fsub_rn(gi, gj[f]))) : 0.f;
#pragma unroll
        for (int f = 0; f < 4; f += 2) {
          const uint32_t p2 = pack_bf16(y[f], y[f + 1]);
          w[(e + f) / 2] = p2;
          if (TWO)
            w2[(e + f) / 2] = pack_bf16(__fsub_rn(y[f], __uint_as_float(p2 << 16)),
                                        __fsub_rn(y[f + 1], __uint_as_float(p2 & 0xffff0000u)));
        }
      }
    }
    // 16 tokens of P take 8 columns; they go where their accumulators were, which this warp has read
    tm_st8(tl + kP + j0, w);
    if (TWO) tm_st8(tl + kP + j0 + 8, w2);
  }
}

// OUT: outputs and last states. Otherwise the first pass over split sequences: what a segment adds to the state.
template <bool OUT>
__global__ void __launch_bounds__(kThreadsLa, 1)
    k_la_chunk(LaParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
  extern __shared__ __align__(1024) char la_smem[];
  Misc& ms = *reinterpret_cast<Misc*>(la_smem + kMisc);
  cudaTriggerProgrammaticLaunchCompletion();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = (int)(blockIdx.x % (unsigned)p.heads), kh = h / p.group;
  const int64_t slot = blockIdx.x / (unsigned)p.heads;
  if (warp == 0) {
    const Piece f = find_piece(p, slot);
    if (lane == 0) ms.piece[0] = f.b, ms.piece[1] = f.begin, ms.piece[2] = f.len, ms.piece[3] = f.i, ms.piece[4] = f.n;
  } else if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ms.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (tid == 64) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.sums[i], 32);
      mbar_init(&ms.oready[i], 256);
      mbar_init(&ms.grown[i], 1);
      mbar_init(&ms.uread[i], 256);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&ms.land[i], 1);
      mbar_init(&ms.full[i], 1);
      mbar_init(&ms.empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ms.vfull[i], 128);
      mbar_init(&ms.vfree[i], 1);
    }
    mbar_init(&ms.qk, 1);
    mbar_init(&ms.qs, 1);
    mbar_init(&ms.pv, 1);
    mbar_init(&ms.pvok, 256);
    mbar_init(&ms.ofree, 256);
    mbar_init(&ms.sready, 256);
    mbar_init(&ms.drain, 1);
    ms.flag = ms.serial = 0;
    ms.halt = Halt{0, 2 * p.wait_ns};
    ms.prod[0] = ms.prod[1] = 1.0;
  }
  tc_before();
  __syncthreads();
  tc_after();
  Piece pc;
  pc.b = ms.piece[0], pc.begin = ms.piece[1], pc.len = ms.piece[2], pc.i = ms.piece[3], pc.n = ms.piece[4];
  const bool last = pc.i == pc.n - 1;
  if (pc.b < 0 || (!OUT && last)) {
    if (warp == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(ms.tmem) : "memory");
    return;
  }
  float2* const serial = serial_note(p, pc, slot, h);
  if (!OUT && pc.i == 0 && tid == 0 && serial) *serial = make_float2(0.f, 0.f);
  // Where the state after the piece goes.
  float* S_out = OUT ? (last && p.S ? p.S + (pc.b * p.heads + h) * (kD * kD) : nullptr)
                     : p.ws_state + (slot * p.heads + h) * (kD * kD);
  const bool in_place = OUT && p.S && p.S == p.S0;
  const int nc = (int)((pc.len + kC - 1) / kC);
  // Where a single chunk is all, o hangs on few weights and one state, whose roundings need not even out: there what
  // rounding P and S takes off goes in as well. (S's lies in the second stage of tiles, which has no other use then.)
  const bool two = OUT && nc == 1, two_s = two && (pc.n > 1 || p.S0);
  const uint32_t tm = ms.tmem, sb = smem_u32(la_smem);
  float* sG = reinterpret_cast<float*>(la_smem + kSums);
  float* sw = sG + 2 * kC;
  Halt* const ab = &ms.halt;
  using Ti = Tiles<OUT>;

  if (OUT ? warp >= 16 && warp < 24 : warp < 8 || (warp >= 16 && warp < 24)) {
    // C: quarters (32 tokens) of a chunk, weighted and in three parts, as rows of the A operand: row 32 (warp & 3) +
    // lane. Warps 16-19 take quarters 0 and 2, warps 20-23 quarters 1 and 3; without outputs A's warps help, and each
    // four have one quarter.
    regs_down<kRegsC>();
    constexpr int kSteps = OUT ? 2 : 1;  // quarters of a chunk for a warp
    const int quad = warp & 3, set = warp < 8 ? 2 + (warp >> 2) : (warp - 16) >> 2, row = 32 * quad + lane;
    const uint32_t Vrow = sb + Ti::kV + (row >> 6) * 16384 + (row & 7) * 2;
    const uint32_t swz = ((row & 63) >> 3) << 4;  // 16-byte chunk of the row's channel, swizzled by the token mod 8
    const uint32_t to = tm + ((uint32_t)(32 * quad) << 16) + kV3<OUT> + 48 * set;
    for (int u = 0; u < kSteps * nc; ++u) {
      const int c = u / kSteps, qt = 2 * (u % kSteps) + set;
      if (u % kSteps == 0) {
        if (!wait_warp(&ms.sums[c & 1], (c >> 1) & 1, ab)) break;
        if (!wait_warp(&ms.full[Ti::at(c)], Ti::phase(c), ab)) break;
      }
      const uint32_t V = Vrow + Ti::offset(c) + qt * 4096;
      const float* w = sw + (c & 1) * kC + 32 * qt;
      uint32_t p0[16], p1[16], p2[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const ulonglong2 w2 = *reinterpret_cast<const ulonglong2*>(w + 4 * (e / 2));
        const uint32_t v0 = lds_u16(V + 256 * e + (swz ^ (((2 * e) & 7) << 4)));
        const uint32_t v1 = lds_u16(V + 256 * e + 128 + (swz ^ (((2 * e + 1) & 7) << 4)));
        // two tokens at once; the top 8 bits, the next 8, the last 8: each difference is exact
        const f32x2 x = f2_mul(f2_bits(v0 << 16, v1 << 16), e & 1 ? w2.y : w2.x);
        const f32x2 r = f2_sub(x, x & 0xffff0000ffff0000ull);
        const f32x2 d = f2_sub(r, r & 0xffff0000ffff0000ull);
        p0[e] = __byte_perm((uint32_t)x, (uint32_t)(x >> 32), 0x7632);
        p1[e] = __byte_perm((uint32_t)r, (uint32_t)(r >> 32), 0x7632);
        p2[e] = __byte_perm((uint32_t)d, (uint32_t)(d >> 32), 0x7632);
      }
      if (u && !wait_warp(&ms.vfree[set], (u - 1) & 1, ab)) break;
      tc_after();
      tm_st16(to, p0);
      tm_st16(to + 16, p1);
      tm_st16(to + 32, p2);
      wait_st();
      tc_before();
      arrive(&ms.vfull[set]);
    }
    roles_done();
    regs_up<kRegs>();
  } else if (warp < 8) {
    regs_down<kRegsA>();
    if (OUT) {
      // A: row i = 32 (warp & 3) + lane of the chunk, columns 64 half .. 64 half + 63
      const int quad = warp & 3, half = warp >> 2, i = 32 * quad + lane;
      const uint32_t tl = tm + ((uint32_t)(32 * quad) << 16);
      bf16* o = static_cast<bf16*>(p.o) + h * kD + 64 * half;
      uint32_t odd = 0;  // a pair of sums of products of outputs: not finite once an output is not (or some pass 1e18)
      for (int c = 0; c < nc; ++c) {
        const float* G = sG + (c & 1) * kC;
        if (!wait_warp(&ms.sums[c & 1], (c >> 1) & 1, ab)) break;
        const float gi = G[i];
        const float ei = ex2(gi);
        if (!wait_warp(&ms.qk, c & 1, ab)) break;
        tc_after();
        if (two) weigh_scores<true>(tl, G, gi, i, quad, half);
        else weigh_scores<false>(tl, G, gi, i, quad, half);
        if (!wait_warp(&ms.qs, c & 1, ab)) break;
        tc_after();
#pragma unroll 1
        for (uint32_t at = tl + kO + 64 * half; at < tl + kO + 64 * half + 64; at += 16) {
          uint32_t x[16];
          tm_ld16(at, x);
          wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__fmul_rn(ei, __uint_as_float(x[e])));
          tm_st16(at, x);
        }
        wait_st();
        tc_before();
        arrive(&ms.pvok);
        if (!wait_warp(&ms.pv, c & 1, ab)) break;
        tc_after();
        // o goes out by way of Q's tile, which nothing reads any more: rows of 128 bytes, swizzled as Q's were
        char* tile = la_smem + Ti::offset(c) + half * 16384;
        const int n = (int)min((int64_t)kC, pc.len - (int64_t)c * kC);
#pragma unroll 1
        for (int blk = 0; blk < 2; ++blk) {
          uint32_t x[32];
          tm_ld32(tl + kO + 64 * half + 32 * blk, x);
          wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = pack_bf16(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(tile + i * 128 + (((4 * blk + e) ^ (i & 7)) << 4)) =
                make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          if (blk) {
            tc_before();
            arrive(&ms.ofree);
          }
          if (i < n) {  // two words an instruction: 332.6 us for 32,768 tokens x 32 heads (one word 334.7, unchecked 330)
            uint32_t t = 0u;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              odd = bf16_fma(x[e], x[e + 1], odd);
              t = bf16_fma(x[e + 2], x[e + 3], t);
            }
            odd = bf16_fma(t, 0x3f803f80u, odd);
          }
        }
        if (n == kC) {
          fence_proxy_async();
          arrive(&ms.oready[c & 1]);
        } else if (!*reinterpret_cast<volatile int*>(&ms.serial)) {
          // the rows past the end are not this sequence's: each warp writes those of its 32 that are
          __syncwarp();
          const int e = lane & 7;
          for (int r = 32 * quad + (lane >> 3); r < min(n, 32 * quad + 32); r += 4)
            *reinterpret_cast<uint4*>(o + (pc.begin + (int64_t)c * kC + r) * p.so + 8 * e) =
                *reinterpret_cast<const uint4*>(tile + r * 128 + ((e ^ (r & 7)) << 4));
        }
      }
      if ((odd & 0x7f80u) == 0x7f80u || (odd & 0x7f800000u) == 0x7f800000u) ms.flag = 1;
      if (in_place) asm volatile("bar.arrive 3, 512;" ::: "memory");
    }
    roles_done();
    regs_up<kRegs>();
  } else if (warp < 16) {
    // B
    regs_up<kRegsB>();
    const int quad = warp & 3, half = (warp - 8) >> 2, row = 32 * quad + lane;
    const uint32_t tl = tm + ((uint32_t)(32 * quad) << 16);
    f32x2 S[32];  // row `row` of the state, columns 64 half .., in pairs
    {
      if (OUT && p.seg) cudaGridDependencySynchronize();
      const float* from = OUT ? start_state(p, pc, slot, h) : nullptr;
      const float note = OUT && serial && tid == 256 ? serial->x : 0.f;
#pragma unroll
      for (int e = 0; e < 32; ++e) S[e] = 0ull;
      if (from) {  // a lane has a row: 32 bytes at a time where the address allows
        from += row * kD + 64 * half;
        if ((uintptr_t)from % 32 == 0) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) ld_32bytes(from + 2 * e, S[e], S[e + 1], S[e + 2], S[e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(from + 2 * e);
            S[e] = x.x, S[e + 1] = x.y;
          }
        }
      }
      // (o waits for this thread's part of S, and looks at this after that)
      if (note != 0.f) *reinterpret_cast<volatile int*>(&ms.serial) = 1;
    }
    char* const s16 = la_smem + kS16 + half * 16384 + row * 128;
    if (two_s) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t x[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          float lo, hi;
          f2_unpack(S[4 * e + f], lo, hi);
          const uint32_t y = pack_bf16(lo, hi);
          x[f] = pack_bf16(__fsub_rn(lo, __uint_as_float(y << 16)), __fsub_rn(hi, __uint_as_float(y & 0xffff0000u)));
        }
        *reinterpret_cast<uint4*>(s16 - kS16 + Ti::kStage + ((e ^ (row & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
    for (int c = 0; c <= nc; ++c) {
      // With the sums comes gamma of this chunk, for the next round.
      if (c < nc && (OUT || c == 0) && !wait_warp(&ms.sums[c & 1], (c >> 1) & 1, ab)) break;
      if (c) {  // S <- gamma S + U
        const float2 g = ms.gamma[(c - 1) & 3];
        const f32x2 g0 = f2_dup(g.x), g1 = f2_dup(g.y);
        // (S's bf16 copy has been read by then, too)
        if (!wait_warp(&ms.grown[(c - 1) & 1], ((c - 1) >> 1) & 1, ab)) break;
        const uint32_t U = tl + kU + 64 * half + (OUT ? 0 : 128 * ((c - 1) & 1));
        tc_after();
#pragma unroll
        for (int blk = 0; blk < 4; ++blk) {
          uint32_t x[16];
          tm_ld16(U + 16 * blk, x);
          wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f32x2& s = S[8 * blk + e];
            s = f2_fma(s, g0, f2_fma(s, g1, f2_bits(x[2 * e], x[2 * e + 1])));
          }
        }
        tc_before();
      }
      if (c == nc) break;
      // (without outputs the next chunk's products need no more than this arrival)
      if (!OUT && c + 1 < nc && !wait_warp(&ms.sums[(c + 1) & 1], ((c + 1) >> 1) & 1, ab)) break;
      arrive(&ms.uread[c & 1]);
      if (OUT) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t x[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            float lo, hi;
            f2_unpack(S[4 * e + f], lo, hi);
            x[f] = pack_bf16(lo, hi);
          }
          *reinterpret_cast<uint4*>(s16 + ((e ^ (row & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
        }
        fence_proxy_async();
        arrive(&ms.sready);
      }
    }
    f32x2 sum = 0ull;  // NaN where an entry is infinite or NaN
#pragma unroll
    for (int e = 0; e < 32; ++e) sum = f2_fma(S[e], 0ull, sum);
    float s0, s1;
    f2_unpack(sum, s0, s1);
    if (s0 != 0.f || s1 != 0.f) ms.flag = 1;
    // (odd decays were flagged before their sums were handed over; what A finds is waited for only where S0 would be lost)
    if (in_place) asm volatile("bar.sync 3, 512;" ::: "memory");
    else asm volatile("bar.sync 1, 256;" ::: "memory");
    if (S_out && !*reinterpret_cast<volatile int*>(&ms.flag) && !*reinterpret_cast<volatile int*>(&ab->abort) &&
        !*reinterpret_cast<volatile int*>(&ms.serial)) {
      float* dst = S_out + row * kD + 64 * half;
      if ((uintptr_t)dst % 32 == 0) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) st_32bytes(dst + 2 * e, S[e], S[e + 1], S[e + 2], S[e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < 32; e += 2) *reinterpret_cast<ulonglong2*>(dst + 2 * e) = make_ulonglong2(S[e], S[e + 1]);
      }
    }
    regs_down<kRegs>();
    roles_done();
  } else {
  regs_down<kRegsRest>();
  if (warp == 24) {
    // Copies. The last chunk's rows past the end are other sequences': they are set to
    // zero in K and V (a weight of zero does not stop an infinity; Q's only reach rows that are not written).
    // Full chunks of o leave from Q's tile before the next Q comes in.
    int issued = 0;
    for (int c = 0; c < nc + Ti::kN; ++c) {
      const int s = Ti::at(c), n = (int)min((int64_t)kC, pc.len - (int64_t)c * kC);  // (n <= 0: nothing more comes in)
      const uint32_t dst = sb + Ti::offset(c);
      const int t0 = (int)(pc.begin + (int64_t)c * kC);
      uint64_t* bar = n == kC ? &ms.full[s] : &ms.land[s];
      if (c >= Ti::kN && !wait_warp(&ms.empty[s], Ti::phase(c - Ti::kN), ab)) break;
      if (n > 0 && lane == 0) {
        mbar_expect_tx(bar, Ti::kStage + p.dbg_tx);
        for (int x = 0; x < 2; ++x) tma_tile(dst + Ti::kK + 16384 * x, &mk, kh * kD + 64 * x, t0, bar);
        for (int x = 0; x < 2; ++x) tma_tile(dst + Ti::kV + 16384 * x, &mv, h * kD + 64 * x, t0, bar);
      }
      if (n > 0) issued = c + 1;
      if (OUT && c >= 2 && pc.len >= (int64_t)(c - 1) * kC) {  // chunk c - 2 is a full one
        if (!wait_warp(&ms.oready[s], ((c - 2) >> 1) & 1, ab)) break;
        if (lane == 0 && !*reinterpret_cast<volatile int*>(&ms.serial)) {
          for (int x = 0; x < 2; ++x) tma_store(&mo, h * kD + 64 * x, t0 - 2 * kC, dst + 16384 * x);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
      }
      if (OUT && n > 0 && lane == 0)
        for (int x = 0; x < 2; ++x) tma_tile(dst + 16384 * x, &mq, kh * kD + 64 * x, t0, bar);
      __syncwarp();
      if (n > 0 && n < kC) {
        if (!wait_warp(&ms.land[s], 0, ab)) break;
        uint4* tile = reinterpret_cast<uint4*>(la_smem + Ti::offset(c) + Ti::kK);
        for (int x = lane; x < (kC - n) * 32; x += 32)  // 8 chunks of 16 bytes x 4 half tiles a row
          tile[((x >> 3) & 3) * 1024 + (n + (x >> 5)) * 8 + (x & 7)] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive(&ms.full[s]);
      }
    }
    if (OUT && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    // A wait gave up: what was asked for still has to land before the CTA ends. (In a chunk whose Q was not asked
    // for, the barrier cannot complete: that wait runs into its limit.)
    Halt ignored = {0, ab->limit_ns};
    if (*reinterpret_cast<volatile int*>(&ab->abort))
      for (int c = max(0, issued - Ti::kN); c < issued; ++c) {
        const bool whole = pc.len >= (int64_t)(c + 1) * kC;
        wait(whole ? &ms.full[Ti::at(c)] : &ms.land[Ti::at(c)], whole ? Ti::phase(c) : 0, &ignored);
      }
  } else if (warp < 27) {
    // Sums of log2 alpha in whole numbers of 2^-40, four tokens to a lane. A decay of
    // zero counts 2^-200: any weight across it is below fp32's smallest number.
    double prod = 1.0;
    bool odd = false;
    float a[4];
    auto load = [&](int c) {  // a chunk ahead of its use
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t t = (int64_t)c * kC + 4 * lane + e;
        a[e] = t < pc.len ? p.alpha[(pc.begin + t) * p.sa + h] : 1.f;
      }
    };
    load(warp - 25);
    for (int c = warp - 25; c < nc; c += 2) {
      // gamma, the product of the decays, in two parts; the same in every lane
      float2 gm = mul2(mul2(make_float2(a[0], 0.f), make_float2(a[1], 0.f)),
                       mul2(make_float2(a[2], 0.f), make_float2(a[3], 0.f)));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
        gm = mul2(gm, make_float2(__shfl_xor_sync(0xffffffffu, gm.x, o), __shfl_xor_sync(0xffffffffu, gm.y, o)));
      prod *= (double)gm.x + (double)gm.y;
      long long g[4], run = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!(a[e] >= 0.f && a[e] <= 1.f)) odd = true;
        const float l = a[e] > 0.f ? fmaxf(log2f(a[e]), -200.f) : -200.f;
        run += __float2ll_rn(__fmul_rn(l, 1099511627776.f));
        g[e] = run;
      }
      load(c + 2);
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
      if (c >= 2 && !wait_warp(&ms.empty[Ti::at(c - 2)], Ti::phase(c - 2), ab)) break;
      *reinterpret_cast<float4*>(sG + (c & 1) * kC + 4 * lane) = make_float4(G[0], G[1], G[2], G[3]);
      *reinterpret_cast<float4*>(sw + (c & 1) * kC + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
      if (lane == 0) ms.gamma[c & 3] = gm;
      if (odd) ms.flag = 1;
      arrive(&ms.sums[c & 1]);
    }
    if (lane == 0) ms.prod[warp - 25] = prod;
  } else {
    // The products.
    const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
    const uint32_t S16 = ((sb + kS16) >> 4) | kByRow;
    if (elect()) {
      for (int c = -1; c < nc; ++c) {
        if (c >= 0) {
          const uint32_t at = (sb + Ti::offset(c)) >> 4;
          const uint32_t Q = at | kByRow, Kc = (at + Ti::kK / 16) | kByChannel, Vc = (at + Ti::kV / 16) | kByChannel;
          if (!OUT && !wait(&ms.full[Ti::at(c)], Ti::phase(c), ab)) break;
          // U is free: read up to the last chunk's, or, where there are two, the one's before. (Chunk 0 waits as well,
          // so that no chunk is through before B has seen its sums.)
          const int r = OUT ? c : max(c - 1, 0);
          if (!wait(&ms.uread[r & 1], (r >> 1) & 1, ab)) break;
          tc_after();
          const uint32_t U = tmu + kU + (OUT ? 0 : 128 * (c & 1));
          bool ok = true;
#pragma unroll
          for (int qt = 0; qt < 4; ++qt) {
            const int buf = OUT ? qt & 1 : qt, use = OUT ? 2 * c + (qt >> 1) : c;
            if (OUT && qt == 2) {  // while quarter 2 is in the making
              if (!(ok = wait(&ms.sready, c & 1, ab))) break;
              if (c && !(ok = wait(&ms.ofree, (c - 1) & 1, ab))) break;
              tc_after();
              product(tmu + kO, Q, S16);
              if (two_s) {
#pragma unroll 1
                for (int s = 0; s < 8; ++s)
                  mma_ss<true>(tmu + kO, Q + (s >> 2) * 1024 + (s & 3) * 2,
                               S16 - kS16 / 16 + Ti::kStage / 16 + (s >> 2) * 1024 + (s & 3) * 2, kIdesc);
              }
              commit(&ms.qs);
            }
            if (!(ok = wait(&ms.vfull[buf], use & 1, ab))) break;
            tc_after();
            const uint32_t a = tmu + kV3<OUT> + 48 * buf, b = Kc + 2 * qt * 128;
            // the small parts first
            if (qt == 0) mma_ts<false>(U, a + 32, b, kIdescMn);
            else mma_ts<true>(U, a + 32, b, kIdescMn);
            mma_ts<true>(U, a + 40, b + 128, kIdescMn);
#pragma unroll
            for (int part = 1; part >= 0; --part)
#pragma unroll
              for (int s = 0; s < 2; ++s) mma_ts<true>(U, a + 16 * part + 8 * s, b + 128 * s, kIdescMn);
            commit(&ms.vfree[buf]);
            if (qt == 3) commit(&ms.grown[c & 1]);
            if (qt == 3 && !OUT) commit(&ms.empty[Ti::at(c)]);
          }
          if (!ok) break;
          if (OUT) {  // while the state is brought up to date
            if (!wait(&ms.pvok, c & 1, ab)) break;
            tc_after();
#pragma unroll
            for (int s = 0; s < 8; ++s)
              mma_ts<true>(tmu + kO, tmu + kP + 16 * s, Vc + s * 128, kIdescMn);
            if (two) {
#pragma unroll 1
              for (int s = 0; s < 8; ++s)
                mma_ts<true>(tmu + kO, tmu + kP + 16 * s + 8, Vc + s * 128, kIdescMn);
            }
            commit(&ms.pv);
            commit(&ms.empty[Ti::at(c)]);
          }
        }
        if (OUT && c + 1 < nc) {  // the next chunk's scores: they follow P's last use in order
          if (!wait(&ms.full[Ti::at(c + 1)], Ti::phase(c + 1), ab)) break;
          tc_after();
          const uint32_t next = (sb + Ti::offset(c + 1)) >> 4;
          product(tmu + kP, next | kByRow, (next + Ti::kK / 16) | kByRow);
          commit(&ms.qk);
        }
      }
      // nothing may be in flight when TMEM is given back
      commit(&ms.drain);
    }
    __syncwarp();
    Halt ignored = {0, ab->limit_ns};
    wait_warp(&ms.drain, 0, &ignored);
  }
  __syncwarp();
  roles_done();
  regs_up<kRegs>();
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  if (OUT && ms.serial) {  // nothing has been written
    if (pc.i) return;
    int64_t begin, len;
    bounds(p, pc.b, begin, len);
    const int64_t at = (pc.b * p.heads + h) * (kD * kD);
    redo<bf16, true, 512, 16>(p, begin, len, h, p.S0 ? p.S0 + at : nullptr, reinterpret_cast<float*>(la_smem),
                              p.S ? p.S + at : nullptr, nullptr);
    return;
  }
  if (ms.halt.abort) {  // a wait gave up: make that visible (nothing of this CTA is in flight any more)
    const bf16 bad = __float2bfloat16_rn(__int_as_float(0x7fc00000));
    if (OUT)
      for (int64_t x = tid; x < pc.len * kD; x += kThreadsLa)
        static_cast<bf16*>(p.o)[(pc.begin + x / kD) * p.so + h * kD + x % kD] = bad;
    if (S_out)
      for (int x = tid; x < kD * kD; x += kThreadsLa) S_out[x] = __int_as_float(0x7fc00000);
    if (!OUT && tid == 0) p.ws_decay[slot * p.heads + h] = make_float2(1.f, 0.f);
    return;
  }
  if (ms.flag) {
    if (OUT && p.seg) cudaGridDependencySynchronize();
    redo<bf16, OUT, 512, 16>(p, pc.begin, pc.len, h, OUT ? start_state(p, pc, slot, h) : nullptr,
                             reinterpret_cast<float*>(la_smem), S_out, OUT ? nullptr : p.ws_decay + slot * p.heads + h);
    return;
  }
  if (!OUT && tid == 0) p.ws_decay[slot * p.heads + h] = in_two(ms.prod[0] * ms.prod[1]);
}

}  // namespace

// A token array as a tensor of heads x 128 channels by tokens, read 64 channels by 128 tokens.
static cudaError_t tile_map(CUtensorMap* m, const void* base, int heads, int64_t stride, int64_t tokens) {
  static PFN_encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_encode>(f);
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)heads * kD, (cuuint64_t)tokens}, pitch[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, kC}, one[2] = {1, 1};
  const CUresult r =
      encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, pitch, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_la_chunk_bf16(const LaParams& p0, cudaStream_t st) {
  LaParams p = p0;
  cudaError_t e;
  CUtensorMap mq = {}, mk = {}, mv = {}, mo = {};
  if (p.n_tokens && ((e = tile_map(&mq, p.q, p.key_heads, p.sq, p.n_tokens)) != cudaSuccess ||
                     (e = tile_map(&mk, p.k, p.key_heads, p.sk, p.n_tokens)) != cudaSuccess ||
                     (e = tile_map(&mv, p.v, p.heads, p.sv, p.n_tokens)) != cudaSuccess ||
                     (e = tile_map(&mo, p.o, p.heads, p.so, p.n_tokens)) != cudaSuccess))
    return e;
  // The roles' shares of registers count on this many at launch.
  static const bool regs = [] {
    cudaFuncAttributes t, f;
    return cudaFuncGetAttributes(&t, k_la_chunk<true>) == cudaSuccess &&
           cudaFuncGetAttributes(&f, k_la_chunk<false>) == cudaSuccess && t.numRegs == kRegs && f.numRegs == kRegs;
  }();
  if (!regs) return cudaErrorLaunchOutOfResources;
  if ((e = set_smem(k_la_chunk<true>, kSmem)) != cudaSuccess) return e;
  const int64_t slots = p.seg ? p.slots : p.n_seqs;
  const unsigned grid = (unsigned)(slots * p.heads);
  if (p.seg) {
    if ((e = set_smem(k_la_chunk<false>, kSmem)) != cudaSuccess) return e;
    k_la_chunk<false><<<grid, kThreadsLa, kSmem, st>>>(p, mq, mk, mv, mo);
    if ((e = cudaGetLastError()) != cudaSuccess || (e = launch_la_scan(p, st)) != cudaSuccess) return e;
  }
  if (la_staged(p)) p.S = p.ws_last;
  if (p.seg) {
    e = launch_upon(k_la_chunk<true>, dim3(grid), kThreadsLa, (int)kSmem, st, p, mq, mk, mv, mo);
  } else {
    k_la_chunk<true><<<grid, kThreadsLa, kSmem, st>>>(p, mq, mk, mv, mo);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return la_staged(p0) ? launch_la_unstage(p0, st) : cudaSuccess;
}

}  // namespace lqi
