// Head-states that follow the hypotheses of beam search (sm_103a): afterwards beam
// b of a group holds what beam parent[b] held. In place, without scratch: the
// beams of a group hold the same planes at different offsets, and a thread owns
// the same 16 bytes of every beam. It reads its 16 bytes of each beam that is a
// source and only then writes those of the beams that move, so no thread ever
// reads what another one writes.
//
// Bound by HBM: the sources are read once (a source of several beams comes from
// L1), the moved beams written once, the rest stays where it is; of the record
// planes only the records held move. 16,384 quantized states in groups of four: 105 to 109 us for
// 603 MB, 81 to 85% of the copy bandwidth; 4,096 fp32 states in groups of eight: 69 to 76 us for
// 398 MB, 77 to 85%. One CTA takes one (outer, group, inner)
// position: it alone reads and rewrites the record counts of its beams, so the
// counts need no second kernel.
#include <cuda_runtime.h>
#include <stdint.h>

#include "lq_device.cuh"
#include "lq_internal.h"

namespace lqi {

namespace {

// Reads the group's parents into smem and says whether any beam moves (1), none
// does (0), or a parent is outside its group (-1). All threads of the CTA call it.
__device__ __forceinline__ int read_parents(const int32_t* parent, int64_t g, int K, int* sp) {
  __shared__ int sbad, smove;
  if (threadIdx.x == 0) sbad = smove = 0;
  __syncthreads();
  if ((int)threadIdx.x < K) {
    const int x = parent[g * K + threadIdx.x];
    sp[threadIdx.x] = x;
    if (x < 0 || x >= K) sbad = 1;
    else if (x != (int)threadIdx.x) smove = 1;
  }
  __syncthreads();
  return sbad ? -1 : smove;
}

// Where vector x of a head-state lies: beam 0's address, the distance from beam to beam in vectors, and how many
// records a source must hold for the vector to be live (0: always).
struct Place {
  uint4* at;
  int64_t pitch;
  int live;
};

// Moves vectors [0, n) as `place` gives them: all loads of a thread come before its first store. One vector of
// each beam at a time; two (for up to four beams) were slower, 126 us for 16,384 states against 107, by their registers.
template <int KM, typename F>
__device__ __forceinline__ void move_all(int n, F place, const int* sn, int K, const int* sp) {
  for (int x = threadIdx.x; x < n; x += blockDim.x) {
    const Place pl = place(x);
    uint4 r[KM];
#pragma unroll
    for (int b = 0; b < KM; ++b)
      if (b < K && sp[b] != b && sn[sp[b]] >= pl.live) r[b] = pl.at[sp[b] * pl.pitch];
#pragma unroll
    for (int b = 0; b < KM; ++b)
      if (b < K && sp[b] != b && sn[sp[b]] >= pl.live) __stcs(pl.at + b * pl.pitch, r[b]);
  }
}

template <int KM>
__global__ void __launch_bounds__(256) k_reorder(Params p, ReorderParams r) {
  __shared__ int sp[kMaxBeams], sn[kMaxBeams], sbad;
  const int K = r.beams;
  const int64_t i = blockIdx.x % r.inner, xg = blockIdx.x / r.inner, g = xg % r.groups;
  const int64_t s0 = xg * K * r.inner + i;  // head-state of beam 0; the beams are r.inner apart
  if (!header_ok(p)) {
    if (threadIdx.x == 0) set_error(p, LQ_ERR_STATE, s0);
    return;
  }
  const int any = read_parents(r.parent, g, K, sp);
  if (any < 0 && threadIdx.x == 0) set_error(p, LQ_ERR_PARENT, s0);
  if (any <= 0) return;
  if (threadIdx.x == 0) sbad = 0;
  __syncthreads();
  if ((int)threadIdx.x < K) {
    const int n = p.counts[s0 + threadIdx.x * r.inner];
    sn[threadIdx.x] = n;
    if (n < 0 || n > p.W) sbad = 1;
  }
  __syncthreads();
  if (sbad) {
    if (threadIdx.x == 0) set_error(p, LQ_ERR_STATE, s0);
    return;
  }
  int nmax = 0;
  for (int b = 0; b < K; ++b)
    if (sp[b] != b) nmax = max(nmax, sn[sp[b]]);

  const int cv = kD * kD * p.bits / 128;  // 16-byte vectors of a head-state's codes
  const int lv = p.C * kD / 4 * (p.comp_fit > 0 ? 2 : 1);
  const int iv = (int)(p.comp_id_stride / 4), rv = nmax * (kD / 4);
  // codes, record keys and corrections (and decays per key), compensators, steps, scales, compensator ids
  const int e0 = cv, e1 = e0 + rv, e2 = e1 + rv, e3 = e2 + (p.kda ? rv : 0), e4 = e3 + lv, e5 = e4 + kD / 4,
            e6 = e5 + kD / 4, n = e6 + iv;
  const int wv = p.W * (kD / 4);
  auto in = [&](void* base, int vecs, int x, bool record) {
    return Place{static_cast<uint4*>(base) + s0 * vecs + x, r.inner * vecs, record ? x / (kD / 4) + 1 : 0};
  };
  move_all<KM>(
      n,
      [&](int x) {
        if (x < e0) return in(p.codes, cv, x, false);
        if (x < e1) return in(p.rec_k, wv, x - e0, true);
        if (x < e2) return in(p.rec_u, wv, x - e1, true);
        if (x < e3) return in(p.rec_alpha, wv, x - e2, true);
        if (x < e4) return in(p.comp_line, lv, x - e3, false);
        if (x < e5) return in(p.sigma, kD / 4, x - e4, false);
        if (x < e6) return in(p.lambda, kD / 4, x - e5, false);
        return in(p.comp_id, iv, x - e6, false);
      },
      sn, K, sp);
  if (!p.kda && (int)threadIdx.x < nmax) {  // one decay per record
    float a[KM];
    float* base = p.rec_alpha + s0 * p.alpha_stride + threadIdx.x;
    const int64_t pitch = r.inner * p.alpha_stride;
#pragma unroll
    for (int b = 0; b < KM; ++b)
      if (b < K && sp[b] != b && (int)threadIdx.x < sn[sp[b]]) a[b] = base[sp[b] * pitch];
#pragma unroll
    for (int b = 0; b < KM; ++b)
      if (b < K && sp[b] != b && (int)threadIdx.x < sn[sp[b]]) base[b * pitch] = a[b];
  }
  if ((int)threadIdx.x < K && sp[threadIdx.x] != (int)threadIdx.x)
    p.counts[s0 + threadIdx.x * r.inner] = sn[sp[threadIdx.x]];
}

template <int KM>
__global__ void __launch_bounds__(256) k_fp32_reorder(float* S, ReorderParams r) {
  __shared__ int sp[kMaxBeams], sn[kMaxBeams];
  const int K = r.beams;
  const int64_t i = blockIdx.x % r.inner, xg = blockIdx.x / r.inner, g = xg % r.groups;
  if (threadIdx.x < kMaxBeams) sn[threadIdx.x] = 0;
  if (read_parents(r.parent, g, K, sp) <= 0) return;
  constexpr int nv = kD * kD / 4;
  uint4* base = reinterpret_cast<uint4*>(S) + (xg * K * r.inner + i) * nv;
  const int64_t pitch = r.inner * nv;
  move_all<KM>(nv, [&](int x) { return Place{base + x, pitch, 0}; }, sn, K, sp);
}

}  // namespace

cudaError_t launch_reorder(const Params& p, const ReorderParams& r, cudaStream_t st) {
  const unsigned grid = (unsigned)(r.outer * r.groups * r.inner);
  if (r.beams <= 4) k_reorder<4><<<grid, 256, 0, st>>>(p, r);
  else if (r.beams <= 8) k_reorder<8><<<grid, 256, 0, st>>>(p, r);
  else if (r.beams <= 16) k_reorder<16><<<grid, 256, 0, st>>>(p, r);
  else k_reorder<32><<<grid, 256, 0, st>>>(p, r);
  return cudaGetLastError();
}

cudaError_t launch_fp32_reorder(float* S, const ReorderParams& r, cudaStream_t st) {
  const unsigned grid = (unsigned)(r.outer * r.groups * r.inner);
  if (r.beams <= 4) k_fp32_reorder<4><<<grid, 256, 0, st>>>(S, r);
  else if (r.beams <= 8) k_fp32_reorder<8><<<grid, 256, 0, st>>>(S, r);
  else if (r.beams <= 16) k_fp32_reorder<16><<<grid, 256, 0, st>>>(S, r);
  else k_fp32_reorder<32><<<grid, 256, 0, st>>>(S, r);
  return cudaGetLastError();
}

}  // namespace lqi
