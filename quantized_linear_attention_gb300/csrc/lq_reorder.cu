// Head-states that follow the hypotheses of beam search (sm_103a): afterwards beam
// b of a group holds what beam parent[b] held. In place, without scratch: the
// beams of a group hold the same planes at different offsets, and a thread owns
// the same 16 bytes of every beam. It reads its 16 bytes of each beam that is a
// source and only then writes those of the beams that move, so no thread ever
// reads what another one writes.
//
// Bound by HBM: the sources are read once (a source of several beams comes from
// L1), the moved beams written once, the rest stays where it is; of the record
// planes only the records held move. One CTA takes one (outer, group, inner)
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

// Moves vectors [0, n) of a plane; beam b's part starts at base + b * pitch (in
// vectors). lim (if not NULL): the vectors of beam b that move, by its source.
template <int KM>
__device__ __forceinline__ void move_plane(uint4* base, int64_t pitch, int n, const int* lim, int per, int K,
                                           const int* sp) {
  for (int x = threadIdx.x; x < n; x += blockDim.x) {
    uint4 r[KM];
#pragma unroll
    for (int b = 0; b < KM; ++b)
      if (b < K && sp[b] != b && (!lim || x < lim[sp[b]] * per)) r[b] = base[sp[b] * pitch + x];
#pragma unroll
    for (int b = 0; b < KM; ++b)
      if (b < K && sp[b] != b && (!lim || x < lim[sp[b]] * per)) base[b * pitch + x] = r[b];
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

  auto plane = [&](void* base, int64_t vecs, int n, const int* lim, int per) {
    move_plane<KM>(static_cast<uint4*>(base) + s0 * vecs, r.inner * vecs, n, lim, per, K, sp);
  };
  const int cv = kD * kD * p.bits / 128;  // 16-byte vectors of a head-state's codes
  const int lv = p.C * kD / 4 * (p.comp_fit > 0 ? 2 : 1);
  plane(p.codes, cv, cv, nullptr, 0);
  plane(p.rec_k, p.W * (kD / 4), nmax * (kD / 4), sn, kD / 4);
  plane(p.rec_u, p.W * (kD / 4), nmax * (kD / 4), sn, kD / 4);
  if (lv) plane(p.comp_line, lv, lv, nullptr, 0);
  plane(p.sigma, kD / 4, kD / 4, nullptr, 0);
  plane(p.lambda, kD / 4, kD / 4, nullptr, 0);
  plane(p.comp_id, p.comp_id_stride / 4, (int)(p.comp_id_stride / 4), nullptr, 0);
  if (p.kda) {
    plane(p.rec_alpha, p.W * (kD / 4), nmax * (kD / 4), sn, kD / 4);
  } else if ((int)threadIdx.x < nmax) {  // one decay per record
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
  __shared__ int sp[kMaxBeams];
  const int K = r.beams;
  const int64_t i = blockIdx.x % r.inner, xg = blockIdx.x / r.inner, g = xg % r.groups;
  if (read_parents(r.parent, g, K, sp) <= 0) return;
  constexpr int nv = kD * kD / 4;
  move_plane<KM>(reinterpret_cast<uint4*>(S) + (xg * K * r.inner + i) * nv, r.inner * nv, nv, nullptr, 0, K, sp);
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
