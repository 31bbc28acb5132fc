// Host side of the C ABI declared in include/lq.h: argument validation, the
// state-buffer layout, and kernel launches. No allocation, no synchronization
// except in lq_get_status.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "lq.h"
#include "lq_internal.h"

using lqi::Header;
using lqi::kD;
using lqi::Params;

namespace {

thread_local char g_err[512] = "";

// Test hook (lq_debug_set_wait): this thread's bound on kernel waits and the
// bytes the append / fold kernels announce beyond those they copy.
constexpr uint64_t kWaitNs = 1000000000ull;  // 1 s
thread_local uint64_t g_wait_ns = kWaitNs;
thread_local int32_t g_tx_append = 0, g_tx_fold = 0;

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}

int ok() {
  g_err[0] = '\0';
  return LQ_OK;
}

int cuda_fail(cudaError_t e, const char* what) {
  (void)cudaGetLastError();
  return fail(LQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int64_t kMaxStates = 0x7fffffff;  // one CTA per head-state, gridDim.x limit

int check_cfg(const lq_config* c) {
  if (!c) return fail(LQ_ERR_INVALID_ARG, "cfg is NULL");
  if (c->d_k != kD || c->d_v != kD)
    return fail(LQ_ERR_UNSUPPORTED, "only d_k = d_v = 128 is built (got d_k=%d d_v=%d)", c->d_k, c->d_v);
  if (c->window < 1 || c->window > lqi::kMaxW)
    return fail(LQ_ERR_UNSUPPORTED, "window must be 1..%d (got %d)", lqi::kMaxW, c->window);
  if (c->n_comp < 0 || c->n_comp > lqi::kMaxC)
    return fail(LQ_ERR_UNSUPPORTED, "n_comp must be 0..%d (got %d)", lqi::kMaxC, c->n_comp);
  if (c->decay_per_key != 0 && c->decay_per_key != 1)
    return fail(LQ_ERR_INVALID_ARG, "decay_per_key must be 0 or 1 (got %d)", c->decay_per_key);
  if (c->smooth != 0 && c->smooth != 1) return fail(LQ_ERR_INVALID_ARG, "smooth must be 0 or 1 (got %d)", c->smooth);
  if (!(c->lambda_floor > 0.0f) || !std::isfinite(c->lambda_floor))
    return fail(LQ_ERR_INVALID_ARG, "lambda_floor must be finite and > 0");
  if (c->comp_fit < 0 || c->comp_fit > 32)
    return fail(LQ_ERR_INVALID_ARG, "comp_fit must be 0..32 (got %d)", c->comp_fit);
  if (c->comp_block != 0 && c->comp_block != 1)
    return fail(LQ_ERR_INVALID_ARG, "comp_block must be 0 or 1 (got %d)", c->comp_block);
  if (c->comp_block && c->comp_fit == 0)
    return fail(LQ_ERR_INVALID_ARG, "comp_block needs fitted factors (comp_fit > 0)");
  if (c->code_bits != 8 && c->code_bits != 6 && c->code_bits != 4) {
    if (c->code_bits >= 2 && c->code_bits <= 7)
      return fail(LQ_ERR_UNSUPPORTED, "code_bits %d: this build runs 8-, 6- and 4-bit codes", c->code_bits);
    return fail(LQ_ERR_INVALID_ARG, "code_bits must be 8, 6 or 4 (got %d)", c->code_bits);
  }
  return LQ_OK;
}

int check_n(int64_t n) {
  if (n < 0 || n > kMaxStates) return fail(LQ_ERR_INVALID_ARG, "n_states must be 0..%lld", (long long)kMaxStates);
  return LQ_OK;
}

uint64_t cfg_hash(const lq_config* c, int64_t n) {
  const int64_t f[10] = {c->d_k,       c->d_v,     c->window,   c->n_comp,     c->decay_per_key,
                         c->smooth,    c->code_bits, c->comp_fit, c->comp_block, n};
  uint32_t fl;
  std::memcpy(&fl, &c->lambda_floor, 4);
  uint64_t h = 1469598103934665603ull;  // FNV-1a
  auto mix = [&](uint64_t v) {
    for (int b = 0; b < 8; ++b) {
      h ^= (v >> (8 * b)) & 0xffu;
      h *= 1099511628211ull;
    }
  };
  for (int64_t v : f) mix((uint64_t)v);
  mix(fl);
  return h;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

void make_layout(const lq_config* c, int64_t n, lq_layout_t* L) {
  const size_t N = (size_t)n, D = kD, W = (size_t)c->window, C = (size_t)c->n_comp;
  std::memset(L, 0, sizeof *L);
  L->comp_id_stride = (int64_t)((C + 3) / 4 * 4);
  if (L->comp_id_stride < 4) L->comp_id_stride = 4;
  L->alpha_stride = c->decay_per_key ? (int64_t)(W * D) : (int64_t)((W + 3) / 4 * 4);
  size_t off = 0;
  L->header = off;
  off = align256(off + sizeof(Header));
  L->counts = off;
  off = align256(off + 4 * N);
  L->full_list = off;
  off = align256(off + 4 * N);
  L->codes = off;
  off = align256(off + N * D * D * (size_t)c->code_bits / 8);
  L->sigma = off;
  off = align256(off + 4 * N * D);
  L->lambda = off;
  off = align256(off + 4 * N * D);
  L->comp_id = off;
  off = align256(off + 4 * N * (size_t)L->comp_id_stride);
  L->comp_line = off;
  off = align256(off + 4 * N * C * D * (c->comp_fit > 0 ? 2 : 1));
  L->rec_k = off;
  off = align256(off + 4 * N * W * D);
  L->rec_u = off;
  off = align256(off + 4 * N * W * D);
  L->rec_alpha = off;
  off = align256(off + 4 * N * (size_t)L->alpha_stride);
  L->total_bytes = off;
  L->boundary_bytes_per_state =
      (int64_t)(D * D * (size_t)c->code_bits / 8 + 4 * D + 4 * D + 4 * C + 4 * C * D * (c->comp_fit > 0 ? 2 : 1));
}

int current_device(int* dev) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  return LQ_OK;
}

int check_stream(lq_stream_t stream, int dev) {
  if (!stream) return LQ_OK;
  // A stream being captured into a CUDA graph may not be queried for its
  // device; its kernels are checked when the graph is instantiated.
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing((cudaStream_t)stream, &cap);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
  if (cap != cudaStreamCaptureStatusNone) return LQ_OK;
  int sdev = -1;
  e = cudaStreamGetDevice((cudaStream_t)stream, &sdev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamGetDevice");
  if (sdev != dev) return fail(LQ_ERR_INVALID_ARG, "stream belongs to device %d, current device is %d", sdev, dev);
  return LQ_OK;
}

// Host-only part of a pointer check: not NULL, aligned.
int check_addr(const void* p, const char* name, size_t align) {
  if (!p) return fail(LQ_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)p % align != 0) return fail(LQ_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
  return LQ_OK;
}

int check_ptr(const void* p, const char* name, size_t align, int dev) {
  int rc = check_addr(p, name, align);
  if (rc) return rc;
  cudaPointerAttributes a;
  cudaError_t e = cudaPointerGetAttributes(&a, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(LQ_ERR_INVALID_ARG, "%s is not a CUDA pointer (%s)", name, cudaGetErrorString(e));
  }
  if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)
    return fail(LQ_ERR_INVALID_ARG, "%s is not device memory", name);
  if (a.type == cudaMemoryTypeDevice && a.device != dev)
    return fail(LQ_ERR_INVALID_ARG, "%s is on device %d, current device is %d", name, a.device, dev);
  return LQ_OK;
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

Params make_params(const lq_config* c, void* state, int64_t n) {
  lq_layout_t L;
  make_layout(c, n, &L);
  char* base = static_cast<char*>(state);
  Params p;
  std::memset(&p, 0, sizeof p);
  p.W = c->window;
  p.C = c->n_comp;
  p.kda = c->decay_per_key;
  p.smooth = c->smooth;
  p.bits = c->code_bits;
  p.comp_fit = c->comp_fit;
  p.comp_block = c->comp_block;
  p.lambda_floor = c->lambda_floor;
  p.phase = -1;
  p.wait_ns = g_wait_ns;
  p.dbg_tx_append = g_tx_append;
  p.dbg_tx_fold = g_tx_fold;
  p.n_states = n;
  p.cfg_hash = cfg_hash(c, n);
  p.comp_id_stride = L.comp_id_stride;
  p.alpha_stride = L.alpha_stride;
  p.hdr = reinterpret_cast<Header*>(base + L.header);
  p.counts = reinterpret_cast<int32_t*>(base + L.counts);
  p.full_list = reinterpret_cast<int32_t*>(base + L.full_list);
  p.codes = reinterpret_cast<int8_t*>(base + L.codes);
  p.sigma = reinterpret_cast<float*>(base + L.sigma);
  p.lambda = reinterpret_cast<float*>(base + L.lambda);
  p.comp_id = reinterpret_cast<int32_t*>(base + L.comp_id);
  p.comp_line = reinterpret_cast<float*>(base + L.comp_line);
  p.rec_k = reinterpret_cast<float*>(base + L.rec_k);
  p.rec_u = reinterpret_cast<float*>(base + L.rec_u);
  p.rec_alpha = reinterpret_cast<float*>(base + L.rec_alpha);
  return p;
}

// Common validation of (cfg, state, n, stream); *dev receives the current device.
// The checks that need no GPU (configuration, size, alignment) come first.
int check_common(const lq_config* cfg, const void* state, int64_t n, lq_stream_t stream, int* dev) {
  int rc = check_cfg(cfg);
  if (rc) return rc;
  if ((rc = check_n(n))) return rc;
  if (n == 0) return LQ_OK;
  if ((rc = check_addr(state, "state", 256))) return rc;
  if ((rc = current_device(dev))) return rc;
  if ((rc = check_stream(stream, *dev))) return rc;
  return check_ptr(state, "state", 256, *dev);
}

// Bytes of the state buffer of (cfg, n): an output must not overlap it.
size_t state_size(const lq_config* cfg, int64_t n) {
  lq_layout_t L;
  make_layout(cfg, n, &L);
  return L.total_bytes;
}

// Host-only checks of a token's inputs and output o: NULL, alignment, and o
// overlapping an input or the state buffer (which the same kernels read and write).
int check_tokens_host(const lq_config* cfg, int64_t n, const void* state, const float* q, const float* k,
                      const float* v, const float* alpha, const float* beta, const float* o) {
  int rc;
  if ((rc = check_addr(q, "q", 16)) || (rc = check_addr(k, "k", 16)) || (rc = check_addr(v, "v", 16)) ||
      (rc = check_addr(alpha, "alpha", cfg->decay_per_key ? 16 : 4)) || (rc = check_addr(beta, "beta", 4)) ||
      (rc = check_addr(o, "o", 16)))
    return rc;
  const size_t vec = (size_t)n * kD * sizeof(float);
  const size_t na = cfg->decay_per_key ? vec : (size_t)n * sizeof(float);
  if (overlaps(o, vec, q, vec) || overlaps(o, vec, k, vec) || overlaps(o, vec, v, vec) ||
      overlaps(o, vec, alpha, na) || overlaps(o, vec, beta, (size_t)n * sizeof(float)))
    return fail(LQ_ERR_INVALID_ARG, "o overlaps an input");
  if (state && overlaps(o, vec, state, state_size(cfg, n)))
    return fail(LQ_ERR_INVALID_ARG, "o overlaps the state buffer");
  return LQ_OK;
}

// The host-only checks of a token call, before anything asks the GPU.
int precheck_tokens(const lq_config* cfg, const void* state, int64_t n, const float* q, const float* k,
                    const float* v, const float* alpha, const float* beta, const float* o) {
  int rc = check_cfg(cfg);
  if (rc || (rc = check_n(n))) return rc;
  if (n == 0) return LQ_OK;
  if ((rc = check_addr(state, "state", 256))) return rc;
  return check_tokens_host(cfg, n, state, q, k, v, alpha, beta, o);
}

int check_tokens(const lq_config* cfg, int64_t n, int dev, const float* q, const float* k, const float* v,
                 const float* alpha, const float* beta, const float* o, const void* state = nullptr) {
  int rc = check_tokens_host(cfg, n, state, q, k, v, alpha, beta, o);
  if (rc) return rc;
  if ((rc = check_ptr(q, "q", 16, dev)) || (rc = check_ptr(k, "k", 16, dev)) || (rc = check_ptr(v, "v", 16, dev)) ||
      (rc = check_ptr(alpha, "alpha", 4, dev)) || (rc = check_ptr(beta, "beta", 4, dev)) ||
      (rc = check_ptr(o, "o", 16, dev)))
    return rc;
  return LQ_OK;
}

// ---- linear attention with a decay per head, beam search

int check_la(const lq_la_config* c) {
  if (!c) return fail(LQ_ERR_INVALID_ARG, "cfg is NULL");
  if (c->d_k != kD || c->d_v != kD)
    return fail(LQ_ERR_UNSUPPORTED, "only d_k = d_v = 128 is built (got d_k=%d d_v=%d)", c->d_k, c->d_v);
  if (c->dtype != LQ_F32 && c->dtype != LQ_BF16 && c->dtype != LQ_F16)
    return fail(LQ_ERR_INVALID_ARG, "dtype must be LQ_F32, LQ_BF16 or LQ_F16 (got %d)", c->dtype);
  if (c->reserved != 0) return fail(LQ_ERR_INVALID_ARG, "reserved must be 0");
  if (c->heads < 1 || c->heads > 65535 || c->key_heads < 1 || c->heads % c->key_heads != 0)
    return fail(LQ_ERR_INVALID_ARG, "heads must be 1..65535 and a multiple of key_heads (got %d, %d)", c->heads,
                c->key_heads);
  const int64_t per16 = c->dtype == LQ_F32 ? 4 : 8;
  const int64_t st[4] = {c->q_stride, c->k_stride, c->v_stride, c->o_stride};
  const char* names[4] = {"q", "k", "v", "o"};
  for (int i = 0; i < 4; ++i) {
    const int64_t least = (int64_t)(i < 2 ? c->key_heads : c->heads) * kD;
    if (st[i] < least || st[i] % per16 != 0 || st[i] > ((int64_t)1 << 38))
      return fail(LQ_ERR_INVALID_ARG, "%s_stride must be at least %lld and a multiple of 16 bytes (got %lld)", names[i],
                  (long long)least, (long long)st[i]);
  }
  if (c->alpha_stride != 0 && (c->alpha_stride < c->heads || c->alpha_stride > ((int64_t)1 << 40)))
    return fail(LQ_ERR_INVALID_ARG, "alpha_stride must be 0 or at least heads (got %lld)", (long long)c->alpha_stride);
  return LQ_OK;
}

size_t la_size(int32_t dtype) { return dtype == LQ_F32 ? 4 : 2; }

// Bytes from the first element of a strided token array to the end of its last token.
size_t la_extent(int64_t tokens, int64_t stride, int64_t row, size_t size) {
  return tokens ? ((size_t)(tokens - 1) * (size_t)stride + (size_t)row) * size : 0;
}

// The token arrays of a call, on the host: NULL, alignment, and o overlapping an input or a state.
int check_la_tokens(const lq_la_config* c, int64_t n, const void* q, const void* k, const void* v, const float* alpha,
                    const void* o) {
  int rc;
  if ((rc = check_addr(q, "q", 16)) || (rc = check_addr(k, "k", 16)) || (rc = check_addr(v, "v", 16)) ||
      (rc = check_addr(alpha, "alpha", 4)) || (rc = check_addr(o, "o", 16)))
    return rc;
  const size_t e = la_size(c->dtype);
  const int64_t kr = (int64_t)c->key_heads * kD, vr = (int64_t)c->heads * kD;
  const size_t no = la_extent(n, c->o_stride, vr, e);
  if (overlaps(o, no, q, la_extent(n, c->q_stride, kr, e)) || overlaps(o, no, k, la_extent(n, c->k_stride, kr, e)) ||
      overlaps(o, no, v, la_extent(n, c->v_stride, vr, e)) ||
      overlaps(o, no, alpha, la_extent(n, c->alpha_stride, c->heads, 4)))
    return fail(LQ_ERR_INVALID_ARG, "o overlaps an input");
  return LQ_OK;
}

int check_la_device(const lq_la_config*, int dev, const void* q, const void* k, const void* v, const float* alpha,
                    const void* o) {
  int rc;
  if ((rc = check_ptr(q, "q", 16, dev)) || (rc = check_ptr(k, "k", 16, dev)) || (rc = check_ptr(v, "v", 16, dev)) ||
      (rc = check_ptr(alpha, "alpha", 4, dev)) || (rc = check_ptr(o, "o", 16, dev)))
    return rc;
  return LQ_OK;
}

int check_prompt_sizes(const lq_la_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len) {
  int rc = check_la(c);
  if (rc) return rc;
  if (n_seqs < 0 || n_tokens < 0 || n_tokens > 0x7fffffff || max_len < 0)
    return fail(LQ_ERR_INVALID_ARG, "n_seqs and max_len must not be negative, n_tokens must be 0..%d", 0x7fffffff);
  if (n_seqs > kMaxStates / 8 / c->heads)
    return fail(LQ_ERR_INVALID_ARG, "n_seqs x heads must be at most %lld", (long long)(kMaxStates / 8));
  return LQ_OK;
}

lqi::LaParams la_params(const lq_la_config* c, const void* q, const void* k, const void* v, const float* alpha,
                        void* o) {
  lqi::LaParams p;
  std::memset(&p, 0, sizeof p);
  p.heads = c->heads;
  p.key_heads = c->key_heads;
  p.group = c->heads / c->key_heads;
  p.dtype = c->dtype;
  p.sq = c->q_stride;
  p.sk = c->k_stride;
  p.sv = c->v_stride;
  p.so = c->o_stride;
  p.sa = c->alpha_stride;
  p.q = q;
  p.k = k;
  p.v = v;
  p.alpha = alpha;
  p.o = o;
  p.wait_ns = g_wait_ns;
  p.dbg_tx = (uint32_t)g_tx_append;
  return p;
}

// Split sequences: what each segment adds to the state, its decay, and the last states where they replace S0.
size_t la_workspace(const lq_la_config* c, int64_t n_seqs, int64_t slots) {
  return align256((size_t)slots * c->heads * kD * kD * sizeof(float)) +
         align256((size_t)slots * c->heads * sizeof(float2)) +
         align256((size_t)n_seqs * c->heads * kD * kD * sizeof(float));
}

int check_beams(int64_t batch, int32_t beams, int64_t vocab, int32_t n_best) {
  if (batch < 0 || beams < 1 || beams > lqi::kMaxBeams)
    return fail(LQ_ERR_INVALID_ARG, "batch must not be negative, beams must be 1..%d (got %lld, %d)", lqi::kMaxBeams,
                (long long)batch, beams);
  if (vocab < 1 || vocab > 0x7fffffff / beams)
    return fail(LQ_ERR_INVALID_ARG, "vocab must be 1..(2^31 - 1) / beams (got %lld)", (long long)vocab);
  if (n_best < 1 || n_best > lqi::kMaxBest || n_best > beams * vocab)
    return fail(LQ_ERR_INVALID_ARG, "n_best must be 1..%d and at most beams x vocab (got %d)", lqi::kMaxBest, n_best);
  // one CTA per slice of a row
  if (batch > kMaxStates / beams / lqi::beam_splits(LQ_F32, vocab))
    return fail(LQ_ERR_INVALID_ARG, "batch %lld is too large", (long long)batch);
  return LQ_OK;
}

int check_reorder(int64_t n_states, int64_t outer, int64_t groups, int32_t beams, int64_t inner) {
  int rc = check_n(n_states);
  if (rc) return rc;
  if (beams < 1 || beams > lqi::kMaxBeams)
    return fail(LQ_ERR_INVALID_ARG, "beams must be 1..%d (got %d)", lqi::kMaxBeams, beams);
  const int64_t f[3] = {outer, groups, inner};
  int64_t n = beams;
  for (int64_t x : f) {
    if (x < 0 || x > kMaxStates) return fail(LQ_ERR_INVALID_ARG, "outer, groups and inner must be 0..%lld",
                                             (long long)kMaxStates);
    n = (n > kMaxStates && x) ? n : n * x;  // (stays above the limit once it is; no overflow: both are below 2^31)
  }
  if (n != n_states)
    return fail(LQ_ERR_INVALID_ARG, "outer x groups x beams x inner must be n_states = %lld", (long long)n_states);
  return LQ_OK;
}

// Sizes of packed prompts.
constexpr int64_t kMaxTokens = 0x7fffff00;  // (tokens are counted in 32 bits, some tiles past the last)

int check_packed(int64_t n_seqs, int64_t n_tokens, int64_t max_len, const int32_t* cu) {
  if (n_seqs < 0 || n_seqs > 0x7fffffff || n_tokens < 0 || n_tokens > kMaxTokens || max_len < 0)
    return fail(LQ_ERR_INVALID_ARG, "n_seqs must be 0..%d, n_tokens 0..%lld, max_len must not be negative", 0x7fffffff,
                (long long)kMaxTokens);
  if (n_seqs == 0) return LQ_OK;
  if (!cu && n_seqs != 1) return fail(LQ_ERR_INVALID_ARG, "cu_seqlens is NULL with n_seqs > 1");
  if (!cu && max_len > 0 && max_len < n_tokens)
    return fail(LQ_ERR_INVALID_ARG, "max_len is less than n_tokens, the length of the only sequence");
  return LQ_OK;
}

int check_dtype(int32_t dtype) {
  if (dtype != LQ_F32 && dtype != LQ_BF16 && dtype != LQ_F16)
    return fail(LQ_ERR_INVALID_ARG, "dtype must be LQ_F32, LQ_BF16 or LQ_F16 (got %d)", dtype);
  return LQ_OK;
}

int check_stride(int64_t stride, int64_t row, const char* name) {
  if (stride < row || stride > ((int64_t)1 << 38))
    return fail(LQ_ERR_INVALID_ARG, "%s must be at least %lld (got %lld)", name, (long long)row, (long long)stride);
  return LQ_OK;
}

constexpr int32_t kMaxChannels = 1 << 20;

int check_conv(const lq_conv_config* c) {
  if (!c) return fail(LQ_ERR_INVALID_ARG, "cfg is NULL");
  if (c->channels < 1 || c->channels > kMaxChannels)
    return fail(LQ_ERR_INVALID_ARG, "channels must be 1..%d (got %d)", kMaxChannels, c->channels);
  if (c->width < 2 || c->width > lqi::kMaxWidth)
    return fail(LQ_ERR_UNSUPPORTED, "width must be 2..%d (got %d)", lqi::kMaxWidth, c->width);
  if (c->silu != 0 && c->silu != 1) return fail(LQ_ERR_INVALID_ARG, "silu must be 0 or 1 (got %d)", c->silu);
  int rc = check_dtype(c->dtype);
  if (rc || (rc = check_stride(c->x_stride, c->channels, "x_stride")) ||
      (rc = check_stride(c->y_stride, c->channels, "y_stride")))
    return rc;
  return LQ_OK;
}

int check_ssm(const lq_ssm_config* c) {
  if (!c) return fail(LQ_ERR_INVALID_ARG, "cfg is NULL");
  if (c->channels < 1 || c->channels > kMaxChannels)
    return fail(LQ_ERR_INVALID_ARG, "channels must be 1..%d (got %d)", kMaxChannels, c->channels);
  if (c->n_state < 1 || c->n_state > lqi::kMaxNState)
    return fail(LQ_ERR_UNSUPPORTED, "n_state must be 1..%d (got %d)", lqi::kMaxNState, c->n_state);
  if (c->groups < 1 || c->channels % c->groups != 0)
    return fail(LQ_ERR_INVALID_ARG, "groups must divide channels (got %d, %d)", c->groups, c->channels);
  if (c->softplus != 0 && c->softplus != 1)
    return fail(LQ_ERR_INVALID_ARG, "softplus must be 0 or 1 (got %d)", c->softplus);
  if (c->reserved != 0) return fail(LQ_ERR_INVALID_ARG, "reserved must be 0");
  int rc = check_dtype(c->dtype);
  const int64_t bc = (int64_t)c->groups * c->n_state;
  if (rc || (rc = check_stride(c->x_stride, c->channels, "x_stride")) ||
      (rc = check_stride(c->dt_stride, c->channels, "dt_stride")) ||
      (rc = check_stride(c->z_stride, c->channels, "z_stride")) ||
      (rc = check_stride(c->y_stride, c->channels, "y_stride")) || (rc = check_stride(c->b_stride, bc, "b_stride")) ||
      (rc = check_stride(c->c_stride, bc, "c_stride")))
    return rc;
  return LQ_OK;
}

// One argument of a call: what it is, where, how long, and whether the call writes it.
struct Arg {
  const void* p;
  const char* name;
  size_t bytes, align;
  bool optional, written;
};

// On the host: NULL, alignment, and written arguments that overlap another. Arguments `in` and
// `out` may be one and the same (a state in place).
int check_args(const Arg* a, int n, int in = -1, int out = -1) {
  int rc;
  for (int i = 0; i < n; ++i)
    if ((a[i].p || !a[i].optional) && a[i].bytes && (rc = check_addr(a[i].p, a[i].name, a[i].align))) return rc;
  for (int i = 0; i < n; ++i) {
    if (!a[i].p || !a[i].written) continue;
    for (int j = 0; j < n; ++j) {
      if (j == i || !a[j].p || (a[j].written && j < i)) continue;
      if (((i == in && j == out) || (i == out && j == in)) && a[i].p == a[j].p) continue;
      if (a[i].bytes && a[j].bytes && overlaps(a[i].p, a[i].bytes, a[j].p, a[j].bytes))
        return fail(LQ_ERR_INVALID_ARG, "%s overlaps %s", a[i].name, a[j].name);
    }
  }
  return LQ_OK;
}

int check_args_device(const Arg* a, int n, int dev) {
  int rc;
  for (int i = 0; i < n; ++i)
    if (a[i].p && a[i].bytes && (rc = check_ptr(a[i].p, a[i].name, a[i].align, dev))) return rc;
  return LQ_OK;
}

// CTAs of a launch: one for each block of channels of each slot.
int check_grid(int64_t slots, int64_t blocks) {
  if (slots > kMaxStates / blocks)
    return fail(LQ_ERR_INVALID_ARG, "too many sequences or tokens for one call (%lld x %lld)", (long long)slots,
                (long long)blocks);
  return LQ_OK;
}

lqi::SsmParams ssm_params(const lq_ssm_config* c, const void* x, const void* dt, const float* A, const void* B,
                          const void* C, const float* D, const void* z, const float* dt_bias, void* y) {
  lqi::SsmParams p;
  std::memset(&p, 0, sizeof p);
  p.channels = c->channels;
  p.n_state = c->n_state;
  p.groups = c->groups;
  p.per_group = c->channels / c->groups;
  p.dtype = c->dtype;
  p.softplus = c->softplus;
  p.sx = c->x_stride;
  p.sdt = c->dt_stride;
  p.sz = c->z_stride;
  p.sb = c->b_stride;
  p.sc = c->c_stride;
  p.sy = c->y_stride;
  p.x = x;
  p.dt = dt;
  p.A = A;
  p.B = B;
  p.C = C;
  p.D = D;
  p.z = z;
  p.dt_bias = dt_bias;
  p.y = y;
  return p;
}

// Split sequences: what a segment adds to the states, and the sum of its steps.
size_t ssm_workspace(const lq_ssm_config* c, int64_t slots) {
  return align256((size_t)slots * c->channels * c->n_state * sizeof(float)) +
         align256((size_t)slots * c->channels * sizeof(float));
}

int launched(cudaError_t e, const char* what) { return e == cudaSuccess ? ok() : cuda_fail(e, what); }

}  // namespace

extern "C" {

const char* lq_last_error(void) { return g_err; }

int lq_version(void) { return 100; }

int lq_debug_set_wait(uint64_t wait_ns, int32_t extra_tx_append, int32_t extra_tx_fold) {
  if (wait_ns > kWaitNs) return fail(LQ_ERR_INVALID_ARG, "wait_ns must be 0..%llu", (unsigned long long)kWaitNs);
  if (extra_tx_append < 0 || extra_tx_append > 1024 || extra_tx_fold < 0 || extra_tx_fold > 1024)
    return fail(LQ_ERR_INVALID_ARG, "extra_tx bytes must be 0..1024");
  g_wait_ns = wait_ns ? wait_ns : kWaitNs;
  g_tx_append = extra_tx_append;
  g_tx_fold = extra_tx_fold;
  return ok();
}

void lq_config_default(lq_config* cfg) {
  if (!cfg) return;
  cfg->d_k = kD;
  cfg->d_v = kD;
  cfg->window = 16;
  cfg->n_comp = 4;
  cfg->decay_per_key = 0;
  cfg->smooth = 1;
  cfg->code_bits = 8;
  cfg->comp_fit = 0;
  cfg->comp_block = 0;
  cfg->lambda_floor = 1e-6f;
}

size_t lq_state_bytes(const lq_config* cfg, int64_t n_states) {
  if (check_cfg(cfg) || check_n(n_states)) return 0;
  lq_layout_t L;
  make_layout(cfg, n_states, &L);
  return L.total_bytes;
}

int lq_layout(const lq_config* cfg, int64_t n_states, lq_layout_t* out) {
  int rc = check_cfg(cfg);
  if (rc) return rc;
  if ((rc = check_n(n_states))) return rc;
  if (!out) return fail(LQ_ERR_INVALID_ARG, "out is NULL");
  make_layout(cfg, n_states, out);
  return ok();
}

int lq_state_init(const lq_config* cfg, void* state, int64_t n_states, const float* S0, lq_stream_t stream) {
  int dev = 0;
  int rc = check_common(cfg, state, n_states, stream, &dev);
  if (rc || n_states == 0) return rc ? rc : ok();
  if (S0 && (rc = check_ptr(S0, "S0", 16, dev))) return rc;
  Params p = make_params(cfg, state, n_states);
  p.S0 = S0;
  return launched(lqi::launch_init(p, (cudaStream_t)stream), "lq_state_init launch");
}

int lq_state_init_range(const lq_config* cfg, void* state, int64_t n_states, int64_t first, int64_t count,
                        const float* S0, lq_stream_t stream) {
  int rc = check_cfg(cfg);
  if (rc) return rc;
  if ((rc = check_n(n_states))) return rc;
  if (first < 0 || count < 0 || first > n_states || count > n_states - first)
    return fail(LQ_ERR_INVALID_ARG, "range [%lld, %lld + %lld) is not inside 0..%lld", (long long)first,
                (long long)first, (long long)count, (long long)n_states);
  if (count == 0) return ok();
  int dev = 0;
  if ((rc = check_common(cfg, state, n_states, stream, &dev))) return rc;
  if (S0 && (rc = check_ptr(S0, "S0", 16, dev))) return rc;
  Params p = make_params(cfg, state, n_states);
  p.S0 = S0;
  p.first = first;
  return launched(lqi::launch_init_range(p, count, (cudaStream_t)stream), "lq_state_init_range launch");
}

int lq_append(const lq_config* cfg, void* state, int64_t n_states, const float* q, const float* k, const float* v,
              const float* alpha, const float* beta, float* o, lq_stream_t stream) {
  int dev = 0;
  int rc = precheck_tokens(cfg, state, n_states, q, k, v, alpha, beta, o);
  if (rc || (rc = check_common(cfg, state, n_states, stream, &dev)) || n_states == 0) return rc ? rc : ok();
  if ((rc = check_tokens(cfg, n_states, dev, q, k, v, alpha, beta, o, state))) return rc;
  Params p = make_params(cfg, state, n_states);
  p.q = q;
  p.k = k;
  p.v = v;
  p.alpha = alpha;
  p.beta = beta;
  p.o = o;
  return launched(lqi::launch_append(p, (cudaStream_t)stream), "lq_append launch");
}

int lq_fold(const lq_config* cfg, void* state, int64_t n_states, lq_stream_t stream) {
  int dev = 0;
  int rc = check_common(cfg, state, n_states, stream, &dev);
  if (rc || n_states == 0) return rc ? rc : ok();
  Params p = make_params(cfg, state, n_states);
  return launched(lqi::launch_fold(p, (cudaStream_t)stream), "lq_fold launch");
}

int lq_decode_step(const lq_config* cfg, void* state, int64_t n_states, int32_t phase, const float* q,
                   const float* k, const float* v, const float* alpha, const float* beta, float* o,
                   lq_stream_t stream) {
  int dev = 0;
  int rc = precheck_tokens(cfg, state, n_states, q, k, v, alpha, beta, o);
  if (rc || (rc = check_common(cfg, state, n_states, stream, &dev))) return rc;
  if (phase != LQ_PHASE_ANY && (phase < 0 || phase >= cfg->window))
    return fail(LQ_ERR_INVALID_ARG, "phase must be LQ_PHASE_ANY or 0..W-1 (got %d)", phase);
  if (n_states == 0) return ok();
  if ((rc = check_tokens(cfg, n_states, dev, q, k, v, alpha, beta, o, state))) return rc;
  Params p = make_params(cfg, state, n_states);
  p.q = q;
  p.k = k;
  p.v = v;
  p.alpha = alpha;
  p.beta = beta;
  p.o = o;
  p.phase = phase;
  // A stated phase below W-1 cannot fill the window: the append-only kernel
  // needs no fold workspace and runs at higher occupancy. At W-1 every
  // head-state folds, in the append kernel. Mixed phases: append (listing the
  // windows filled), then fold the list.
  if (phase == LQ_PHASE_ANY) {
    p.push_full = 1;
    cudaError_t e = lqi::launch_append(p, (cudaStream_t)stream);
    if (e == cudaSuccess) e = lqi::launch_fold_listed(p, (cudaStream_t)stream);
    return launched(e, "lq_decode_step launch");
  }
  if (phase < cfg->window - 1)
    return launched(lqi::launch_append(p, (cudaStream_t)stream), "lq_decode_step launch");
  return launched(lqi::launch_step(p, (cudaStream_t)stream), "lq_decode_step launch");
}

int lq_decode_step_noalloc(const lq_config* cfg, void* state, int64_t n_states, const float* q, const float* k,
                           const float* v, const float* alpha, const float* beta, float* o, lq_stream_t stream) {
  int rc = check_cfg(cfg);
  if (rc) return rc;
  if (cfg->code_bits != 8 || cfg->comp_fit != 0)
    return fail(LQ_ERR_UNSUPPORTED, "lq_decode_step_noalloc runs 8-bit codes with line compensators only");
  if (n_states > lqi::kNoAllocMaxStates)
    return fail(LQ_ERR_INVALID_ARG, "lq_decode_step_noalloc: n_states %lld exceeds the %d head-states its fixed "
                "work list holds", (long long)n_states, lqi::kNoAllocMaxStates);
  int dev = 0;
  if ((rc = precheck_tokens(cfg, state, n_states, q, k, v, alpha, beta, o)) ||
      (rc = check_common(cfg, state, n_states, stream, &dev)))
    return rc;
  if (n_states == 0) return ok();
  if ((rc = check_tokens(cfg, n_states, dev, q, k, v, alpha, beta, o, state))) return rc;
  Params p = make_params(cfg, state, n_states);
  p.q = q;
  p.k = k;
  p.v = v;
  p.alpha = alpha;
  p.beta = beta;
  p.o = o;
  p.phase = LQ_PHASE_ANY;
  return launched(lqi::launch_decode_noalloc(p, dev, (cudaStream_t)stream), "lq_decode_step_noalloc launch");
}

int lq_decode_step2(const lq_config* cfg, void* state, int64_t n_states, int32_t phase, const float* q,
                    const float* k1, const float* v1, const float* beta1, const float* k2, const float* v2,
                    const float* beta2, const float* alpha, float* o, lq_stream_t stream) {
  int dev = 0;
  int rc = precheck_tokens(cfg, state, n_states, q, k1, v1, alpha, beta1, o);
  if (rc || (rc = check_common(cfg, state, n_states, stream, &dev))) return rc;
  if (cfg->window < 2) return fail(LQ_ERR_UNSUPPORTED, "two-record tokens need a window of at least 2 records");
  if (phase != LQ_PHASE_ANY && (phase < 0 || phase > cfg->window - 2))
    return fail(LQ_ERR_INVALID_ARG, "phase must be LQ_PHASE_ANY or 0..W-2 (got %d)", phase);
  if (n_states == 0) return ok();
  if ((rc = check_tokens(cfg, n_states, dev, q, k1, v1, alpha, beta1, o, state))) return rc;
  if ((rc = check_ptr(k2, "k2", 16, dev)) || (rc = check_ptr(v2, "v2", 16, dev)) ||
      (rc = check_ptr(beta2, "beta2", 4, dev)))
    return rc;
  const size_t vec = (size_t)n_states * kD * sizeof(float);
  if (overlaps(o, vec, k2, vec) || overlaps(o, vec, v2, vec) || overlaps(o, vec, beta2, (size_t)n_states * 4))
    return fail(LQ_ERR_INVALID_ARG, "o overlaps an input");
  Params p = make_params(cfg, state, n_states);
  p.q = q;
  p.k = k1;
  p.v = v1;
  p.beta = beta1;
  p.k2 = k2;
  p.v2 = v2;
  p.beta2 = beta2;
  p.alpha = alpha;
  p.o = o;
  p.phase = phase;
  // The window can fill only at phase W-2 (or at any phase when not stated):
  // then the filled head-states are listed and folded by a second kernel.
  p.push_full = (phase == LQ_PHASE_ANY || phase == cfg->window - 2) ? 1 : 0;
  cudaError_t e = lqi::launch_append2(p, (cudaStream_t)stream);
  if (e == cudaSuccess && p.push_full) e = lqi::launch_fold_listed(p, (cudaStream_t)stream);
  return launched(e, "lq_decode_step2 launch");
}

int lq_decode_step_rwkv7(const lq_config* cfg, void* state, int64_t n_states, int32_t phase, const float* r,
                         const float* w, const float* kh, const float* a, const float* k, const float* v, float* o,
                         lq_stream_t stream) {
  int dev = 0;
  int rc = check_common(cfg, state, n_states, stream, &dev);
  if (rc) return rc;
  if (!cfg->decay_per_key) return fail(LQ_ERR_UNSUPPORTED, "RWKV7 tokens need per-key decay (decay_per_key = 1)");
  if (cfg->window < 2) return fail(LQ_ERR_UNSUPPORTED, "two-record tokens need a window of at least 2 records");
  if (phase != LQ_PHASE_ANY && (phase < 0 || phase > cfg->window - 2))
    return fail(LQ_ERR_INVALID_ARG, "phase must be LQ_PHASE_ANY or 0..W-2 (got %d)", phase);
  if (n_states == 0) return ok();
  const void* in[6] = {r, w, kh, a, k, v};
  const char* names[6] = {"r", "w", "kh", "a", "k", "v"};
  for (int t = 0; t < 6; ++t)
    if ((rc = check_ptr(in[t], names[t], 16, dev))) return rc;
  if ((rc = check_ptr(o, "o", 16, dev))) return rc;
  const size_t vec = (size_t)n_states * kD * sizeof(float);
  for (int t = 0; t < 6; ++t)
    if (overlaps(o, vec, in[t], vec)) return fail(LQ_ERR_INVALID_ARG, "o overlaps an input");
  if (overlaps(o, vec, state, state_size(cfg, n_states)))
    return fail(LQ_ERR_INVALID_ARG, "o overlaps the state buffer");
  Params p = make_params(cfg, state, n_states);
  p.q = r;
  p.alpha = w;
  p.kh = kh;
  p.ka = a;
  p.k = k;
  p.v = v;
  p.o = o;
  p.phase = phase;
  p.push_full = (phase == LQ_PHASE_ANY || phase == cfg->window - 2) ? 1 : 0;
  cudaError_t e = lqi::launch_append_rwkv(p, (cudaStream_t)stream);
  if (e == cudaSuccess && p.push_full) e = lqi::launch_fold_listed(p, (cudaStream_t)stream);
  return launched(e, "lq_decode_step_rwkv7 launch");
}

int lq_export_state(const lq_config* cfg, const void* state, int64_t n_states, float* S_out, lq_stream_t stream) {
  int dev = 0;
  int rc = check_common(cfg, state, n_states, stream, &dev);
  if (rc || n_states == 0) return rc ? rc : ok();
  if ((rc = check_ptr(S_out, "S_out", 16, dev))) return rc;
  if (overlaps(S_out, (size_t)n_states * kD * kD * sizeof(float), state, state_size(cfg, n_states)))
    return fail(LQ_ERR_INVALID_ARG, "S_out overlaps the state buffer");
  Params p = make_params(cfg, const_cast<void*>(state), n_states);
  p.S_out = S_out;
  return launched(lqi::launch_export(p, (cudaStream_t)stream), "lq_export_state launch");
}

int lq_fp32_decode_step(const lq_config* cfg, float* S, int64_t n_states, const float* q, const float* k,
                        const float* v, const float* alpha, const float* beta, float* o, lq_stream_t stream) {
  int rc = check_cfg(cfg);
  if (rc) return rc;
  if ((rc = check_n(n_states))) return rc;
  if (n_states == 0) return ok();
  int dev = 0;
  if ((rc = current_device(&dev)) || (rc = check_stream(stream, dev))) return rc;
  if ((rc = check_ptr(S, "S", 16, dev))) return rc;
  if ((rc = check_tokens(cfg, n_states, dev, q, k, v, alpha, beta, o))) return rc;
  const size_t sb = (size_t)n_states * kD * kD * sizeof(float), vec = (size_t)n_states * kD * sizeof(float);
  if (overlaps(S, sb, o, vec) || overlaps(S, sb, q, vec) || overlaps(S, sb, k, vec) || overlaps(S, sb, v, vec))
    return fail(LQ_ERR_INVALID_ARG, "S overlaps a token input or o");
  lqi::Fp32Params p;
  p.n_states = n_states;
  p.kda = cfg->decay_per_key;
  p.S = S;
  p.q = q;
  p.k = k;
  p.v = v;
  p.alpha = alpha;
  p.beta = beta;
  p.o = o;
  return launched(lqi::launch_fp32_step(p, (cudaStream_t)stream), "lq_fp32_decode_step launch");
}

void lq_la_config_default(lq_la_config* cfg, int32_t heads, int32_t key_heads, int32_t dtype) {
  if (!cfg) return;
  std::memset(cfg, 0, sizeof *cfg);
  cfg->d_k = kD;
  cfg->d_v = kD;
  cfg->heads = heads;
  cfg->key_heads = key_heads;
  cfg->dtype = dtype;
  cfg->q_stride = cfg->k_stride = (int64_t)key_heads * kD;
  cfg->v_stride = cfg->o_stride = (int64_t)heads * kD;
  cfg->alpha_stride = heads;
}

size_t lq_la_workspace_bytes(const lq_la_config* cfg, int64_t n_seqs, int64_t n_tokens, int64_t max_len) {
  if (check_prompt_sizes(cfg, n_seqs, n_tokens, max_len) || n_seqs == 0) return 0;
  const int64_t slots = lqi::la_most_slots(cfg, n_seqs, n_tokens, max_len);
  return slots ? la_workspace(cfg, n_seqs, slots) : 0;
}

int lq_la_prefill(const lq_la_config* cfg, int64_t n_seqs, int64_t n_tokens, int64_t max_len,
                  const int32_t* cu_seqlens, const void* q, const void* k, const void* v, const float* alpha,
                  const float* S0, float* S_out, void* o, void* workspace, size_t workspace_bytes,
                  lq_stream_t stream) {
  int rc = check_prompt_sizes(cfg, n_seqs, n_tokens, max_len);
  if (rc) return rc;
  if (n_seqs == 0) return ok();
  if (!cu_seqlens && n_seqs != 1) return fail(LQ_ERR_INVALID_ARG, "cu_seqlens is NULL with n_seqs > 1");
  if (!cu_seqlens && max_len > 0 && max_len < n_tokens)
    return fail(LQ_ERR_INVALID_ARG, "max_len is less than n_tokens, the length of the only sequence");
  if (cu_seqlens && (rc = check_addr(cu_seqlens, "cu_seqlens", 4))) return rc;
  if (n_tokens && (rc = check_la_tokens(cfg, n_tokens, q, k, v, alpha, o))) return rc;
  if (S0 && (rc = check_addr(S0, "S0", 16))) return rc;
  if (S_out && (rc = check_addr(S_out, "S_out", 16))) return rc;
  const size_t sb = (size_t)n_seqs * cfg->heads * kD * kD * sizeof(float), e = la_size(cfg->dtype);
  const size_t nq = la_extent(n_tokens, cfg->q_stride, (int64_t)cfg->key_heads * kD, e);
  const size_t nk = la_extent(n_tokens, cfg->k_stride, (int64_t)cfg->key_heads * kD, e);
  const size_t nv = la_extent(n_tokens, cfg->v_stride, (int64_t)cfg->heads * kD, e);
  const size_t no = la_extent(n_tokens, cfg->o_stride, (int64_t)cfg->heads * kD, e);
  const size_t na = la_extent(n_tokens, cfg->alpha_stride, cfg->heads, 4), nc = cu_seqlens ? (size_t)(n_seqs + 1) * 4 : 0;
  if (S_out && S_out != S0 && S0 && overlaps(S_out, sb, S0, sb))
    return fail(LQ_ERR_INVALID_ARG, "S_out overlaps S0 (it may only be S0 itself)");
  if (S_out && (overlaps(S_out, sb, q, nq) || overlaps(S_out, sb, k, nk) || overlaps(S_out, sb, v, nv) ||
                overlaps(S_out, sb, o, no) || overlaps(S_out, sb, alpha, na)))
    return fail(LQ_ERR_INVALID_ARG, "S_out overlaps a token array");
  if (overlaps(cu_seqlens, nc, o, no) || (S_out && overlaps(cu_seqlens, nc, S_out, sb)))
    return fail(LQ_ERR_INVALID_ARG, "cu_seqlens overlaps o or S_out");
  if (S0 && overlaps(S0, sb, o, no)) return fail(LQ_ERR_INVALID_ARG, "o overlaps S0");
  lqi::LaParams p = la_params(cfg, q, k, v, alpha, o);
  lqi::la_plan(cfg, n_seqs, n_tokens, max_len, &p.seg, &p.slots);
  const size_t need = p.slots ? la_workspace(cfg, n_seqs, p.slots) : 0;
  if (need) {
    if ((rc = check_addr(workspace, "workspace", 256))) return rc;
    if (workspace_bytes < need)
      return fail(LQ_ERR_INVALID_ARG, "workspace has %zu bytes, %zu are needed", workspace_bytes, need);
    if (overlaps(workspace, need, o, no) || (S_out && overlaps(workspace, need, S_out, sb)) ||
        (S0 && overlaps(workspace, need, S0, sb)) || overlaps(workspace, need, q, nq) ||
        overlaps(workspace, need, k, nk) || overlaps(workspace, need, v, nv) || overlaps(workspace, need, alpha, na) ||
        overlaps(workspace, need, cu_seqlens, nc))
      return fail(LQ_ERR_INVALID_ARG, "workspace overlaps another argument");
  }
  int dev = 0;
  if ((rc = current_device(&dev)) || (rc = check_stream(stream, dev))) return rc;
  if (n_tokens && (rc = check_la_device(cfg, dev, q, k, v, alpha, o))) return rc;
  if ((cu_seqlens && (rc = check_ptr(cu_seqlens, "cu_seqlens", 4, dev))) ||
      (S0 && (rc = check_ptr(S0, "S0", 16, dev))) || (S_out && (rc = check_ptr(S_out, "S_out", 16, dev))) ||
      (need && (rc = check_ptr(workspace, "workspace", 256, dev))))
    return rc;
  p.n_seqs = n_seqs;
  p.n_tokens = n_tokens;
  p.max_len = max_len;
  p.cu = cu_seqlens;
  p.S0 = S0;
  p.S = S_out;
  char* ws = static_cast<char*>(workspace);
  p.ws_state = reinterpret_cast<float*>(ws);
  ws += align256((size_t)p.slots * cfg->heads * kD * kD * sizeof(float));
  p.ws_decay = reinterpret_cast<float2*>(ws);
  ws += align256((size_t)p.slots * cfg->heads * sizeof(float2));
  p.ws_last = reinterpret_cast<float*>(ws);
  return launched(lqi::launch_la_prefill(p, (cudaStream_t)stream), "lq_la_prefill launch");
}

int lq_la_decode_step(const lq_la_config* cfg, float* S, int64_t n_seqs, const void* q, const void* k, const void* v,
                      const float* alpha, void* o, lq_stream_t stream) {
  int rc = check_prompt_sizes(cfg, n_seqs, n_seqs, 0);
  if (rc) return rc;
  if (n_seqs == 0) return ok();
  if ((rc = check_addr(S, "S", 16)) || (rc = check_la_tokens(cfg, n_seqs, q, k, v, alpha, o))) return rc;
  const size_t sb = (size_t)n_seqs * cfg->heads * kD * kD * sizeof(float), e = la_size(cfg->dtype);
  const int64_t kr = (int64_t)cfg->key_heads * kD, vr = (int64_t)cfg->heads * kD;
  if (overlaps(S, sb, q, la_extent(n_seqs, cfg->q_stride, kr, e)) ||
      overlaps(S, sb, k, la_extent(n_seqs, cfg->k_stride, kr, e)) ||
      overlaps(S, sb, v, la_extent(n_seqs, cfg->v_stride, vr, e)) ||
      overlaps(S, sb, o, la_extent(n_seqs, cfg->o_stride, vr, e)) ||
      overlaps(S, sb, alpha, la_extent(n_seqs, cfg->alpha_stride, cfg->heads, 4)))
    return fail(LQ_ERR_INVALID_ARG, "S overlaps a token input or o");
  int dev = 0;
  if ((rc = current_device(&dev)) || (rc = check_stream(stream, dev))) return rc;
  if ((rc = check_ptr(S, "S", 16, dev)) || (rc = check_la_device(cfg, dev, q, k, v, alpha, o))) return rc;
  lqi::LaParams p = la_params(cfg, q, k, v, alpha, o);
  p.n_seqs = n_seqs;
  p.n_tokens = n_seqs;
  p.S = S;
  return launched(lqi::launch_la_step(p, (cudaStream_t)stream), "lq_la_decode_step launch");
}

size_t lq_beam_workspace_bytes(int64_t batch, int32_t beams, int64_t vocab, int32_t n_best) {
  if (check_beams(batch, beams, vocab, n_best) || batch == 0) return 0;
  return lqi::beam_workspace(batch, beams, vocab, n_best);
}

int lq_beam_select(int32_t dtype, int64_t batch, int32_t beams, int64_t vocab, int32_t n_best, const void* logits,
                   int64_t row_stride, const float* scores, float* out_scores, int32_t* out_parent,
                   int32_t* out_token, void* workspace, size_t workspace_bytes, lq_stream_t stream) {
  if (dtype != LQ_F32 && dtype != LQ_BF16 && dtype != LQ_F16)
    return fail(LQ_ERR_INVALID_ARG, "dtype must be LQ_F32, LQ_BF16 or LQ_F16 (got %d)", dtype);
  int rc = check_beams(batch, beams, vocab, n_best);
  if (rc) return rc;
  if (batch == 0) return ok();
  if (row_stride < vocab || row_stride > ((int64_t)1 << 40))
    return fail(LQ_ERR_INVALID_ARG, "row_stride must be at least vocab (got %lld)", (long long)row_stride);
  const size_t e = la_size(dtype);
  if ((rc = check_addr(logits, "logits", e)) || (rc = check_addr(scores, "scores", 4)) ||
      (rc = check_addr(out_scores, "out_scores", 4)) || (rc = check_addr(out_parent, "out_parent", 4)) ||
      (rc = check_addr(out_token, "out_token", 4)) || (rc = check_addr(workspace, "workspace", 256)))
    return rc;
  const size_t need = lqi::beam_workspace(batch, beams, vocab, n_best);
  if (workspace_bytes < need)
    return fail(LQ_ERR_INVALID_ARG, "workspace has %zu bytes, %zu are needed", workspace_bytes, need);
  const size_t nl = la_extent(batch * beams, row_stride, vocab, e), ns = (size_t)batch * beams * 4,
               no = (size_t)batch * n_best * 4;
  const void* out[4] = {out_scores, out_parent, out_token, workspace};
  const size_t nout[4] = {no, no, no, need};
  for (int i = 0; i < 4; ++i) {
    if (overlaps(out[i], nout[i], logits, nl) || overlaps(out[i], nout[i], scores, ns))
      return fail(LQ_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], nout[i], out[j], nout[j]))
        return fail(LQ_ERR_INVALID_ARG, "the outputs and the workspace overlap");
  }
  int dev = 0;
  if ((rc = current_device(&dev)) || (rc = check_stream(stream, dev))) return rc;
  if ((rc = check_ptr(logits, "logits", e, dev)) || (rc = check_ptr(scores, "scores", 4, dev)) ||
      (rc = check_ptr(out_scores, "out_scores", 4, dev)) || (rc = check_ptr(out_parent, "out_parent", 4, dev)) ||
      (rc = check_ptr(out_token, "out_token", 4, dev)) || (rc = check_ptr(workspace, "workspace", 256, dev)))
    return rc;
  lqi::BeamParams p;
  std::memset(&p, 0, sizeof p);
  p.dtype = dtype;
  p.beams = beams;
  p.n_best = n_best;
  p.splits = lqi::beam_splits(dtype, vocab);
  p.batch = batch;
  p.vocab = vocab;
  p.row_stride = row_stride;
  p.logits = logits;
  p.scores = scores;
  p.out_scores = out_scores;
  p.out_parent = out_parent;
  p.out_token = out_token;
  p.ws = workspace;
  return launched(lqi::launch_beam_select(p, (cudaStream_t)stream), "lq_beam_select launch");
}

int lq_state_reorder(const lq_config* cfg, void* state, int64_t n_states, int64_t outer, int64_t groups,
                     int32_t beams, int64_t inner, const int32_t* parent, lq_stream_t stream) {
  int rc = check_cfg(cfg);
  if (rc || (rc = check_reorder(n_states, outer, groups, beams, inner))) return rc;
  if (n_states == 0) return ok();
  if ((rc = check_addr(state, "state", 256)) || (rc = check_addr(parent, "parent", 4))) return rc;
  if (overlaps(parent, (size_t)groups * beams * 4, state, state_size(cfg, n_states)))
    return fail(LQ_ERR_INVALID_ARG, "parent overlaps the state buffer");
  int dev = 0;
  if ((rc = check_common(cfg, state, n_states, stream, &dev)) || (rc = check_ptr(parent, "parent", 4, dev))) return rc;
  Params p = make_params(cfg, state, n_states);
  const lqi::ReorderParams r = {outer, groups, inner, beams, parent};
  return launched(lqi::launch_reorder(p, r, (cudaStream_t)stream), "lq_state_reorder launch");
}

int lq_fp32_state_reorder(float* S, int64_t n_states, int64_t outer, int64_t groups, int32_t beams, int64_t inner,
                          const int32_t* parent, lq_stream_t stream) {
  int rc = check_reorder(n_states, outer, groups, beams, inner);
  if (rc) return rc;
  if (n_states == 0) return ok();
  if ((rc = check_addr(S, "S", 16)) || (rc = check_addr(parent, "parent", 4))) return rc;
  if (overlaps(parent, (size_t)groups * beams * 4, S, (size_t)n_states * kD * kD * sizeof(float)))
    return fail(LQ_ERR_INVALID_ARG, "parent overlaps S");
  int dev = 0;
  if ((rc = current_device(&dev)) || (rc = check_stream(stream, dev))) return rc;
  if ((rc = check_ptr(S, "S", 16, dev)) || (rc = check_ptr(parent, "parent", 4, dev))) return rc;
  const lqi::ReorderParams r = {outer, groups, inner, beams, parent};
  return launched(lqi::launch_fp32_reorder(S, r, (cudaStream_t)stream), "lq_fp32_state_reorder launch");
}

void lq_conv_config_default(lq_conv_config* cfg, int32_t channels, int32_t width, int32_t dtype, int32_t silu) {
  if (!cfg) return;
  std::memset(cfg, 0, sizeof *cfg);
  cfg->channels = channels;
  cfg->width = width;
  cfg->dtype = dtype;
  cfg->silu = silu;
  cfg->x_stride = cfg->y_stride = channels;
}

int lq_conv_prefill(const lq_conv_config* cfg, int64_t n_seqs, int64_t n_tokens, int64_t max_len,
                    const int32_t* cu_seqlens, const void* x, const float* weight, const float* bias, const void* S0,
                    void* S_out, void* y, lq_stream_t stream) {
  int rc = check_conv(cfg);
  if (rc || (rc = check_packed(n_seqs, n_tokens, max_len, cu_seqlens))) return rc;
  if (n_seqs == 0) return ok();
  const size_t e = la_size(cfg->dtype), C = (size_t)cfg->channels;
  const size_t sb = (size_t)n_seqs * (cfg->width - 1) * C * e;
  const Arg a[7] = {{x, "x", la_extent(n_tokens, cfg->x_stride, cfg->channels, e), e, false, false},
                    {y, "y", la_extent(n_tokens, cfg->y_stride, cfg->channels, e), e, false, true},
                    {weight, "weight", C * cfg->width * 4, 4, false, false},
                    {bias, "bias", C * 4, 4, true, false},
                    {S0, "S0", sb, e, true, false},
                    {S_out, "S_out", sb, e, true, true},
                    {cu_seqlens, "cu_seqlens", cu_seqlens ? (size_t)(n_seqs + 1) * 4 : 0, 4, true, false}};
  if ((rc = check_args(a, 7, 4, 5))) return rc;
  lqi::ConvParams p;
  std::memset(&p, 0, sizeof p);
  p.channels = cfg->channels;
  p.width = cfg->width;
  p.dtype = cfg->dtype;
  p.silu = cfg->silu;
  p.sx = cfg->x_stride;
  p.sy = cfg->y_stride;
  p.n_seqs = n_seqs;
  p.n_tokens = n_tokens;
  p.max_len = max_len;
  p.cu = cu_seqlens;
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.S0 = S0;
  p.S = S_out;
  p.y = y;
  lqi::conv_plan(p);
  if ((rc = check_grid(p.slots, (cfg->channels + 127) / 128))) return rc;
  int dev = 0;
  if ((rc = current_device(&dev)) || (rc = check_stream(stream, dev)) || (rc = check_args_device(a, 7, dev))) return rc;
  return launched(lqi::launch_conv_prefill(p, (cudaStream_t)stream), "lq_conv_prefill launch");
}

int lq_conv_decode_step(const lq_conv_config* cfg, void* S, int64_t n_seqs, const void* x, const float* weight,
                        const float* bias, void* y, lq_stream_t stream) {
  int rc = check_conv(cfg);
  if (rc) return rc;
  if (n_seqs < 0) return fail(LQ_ERR_INVALID_ARG, "n_seqs must not be negative");
  if ((rc = check_grid(n_seqs, (cfg->channels + 127) / 128))) return rc;
  if (n_seqs == 0) return ok();
  const size_t e = la_size(cfg->dtype), C = (size_t)cfg->channels;
  const Arg a[5] = {{x, "x", la_extent(n_seqs, cfg->x_stride, cfg->channels, e), e, false, false},
                    {y, "y", la_extent(n_seqs, cfg->y_stride, cfg->channels, e), e, false, true},
                    {weight, "weight", C * cfg->width * 4, 4, false, false},
                    {bias, "bias", C * 4, 4, true, false},
                    {S, "S", (size_t)n_seqs * (cfg->width - 1) * C * e, e, false, true}};
  if ((rc = check_args(a, 5))) return rc;
  int dev = 0;
  if ((rc = current_device(&dev)) || (rc = check_stream(stream, dev)) || (rc = check_args_device(a, 5, dev))) return rc;
  lqi::ConvParams p;
  std::memset(&p, 0, sizeof p);
  p.channels = cfg->channels;
  p.width = cfg->width;
  p.dtype = cfg->dtype;
  p.silu = cfg->silu;
  p.sx = cfg->x_stride;
  p.sy = cfg->y_stride;
  p.n_seqs = p.n_tokens = n_seqs;
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.S = S;
  p.y = y;
  return launched(lqi::launch_conv_step(p, (cudaStream_t)stream), "lq_conv_decode_step launch");
}

void lq_ssm_config_default(lq_ssm_config* cfg, int32_t channels, int32_t n_state, int32_t groups, int32_t dtype,
                           int32_t softplus) {
  if (!cfg) return;
  std::memset(cfg, 0, sizeof *cfg);
  cfg->channels = channels;
  cfg->n_state = n_state;
  cfg->groups = groups;
  cfg->dtype = dtype;
  cfg->softplus = softplus;
  cfg->x_stride = cfg->dt_stride = cfg->z_stride = cfg->y_stride = channels;
  cfg->b_stride = cfg->c_stride = (int64_t)groups * n_state;
}

size_t lq_ssm_workspace_bytes(const lq_ssm_config* cfg, int64_t n_seqs, int64_t n_tokens, int64_t max_len) {
  const int32_t some = 0;
  if (check_ssm(cfg) || check_packed(n_seqs, n_tokens, max_len, &some) || n_seqs == 0) return 0;
  const int64_t slots = lqi::ssm_most_slots(cfg, n_seqs, n_tokens, max_len);
  return slots ? ssm_workspace(cfg, slots) : 0;
}

int lq_ssm_prefill(const lq_ssm_config* cfg, int64_t n_seqs, int64_t n_tokens, int64_t max_len,
                   const int32_t* cu_seqlens, const void* x, const void* dt, const float* A, const void* B,
                   const void* C, const float* D, const void* z, const float* dt_bias, const float* S0, float* S_out,
                   void* y, void* workspace, size_t workspace_bytes, lq_stream_t stream) {
  int rc = check_ssm(cfg);
  if (rc || (rc = check_packed(n_seqs, n_tokens, max_len, cu_seqlens))) return rc;
  if (n_seqs == 0) return ok();
  lqi::SsmParams p = ssm_params(cfg, x, dt, A, B, C, D, z, dt_bias, y);
  lqi::SsmPlan plan;
  lqi::ssm_plan(cfg, n_seqs, n_tokens, max_len, &plan);
  p.spt = plan.spt;
  p.lpc = plan.lpc;
  p.seg = plan.seg;
  p.slots = plan.slots;
  const size_t need = p.seg ? ssm_workspace(cfg, p.slots) : 0;
  const size_t e = la_size(cfg->dtype), ch = (size_t)cfg->channels, N = (size_t)cfg->n_state;
  const int64_t row = cfg->channels, bc = (int64_t)cfg->groups * cfg->n_state;
  const size_t sb = (size_t)n_seqs * ch * N * 4;
  const Arg a[13] = {{x, "x", la_extent(n_tokens, cfg->x_stride, row, e), e, false, false},
                     {dt, "dt", la_extent(n_tokens, cfg->dt_stride, row, e), e, false, false},
                     {z, "z", la_extent(n_tokens, cfg->z_stride, row, e), e, true, false},
                     {B, "B", la_extent(n_tokens, cfg->b_stride, bc, e), e, false, false},
                     {C, "C", la_extent(n_tokens, cfg->c_stride, bc, e), e, false, false},
                     {y, "y", la_extent(n_tokens, cfg->y_stride, row, e), e, false, true},
                     {A, "A", ch * N * 4, 4, false, false},
                     {D, "D", ch * 4, 4, true, false},
                     {dt_bias, "dt_bias", ch * 4, 4, true, false},
                     {S0, "S0", sb, 4, true, false},
                     {S_out, "S_out", sb, 4, true, true},
                     {cu_seqlens, "cu_seqlens", cu_seqlens ? (size_t)(n_seqs + 1) * 4 : 0, 4, true, false},
                     {need ? workspace : nullptr, "workspace", need, 256, false, true}};
  if ((rc = check_args(a, 13, 9, 10))) return rc;
  if (need && workspace_bytes < need)
    return fail(LQ_ERR_INVALID_ARG, "workspace has %zu bytes, %zu are needed", workspace_bytes, need);
  if ((rc = check_grid(p.slots, plan.blocks)) ||
      (p.seg && (rc = check_grid(n_seqs, (int64_t)(ch * N + 255) / 256))))
    return rc;
  int dev = 0;
  if ((rc = current_device(&dev)) || (rc = check_stream(stream, dev)) || (rc = check_args_device(a, 13, dev)))
    return rc;
  p.n_seqs = n_seqs;
  p.n_tokens = n_tokens;
  p.max_len = max_len;
  p.cu = cu_seqlens;
  p.S0 = S0;
  p.S = S_out;
  p.ws_state = static_cast<float*>(workspace);
  p.ws_step = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256((size_t)p.slots * ch * N * 4));
  return launched(lqi::launch_ssm_prefill(p, (cudaStream_t)stream), "lq_ssm_prefill launch");
}

int lq_ssm_decode_step(const lq_ssm_config* cfg, float* S, int64_t n_seqs, const void* x, const void* dt,
                       const float* A, const void* B, const void* C, const float* D, const void* z,
                       const float* dt_bias, void* y, lq_stream_t stream) {
  int rc = check_ssm(cfg);
  if (rc) return rc;
  if (n_seqs < 0) return fail(LQ_ERR_INVALID_ARG, "n_seqs must not be negative");
  if ((rc = check_grid(n_seqs, (int64_t)cfg->channels))) return rc;
  if (n_seqs == 0) return ok();
  const size_t e = la_size(cfg->dtype), ch = (size_t)cfg->channels, N = (size_t)cfg->n_state;
  const int64_t row = cfg->channels, bc = (int64_t)cfg->groups * cfg->n_state;
  const Arg a[10] = {{x, "x", la_extent(n_seqs, cfg->x_stride, row, e), e, false, false},
                     {dt, "dt", la_extent(n_seqs, cfg->dt_stride, row, e), e, false, false},
                     {z, "z", la_extent(n_seqs, cfg->z_stride, row, e), e, true, false},
                     {B, "B", la_extent(n_seqs, cfg->b_stride, bc, e), e, false, false},
                     {C, "C", la_extent(n_seqs, cfg->c_stride, bc, e), e, false, false},
                     {y, "y", la_extent(n_seqs, cfg->y_stride, row, e), e, false, true},
                     {A, "A", ch * N * 4, 4, false, false},
                     {D, "D", ch * 4, 4, true, false},
                     {dt_bias, "dt_bias", ch * 4, 4, true, false},
                     {S, "S", (size_t)n_seqs * ch * N * 4, 4, false, true}};
  if ((rc = check_args(a, 10))) return rc;
  int dev = 0;
  if ((rc = current_device(&dev)) || (rc = check_stream(stream, dev)) || (rc = check_args_device(a, 10, dev)))
    return rc;
  lqi::SsmParams p = ssm_params(cfg, x, dt, A, B, C, D, z, dt_bias, y);
  p.n_seqs = p.n_tokens = n_seqs;
  p.S = S;
  return launched(lqi::launch_ssm_step(p, (cudaStream_t)stream), "lq_ssm_decode_step launch");
}

int lq_token_logprobs(int32_t dtype, int64_t rows, int64_t vocab, int32_t n_top, const void* logits,
                      int64_t row_stride, const int32_t* tokens, float* logprob, float* entropy, float* top_logprob,
                      int32_t* top_token, lq_stream_t stream) {
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (rows < 0 || rows > kMaxStates / 8)
    return fail(LQ_ERR_INVALID_ARG, "rows must be 0..%lld (got %lld)", (long long)(kMaxStates / 8), (long long)rows);
  if (vocab < 1 || vocab > 0x7fffffff)
    return fail(LQ_ERR_INVALID_ARG, "vocab must be 1..%d (got %lld)", 0x7fffffff, (long long)vocab);
  if (n_top < 0 || n_top > lqi::kMaxTop || n_top > vocab)
    return fail(LQ_ERR_INVALID_ARG, "n_top must be 0..%d and at most vocab (got %d)", lqi::kMaxTop, n_top);
  if (row_stride < vocab || row_stride > ((int64_t)1 << 40))
    return fail(LQ_ERR_INVALID_ARG, "row_stride must be at least vocab (got %lld)", (long long)row_stride);
  if ((tokens == nullptr) != (logprob == nullptr))
    return fail(LQ_ERR_INVALID_ARG, "tokens and logprob go together: one of them is NULL");
  if (n_top == 0 && (top_logprob || top_token))
    return fail(LQ_ERR_INVALID_ARG, "top_logprob and top_token must be NULL where n_top is 0");
  if (rows == 0) return ok();
  if (!logprob && !entropy && !n_top) return fail(LQ_ERR_INVALID_ARG, "no output is asked for");
  const size_t e = la_size(dtype), r4 = (size_t)rows * 4;
  const Arg a[6] = {{logits, "logits", la_extent(rows, row_stride, vocab, e), e, false, false},
                    {tokens, "tokens", r4, 4, true, false},
                    {logprob, "logprob", r4, 4, true, true},
                    {entropy, "entropy", r4, 4, true, true},
                    {top_logprob, "top_logprob", r4 * n_top, 4, false, true},
                    {top_token, "top_token", r4 * n_top, 4, false, true}};
  if ((rc = check_args(a, 6))) return rc;
  int dev = 0;
  if ((rc = current_device(&dev)) || (rc = check_stream(stream, dev)) || (rc = check_args_device(a, 6, dev))) return rc;
  lqi::LogprobParams p;
  std::memset(&p, 0, sizeof p);
  p.dtype = dtype;
  p.n_top = n_top;
  p.rows = rows;
  p.vocab = vocab;
  p.row_stride = row_stride;
  p.logits = logits;
  p.tokens = tokens;
  p.logprob = logprob;
  p.entropy = entropy;
  p.top_logprob = top_logprob;
  p.top_token = top_token;
  return launched(lqi::launch_token_logprobs(p, (cudaStream_t)stream), "lq_token_logprobs launch");
}

int lq_get_status(const void* state, int64_t* bad_state, lq_stream_t stream) {
  int dev = 0;
  int rc = current_device(&dev);
  if (rc) return rc;
  if ((rc = check_stream(stream, dev))) return rc;
  if ((rc = check_ptr(state, "state", 256, dev))) return rc;
  Header h;
  cudaError_t e = cudaMemcpyAsync(&h, state, sizeof h, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "reading the status word");
  e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  if (bad_state) *bad_state = h.bad_state;
  if (h.magic != lqi::kMagic) return fail(LQ_ERR_STATE, "state buffer is not initialised");
  ok();
  return h.status;
}

int lq_clear_status(void* state, lq_stream_t stream) {
  int dev = 0;
  int rc = current_device(&dev);
  if (rc) return rc;
  if ((rc = check_stream(stream, dev))) return rc;
  if ((rc = check_ptr(state, "state", 256, dev))) return rc;
  char* base = static_cast<char*>(state);
  cudaError_t e = cudaMemsetAsync(base + offsetof(Header, status), 0, sizeof(int32_t), (cudaStream_t)stream);
  if (e == cudaSuccess)
    e = cudaMemsetAsync(base + offsetof(Header, bad_state), 0xff, sizeof(int64_t), (cudaStream_t)stream);
  return e == cudaSuccess ? ok() : cuda_fail(e, "lq_clear_status");
}

}  // extern "C"
