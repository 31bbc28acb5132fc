// Internal declarations shared by the host API (lq_api.cu) and the kernels (lq_kernels.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lq.h"

namespace lqi {

constexpr uint32_t kMagic = 0x4C513847u;  // "GQ8L"
constexpr uint32_t kLayoutVersion = 2;
constexpr int kD = 128;       // d_k = d_v
constexpr int kMaxW = 32;     // records per window
constexpr int kMaxC = 8;      // compensators per head-state
constexpr int kThreads = 256; // threads per CTA; one CTA per head-state
// lq_decode_step_noalloc: head-states its fixed work list holds, and the int32
// offset of the list in the array (the two counters sit before it).
constexpr int kNoAllocMaxStates = 65536;
constexpr int kNoAllocListOffset = 64;

// Device-resident header at offset 0 of every state buffer (256 bytes).
struct Header {
  uint32_t magic;
  uint32_t version;
  uint64_t cfg_hash;
  int64_t n_states;
  int32_t status;     // first device-side error (lq_status), 0 when clean
  int32_t reserved0;
  int64_t bad_state;  // head-state index that set `status`
  int32_t full_n;     // entries on the full-window list (mixed-phase decode step)
  int32_t fold_done;  // CTAs of the list fold that have finished
  uint8_t pad[256 - 48];
};
static_assert(sizeof(Header) == 256, "header is 256 bytes");

// Byte offsets of one head-state's working set in dynamic shared memory
// (computed on the host for the kernel being launched).
struct Stage {
  // staged by bulk copies, dense
  int codes, sigma, lambda, comp_id, comp_line, rec_k, rec_u, rec_alpha;
  // computed, blocked layout
  int kn_b, qn_b, zk_b, zq_b, lam_b, kd_b, bd_b, P_b;
  // computed, dense
  int basek, baseq, P, g, h, ec, eq;
  // two-record tokens: the second record's key, read vector and sums
  int k2n_b, zk2_b, basek2, g2, ec2;
  // RWKV7 tokens: the erase key and the decay products of the held records
  int en_b, Pp_b;
  // append-only step: the smoothed read vectors as duplicated pairs
  int zdk, zdq;
  int end;
};

// Everything a kernel needs, passed by value.
struct Params {
  int W, C, kda, smooth;
  int bits;      // code width: 8 or 4
  int comp_fit;  // 0: outlier-line compensators; s > 0: factors fitted by s sweeps
  int comp_block;  // fitted factors: 1 = block fit from the previous window's factors
  float lambda_floor;
  int phase;  // expected record count before the call, or -1
  int push_full;  // append: list the head-states whose window this token fills
  int64_t n_states;
  int64_t first;  // range init: first head-state of the range
  uint64_t cfg_hash;
  int64_t comp_id_stride, alpha_stride;
  Header* hdr;
  int32_t* counts;
  int32_t* full_list;
  int32_t* list_ctr;  // lq_decode_step_noalloc: [0] entries on the list, [1] list-fold CTAs done
  uint64_t wait_ns;   // bound on a wait for staged copies (1 s; shorter only under lq_debug_set_wait)
  int32_t dbg_tx_append, dbg_tx_fold;  // test hook: bytes announced beyond those copied (0 normally)
  int8_t* codes;
  float* sigma;
  float* lambda;
  int32_t* comp_id;
  float* comp_line;
  float* rec_k;
  float* rec_u;
  float* rec_alpha;
  const float* q;
  const float* k;
  const float* v;
  const float* alpha;
  const float* beta;
  const float* k2;  // two-record tokens: the second record's key, value and step
  const float* v2;
  const float* beta2;
  const float* kh;  // RWKV7 tokens: the erase direction and its per-key rate
  const float* ka;
  float* o;
  const float* S0;  // init source (NULL: zero)
  float* S_out;     // export target
  Stage st;         // shared-memory layout of the launched kernel
  int r1;           // bytes of the staging / state-tile region
};

// The fp32-state baseline decode step (lq_fp32_decode_step).
struct Fp32Params {
  int64_t n_states;
  int kda;
  float* S;  // [n][d_v][d_k], updated in place
  const float* q;
  const float* k;
  const float* v;
  const float* alpha;
  const float* beta;
  float* o;
};

// Linear attention with a decay per head (lq_la_prefill, lq_la_decode_step).
constexpr int kMaxBeams = 32;
constexpr int kMaxBest = 64;

struct LaParams {
  int heads, key_heads, group;  // group: heads per key head
  int dtype;
  int64_t sq, sk, sv, so, sa;  // elements between tokens
  int64_t n_seqs, n_tokens, max_len;
  int64_t seg;        // tokens per segment of a split sequence; 0: sequences are not split
  int64_t slots;      // upper bound of the segments of all sequences
  const int32_t* cu;  // NULL: one sequence of n_tokens
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* S0;
  float* S;  // prefill: final states (may be NULL); decode step: states, in place
  void* o;
  float* ws_state;  // [slots][heads][128][128]: what a segment adds to the state
  float2* ws_decay; // [slots][heads]: the product of a segment's decays, in two parts
  float* ws_last;   // [n_seqs][heads][128][128]: last states on their way into S where that is S0
  uint64_t wait_ns;  // half the bound on a wait of the chunked form
  uint32_t dbg_tx;   // test hook: bytes announced beyond those copied (0 normally)
};

// Short causal convolution (lq_conv_prefill, lq_conv_decode_step).
struct ConvParams {
  int channels, width, dtype, silu;
  int64_t sx, sy;  // elements between tokens
  int64_t n_seqs, n_tokens, max_len;
  int64_t seg;     // tokens per tile
  int64_t slots;   // upper bound of the tiles of all sequences
  const int32_t* cu;  // NULL: one sequence of n_tokens
  const void* x;
  const float* weight;  // [channels][width]
  const float* bias;    // may be NULL
  const void* S0;       // may be NULL (zero)
  void* S;              // prefill: last inputs (may be NULL); decode step: in place
  void* y;
};

// Selective state space scan (lq_ssm_prefill, lq_ssm_decode_step).
struct SsmPlan {
  int spt, lpc;    // states a thread, lanes a channel
  int64_t seg;     // tokens per segment of a split sequence; 0: sequences are not split
  int64_t slots;   // upper bound of the segments of all sequences
  int64_t blocks;  // CTAs of a segment
};

struct SsmParams {
  int channels, n_state, groups, per_group;  // per_group: channels of a group
  int dtype, softplus;
  int spt, lpc;  // states a thread, lanes a channel
  int64_t sx, sdt, sz, sb, sc, sy;  // elements between tokens
  int64_t n_seqs, n_tokens, max_len;
  int64_t seg;    // tokens per segment of a split sequence; 0: sequences are not split
  int64_t slots;  // upper bound of the segments of all sequences
  const int32_t* cu;  // NULL: one sequence of n_tokens
  const void* x;
  const void* dt;
  const void* z;  // may be NULL
  const void* B;
  const void* C;
  const float* A;        // [channels][n_state]
  const float* D;        // may be NULL
  const float* dt_bias;  // may be NULL
  const float* S0;       // may be NULL (zero)
  float* S;              // prefill: last states (may be NULL); decode step: in place
  void* y;
  float* ws_state;  // [slots][channels][n_state]
  float* ws_step;   // [slots][channels]
};

constexpr int kMaxWidth = 4;    // taps of a convolution
constexpr int kMaxNState = 64;  // states of a channel
constexpr int kMaxTop = 32;     // alternatives of a row

// Log probabilities of given tokens (lq_token_logprobs).
struct LogprobParams {
  int dtype, n_top;
  int64_t rows, vocab, row_stride;
  const void* logits;
  const int32_t* tokens;  // may be NULL
  float* logprob;         // NULL with tokens
  float* entropy;         // may be NULL
  float* top_logprob;     // [rows][n_top]
  int32_t* top_token;
};

struct BeamParams {
  int dtype, beams, n_best, splits;
  int64_t batch, vocab, row_stride;
  const void* logits;
  const float* scores;
  float* out_scores;
  int32_t* out_parent;
  int32_t* out_token;
  void* ws;
};

struct ReorderParams {
  int64_t outer, groups, inner;
  int beams;
  const int32_t* parent;
};

// Tokens per segment (0: whole sequences) and the segments there can be, by size.
void la_plan(const lq_la_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len, int64_t* seg, int64_t* slots);
// No call of these sizes or smaller ones has more segments.
int64_t la_most_slots(const lq_la_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len);
size_t beam_workspace(int64_t batch, int beams, int64_t vocab, int n_best);
int beam_splits(int dtype, int64_t vocab);

// How a scan of these sizes runs; and the most segments of any call of these sizes or smaller ones (0: none is split).
void ssm_plan(const lq_ssm_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len, SsmPlan* plan);
int64_t ssm_most_slots(const lq_ssm_config* c, int64_t n_seqs, int64_t n_tokens, int64_t max_len);

void conv_plan(ConvParams& p);  // seg and slots, by size

cudaError_t launch_conv_prefill(const ConvParams& p, cudaStream_t st);
cudaError_t launch_conv_step(const ConvParams& p, cudaStream_t st);
cudaError_t launch_ssm_prefill(const SsmParams& p, cudaStream_t st);
cudaError_t launch_ssm_step(const SsmParams& p, cudaStream_t st);
cudaError_t launch_token_logprobs(const LogprobParams& p, cudaStream_t st);
cudaError_t launch_la_prefill(const LaParams& p, cudaStream_t st);
cudaError_t launch_la_step(const LaParams& p, cudaStream_t st);
cudaError_t launch_beam_select(const BeamParams& p, cudaStream_t st);
cudaError_t launch_reorder(const Params& p, const ReorderParams& r, cudaStream_t st);
cudaError_t launch_fp32_reorder(float* S, const ReorderParams& r, cudaStream_t st);
cudaError_t launch_init(const Params& p, cudaStream_t st);
cudaError_t launch_append(const Params& p, cudaStream_t st);
cudaError_t launch_append_slist(const Params& p, cudaStream_t st);
cudaError_t launch_append2(const Params& p, cudaStream_t st);
cudaError_t launch_append_rwkv(const Params& p, cudaStream_t st);
cudaError_t launch_step(const Params& p, cudaStream_t st);
cudaError_t launch_fold(const Params& p, cudaStream_t st);
cudaError_t launch_init_range(const Params& p, int64_t count, cudaStream_t st);
cudaError_t launch_fold_listed(const Params& p, cudaStream_t st);
cudaError_t launch_decode_noalloc(const Params& p, int dev, cudaStream_t st);
cudaError_t launch_export(const Params& p, cudaStream_t st);
cudaError_t launch_fp32_step(const Fp32Params& p, cudaStream_t st);

}  // namespace lqi
