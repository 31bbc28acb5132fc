// The scan's kernels for bf16 tokens (a file for each type, to compile side by side).
#include "lq_ssm.cuh"

namespace lqi {

cudaError_t launch_ssm_prefill_bf16(const SsmParams& p, cudaStream_t st) { return launch<__nv_bfloat16>(p, st); }

}  // namespace lqi
