// The scan's kernels for f32 tokens (a file for each type, to compile side by side).
#include "lq_ssm.cuh"

namespace lqi {

cudaError_t launch_ssm_prefill_f32(const SsmParams& p, cudaStream_t st) { return launch<float>(p, st); }

}  // namespace lqi
