#include "rn_logprob.cuh"

namespace rn {
cudaError_t logprob_fwd_bf16(const LogprobParams& p, cudaStream_t s) {
    return logprob_fwd_t<__nv_bfloat16>(p, s);
}
}  // namespace rn
