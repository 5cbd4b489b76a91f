#include "rn_logprob.cuh"

namespace rn {
cudaError_t logprob_fwd_f32(const LogprobParams& p, cudaStream_t s) {
    return logprob_fwd_t<float>(p, s);
}
}  // namespace rn
