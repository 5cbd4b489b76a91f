#include "rn_logprob.cuh"

namespace rn {
cudaError_t logprob_fwd_f16(const LogprobParams& p, cudaStream_t s) {
    return logprob_fwd_t<__half>(p, s);
}
}  // namespace rn
