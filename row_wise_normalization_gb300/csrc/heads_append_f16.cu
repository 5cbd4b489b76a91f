// heads_append_f16.cu -- the same into a paged cache of f16 rows.
#include "rn_heads.cuh"

namespace rn {
cudaError_t heads_append_f16(HeadShape sh, const HeadsParams& p, cudaStream_t s) {
    return heads_fwd_t<__half, true, false>(sh, p, s);
}
}  // namespace rn
