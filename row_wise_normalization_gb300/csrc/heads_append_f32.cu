// heads_append_f32.cu -- the same into a paged cache of f32 rows.
#include "rn_heads.cuh"

namespace rn {
cudaError_t heads_append_f32(HeadShape sh, const HeadsParams& p, cudaStream_t s) {
    return heads_fwd_t<float, true, false>(sh, p, s);
}
}  // namespace rn
