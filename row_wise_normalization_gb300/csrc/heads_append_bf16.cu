// heads_append_bf16.cu -- the same into a paged cache of bf16 rows.
#include "rn_heads.cuh"

namespace rn {
cudaError_t heads_append_bf16(HeadShape sh, const HeadsParams& p, cudaStream_t s) {
    return heads_fwd_t<__nv_bfloat16, true, false>(sh, p, s);
}
}  // namespace rn
