// heads_append8_bf16.cu -- the same from bf16 rows into an 8-bit paged cache.
#include "rn_heads.cuh"

namespace rn {
cudaError_t heads_append8_bf16(HeadShape sh, const HeadsParams& p, cudaStream_t s) {
    return heads_fwd_t<__nv_bfloat16, true, true>(sh, p, s);
}
}  // namespace rn
