// heads_append8_f32.cu -- the same from f32 rows into an 8-bit paged cache.
#include "rn_heads.cuh"

namespace rn {
cudaError_t heads_append8_f32(HeadShape sh, const HeadsParams& p, cudaStream_t s) {
    return heads_fwd_t<float, true, true>(sh, p, s);
}
}  // namespace rn
