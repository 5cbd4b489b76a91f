// heads_append8_f16.cu -- the same from f16 rows into an 8-bit paged cache.
#include "rn_heads.cuh"

namespace rn {
cudaError_t heads_append8_f16(HeadShape sh, const HeadsParams& p, cudaStream_t s) {
    return heads_fwd_t<__half, true, true>(sh, p, s);
}
}  // namespace rn
