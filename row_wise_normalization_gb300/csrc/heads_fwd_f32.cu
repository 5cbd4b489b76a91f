// heads_fwd_f32.cu -- norms of queries and keys with the position rotation, f32 rows.
#include "rn_heads.cuh"

namespace rn {
cudaError_t heads_fwd_f32(HeadShape sh, const HeadsParams& p, cudaStream_t s) {
    return heads_fwd_t<float, false, false>(sh, p, s);
}
}  // namespace rn
