// heads_fwd_f16.cu -- norms of queries and keys with the position rotation, f16 rows.
#include "rn_heads.cuh"

namespace rn {
cudaError_t heads_fwd_f16(HeadShape sh, const HeadsParams& p, cudaStream_t s) {
    return heads_fwd_t<__half, false, false>(sh, p, s);
}
}  // namespace rn
