// heads_fwd_bf16.cu -- norms of queries and keys with the position rotation, bf16 rows.
#include "rn_heads.cuh"

namespace rn {
cudaError_t heads_fwd_bf16(HeadShape sh, const HeadsParams& p, cudaStream_t s) {
    return heads_fwd_t<__nv_bfloat16, false, false>(sh, p, s);
}
}  // namespace rn
