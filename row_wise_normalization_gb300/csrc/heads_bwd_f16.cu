// heads_bwd_f16.cu -- the gradient of norms of queries and keys with the position rotation, f16 rows.
#include "rn_heads.cuh"

namespace rn {
cudaError_t heads_bwd_f16(HeadShape sh, const HeadsParams& p, int ctas, void* dwq,
                          void* dwk, cudaStream_t s) {
    return heads_bwd_t<__half>(sh, p, ctas, dwq, dwk, s);
}
}  // namespace rn
