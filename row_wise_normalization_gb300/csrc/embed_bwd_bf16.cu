#include "embed_bwd.cuh"

namespace rn {
cudaError_t embed_bwd_bf16(int gtype, int ne, bool few, const SortParams& z, int sms,
                           const EmbedBwdParams& p, cudaStream_t s) {
    if (gtype != DT_F32) return embed_bwd_t<__nv_bfloat16, __nv_bfloat16>(ne, few, z, sms, p, s);
    return embed_bwd_t<__nv_bfloat16, float>(ne, few, z, sms, p, s);
}
}  // namespace rn
