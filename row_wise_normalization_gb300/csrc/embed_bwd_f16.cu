#include "embed_bwd.cuh"

namespace rn {
cudaError_t embed_bwd_f16(int gtype, int ne, bool few, const SortParams& z, int sms,
                          const EmbedBwdParams& p, cudaStream_t s) {
    if (gtype != DT_F32) return embed_bwd_t<__half, __half>(ne, few, z, sms, p, s);
    return embed_bwd_t<__half, float>(ne, few, z, sms, p, s);
}
}  // namespace rn
