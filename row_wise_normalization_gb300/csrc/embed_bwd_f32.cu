#include "embed_bwd.cuh"

namespace rn {
cudaError_t embed_bwd_f32(int gtype, int ne, bool few, const SortParams& z, int sms,
                          const EmbedBwdParams& p, cudaStream_t s) {
    (void)gtype;
    return embed_bwd_t<float, float>(ne, few, z, sms, p, s);
}
}  // namespace rn
