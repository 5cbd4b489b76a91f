// embed_fwd.cu -- embedding rows: out[i] = scale * table[tokens[i]].
//
// Nothing is computed but one product an element, so the bytes bound it: each
// different table row read once (repeats come from L2), every output row
// written. The work is the flat list of 16-byte vectors of the output (narrower
// ones where the rows' alignment asks for it), kEmbedU of them a thread, so
// that a few long rows and many short ones fill the GPU alike. The
// loads of a thread's ids come first, then its row loads together, then its
// stores: two waits for memory whatever the width.
#include "rn_tokens.cuh"

namespace rn {

constexpr int kEmbedThreads = 256;
constexpr int kEmbedU = 4;

template <typename T, int NE>
__global__ void __launch_bounds__(kEmbedThreads) embed_fwd_kernel(const EmbedParams p, int itype) {
    pdl_launch_dependents();
    const int64_t base = (int64_t)blockIdx.x * (kEmbedThreads * kEmbedU);
    // the CTA's first vector: one 64-bit division; from there 32 bits suffice
    const int64_t row0 = base / p.vpr.d;
    const uint32_t col0 = (uint32_t)(base - row0 * p.vpr.d);
    int64_t row[kEmbedU], id[kEmbedU];
    uint32_t col[kEmbedU];
    pdl_wait();
#pragma unroll
    for (int u = 0; u < kEmbedU; ++u) {
        const uint32_t k = u * kEmbedThreads + threadIdx.x;
        const uint32_t q = fast_quot(col0 + k, p.vpr);
        row[u] = row0 + q;
        col[u] = col0 + k - q * p.vpr.d;
        id[u] = base + k < p.total ? ld_id(p.tokens, row[u], itype) : -1;
    }
    Raw<NE * (int)sizeof(T)> r[kEmbedU];
#pragma unroll
    for (int u = 0; u < kEmbedU; ++u) {
        if (id[u] >= 0 && id[u] < p.vocab) {
            r[u] = ld_raw<NE * (int)sizeof(T)>((const T*)p.table + id[u] * p.ldt +
                                               (int64_t)col[u] * NE);
        } else {
#pragma unroll
            for (int k = 0; k < (int)(sizeof(r[u].w) / 4); ++k) r[u].w[k] = 0;
        }
    }
#pragma unroll
    for (int u = 0; u < kEmbedU; ++u) {
        if (base + u * kEmbedThreads + threadIdx.x < p.total) {
            float v[NE];
            unpack<T, NE>(v, r[u]);
            const bool there = id[u] >= 0 && id[u] < p.vocab;
            // (an absent id gives +0 whatever the sign of the scale)
#pragma unroll
            for (int k = 0; k < NE; ++k) v[k] = there ? v[k] * p.scale : 0.f;
            st_elems<T, NE>((T*)p.out + row[u] * p.ldo + (int64_t)col[u] * NE, v);
        }
    }
}

template <typename T, int NE>
static cudaError_t embed_fwd_go(int itype, const EmbedParams& p, cudaStream_t s) {
    const int64_t per = kEmbedThreads * kEmbedU;
    return launch_pdl(embed_fwd_kernel<T, NE>, (unsigned)((p.total + per - 1) / per),
                      kEmbedThreads, 0, s, p, itype);
}

cudaError_t embed_fwd_launch(int dtype, int itype, int ne, const EmbedParams& p, cudaStream_t s) {
    if (dtype == DT_F32) {
        if (ne == 4) return embed_fwd_go<float, 4>(itype, p, s);
        if (ne == 2) return embed_fwd_go<float, 2>(itype, p, s);
        return embed_fwd_go<float, 1>(itype, p, s);
    }
#define RN_GO(T)                                                \
    {                                                           \
        if (ne == 8) return embed_fwd_go<T, 8>(itype, p, s);    \
        if (ne == 4) return embed_fwd_go<T, 4>(itype, p, s);    \
        if (ne == 2) return embed_fwd_go<T, 2>(itype, p, s);    \
        return embed_fwd_go<T, 1>(itype, p, s);                 \
    }
    if (dtype == DT_BF16) RN_GO(__nv_bfloat16)
    RN_GO(__half)
#undef RN_GO
}

}  // namespace rn
