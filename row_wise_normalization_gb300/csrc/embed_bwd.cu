// embed_bwd.cu -- gradient of embedding rows from the sorted ids:
//   dtable[v] = (accumulate ? dtable[v] : 0) + scale * sum_{i: id_i = v} dout[i].
//
// Bytes bound it: dout read once, every row of the gradient written once (most
// ids of a vocabulary are absent from a batch, so most of the time goes into
// rows of zeros). The sorted positions are cut into chunks of kEmbedChunk. A
// group of threads takes one chunk and a slice of the columns, adds the chunk's
// rows in registers (FP32) and, where the id changes, writes the id's row. An
// id whose positions run over a chunk's edge leaves its sum of each chunk in
// the workspace, and a second kernel adds those in chunk order, so that an id
// which fills half of a batch is summed by as many groups as its rows fill.
// CTAs beside them clear the rows of the ids that the sort did not mark
// present. Every sum has a fixed order: results repeat bit for bit.
#include "rn_tokens.cuh"

namespace rn {

constexpr int kSegThreads = 256;
constexpr int kZeroRowsPerCta = 64;

template <typename T, typename G, int NE>
__global__ void __launch_bounds__(kSegThreads) embed_bwd_kernel(const EmbedBwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    G* const DG = (G*)p.dtable;
    if ((int)blockIdx.x >= p.seg_ctas) {
        // rows of absent ids: a warp for each row
        const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
        float z[NE];
#pragma unroll
        for (int k = 0; k < NE; ++k) z[k] = 0.f;
        const int64_t r0 = (int64_t)((int)blockIdx.x - p.seg_ctas) * kZeroRowsPerCta;
        for (int k = w; k < kZeroRowsPerCta; k += kSegThreads / 32) {
            const int64_t v = r0 + k;
            if (v >= p.vocab) return;
            if ((ld_u32(p.present + (v >> 5)) >> (v & 31)) & 1u) continue;
            G* row = DG + v * p.ldg;
            for (int64_t j = (int64_t)lane * NE; j < p.d; j += 32 * NE) st_elems<G, NE>(row + j, z);
        }
        return;
    }
    const int tx = (int)threadIdx.x % p.tx, ty = (int)threadIdx.x / p.tx;
    const int slice = (int)blockIdx.x % p.slices;
    const int64_t c = (int64_t)((int)blockIdx.x / p.slices) * p.ty + ty;
    const int64_t j = ((int64_t)slice * p.tx + tx) * NE;
    if (c >= p.chunks || j >= p.d) return;
    const T* const X = (const T*)p.dout + j;
    const int64_t i0 = c * kEmbedChunk;
    const int64_t i1 = i0 + kEmbedChunk < p.n ? i0 + kEmbedChunk : p.n;
    uint32_t cur = ld_u32(p.key + i0);
    bool open = i0 > 0 && ld_u32(p.key + i0 - 1) == cur;   // cur began in an earlier chunk
    const bool on = i1 < p.n && ld_u32(p.key + i1) == ld_u32(p.key + i1 - 1);
    float acc[NE];
#pragma unroll
    for (int k = 0; k < NE; ++k) acc[k] = 0.f;
    auto put = [&](bool last) {
        if (cur >= (uint32_t)p.vocab) return;   // ids outside the vocabulary
        if (open || (last && on)) {
            float* w = p.part + (2 * c + (open ? 0 : 1)) * p.dpad + j;
            st_elems<float, NE>(w, acc);
        } else {
            G* g = DG + (int64_t)cur * p.ldg + j;
            float o[NE];
            if (p.accumulate) {
                ld_elems<G, NE>(o, g);
#pragma unroll
                for (int k = 0; k < NE; ++k) o[k] = fmaf(p.scale, acc[k], o[k]);
            } else {
#pragma unroll
                for (int k = 0; k < NE; ++k) o[k] = p.scale * acc[k];
            }
            st_elems<G, NE>(g, o);
        }
    };
    for (int64_t i = i0; i < i1; i += 4) {
        uint32_t key[4];
        float v[4][NE];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (i + u < i1) {
                key[u] = ld_u32(p.key + i + u);
                const int64_t r = (int64_t)ld_u32((const uint32_t*)p.pos + i + u);
                if (key[u] < (uint32_t)p.vocab) ld_elems<T, NE>(v[u], X + r * p.lddo);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (i + u < i1) {
                if (key[u] != cur) {
                    put(false);
                    cur = key[u];
                    open = false;
#pragma unroll
                    for (int k = 0; k < NE; ++k) acc[k] = 0.f;
                }
                if (cur < (uint32_t)p.vocab) {
#pragma unroll
                    for (int k = 0; k < NE; ++k) acc[k] += v[u][k];
                }
            }
        }
    }
    put(true);
}

// The ids whose positions run over a chunk's edge: the CTA of the chunk that
// such an id begins in adds its sums, 8 warps taking every 8th chunk, then the
// 8 sums in order.
constexpr int kJoinWarps = 8;

template <typename G, int NE>
__global__ void __launch_bounds__(kJoinWarps * 32) embed_join_kernel(const EmbedBwdParams p) {
    __shared__ float sum[kJoinWarps][32 * NE];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t c = blockIdx.x;
    const int64_t i0 = c * kEmbedChunk, i1 = i0 + kEmbedChunk;
    if (i1 >= p.n) return;
    const uint32_t cur = ld_u32(p.key + i1 - 1);
    if (cur >= (uint32_t)p.vocab || ld_u32(p.key + i1) != cur) return;
    if (ld_u32(p.key + i0) == cur && i0 > 0 && ld_u32(p.key + i0 - 1) == cur) return;
    // the first position after the id's
    int64_t lo = i1, hi = p.n;
    while (lo < hi) {
        const int64_t m = (lo + hi) >> 1;
        if (ld_u32(p.key + m) == cur)
            lo = m + 1;
        else
            hi = m;
    }
    const int64_t last = (lo - 1) / kEmbedChunk;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t jb = (int64_t)blockIdx.y * 32 * NE; jb < p.d; jb += (int64_t)gridDim.y * 32 * NE) {
        const int64_t j = jb + lane * NE;
        float acc[NE];
#pragma unroll
        for (int k = 0; k < NE; ++k) acc[k] = 0.f;
        if (j < p.d) {
            for (int64_t q = c + w; q <= last; q += kJoinWarps) {
                float v[NE];
                ld_elems<float, NE>(v, p.part + (2 * q + (q == c ? 1 : 0)) * p.dpad + j);
#pragma unroll
                for (int k = 0; k < NE; ++k) acc[k] += v[k];
            }
        }
#pragma unroll
        for (int k = 0; k < NE; ++k) sum[w][lane * NE + k] = acc[k];
        __syncthreads();
        if (w == 0 && j < p.d) {
            float o[NE];
            G* g = (G*)p.dtable + (int64_t)cur * p.ldg + j;
            if (p.accumulate) ld_elems<G, NE>(o, g);
#pragma unroll
            for (int k = 0; k < NE; ++k) {
                float s = sum[0][lane * NE + k];
#pragma unroll
                for (int q = 1; q < kJoinWarps; ++q) s += sum[q][lane * NE + k];
                o[k] = p.accumulate ? fmaf(p.scale, s, o[k]) : p.scale * s;
            }
            st_elems<G, NE>(g, o);
        }
        __syncthreads();
    }
}

template <typename T, typename G, int NE>
static cudaError_t embed_bwd_go(const EmbedBwdParams& p, cudaStream_t s) {
    cudaError_t err = launch_pdl(embed_bwd_kernel<T, G, NE>, (unsigned)(p.seg_ctas + p.zero_ctas),
                                 kSegThreads, 0, s, p);
    if (err != cudaSuccess || p.chunks < 2) return err;
    return launch_pdl(embed_join_kernel<G, NE>, (unsigned)p.chunks, kJoinWarps * 32, 0, s, p);
}

cudaError_t embed_bwd_launch(int dtype, int gtype, int ne, const EmbedBwdParams& q,
                             cudaStream_t s) {
    EmbedBwdParams p = q;
    const int64_t vpr = p.d / ne;
    p.tx = 32;
    while (p.tx < kSegThreads && p.tx < vpr) p.tx *= 2;
    p.ty = kSegThreads / p.tx;
    p.slices = (int)((vpr + p.tx - 1) / p.tx);
    p.chunks = (p.n + kEmbedChunk - 1) / kEmbedChunk;
    p.seg_ctas = (int)((p.chunks + p.ty - 1) / p.ty * p.slices);
    p.zero_ctas =
        p.accumulate ? 0 : (int)((p.vocab + kZeroRowsPerCta - 1) / kZeroRowsPerCta);
#define RN_GO(T, G)                                           \
    {                                                         \
        if (ne == 8) return embed_bwd_go<T, G, 8>(p, s);      \
        if (ne == 4) return embed_bwd_go<T, G, 4>(p, s);      \
        if (ne == 2) return embed_bwd_go<T, G, 2>(p, s);      \
        return embed_bwd_go<T, G, 1>(p, s);                   \
    }
    if (dtype == DT_F32) {
        if (ne == 4) return embed_bwd_go<float, float, 4>(p, s);
        if (ne == 2) return embed_bwd_go<float, float, 2>(p, s);
        return embed_bwd_go<float, float, 1>(p, s);
    }
    if (dtype == DT_BF16) {
        if (gtype == DT_BF16) RN_GO(__nv_bfloat16, __nv_bfloat16)
        RN_GO(__nv_bfloat16, float)
    }
    if (gtype == DT_F16) RN_GO(__half, __half)
    RN_GO(__half, float)
#undef RN_GO
}

}  // namespace rn
