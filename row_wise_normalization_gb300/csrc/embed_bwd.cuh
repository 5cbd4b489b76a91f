// embed_bwd.cuh -- gradient of embedding rows from the sorted ids:
//   dtable[v] = (accumulate ? dtable[v] : 0) + scale * sum_{i: id_i = v} dout[i]
// for the ids that occur (embed_sort.cu clears the rows of the others).
//
// Bytes bound it: dout read once, every row of the gradient written once. The
// sorted positions are cut into chunks of 8 to 32, a lane for each position.
// A group of threads takes one chunk and a slice of the columns, has 8 of the chunk's
// rows in flight at a time, adds them in registers (FP32) and, where the id changes,
// writes the id's row. An id whose positions run over a chunk's edge leaves its sum of
// each chunk in the workspace, and a second kernel adds those in chunk order, so that an
// id which fills half of a batch is summed by as many groups as its rows fill.
// Every sum has a fixed order: results repeat bit for bit.
#pragma once

#include "rn_embed.cuh"

namespace rn {

template <typename T, typename G, int NE>
__global__ void __launch_bounds__(kSegThreads, 4) embed_bwd_kernel(const EmbedBwdParams p) {
    pdl_launch_dependents();
    const int64_t c = (int64_t)((int)blockIdx.x / p.slices) * p.ty + (int)threadIdx.x / p.tx;
    if (c >= p.chunks) return;          // whole warps: p.tx is a multiple of 32
    pdl_wait();
    sum_chunk<T, G, NE>(p, c, (int)blockIdx.x % p.slices, (int)threadIdx.x % p.tx);
}

template <typename G>
__global__ void __launch_bounds__(kJoinWarps * 32, 4)
    embed_join_kernel(const EmbedBwdParams p, bool vec, bool once) {
    __shared__ float sum[kJoinWarps][kJoinBlock];
    __shared__ JoinState st;
    pdl_launch_dependents();
    pdl_wait();
    join_chunks<G, kJoinWarps>(p, vec, once, (int64_t)blockIdx.x * kJoinWarps, blockIdx.y, gridDim.y,
                               st, sum);
}

template <typename G>
__global__ void __launch_bounds__(kJoinWarps * 32)
    embed_long_kernel(const EmbedBwdParams p, bool vec) {
    __shared__ float sum[kJoinWarps][kJoinBlock];
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t n = ld_u32(p.longs);
    for (uint32_t i = blockIdx.x; i < n; i += gridDim.x) {
        const Raw<16> r = ld_raw<16>((const LongId*)(p.longs + 4) + i);
        join_long<G, kJoinWarps>(p, vec, true, LongId{r.w[0], r.w[1], r.w[2], 0}, sum, blockIdx.y,
                                 gridDim.y);
    }
}

template <typename T, typename G, int NE>
cudaError_t embed_bwd_go(const EmbedBwdParams& p, cudaStream_t s) {
    cudaError_t err = launch_pdl(embed_bwd_kernel<T, G, NE>,
                                 (unsigned)((p.chunks + p.ty - 1) / p.ty * p.slices), kSegThreads,
                                 0, s, p);
    if (err != cudaSuccess || p.chunks < 2) return err;
    const int64_t blocks = (p.d + kJoinBlock - 1) / kJoinBlock;
    const int64_t ctas = (p.chunks - 1 + kJoinWarps - 1) / kJoinWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool vec = NE % 4 == 0, once = p.chunks <= kJoinOnce;
    // (kJoinCols blocks a step; one launch that has long ids to do as well: a block each)
    const int64_t wide = once ? blocks : (blocks + kJoinCols - 1) / kJoinCols;
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)(wide < 8 ? wide : 8), 1);
    err = cudaLaunchKernelEx(&cfg, embed_join_kernel<G>, p, vec, once);
    if (err != cudaSuccess || once) return err;
    // (an id is long if it fills a CTA's chunks: there are at most as many as CTAs)
    cfg.gridDim = dim3((unsigned)(ctas < 32 ? ctas : 32), (unsigned)(blocks < 32 ? blocks : 32), 1);
    return cudaLaunchKernelEx(&cfg, embed_long_kernel<G>, p, vec);
}

// One type of rows and of the gradient.
template <typename T, typename G>
cudaError_t embed_bwd_t(int ne, const EmbedBwdParams& p, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (ne == 8) return embed_bwd_go<T, G, 8>(p, s);
    if (ne == 4) return embed_bwd_go<T, G, 4>(p, s);
    if (ne == 2) return embed_bwd_go<T, G, 2>(p, s);
    return embed_bwd_go<T, G, 1>(p, s);
}

}  // namespace rn
