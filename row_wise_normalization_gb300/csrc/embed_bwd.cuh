// embed_bwd.cuh -- gradient of embedding rows from the sorted ids:
//   dtable[v] = (accumulate ? dtable[v] : 0) + scale * sum_{i: id_i = v} dout[i]
// for the ids that occur; the rows of the others are zeros.
//
// Bytes bound it: dout read once, every row of the gradient written once. The
// sorted positions are cut into chunks of 8 to 32, a lane for each position.
// A group of threads takes one chunk and a slice of the columns, has 8 of the chunk's
// rows in flight at a time, adds them in registers (FP32) and, where the id changes,
// writes the id's row. An id whose positions run over a chunk's edge leaves its sum of
// each chunk in the workspace, and a second kernel adds those in chunk order, so that an
// id which fills half of a batch is summed by as many groups as its rows fill.
// Every sum has a fixed order: results repeat bit for bit.
//
// The rows of ids that do not occur are most of a gradient's bytes, and which they are the ids alone
// say. The first CTAs of the launch clear them: each owns a range of the vocabulary, reads all ids
// (from L2) and marks those of its range in shared memory. They need not wait for the sort and run
// beside it and then beside the sums. (In a kernel of their own between the two, for which the
// sums had to wait: 16383 x 771 FP16 into 50001 rows 54 us, not 49; 16383 x 256 25, not 22.)
//
// 65536 x 4096 BF16 into 128000 rows (19851 of them occur): 277 us where the bytes alone
// take 234: rows of zeros 142 and sums 107 by themselves, joins 20, most of it the latency of two
// launches. 16383 x 771 FP16 into FP32, a third of it one id: 49 us (bytes 26): sort 16, joins 10,
// sums 17, which at odd widths, an access 2 bytes, are bound by instructions.
#pragma once

#include "rn_embed.cuh"

namespace rn {

// The first zero_ctas CTAs clear the rows of absent ids, beside the sort: what they touch no kernel
// of the call before touches, and the sort lets this kernel start only after its own wait, when
// all work ahead of the call has completed (the exception that rn_device.cuh names).
template <typename T, typename G, int NE>
__global__ void __launch_bounds__(kSegThreads, 4)
    embed_bwd_kernel(const SortParams z, const EmbedBwdParams p, int zero_ctas) {
    __shared__ __align__(16) uint32_t mem[kClearWords];
    if ((int)blockIdx.x < zero_ctas) {
        clear_absent<kSegThreads, false>(z, (int)blockIdx.x, zero_ctas, mem);
        return;
    }
    pdl_launch_dependents();
    const int at = (int)blockIdx.x - zero_ctas;
    const int64_t c = (int64_t)(at / p.slices) * p.ty + (int)threadIdx.x / p.tx;
    if (c >= p.chunks) return;          // whole warps: p.tx is a multiple of 32
    pdl_wait();
    sum_chunk<T, G, NE>(p, c, at % p.slices, (int)threadIdx.x % p.tx);
}

template <typename G>
__global__ void __launch_bounds__(kJoinWarps * 32, 4)
    embed_join_kernel(const EmbedBwdParams p, bool vec, bool once) {
    __shared__ float sum[kJoinWarps][kJoinBlock];
    __shared__ JoinState st;
    pdl_launch_dependents();
    pdl_wait();
    join_chunks<G>(p, vec, once, (int64_t)blockIdx.x * kJoinWarps, blockIdx.y, gridDim.y,
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
        join_long<G>(p, vec, true, LongId{r.w[0], r.w[1], r.w[2], 0}, sum, blockIdx.y,
                                 gridDim.y);
    }
}

template <typename T, typename G, int NE>
cudaError_t embed_bwd_go(const SortParams& z, const EmbedBwdParams& p, int sms, cudaStream_t s) {
    const int zero_ctas = z.zero ? (embed_zeros_many(p.n, z) ? 4 : 2) * sms : 0;
    const unsigned sum_ctas = (unsigned)((p.chunks + p.ty - 1) / p.ty * p.slices);
    cudaError_t err = launch_pdl(embed_bwd_kernel<T, G, NE>, (unsigned)zero_ctas + sum_ctas,
                                 kSegThreads, 0, s, z, p, zero_ctas);
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

// Few ids: one launch, without a sort. A CTA takes one position and a block of columns (a warp's),
// compares all ids with the position's and leaves if an earlier position has the same id. Else it
// lists the id's positions in order, its 8 warps add every 8th row each, and the warps' sums are
// added in order. Other CTAs of the launch clear the rows of absent ids, and let the next kernel
// start only once they are done: its CTAs would all go to the SMs that are free first (64 x 768
// FP32 into 32000 rows by one such CTA an SM, call behind call: 42 us, not 23; by four 16).
constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
static_assert(kFewIds <= 32 * 32, "a lane for each word of the marks");

template <typename T, typename G, int NE>
__global__ void __launch_bounds__(kFewThreads, 4)
    embed_few_kernel(const SortParams z, const EmbedBwdParams p, int zero_ctas, FastDiv blocks) {
    constexpr int M = seg_vectors<T, NE>();
    constexpr int B = NE * (int)sizeof(T);
    constexpr int E = M * NE;
    constexpr int kCols = 32 * E;           // columns of a block
    static_assert(kFewWarps * kCols <= kClearWords, "the warps' sums");
    __shared__ __align__(16) uint32_t raw[kClearWords];
    __shared__ uint32_t mask[32];
    __shared__ uint16_t list[kFewIds];
    pdl_wait();
    if ((int)blockIdx.x < zero_ctas) {
        clear_absent<kFewThreads, true>(z, (int)blockIdx.x, zero_ctas, raw);
        pdl_launch_dependents();
        return;
    }
    pdl_launch_dependents();
    const int t = threadIdx.x, w = t >> 5, lane = t & 31, n = (int)p.n;
    const uint32_t at = blockIdx.x - (unsigned)zero_ctas;
    const int i = (int)fast_quot(at, blocks);
    const int64_t col = (int64_t)(at - (uint32_t)i * blocks.d) * kCols;
    const int64_t id = ld_id(z.tokens, i, z.itype);
    if (id < 0 || id >= p.vocab) return;
    // the positions that hold the id: a bit each
    if (t < 32) mask[t] = 0;
    __syncthreads();
    for (int j0 = 0; j0 < n; j0 += kFewThreads) {
        const int j = j0 + t;
        const unsigned m = __ballot_sync(0xffffffffu, j < n && ld_id(z.tokens, j, z.itype) == id);
        if (lane == 0) mask[j >> 5] = m;
    }
    __syncthreads();
    const uint32_t mine = mask[lane];
    const int word = i >> 5;
    if (__any_sync(0xffffffffu, lane < word ? mine != 0
                                            : lane == word && (mine & ((1u << (i & 31)) - 1)) != 0))
        return;                             // an earlier position has it: the same in every warp
    int before = __popc(mine);              // inclusive, then exclusive sum over the words
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int q = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += q;
    }
    const int rows = __shfl_sync(0xffffffffu, before, 31);
    before -= __popc(mine);
    for (int k = w; k < 32; k += kFewWarps) {
        const uint32_t m = __shfl_sync(0xffffffffu, mine, k);
        const int first = __shfl_sync(0xffffffffu, before, k);
        if (m >> lane & 1u) list[first + __popc(m & ((1u << lane) - 1))] = (uint16_t)(k * 32 + lane);
    }
    __syncthreads();
    const int64_t j0 = col + lane * NE;
    constexpr int step = 32 * NE;
    const int cols = (int)max((int64_t)-1, min((int64_t)kCols, p.d - j0));
    const T* const X = (const T*)p.dout + j0;
    F2 acc[E / 2];
#pragma unroll
    for (int k = 0; k < E / 2; ++k) acc[k] = f2s(0.f);
    for (int r0 = w; r0 < rows; r0 += kSegU * kFewWarps) {
        Raw<B> r[kSegU][M];
#pragma unroll
        for (int u = 0; u < kSegU; ++u) {
            if (r0 + u * kFewWarps < rows) {
                const int64_t pos = list[r0 + u * kFewWarps];
#pragma unroll
                for (int m = 0; m < M; ++m)
                    if (m * step < cols) r[u][m] = ld_raw<B>(X + pos * p.lddo + m * step);
            }
        }
#pragma unroll
        for (int u = 0; u < kSegU; ++u) {
            if (r0 + u * kFewWarps < rows) {
                float v[E];
#pragma unroll
                for (int m = 0; m < M; ++m) unpack<T, NE>(v + m * NE, r[u][m]);
#pragma unroll
                for (int k = 0; k < E / 2; ++k) acc[k] = add2(acc[k], f2(v[2 * k], v[2 * k + 1]));
            }
        }
    }
    float s[E];
#pragma unroll
    for (int k = 0; k < E / 2; ++k) f2_get(acc[k], s[2 * k], s[2 * k + 1]);
    G* const g = (G*)p.dtable + id * p.ldg + col;
    if (rows == 1) {
        if (w != 0) return;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            if (m * step < cols) {
                G* const o = g + lane * NE + m * step;
                float v[NE];
                if (p.accumulate) ld_elems<G, NE>(v, o);
#pragma unroll
                for (int k = 0; k < NE; ++k)
                    v[k] = p.accumulate ? fmaf(p.scale, s[m * NE + k], v[k]) : p.scale * s[m * NE + k];
                st_elems<G, NE>(o, v);
            }
        }
        return;
    }
    float(*const red)[kCols] = (float(*)[kCols])raw;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int k = 0; k < NE; ++k) red[w][m * step + lane * NE + k] = s[m * NE + k];
    __syncthreads();
    const int warps = rows < kFewWarps ? rows : kFewWarps;
    for (int c = t; c < kCols && col + c < p.d; c += kFewThreads) {
        float v = red[0][c], o[1];
        for (int q = 1; q < warps; ++q) v += red[q][c];
        if (p.accumulate) ld_elems<G, 1>(o, g + c);
        o[0] = p.accumulate ? fmaf(p.scale, v, o[0]) : p.scale * v;
        st_elems<G, 1>(g + c, o);
    }
}

template <typename T, typename G, int NE>
cudaError_t embed_few_go(const SortParams& z, const EmbedBwdParams& p, int sms, cudaStream_t s) {
    const uint32_t blocks = (uint32_t)((p.d + 32 * seg_vectors<T, NE>() * NE - 1) /
                                       (32 * seg_vectors<T, NE>() * NE));
    const int zero_ctas = z.zero ? 4 * sms : 0;
    return launch_pdl(embed_few_kernel<T, G, NE>, (unsigned)zero_ctas + (unsigned)p.n * blocks,
                      kFewThreads, 0, s, z, p, zero_ctas, fast_div(blocks));
}

// One type of rows and of the gradient.
template <typename T, typename G, int NE>
cudaError_t embed_bwd_one(bool few, const SortParams& z, int sms, const EmbedBwdParams& p,
                          cudaStream_t s) {
    return few ? embed_few_go<T, G, NE>(z, p, sms, s) : embed_bwd_go<T, G, NE>(z, p, sms, s);
}
template <typename T, typename G>
cudaError_t embed_bwd_t(int ne, bool few, const SortParams& z, int sms, const EmbedBwdParams& p,
                        cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (ne == 8) return embed_bwd_one<T, G, 8>(few, z, sms, p, s);
    if (ne == 4) return embed_bwd_one<T, G, 4>(few, z, sms, p, s);
    if (ne == 2) return embed_bwd_one<T, G, 2>(few, z, sms, p, s);
    return embed_bwd_one<T, G, 1>(few, z, sms, p, s);
}

}  // namespace rn
