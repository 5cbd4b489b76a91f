// embed_sort.cu -- the ids of an embedding gradient in order, with their
// positions (a stable radix sort, lowest digit first).
//
// A vocabulary needs 10 to 18 bits, so two digits of at most 9 bits sort it. Ranks
// are stable: a warp owns consecutive ids and takes 32 at a time; equal digits
// among the 32 are found by a ballot a bit and numbered by lane, and a table of counts
// for each warp carries the number from one 32 to the next. Nothing depends on the
// order in which CTAs or atomics run.
//
// Up to 163840 ids (10240 a CTA of the largest cluster that the GPU places, 16 on a whole
// GB300) are sorted by one thread-block cluster of 1 to 16 CTAs that keeps them in its CTAs'
// shared memory: a pass counts its digits, the CTAs read each other's counts, and every id goes
// straight to its place in the shared memory of the CTA that owns it (the last pass writes to
// global memory). One launch. More ids are sorted in global memory, three launches a digit; one
// CTA there scans the counts. With the sums of 8 columns into 128000 rows, by the cluster and in
// global memory: 16383 ids 24 and 35 us, 65536 ids 44 and 48, 100000 ids 53 and 51, 163840 ids 68
// and 62; 1000000 ids 171 in global memory.
#include "rn_embed.cuh"

namespace rn {

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SortParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ uint32_t wsum[kSortWarps];
    pdl_wait();
    pdl_launch_dependents();   // in this order: see embed_bwd_kernel
    cluster_sort(p, smem, wsum, (int)blockIdx.x);
}

// ---- more ids: in global memory -------------------------------------------------
// Counts of the tile's digits. The first pass reads the ids themselves.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads)
    sort_hist_kernel(const SortParams p, int src, int shift) {
    __shared__ uint32_t h[kSortBins];
    pdl_launch_dependents();
    const int t = threadIdx.x;
    h[t] = 0;
    __syncthreads();
    pdl_wait();
    if (FIRST && blockIdx.x == 0 && t == 0) *p.zeroed = 0;
    const uint32_t mask = (1u << p.bits) - 1;
    const int64_t base = (int64_t)blockIdx.x * kSortTile;
    uint32_t k[kSortPerThread];
#pragma unroll
    for (int j = 0; j < kSortPerThread; ++j) {
        const int64_t i = base + j * kSortThreads + t;
        k[j] = i < p.n ? (FIRST ? id_key(p, i) : ld_u32(p.key[src] + i)) : ~0u;
    }
#pragma unroll
    for (int j = 0; j < kSortPerThread; ++j)
        if (base + j * kSortThreads + t < p.n) atomicAdd(&h[(k[j] >> shift) & mask], 1u);
    __syncthreads();
    p.hist[(int64_t)blockIdx.x * kSortBins + t] = h[t];
}

// Exclusive sums of the counts, over the digits and within a digit over the tiles, in
// place: one CTA, a thread for each digit.
__global__ void __launch_bounds__(kSortThreads) sort_scan_kernel(const SortParams p) {
    __shared__ uint32_t wsum[kSortWarps];
    pdl_launch_dependents();
    const int t = threadIdx.x;
    pdl_wait();
    uint32_t total = 0;
#pragma unroll 8
    for (int k = 0; k < p.tiles; ++k) total += ld_u32(p.hist + (int64_t)k * kSortBins + t);
    uint32_t run = sum_before(total, wsum);
    for (int k0 = 0; k0 < p.tiles; k0 += 8) {   // loads of a step together
        uint32_t c[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            c[u] = k0 + u < p.tiles ? ld_u32(p.hist + (int64_t)(k0 + u) * kSortBins + t) : 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (k0 + u < p.tiles) p.hist[(int64_t)(k0 + u) * kSortBins + t] = run;
            run += c[u];
        }
    }
}

template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads)
    sort_scatter_kernel(const SortParams p, int src, int shift) {
    __shared__ uint32_t cnt[kSortWarps][kSortBins];
    const int t = threadIdx.x, w = t >> 5, lane = t & 31;
    for (int k = 0; k < kSortWarps; ++k) cnt[k][t] = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();   // in this order: see embed_bwd_kernel
    const uint32_t mask = (1u << p.bits) - 1;
    const int64_t base = (int64_t)blockIdx.x * kSortTile + w * (kSortPerThread * 32);
    uint32_t key[kSortPerThread], rank[kSortPerThread];
    int32_t pos[kSortPerThread];
#pragma unroll
    for (int j = 0; j < kSortPerThread; ++j) {
        const int64_t i = base + j * 32 + lane;
        if (i < p.n) {
            key[j] = FIRST ? id_key(p, i) : ld_u32(p.key[src] + i);
            pos[j] = FIRST ? (int32_t)i : (int32_t)ld_u32((const uint32_t*)p.pos[src] + i);
        } else {
            key[j] = 0;
            pos[j] = -1;
        }
    }
    uint32_t run = ld_u32(p.hist + (int64_t)blockIdx.x * kSortBins + t);
#pragma unroll
    for (int j = 0; j < kSortPerThread; ++j)
        rank[j] = warp_rank(cnt[w], (key[j] >> shift) & mask,
                            same_digit((key[j] >> shift) & mask, pos[j] >= 0), pos[j] >= 0, lane);
    __syncthreads();
    for (int k = 0; k < kSortWarps; ++k) {
        const uint32_t c = cnt[k][t];
        cnt[k][t] = run;
        run += c;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortPerThread; ++j) {
        if (pos[j] >= 0) {
            const uint32_t at = cnt[w][(key[j] >> shift) & mask] + rank[j];
            p.key[src ^ 1][at] = key[j];
            p.pos[src ^ 1][at] = pos[j];
        }
    }
}

static cudaError_t sort_in_cluster(SortParams& p, int ctas, cudaStream_t s) {
    p.cluster = ctas;
    const int64_t per = (p.n + p.cluster - 1) / p.cluster;
    p.share = (int)((per + kSortThreads - 1) / kSortThreads * kSortThreads);
    p.owner = fast_div((uint32_t)p.share);
    const int smem = cluster_bytes(p.share, p.passes);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.cluster, 1, 1);
    cfg.blockDim = dim3(kSortThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, embed_sort_kernel, p);
}

static cudaError_t sort_in_memory(const SortParams& p, cudaStream_t s) {
    const unsigned grid = (unsigned)p.tiles;
    for (int k = 0; k < p.passes; ++k) {
        // from one pair of arrays to the other, so that the last pass ends in [0]
        const int shift = k * p.bits, src = (p.passes - k) & 1;
        cudaError_t err =
            k == 0 ? launch_pdl(sort_hist_kernel<true>, grid, kSortThreads, 0, s, p, src, shift)
                   : launch_pdl(sort_hist_kernel<false>, grid, kSortThreads, 0, s, p, src, shift);
        if (err == cudaSuccess) err = launch_pdl(sort_scan_kernel, 1, kSortThreads, 0, s, p);
        if (err == cudaSuccess)
            err = k == 0 ? launch_pdl(sort_scatter_kernel<true>, grid, kSortThreads, 0, s, p, src,
                                      shift)
                         : launch_pdl(sort_scatter_kernel<false>, grid, kSortThreads, 0, s, p, src,
                                      shift);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

// The largest cluster of the sort that the GPU places, with all the shared memory a CTA may need.
static cudaError_t sort_most(int* most) {
    static thread_local unsigned long long prepared = 0;
    static thread_local int found = 1;
    unsigned long long ctx = 0;
    const cudaError_t err = current_context_id(&ctx);
    if (err != cudaSuccess) return err;
    const cudaError_t set = once_in_context(ctx, prepared, [] {
        constexpr int smem = cluster_bytes(kSortMaxShare, 2);
        cudaError_t e = cudaFuncSetAttribute(
            embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(embed_sort_kernel,
                                     cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            found = placeable_cluster(kSortMaxCluster, [](int c) {
                return resident_clusters((const void*)embed_sort_kernel, c, kSortThreads, smem);
            });
        return e;
    });
    *most = found;
    return set;
}

cudaError_t embed_sort_launch(SortParams p, cudaStream_t s) {
    p.passes = sort_passes(p.vocab);
    p.bits = (sort_key_bits(p.vocab) + p.passes - 1) / p.passes;
    int most = 1;
    const cudaError_t err = sort_most(&most);
    if (err != cudaSuccess) return err;
    const int ctas = sort_cluster(p.n, most);
    return ctas > 0 ? sort_in_cluster(p, ctas, s) : sort_in_memory(p, s);
}

}  // namespace rn
