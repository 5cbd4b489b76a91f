// embed_sort.cu -- the ids of an embedding gradient in order, with their
// positions: a stable radix sort, lowest digit first.
//
// A vocabulary needs 10 to 18 bits, so two digits of at most 9 bits sort it.
// A CTA takes a tile of 4096 ids. Each pass counts the tile's digits
// (hist kernel), then every scatter CTA finds its own bases from the counts of
// all tiles (there are few: 16 for 65536 ids, so that reading them again costs
// less than a scan kernel of its own), ranks its ids and writes them out.
// Ranks are stable: a warp owns 256 consecutive ids and takes 32 at a time;
// equal digits among the 32 are found by a warp match and numbered by lane,
// and a table of counts for each warp carries the number from one 32 to the
// next. Nothing depends on the order in which CTAs or atomics run.
#include "rn_tokens.cuh"

namespace rn {

constexpr int kSortWarps = kSortThreads / 32;

// The sort key of the id at position i.
__device__ __forceinline__ uint32_t id_key(const SortParams& p, int64_t i, int itype) {
    const int64_t id = ld_id(p.tokens, i, itype);
    return (uint32_t)((id >= 0 && id < p.vocab) ? id : p.vocab);
}

// Counts of the tile's digits. The first pass reads the ids themselves and
// clears the bits of the ids present.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads)
    sort_hist_kernel(const SortParams p, int itype, int src, int shift) {
    __shared__ uint32_t h[kSortBins];
    pdl_launch_dependents();
    const int t = threadIdx.x;
    for (int b = t; b < kSortBins; b += kSortThreads) h[b] = 0;
    __syncthreads();
    pdl_wait();
    const uint32_t mask = (1u << p.bits) - 1;
    const int64_t base = (int64_t)blockIdx.x * kSortTile;
    uint32_t k[kSortPerThread];
#pragma unroll
    for (int j = 0; j < kSortPerThread; ++j) {
        const int64_t i = base + j * kSortThreads + t;
        k[j] = i < p.n ? (FIRST ? id_key(p, i, itype) : ld_u32(p.key[src] + i)) : ~0u;
    }
#pragma unroll
    for (int j = 0; j < kSortPerThread; ++j)
        if (base + j * kSortThreads + t < p.n) atomicAdd(&h[(k[j] >> shift) & mask], 1u);
    if (FIRST && p.present) {
        const int64_t words = (p.vocab + 31) / 32;
        for (int64_t w = (int64_t)blockIdx.x * kSortThreads + t; w < words;
             w += (int64_t)gridDim.x * kSortThreads)
            p.present[w] = 0;
    }
    __syncthreads();
    for (int b = t; b < kSortBins; b += kSortThreads)
        p.hist[(int64_t)blockIdx.x * kSortBins + b] = h[b];
}

template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads)
    sort_scatter_kernel(const SortParams p, int itype, int src, int shift) {
    static_assert(kSortThreads == kSortBins, "one thread for each digit");
    __shared__ uint32_t cnt[kSortWarps][kSortBins];
    __shared__ uint32_t wsum[kSortWarps];
    pdl_launch_dependents();
    const int t = threadIdx.x, w = t >> 5, lane = t & 31;
    for (int k = 0; k < kSortWarps; ++k) cnt[k][t] = 0;
    __syncthreads();
    pdl_wait();
    const uint32_t mask = (1u << p.bits) - 1;
    const int64_t base = (int64_t)blockIdx.x * kSortTile + w * (kSortPerThread * 32);
    uint32_t key[kSortPerThread], rank[kSortPerThread];
    int32_t pos[kSortPerThread];
#pragma unroll
    for (int j = 0; j < kSortPerThread; ++j) {
        const int64_t i = base + j * 32 + lane;
        if (i < p.n) {
            key[j] = FIRST ? id_key(p, i, itype) : ld_u32(p.key[src] + i);
            pos[j] = FIRST ? (int32_t)i : (int32_t)ld_u32((const uint32_t*)p.pos[src] + i);
        } else {
            key[j] = 0;
            pos[j] = -1;
        }
    }
    // this thread's digit: its count before this tile, and in all tiles
    uint32_t before = 0, total = 0;
    for (int k = 0; k < p.tiles; ++k) {
        const uint32_t c = ld_u32(p.hist + (int64_t)k * kSortBins + t);
        if (k < (int)blockIdx.x) before += c;
        total += c;
    }
    // exclusive sum of the totals over the digits
    uint32_t incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[w] = incl;
    // ranks within the warp's ids
#pragma unroll
    for (int j = 0; j < kSortPerThread; ++j) {
        const bool in = pos[j] >= 0;
        const uint32_t dg = in ? (key[j] >> shift) & mask : (uint32_t)kSortBins;
        const unsigned same = __match_any_sync(0xffffffffu, dg);
        const int lead = __ffs(same) - 1;
        uint32_t r = 0;
        if (in && lane == lead) {
            r = cnt[w][dg];
            cnt[w][dg] = r + __popc(same);
        }
        r = __shfl_sync(0xffffffffu, r, lead);
        rank[j] = r + __popc(same & ((1u << lane) - 1));
        __syncwarp();
    }
    __syncthreads();
    uint32_t run = before + incl - total;
    for (int k = 0; k < w; ++k) run += wsum[k];
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
            if (FIRST && p.present && key[j] < (uint32_t)p.vocab)
                atomicOr(&p.present[key[j] >> 5], 1u << (key[j] & 31));
        }
    }
}

cudaError_t embed_sort_launch(int itype, SortParams p, cudaStream_t s) {
    const int passes = sort_passes(p.vocab);
    p.bits = (sort_key_bits(p.vocab) + passes - 1) / passes;
    const unsigned grid = (unsigned)p.tiles;
    for (int k = 0; k < passes; ++k) {
        const int shift = k * p.bits, src = k & 1;
        cudaError_t err =
            k == 0 ? launch_pdl(sort_hist_kernel<true>, grid, kSortThreads, 0, s, p, itype, src,
                                shift)
                   : launch_pdl(sort_hist_kernel<false>, grid, kSortThreads, 0, s, p, itype, src,
                                shift);
        if (err != cudaSuccess) return err;
        err = k == 0 ? launch_pdl(sort_scatter_kernel<true>, grid, kSortThreads, 0, s, p, itype,
                                  src, shift)
                     : launch_pdl(sort_scatter_kernel<false>, grid, kSortThreads, 0, s, p, itype,
                                  src, shift);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace rn
