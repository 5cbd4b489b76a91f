// rn_tokens.h -- kernel arguments of the token operators (embedding rows and
// their gradient, log probabilities and their gradient), shared by the C-ABI
// unit and the kernel units.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "rn_params.h"

namespace rn {

// Ids (tokens, targets) are 32- or 64-bit signed integers.
enum IndexType : int { IT_I32 = 0, IT_I64 = 1 };
constexpr int index_size(int it) { return it == IT_I64 ? 8 : 4; }

// Division of a 32-bit number below 2^31 by a fixed divisor: a multiplication
// and a shift (Granlund and Montgomery, "Division by invariant integers using
// multiplication"). With s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1,
// n / d = (umulhi(m, n) + n) >> s; n < 2^31 keeps the sum within 32 bits.
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f;
    f.d = d;
    f.s = 0;
    while (((uint64_t)1 << f.s) < d) ++f.s;
    f.m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.s) - d)) / d + 1);
    return f;
}

// Function attributes belong to a context: `set` runs once in each, in each thread, and again after
// it has failed. `done`: the context it last succeeded in (a thread's own); ctx 0: none is current.
template <typename Set>
inline cudaError_t once_in_context(unsigned long long ctx, unsigned long long& done, Set set) {
    if (ctx != 0 && done == ctx) return cudaSuccess;
    const cudaError_t err = set();
    if (err == cudaSuccess) done = ctx;
    return err;
}

// The largest cluster that the context's GPU can place, a power of two up to `most`: fits(c) says
// how many clusters of c CTAs can be resident (cudaOccupancyMaxActiveClusters; a partition of a GPU
// may have no 16 SMs side by side). 1 where nothing larger fits.
template <typename Fits>
inline int placeable_cluster(int most, Fits fits) {
    while (most > 1 && fits(most) < 1) most /= 2;
    return most;
}
inline int resident_clusters(const void* kernel, int ctas, int threads, int smem) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return n;
}

// out[i] = scale * table[tokens[i]], zeros where the id is outside [0, vocab).
struct EmbedParams {
    const void* tokens;
    const void* table;
    void* out;
    int64_t n, vocab;
    int64_t ldt, ldo;     // row strides in elements
    int64_t total;        // n * vectors per row
    FastDiv vpr;          // vectors per row
    float scale;
};
// ne: elements of the widest access that table and out are aligned for; d: the width.
cudaError_t embed_fwd_launch(int dtype, int itype, int ne, int64_t d, const EmbedParams& p,
                             cudaStream_t s);

// An output row of d elements of `es` bytes, written by aligned 16-byte vectors that are each
// put together from the two aligned 16-byte vectors of the source row that hold their elements:
// elements [head, head + nv * (16 / es)) are written so, the rest one at a time. A vector whose two
// would reach beyond the source row is left to those: fewer than 4 * 16 / es of them, a warp's.
struct ShiftSpan {
    int64_t head, nv;
    uint32_t phase;       // bytes from the source's aligned vector to the first vector's elements
};
#ifdef __CUDACC__
__host__ __device__
#endif
constexpr ShiftSpan shift_span(uintptr_t out, uintptr_t src, int64_t d, int es) {
    const int64_t vec = 16 / es;
    int64_t head = (int64_t)((0u - (uint32_t)out) & 15u) / es;
    if (head > d) head = d;
    int64_t nv = (d - head) / vec;
    const uint32_t phase = ((uint32_t)src + (uint32_t)(head * es)) & 15u;
    if (phase != 0 && nv > 0 && (int64_t)phase > head * es) {   // its first vector begins before the row
        head += vec;
        nv -= 1;
    }
    if (phase != 0 && nv > 0 && (int64_t)(16 - phase) > (d - head - nv * vec) * es)   // ends behind it
        nv -= 1;
    return {head, nv, phase};
}

// Stable sort of the n ids by value, with their positions. Ids outside
// [0, vocab) are given the key `vocab`, so that they come last.
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortPerThread = 8;
constexpr int kSortTile = kSortThreads * kSortPerThread;   // ids of a CTA, sorting in global memory
constexpr int kSortBits = 9;                               // bits of a digit, at most
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortMaxCluster = 16;
constexpr int kSortMaxShare = 10240;   // ids of a CTA, sorting in shared memory
// CTAs of the cluster that sorts n ids, where the GPU places up to `most` (a power of two): 0, more
// ids than it holds, for the sort in global memory. 512 ids a CTA, one for each thread, up to 8
// CTAs, and 1024 before there are 16, whose barriers cost more: with the sums of 8 columns 2048 ids
// 12.7 us, 16.0 by one CTA; 4096 ids 13.3, 16.6 by two; 8192 ids 16.2, 17.0 by 16 CTAs, 18.3 by
// four; 16383 ids 18.9, 20.1 by 8.
constexpr int sort_cluster(int64_t n, int most) {
    if (n > (int64_t)most * kSortMaxShare) return 0;
    int c = 1;
    while (c < most && n > (int64_t)c * (c < 8 ? 512 : 1024)) c *= 2;
    return c;
}
// Whether some GPU (one that places no cluster at all) sorts n ids in global memory.
constexpr bool sort_may_use_memory(int64_t n) { return sort_cluster(n, 1) == 0; }
struct SortParams {
    const void* tokens;
    int64_t n, vocab;
    uint32_t* key[2];     // [n] each: the result in [0]; [1] where sort_may_use_memory only
    int32_t* pos[2];
    uint32_t* hist;       // [tiles][kSortBins], where sort_may_use_memory
    uint32_t* zeroed;     // a word that the sort clears for the kernels after it
    int tiles;
    int bits, passes;     // bits of a digit, digits
    int itype;
    int cluster, share;   // CTAs that sort in shared memory, ids of each
    FastDiv owner;        // division by share
    // Rows of ids that do not occur, cleared beside sort and sums (NULL: left as they are)
    char* zero;
    int64_t zero_pitch, zero_bytes;   // bytes from row to row, and of a row
    bool bulk;            // long rows, in device memory (embed_few_kernel)
};
constexpr int64_t kZeroBulk = 512;    // bytes of a row from which the bulk-copy engine clears it
constexpr int sort_key_bits(int64_t vocab) {
    int b = 0;
    while (((int64_t)1 << b) <= vocab) ++b;   // keys 0 .. vocab
    return b;
}
constexpr int sort_passes(int64_t vocab) { return (sort_key_bits(vocab) + kSortBits - 1) / kSortBits; }
// Sorts into key[0], pos[0].
cudaError_t embed_sort_launch(SortParams p, cudaStream_t s);

// dtable[v] = (accumulate ? dtable[v] : 0) + scale * sum of dout[i] over the
// positions i with tokens[i] == v, for the ids v that occur, from the sorted ids.
// Sorted positions one thread group sums, 8 to 32 (a lane each): as many as leave 2048 groups
// of CTA size, several rounds of what the GPU holds at once.
constexpr int embed_chunk(int64_t n, int64_t d) {
    int c = 8;
    while (c < 32 && n / (2 * c) * ((d + 2047) / 2048) >= 2048) c *= 2;
    return c;
}
struct EmbedBwdParams {
    const void* dout;
    void* dtable;
    const uint32_t* key;
    const int32_t* pos;
    float* part;               // [2 * chunks][dpad]
    uint32_t* longs;           // ids of many chunks: their number, and from [4] on 4 words each
    int64_t n, vocab, d, dpad;
    int64_t lddo, ldg;
    int64_t chunks;
    int chunk;                 // positions of a chunk
    int tx, ty;                // threads across a row, chunks of a CTA
    int slices;                // CTAs across a row
    float scale;
    int accumulate;
};
// Whether the zeros are many beside the sums (128 MB at least): 4 clearing CTAs an SM, which take
// all of it until they end, rather than 2. Measured on GB300, 4 against 2: 65536 x 4096 BF16 into
// 128000 rows 277 against 281 to 306 us, 16383 x 768 into FP32 (343 MB) 71 against 86, 4096 x 768
// into 50001 rows (141 MB) 32 against 37; 16383 x 771 into 50001 (104 MB) 50.5 against 49, 16383 x
// 256 27 against 22, 200000 x 1024 into 128000 182 against 157.
constexpr int64_t kZerosMany = 128 << 20;
constexpr bool embed_zeros_many(int64_t n, const SortParams& z) {
    return (z.vocab - n) * z.zero_bytes >= kZerosMany;
}
// Few ids (embed_few_kernel): at most kFewIds, and rows of kFewBytes together. Measured on GB300,
// added to a gradient, one launch against the sort's four: FP32 64 x 768 2.8 against 9.7 us,
// 512 x 768 10.4 against 11.5, 1024 x 512 (2 MB) 14.7 against 14.4, 512 x 2048 24.0 against 12.0;
// BF16 512 x 1024 8.2 against 12.1, 512 x 2048 (2 MB) 13.9 against 12.3, 512 x 4096 25.0
// against 13.1. (The host's time for three launches, 6 us, comes to that.)
constexpr int kFewIds = 1024;
constexpr int64_t kFewBytes = 2 << 20;
constexpr bool embed_few(int64_t n, int64_t d, int es) {
    return n <= kFewIds && n * d * es <= kFewBytes;
}
// The whole gradient.
cudaError_t embed_bwd_launch(int dtype, int gtype, int ne, const SortParams& sp,
                             const EmbedBwdParams& p, cudaStream_t s);

// Log probabilities over the rows of a matrix of logits.
constexpr int kMaxTop = 32;
struct LogprobParams {
    const void* logits;
    const void* targets;    // may be NULL
    float* logp;            // may be NULL, as every output
    float* entropy;
    float* lse;
    void* top_ids;
    float* top_logp;
    int64_t rows, ld;
    int vocab, top, itype;
    int split;              // CTAs of a row
    float scale;
};
constexpr int kLpThreads = 256;
constexpr int kLpU = 4;              // vectors a thread holds of a batch
constexpr int kLpMaxCluster = 16;
// CTAs a row is split over: as many as keep every SM at its four resident CTAs, while each still
// has a whole batch of its threads to read. A power of two up to `most`, what the GPU places.
constexpr int logprob_split(int64_t rows, int vocab, int vec, int sms, int most) {
    const int64_t batches = (vocab / vec + kLpThreads * kLpU - 1) / (kLpThreads * kLpU);
    int c = 1;
    while (c < most && rows * c * 2 <= 4 * (int64_t)sms && c * 2 <= batches) c *= 2;
    return c;
}
cudaError_t logprob_fwd_launch(int dtype, const LogprobParams& p, cudaStream_t s);

struct LogprobBwdParams {
    const float* dlogp;       // may be NULL
    const float* dentropy;    // may be NULL
    const void* logits;
    const void* targets;      // may be NULL (with dlogp NULL)
    const float* lse;
    const float* entropy;     // with dentropy
    void* dlogits;
    int64_t rows, ld, ldd;
    FastDiv tiles;            // tiles of a row
    int vocab, itype;
    float scale;
};
// vec: logits and dlogits of every row share a 16-byte phase.
cudaError_t logprob_bwd_launch(int dtype, bool vec, const LogprobBwdParams& p, cudaStream_t s);

}  // namespace rn
