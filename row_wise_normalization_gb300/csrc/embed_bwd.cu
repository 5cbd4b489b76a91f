// embed_bwd.cu -- gradient of embedding rows from the sorted ids:
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
#include "rn_tokens.cuh"

namespace rn {

constexpr int kSegThreads = 256;
constexpr int kSegU = 8;            // rows in flight

// Vectors of NE elements a thread has of a row: 16 bytes, at most 4.
template <typename T, int NE>
constexpr int seg_vectors() {
    return 16 / (NE * (int)sizeof(T)) < 4 ? 16 / (NE * (int)sizeof(T)) : 4;
}

template <typename T, typename G, int NE>
__global__ void __launch_bounds__(kSegThreads, 4) embed_bwd_kernel(const EmbedBwdParams p) {
    constexpr int M = seg_vectors<T, NE>();
    constexpr int B = NE * (int)sizeof(T);
    pdl_launch_dependents();
    G* const DG = (G*)p.dtable;
    const int tx = (int)threadIdx.x % p.tx, ty = (int)threadIdx.x / p.tx, lane = tx & 31;
    const int slice = (int)blockIdx.x % p.slices;
    const int64_t c = (int64_t)((int)blockIdx.x / p.slices) * p.ty + ty;
    if (c >= p.chunks) return;          // whole warps: tx is a multiple of 32
    // this thread's vectors: every 32nd of its warp's, from column j0 on
    const int64_t j0 = (((int64_t)slice * p.tx + (tx - lane)) * M + lane) * NE;
    constexpr int step = 32 * NE;
    const int cols = (int)max((int64_t)-1, min((int64_t)(M * step), p.d - j0));   // of them in the row
    const T* const X = (const T*)p.dout + j0;
    const int64_t i0 = c * p.chunk;
    const int len = (int)min((int64_t)p.chunk, p.n - i0);
    pdl_wait();
    const uint32_t prev = i0 > 0 ? ld_u32(p.key + i0 - 1) : 0xffffffffu;
    const uint32_t next = i0 + len < p.n ? ld_u32(p.key + i0 + len) : 0xffffffffu;
    uint32_t my_key = 0xffffffffu;
    int32_t my_pos = 0;
    if (lane < len) {
        my_key = ld_u32(p.key + i0 + lane);
        my_pos = (int32_t)ld_u32((const uint32_t*)p.pos + i0 + lane);
    }
    // positions of ids outside the vocabulary come last: cnt without them
    const int cnt = __popc(__ballot_sync(0xffffffffu, my_key < (uint32_t)p.vocab));
    if (cnt == 0) return;
    // bit i: position i begins an id; `open`: the chunk's first began in an earlier chunk
    const uint32_t left = __shfl_up_sync(0xffffffffu, my_key, 1);
    const unsigned heads = __ballot_sync(0xffffffffu, lane > 0 && my_key != left);
    bool open = prev == __shfl_sync(0xffffffffu, my_key, 0);
    constexpr int E = M * NE;           // elements of this thread, in pairs
    F2 acc[E / 2];
    auto clear = [&]() {
#pragma unroll
        for (int k = 0; k < E / 2; ++k) acc[k] = f2s(0.f);
    };
    clear();
    // The sum of the id of position i, complete as far as this chunk goes; `on`: it goes on in
    // the next.
    auto put = [&](int i, bool on) {
        const uint32_t id = __shfl_sync(0xffffffffu, my_key, i);
        float* const w = p.part + (2 * c + (open ? 0 : 1)) * p.dpad + j0;
        G* const g = DG + (int64_t)id * p.ldg + j0;
        float s[E];
#pragma unroll
        for (int k = 0; k < E / 2; ++k) f2_get(acc[k], s[2 * k], s[2 * k + 1]);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            if (m * step < cols) {
                if (open || on) {
                    st_elems<float, NE>(w + m * step, s + m * NE);
                } else {
                    float o[NE];
                    if (p.accumulate) ld_elems<G, NE>(o, g + m * step);
#pragma unroll
                    for (int k = 0; k < NE; ++k)
                        o[k] = p.accumulate ? fmaf(p.scale, s[m * NE + k], o[k])
                                            : p.scale * s[m * NE + k];
                    st_elems<G, NE>(g + m * step, o);
                }
            }
        }
        open = false;
    };
    auto add = [&](const Raw<B>(&r)[M]) {
        float v[E];
#pragma unroll
        for (int m = 0; m < M; ++m) unpack<T, NE>(v + m * NE, r[m]);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) acc[k] = add2(acc[k], f2(v[2 * k], v[2 * k + 1]));
    };
    for (int i = 0; i < cnt; i += kSegU) {
        Raw<B> r[kSegU][M];
#pragma unroll
        for (int u = 0; u < kSegU; ++u) {
            const int64_t at = __shfl_sync(0xffffffffu, my_pos, (i + u) & 31);
            if (i + u < cnt) {
#pragma unroll
                for (int m = 0; m < M; ++m)
                    if (m * step < cols) r[u][m] = ld_raw<B>(X + at * p.lddo + m * step);
            }
        }
        const unsigned h = heads >> i;
#pragma unroll
        for (int u = 0; u < kSegU; ++u) {
            if (i + u < cnt) {
                if (h >> u & 1u) {
                    put(i + u - 1, false);
                    clear();
                }
                add(r[u]);
            }
        }
    }
    put(cnt - 1, next == __shfl_sync(0xffffffffu, my_key, cnt - 1));
}

// The ids whose positions run over a chunk's edge. Each warp of a CTA looks at one
// chunk and, if such an id begins in it and ends within kJoinWarps chunks, adds the id's sums of
// the chunks in order, kJoinCols blocks of 128 columns at a time so that enough loads are in
// flight. A longer id is left to the whole CTA, whose warps take its sums in turn; the
// warps' sums are added in order. blockIdx.y takes the blocks of columns in turn.
// In long batches an id may have thousands of sums, and it takes two launches: the
// first also adds the kJoinWarps sums of every CTA whose chunks lie within one id, and lists the
// long ids; the second does those, in any order, with the CTAs' sums.
// (The sums lie in rows of their own, 16-byte aligned whatever the gradient's rows are;
// `vec` says whether those are.)
constexpr int kJoinWarps = 8;
constexpr int kJoinCols = 4;
constexpr int kJoinBlock = 128;
constexpr int kJoinOnce = 64;       // chunks up to which one launch does
struct alignas(16) LongId {          // its first and last chunk
    uint32_t first, last, id, pad;
};

template <typename G>
__device__ __forceinline__ void join_put(const EmbedBwdParams& p, bool vec, uint32_t id, int64_t j,
                                         const float* acc) {
    G* const g = (G*)p.dtable + (int64_t)id * p.ldg + j;
    auto value = [&](float old, float s) {
        return p.accumulate ? fmaf(p.scale, s, old) : p.scale * s;
    };
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    if (vec) {
        if (p.accumulate) ld_elems<G, 4>(o, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = value(o[k], acc[k]);
        st_elems<G, 4>(g, o);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (j + k < p.d) {
                if (p.accumulate) ld_elems<G, 1>(o + k, g + k);
                o[k] = value(o[k], acc[k]);
                st_elems<G, 1>(g + k, o + k);
            }
    }
}

// A block's 128 columns of row q of the sums, 4 a lane.
__device__ __forceinline__ void join_load(const EmbedBwdParams& p, float* v, int64_t q, int64_t b,
                                          int lane) {
    const int64_t j = b * kJoinBlock + lane * 4;
    if (j < p.d) {
        ld_elems<float, 4>(v, p.part + q * p.dpad + j);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = 0.f;
    }
}

// The sum of a long id, by a CTA: its sums are the first chunk's second row, the chunks up to
// the next CTA's, the CTAs' that lie within it (`grouped`), and the chunks that remain.
template <typename G>
__device__ __forceinline__ void join_long(const EmbedBwdParams& p, bool vec, bool grouped,
                                          const LongId& id, float (*sum)[kJoinBlock]) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = id.first, end = id.last;
    const int64_t ga = grouped ? first / kJoinWarps + 1 : 0;
    const int64_t gb = grouped ? end / kJoinWarps : 0;   // (ga <= gb: it spans kJoinWarps chunks more)
    const int64_t head = grouped ? ga * kJoinWarps - first : end + 1 - first;
    const int64_t terms = grouped ? head + (gb - ga) + (end + 1 - gb * kJoinWarps) : head;
    auto row = [&](int64_t t) {
        if (t == 0) return 2 * first + 1;
        if (t < head) return 2 * (first + t);
        if (t < head + (gb - ga)) return 2 * (ga + t - head) * kJoinWarps;
        return 2 * (gb * kJoinWarps + t - head - (gb - ga));
    };
    const int64_t blocks = (p.d + kJoinBlock - 1) / kJoinBlock;
    for (int64_t b = blockIdx.y; b < blocks; b += gridDim.y) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int64_t t = w; t < terms; t += 8 * kJoinWarps) {
            float v[8][4];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (t + u * kJoinWarps < terms) {
                    join_load(p, v[u], row(t + u * kJoinWarps), b, lane);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[u][k] = 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[k] += v[u][k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[w][lane * 4 + k] = acc[k];
        __syncthreads();
        const int64_t j = b * kJoinBlock + lane * 4;
        if (w == 0 && j < p.d) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[k] = sum[0][lane * 4 + k];
#pragma unroll
                for (int r = 1; r < kJoinWarps; ++r) acc[k] += sum[r][lane * 4 + k];
            }
            join_put<G>(p, vec, id.id, j, acc);
        }
    }
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
        join_long<G>(p, vec, true, LongId{r.w[0], r.w[1], r.w[2], 0}, sum);
    }
}

// `once`: the only launch, which does the long ids as well.
template <typename G>
__global__ void __launch_bounds__(kJoinWarps * 32, 4)
    embed_join_kernel(const EmbedBwdParams p, bool vec, bool once) {
    __shared__ float sum[kJoinWarps][kJoinBlock];
    __shared__ LongId longid;           // a long id that begins here (there is one at most)
    __shared__ bool any;
    pdl_launch_dependents();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c0 = (int64_t)blockIdx.x * kJoinWarps, c = c0 + w;
    const int64_t i0 = c * p.chunk, i1 = i0 + p.chunk;
    const int64_t blocks = (p.d + kJoinBlock - 1) / kJoinBlock;
    if (threadIdx.x == 0) any = false;
    pdl_wait();
    int64_t last = -1;
    uint32_t cur = 0xffffffffu;
    bool within = false;                // the CTA's chunks lie within one id
    if (i1 < p.n) {
        // (loads together: most chunks need no more)
        const uint32_t before = i0 > 0 ? ld_u32(p.key + i0 - 1) : 0xffffffffu;
        const uint32_t begin = ld_u32(p.key + i0), after = ld_u32(p.key + i1);
        const int64_t e = min(i1 + p.chunk, p.n) - 1;
        const uint32_t far = ld_u32(p.key + e);
        cur = ld_u32(p.key + i1 - 1);
        if (!once) {
            const int64_t g0 = c0 * p.chunk, g1 = g0 + (int64_t)kJoinWarps * p.chunk;
            within = g0 > 0 && g1 < p.n && ld_u32(p.key + g0 - 1) == cur &&
                     ld_u32(p.key + g1) == cur && cur < (uint32_t)p.vocab;
        }
        if (cur < (uint32_t)p.vocab && after == cur && !(begin == cur && before == cur)) {
            last = c + 1;
            if (far == cur && e + 1 < p.n) {
                // the first position after the id's, in [lo, hi]: 32 places at a time
                int64_t lo = e + 1, hi = p.n;
                while (lo < hi) {
                    const int64_t w32 = (hi - lo + 31) / 32;
                    const int64_t at = min(lo + (lane + 1) * w32, hi) - 1;
                    const unsigned same = __ballot_sync(0xffffffffu, ld_u32(p.key + at) == cur);
                    const int k = __popc(same);      // the first k places are the id's
                    const int64_t from = lo + k * w32;
                    lo = k == 32 ? hi : from;
                    if (k < 32) hi = min(from + w32, hi) - 1;
                }
                last = (lo - 1) / p.chunk;
            }
        }
    }
    const bool many = last - c >= kJoinWarps;
    __syncthreads();
    if (many && lane == 0) {
        any = true;
        longid = LongId{(uint32_t)c, (uint32_t)last, cur, 0};
        if (!once && blockIdx.y == 0)
            ((LongId*)(p.longs + 4))[atomicAdd(p.longs, 1u)] = longid;
    }
    if (last >= 0 && !many) {
        for (int64_t b0 = blockIdx.y; b0 < blocks; b0 += (int64_t)gridDim.y * kJoinCols) {
            float acc[kJoinCols][4], two[kJoinCols][4];
            // (the first two chunks, which every such id has, in one go)
#pragma unroll
            for (int u = 0; u < kJoinCols; ++u)
                join_load(p, acc[u], 2 * c + 1, b0 + u * gridDim.y, lane);
#pragma unroll
            for (int u = 0; u < kJoinCols; ++u)
                join_load(p, two[u], 2 * (c + 1), b0 + u * gridDim.y, lane);
            for (int64_t q = c + 2;; ++q) {
#pragma unroll
                for (int u = 0; u < kJoinCols; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[u][k] += two[u][k];
                if (q > last) break;
#pragma unroll
                for (int u = 0; u < kJoinCols; ++u)
                    join_load(p, two[u], 2 * q, b0 + u * gridDim.y, lane);
            }
#pragma unroll
            for (int u = 0; u < kJoinCols; ++u) {
                const int64_t j = (b0 + u * gridDim.y) * kJoinBlock + lane * 4;
                if (j < p.d) join_put<G>(p, vec, cur, j, acc[u]);
            }
        }
    }
    if (within) {
        // the sum of the CTA's chunks, in the place of the first one's
        for (int64_t b = blockIdx.y + (int64_t)w * gridDim.y; b < blocks;
             b += (int64_t)kJoinWarps * gridDim.y) {
            float v[kJoinWarps][4];
#pragma unroll
            for (int u = 0; u < kJoinWarps; ++u) join_load(p, v[u], 2 * (c0 + u), b, lane);
#pragma unroll
            for (int u = 1; u < kJoinWarps; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[0][k] += v[u][k];
            const int64_t j = b * kJoinBlock + lane * 4;
            if (j < p.d) st_elems<float, 4>(p.part + 2 * c0 * p.dpad + j, v[0]);
        }
    }
    if (!once) return;
    __syncthreads();
    if (any) join_long<G>(p, vec, false, longid, sum);
}

template <typename T, typename G, int NE>
static cudaError_t embed_bwd_go(const EmbedBwdParams& p, cudaStream_t s) {
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

cudaError_t embed_bwd_launch(int dtype, int gtype, int ne, const EmbedBwdParams& q,
                             cudaStream_t s) {
    EmbedBwdParams p = q;
    const int bytes = ne * dtype_size(dtype);
    const int m = 16 / bytes < 4 ? 16 / bytes : 4;      // seg_vectors
    const int64_t vpt = (p.d / ne + m - 1) / m;         // threads a row could use
    p.tx = 32;
    while (p.tx < kSegThreads && p.tx < vpt) p.tx *= 2;
    p.ty = kSegThreads / p.tx;
    p.slices = (int)((vpt + p.tx - 1) / p.tx);
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
