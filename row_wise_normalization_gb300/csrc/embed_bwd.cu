// embed_bwd.cu -- gradient of embedding rows from the sorted ids:
//   dtable[v] = (accumulate ? dtable[v] : 0) + scale * sum_{i: id_i = v} dout[i]
// for the ids that occur (embed_sort.cu clears the rows of the others).
//
// Bytes bound it: dout read once, every row of the gradient written once. The
// sorted positions are cut into chunks of 32 (8 in short batches), a lane for each of a
// chunk's ids.
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

template <typename T, typename G, int NE>
__global__ void __launch_bounds__(kSegThreads, 3) embed_bwd_kernel(const EmbedBwdParams p) {
    static_assert(kEmbedChunkMax <= 32, "a lane for each position");
    constexpr int B = NE * (int)sizeof(T);
    pdl_launch_dependents();
    G* const DG = (G*)p.dtable;
    const int tx = (int)threadIdx.x % p.tx, ty = (int)threadIdx.x / p.tx, lane = tx & 31;
    const int slice = (int)blockIdx.x % p.slices;
    const int64_t c = (int64_t)((int)blockIdx.x / p.slices) * p.ty + ty;
    const int64_t j = ((int64_t)slice * p.tx + tx) * NE;
    if (c >= p.chunks) return;          // whole warps: tx is a multiple of 32
    const bool on_row = j < p.d;
    const T* const X = (const T*)p.dout + (on_row ? j : 0);
    const int64_t i0 = c * p.chunk;
    const int cnt = (int)min((int64_t)p.chunk, p.n - i0);
    pdl_wait();
    uint32_t my_key = 0xffffffffu;
    int32_t my_pos = 0;
    if (lane < cnt) {
        my_key = ld_u32(p.key + i0 + lane);
        my_pos = (int32_t)ld_u32((const uint32_t*)p.pos + i0 + lane);
    }
    const uint32_t prev = i0 > 0 ? ld_u32(p.key + i0 - 1) : 0xffffffffu;
    const uint32_t next = i0 + cnt < p.n ? ld_u32(p.key + i0 + cnt) : 0xffffffffu;
    uint32_t cur = __shfl_sync(0xffffffffu, my_key, 0);
    bool open = prev == cur;            // cur began in an earlier chunk
    float acc[NE];
#pragma unroll
    for (int k = 0; k < NE; ++k) acc[k] = 0.f;
    // cur's sum is complete as far as this chunk goes; `on`: it goes on in the next
    auto put = [&](bool on) {
        if (cur >= (uint32_t)p.vocab || !on_row) return;   // (ids outside the vocabulary)
        if (open || on) {
            st_elems<float, NE>(p.part + (2 * c + (open ? 0 : 1)) * p.dpad + j, acc);
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
    for (int i = 0; i < cnt; i += kSegU) {
        uint32_t key[kSegU];
        Raw<B> r[kSegU];
#pragma unroll
        for (int u = 0; u < kSegU; ++u) {
            key[u] = __shfl_sync(0xffffffffu, my_key, i + u);
            const int64_t at = __shfl_sync(0xffffffffu, my_pos, i + u);
            if (key[u] < (uint32_t)p.vocab) r[u] = ld_raw<B>(X + at * p.lddo);
        }
#pragma unroll
        for (int u = 0; u < kSegU; ++u) {
            if (i + u < cnt) {
                if (key[u] != cur) {
                    put(false);
                    cur = key[u];
                    open = false;
#pragma unroll
                    for (int k = 0; k < NE; ++k) acc[k] = 0.f;
                }
                if (cur < (uint32_t)p.vocab) {
                    float v[NE];
                    unpack<T, NE>(v, r[u]);
#pragma unroll
                    for (int k = 0; k < NE; ++k) acc[k] += v[k];
                }
            }
        }
    }
    put(next == cur);
}

// The ids whose positions run over a chunk's edge. Each warp of a CTA looks at one
// chunk and, if such an id begins in it, adds the id's sums of the chunks in order, kJoinCols
// blocks of 128 columns at a time so that enough loads are in flight. An id
// of more than kJoinMany chunks is left to the whole CTA: each warp takes every
// kJoinWarps-th chunk, and the warps' sums are added in order. blockIdx.y takes the
// blocks of columns in turn. (The sums lie in rows of their own, 16-byte aligned whatever
// the gradient's rows are; `vec` says whether those are.)
constexpr int kJoinWarps = 8;
constexpr int kJoinMany = 16;
constexpr int kJoinCols = 4;
constexpr int kJoinBlock = 128;

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

template <typename G>
__global__ void __launch_bounds__(kJoinWarps * 32)
    embed_join_kernel(const EmbedBwdParams p, bool vec) {
    __shared__ float sum[kJoinWarps][kJoinBlock];
    __shared__ int64_t ends[kJoinWarps];      // last chunk of a long id (or -1)
    __shared__ uint32_t ids[kJoinWarps];
    pdl_launch_dependents();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c0 = (int64_t)blockIdx.x * kJoinWarps, c = c0 + w;
    const int64_t i0 = c * p.chunk, i1 = i0 + p.chunk;
    pdl_wait();
    int64_t last = -1;
    uint32_t cur = 0xffffffffu;
    if (i1 < p.n) {
        // (loads together: most chunks need no more)
        const uint32_t before = i0 > 0 ? ld_u32(p.key + i0 - 1) : 0xffffffffu;
        const uint32_t begin = ld_u32(p.key + i0), after = ld_u32(p.key + i1);
        const int64_t e = min(i1 + p.chunk, p.n) - 1;
        const uint32_t far = ld_u32(p.key + e);
        cur = ld_u32(p.key + i1 - 1);
        if (cur < (uint32_t)p.vocab && after == cur && !(begin == cur && before == cur)) {
            last = c + 1;
            if (far == cur && e + 1 < p.n) {
                // the first position after the id's
                int64_t lo = e + 1, hi = p.n;
                while (lo < hi) {
                    const int64_t m = (lo + hi) >> 1;
                    if (ld_u32(p.key + m) == cur)
                        lo = m + 1;
                    else
                        hi = m;
                }
                last = (lo - 1) / p.chunk;
            }
        }
    }
    const bool many = last - c > kJoinMany;
    if (lane == 0) {
        ends[w] = many ? last : -1;
        ids[w] = cur;
    }
    const int64_t blocks = (p.d + kJoinBlock - 1) / kJoinBlock;
    // chunk q's sum of the id that begins in chunk o, at block b
    auto load = [&](float* v, int64_t q, int64_t o, int64_t b) {
        const int64_t j = b * kJoinBlock + lane * 4;
        if (j < p.d) {
            ld_elems<float, 4>(v, p.part + (2 * q + (q == o ? 1 : 0)) * p.dpad + j);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = 0.f;
        }
    };
    if (last >= 0 && !many) {
        for (int64_t b0 = blockIdx.y; b0 < blocks; b0 += (int64_t)gridDim.y * kJoinCols) {
            float acc[kJoinCols][4];
            // (the first two chunks, which every such id has, in one go)
            float two[kJoinCols][4];
#pragma unroll
            for (int u = 0; u < kJoinCols; ++u) load(acc[u], c, c, b0 + u * gridDim.y);
#pragma unroll
            for (int u = 0; u < kJoinCols; ++u) load(two[u], c + 1, c, b0 + u * gridDim.y);
            for (int64_t q = c + 2;; ++q) {
#pragma unroll
                for (int u = 0; u < kJoinCols; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[u][k] += two[u][k];
                if (q > last) break;
#pragma unroll
                for (int u = 0; u < kJoinCols; ++u) load(two[u], q, c, b0 + u * gridDim.y);
            }
#pragma unroll
            for (int u = 0; u < kJoinCols; ++u) {
                const int64_t j = (b0 + u * gridDim.y) * kJoinBlock + lane * 4;
                if (j < p.d) join_put<G>(p, vec, cur, j, acc[u]);
            }
        }
    }
    __syncthreads();
    for (int m = 0; m < kJoinWarps; ++m) {
        if (ends[m] < 0) continue;
        for (int64_t b = blockIdx.y; b < blocks; b += gridDim.y) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            for (int64_t q = c0 + m + w; q <= ends[m]; q += 8 * kJoinWarps) {
                float v[8][4];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (q + u * kJoinWarps <= ends[m]) {
                        load(v[u], q + u * kJoinWarps, c0 + m, b);
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
                join_put<G>(p, vec, ids[m], j, acc);
            }
        }
    }
}

template <typename T, typename G, int NE>
static cudaError_t embed_bwd_go(const EmbedBwdParams& p, cudaStream_t s) {
    const int64_t ctas = (p.chunks + p.ty - 1) / p.ty * p.slices;
    cudaError_t err =
        launch_pdl(embed_bwd_kernel<T, G, NE>, (unsigned)ctas, kSegThreads, 0, s, p);
    if (err != cudaSuccess || p.chunks < 2) return err;
    const int64_t blocks = (p.d + kJoinBlock - 1) / kJoinBlock;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.chunks - 1 + kJoinWarps - 1) / kJoinWarps),
                       (unsigned)(blocks < 8 ? blocks : 8), 1);
    cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, embed_join_kernel<G>, p, NE % 4 == 0);
}

cudaError_t embed_bwd_launch(int dtype, int gtype, int ne, const EmbedBwdParams& q,
                             cudaStream_t s) {
    EmbedBwdParams p = q;
    const int64_t vpr = p.d / ne;
    p.tx = 32;
    while (p.tx < kSegThreads && p.tx < vpr) p.tx *= 2;
    p.ty = kSegThreads / p.tx;
    p.slices = (int)((vpr + p.tx - 1) / p.tx);
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
