// embed_fwd.cu -- embedding rows: out[i] = scale * table[tokens[i]].
//
// Nothing is computed but one product an element, so the bytes bound it: each
// different table row read once (repeats come from L2), every output row
// written. Where rows are 16-byte aligned the work is the flat list of the output's 16-byte
// vectors, kEmbedU of them a thread, so that a few long rows and many short ones fill the
// GPU alike. The
// loads of a thread's ids come first, then its row loads together, then its
// stores: two waits for memory whatever the width.
#include <type_traits>

#include "rn_tokens.cuh"

namespace rn {

constexpr int kEmbedThreads = 256;
constexpr int kEmbedU = 4;

// The NE elements of r times `scale`, rounded once. (A scale of 1 leaves the bits: no arithmetic.)
template <typename T, int NE>
__device__ __forceinline__ void scale_raw(Raw<NE * (int)sizeof(T)>& r, float scale) {
    float v[NE];
    unpack<T, NE>(v, r);
    const F2 k = f2s(scale);
#pragma unroll
    for (int i = 0; i < NE; i += 2) f2_get(mul2(f2(v[i], v[i + 1]), k), v[i], v[i + 1]);
    r = pack<T, NE>(v);
}

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
            // (an absent id gives +0 whatever the sign of the scale)
            if (p.scale != 1.f)
                scale_raw<T, NE>(r[u], id[u] >= 0 && id[u] < p.vocab ? p.scale : 0.f);
            st_raw((T*)p.out + row[u] * p.ldo + (int64_t)col[u] * NE, r[u]);
        }
    }
}

// Rows at any phase (odd widths or strides, offset bases): 16-byte stores to the aligned part of
// the output row, each from the two aligned 16-byte vectors of the table row that hold its
// elements, shifted by the row's common phase. Nothing beside the row is read: where an end vector's
// two would reach beyond it, its elements are copied one at a time with the row's unaligned head
// and tail, by the row's first warp. A warp takes 128 vectors of a row. (4097 x 771 FP16 3.0 us,
// one element an access throughout 8.1. With whole vectors at the row's ends, which read up to 14
// bytes of what lies beside it, 65536 x 37 BF16 took 17.3 us, not 18.6; the wider ones gained nothing.)
constexpr int kShiftVectors = 32 * kEmbedU;

template <typename T>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_shift_kernel(const EmbedParams p, int itype, int64_t d, FastDiv pieces) {
    constexpr int VEC = Elem<T>::kVec;
    pdl_launch_dependents();
    const uint32_t k = blockIdx.x * (kEmbedThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const uint32_t row = fast_quot(k, pieces), piece = k - row * pieces.d;
    if (row >= p.n) return;
    T* const O = (T*)p.out + row * p.ldo;
    pdl_wait();
    const int64_t id = ld_id(p.tokens, row, itype);
    const bool there = id >= 0 && id < p.vocab;
    const T* const S = (const T*)p.table + (there ? id : 0) * p.ldt;
    const ShiftSpan span = shift_span((uintptr_t)O, (uintptr_t)S, d, (int)sizeof(T));
    const int64_t head = span.head, nv = span.nv, tail = head + nv * VEC;
    // the phase of every vector's source
    const uint32_t q = span.phase;
    const char* const A = (const char*)(S + head) - q;
    const int64_t v0 = (int64_t)piece * kShiftVectors + lane;
    Raw<16> a[kEmbedU], b[kEmbedU];
#pragma unroll
    for (int u = 0; u < kEmbedU; ++u) {
        const int64_t v = v0 + u * 32;
        a[u] = b[u] = Raw<16>{};
        if (v < nv && there) {
            a[u] = ld_raw<16>(A + v * 16);
            if (q) b[u] = ld_raw<16>(A + v * 16 + 16);
        }
    }
    // an element of the row's ends
    const int64_t j = lane < head ? lane : tail + lane - head;
    const bool ends = piece == 0 && j < d;
    Raw<(int)sizeof(T)> e = {};
    if (ends && there) e = ld_raw<(int)sizeof(T)>(S + j);
#pragma unroll
    for (int u = 0; u < kEmbedU; ++u) {
        const int64_t v = v0 + u * 32;
        if (v < nv) {
            const uint32_t w[8] = {a[u].w[0], a[u].w[1], a[u].w[2], a[u].w[3],
                                   b[u].w[0], b[u].w[1], b[u].w[2], b[u].w[3]};
            Raw<16> r;
            auto pick = [&](auto first) {      // words from `first` on, and half a word more
                constexpr int s = decltype(first)::value;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    r.w[i] = q & 2u ? __funnelshift_r(w[i + s], w[i + s + 1 < 8 ? i + s + 1 : 7], 16)
                                    : w[i + s];
            };
            switch (q >> 2) {
                case 0: pick(std::integral_constant<int, 0>{}); break;
                case 1: pick(std::integral_constant<int, 1>{}); break;
                case 2: pick(std::integral_constant<int, 2>{}); break;
                default: pick(std::integral_constant<int, 3>{}); break;
            }
            // (an absent id gives +0 whatever the sign of the scale)
            if (p.scale != 1.f) scale_raw<T, VEC>(r, there ? p.scale : 0.f);
            st_raw(O + head + v * VEC, r);
        }
    }
    if (ends) {
        if (p.scale != 1.f) {
            float x[1];
            unpack<T, 1>(x, e);
            x[0] = there ? x[0] * p.scale : 0.f;
            e = pack<T, 1>(x);
        }
        st_raw(O + j, e);
    }
}

template <typename T>
static cudaError_t embed_shift_go(int itype, const EmbedParams& p, int64_t d, cudaStream_t s) {
    const int64_t pieces = (d / Elem<T>::kVec + kShiftVectors) / kShiftVectors;
    constexpr int64_t per = kEmbedThreads / 32;
    return launch_pdl(embed_shift_kernel<T>, (unsigned)((p.n * pieces + per - 1) / per),
                      kEmbedThreads, 0, s, p, itype, d, fast_div((uint32_t)pieces));
}

template <typename T, int NE>
static cudaError_t embed_fwd_go(int itype, const EmbedParams& p, cudaStream_t s) {
    const int64_t per = kEmbedThreads * kEmbedU;
    return launch_pdl(embed_fwd_kernel<T, NE>, (unsigned)((p.total + per - 1) / per),
                      kEmbedThreads, 0, s, p, itype);
}

cudaError_t embed_fwd_launch(int dtype, int itype, int ne, int64_t d, const EmbedParams& p,
                             cudaStream_t s) {
    if (ne * dtype_size(dtype) == 16) {
        if (dtype == DT_F32) return embed_fwd_go<float, 4>(itype, p, s);
        if (dtype == DT_BF16) return embed_fwd_go<__nv_bfloat16, 8>(itype, p, s);
        return embed_fwd_go<__half, 8>(itype, p, s);
    }
    if (dtype == DT_F32) return embed_shift_go<float>(itype, p, d, s);
    if (dtype == DT_BF16) return embed_shift_go<__nv_bfloat16>(itype, p, d, s);
    return embed_shift_go<__half>(itype, p, d, s);
}

}  // namespace rn
