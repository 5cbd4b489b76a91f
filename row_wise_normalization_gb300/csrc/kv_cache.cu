// kv_cache.cu -- slots of a paged cache's tokens, and the rows of slots out of it.
#include <type_traits>

#include "rn_heads.cuh"

namespace rn {

// ---- slots ---------------------------------------------------------------------
// Token t of the batch belongs to the sequence b with offsets_b <= t < offsets_{b+1}; its
// position is starts_b + t - offsets_b, and the page table gives the page of that position.
// A few bytes a token, so latency bounds it: the offsets are brought into shared memory in one
// round, in which a thread then finds its sequence by bisection (from L2 every step of that would
// wait by itself), and the page table's entry is the one load that has to wait for it.
constexpr int kSlotsThreads = 256;
constexpr int kSlotsHeld = 4096;     // offsets in shared memory; longer batches bisect in L2

__device__ __forceinline__ void st_id(void* p, int64_t i, int64_t v, int itype) {
    if (itype == IT_I64)
        ((long long*)p)[i] = v;
    else
        ((int*)p)[i] = (int)v;
}

__global__ void __launch_bounds__(kSlotsThreads) kv_slots_kernel(const SlotsParams p,
                                                                 FastDiv page, bool held) {
    __shared__ int64_t off[kSlotsHeld];
    pdl_launch_dependents();
    pdl_wait();
    if (held) {
        for (int i = threadIdx.x; i <= p.seqs; i += kSlotsThreads) off[i] = ld_id(p.offsets, i, p.itype);
        __syncthreads();
    }
    const int64_t t = (int64_t)blockIdx.x * kSlotsThreads + threadIdx.x;
    if (t >= p.n) return;
    auto at = [&](int i) { return held ? off[i] : ld_id(p.offsets, i, p.itype); };
    // the first end beyond t
    const int lo = first_beyond(at, p.seqs, t);
    int64_t pos = -1, slot = -1;
    if (lo <= p.seqs) {
        const int64_t first = at(lo - 1);
        const int64_t q = ld_id(p.starts, lo - 1, p.itype) + (t - first);
        if (first <= t && q >= 0 && q <= 0x7fffffff) {
            pos = q;
            const uint32_t col = fast_quot((uint32_t)q, page);
            if (col < p.width) {
                const int64_t g = ld_id(p.page_table, (lo - 1) * p.ld + col, p.itype);
                if (g >= 0 && g < p.pages)
                    slot = g * page.d + (int64_t)((uint32_t)q - col * page.d);
            }
        }
    }
    st_id(p.slots, t, slot, p.itype);
    if (p.positions) st_id(p.positions, t, pos, p.itype);
}

cudaError_t kv_slots_launch(const SlotsParams& p, cudaStream_t s) {
    return launch_pdl(kv_slots_kernel, (unsigned)((p.n + kSlotsThreads - 1) / kSlotsThreads),
                      kSlotsThreads, 0, s, p, fast_div((uint32_t)p.page), p.seqs < kSlotsHeld);
}

// ---- gather --------------------------------------------------------------------
// out[t][h] = scale * cache[slot_t][h], zeros where there is no slot. Bytes bound it: the work is
// the flat list of the output's vectors, kGatherU of them a thread, whose slots are loaded first,
// then all their rows, then all are stored: two waits for memory whatever the widths.
constexpr int kGatherThreads = 256;
constexpr int kGatherU = 4;          // (131072 x 8 x 128 from e4m3 130 us; 2 144, 8 137)

// NE e4m3 values, each an FP32 one times scale, rounded once. Pairs go through FP16, which holds
// every e4m3 value: one conversion for two (131072 x 8 x 128 to BF16 with one for each value 146 us,
// bound by instructions).
template <typename T, int NE>
__device__ __forceinline__ void store_from_e4m3(T* out, const Raw<NE>& r, float scale) {
    float v[NE];
    if constexpr (NE == 1) {
        v[0] = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)r.w[0], __NV_E4M3))) *
               scale;
    } else {
        const F2 k = f2s(scale);
#pragma unroll
        for (int i = 0; i < NE; i += 2) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)(r.w[i / 4] >> (8 * (i % 4))), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            f2_get(mul2(f2(f.x, f.y), k), v[i], v[i + 1]);
        }
    }
    st_elems<T, NE>(out, v);
}

// One byte is no Raw of the accesses above.
template <int B>
__device__ __forceinline__ Raw<B> ld_bytes(const void* p) {
    if constexpr (B == 1) {
        Raw<B> r;
        uint16_t v;
        asm volatile("ld.global.L1::no_allocate.u8 %0, [%1];" : "=h"(v) : "l"(p));
        r.w[0] = v;
        return r;
    } else {
        return ld_raw<B>(p);
    }
}

// T void: elements of ES bytes, copied.
template <typename T, int NE, int ES>
__global__ void __launch_bounds__(kGatherThreads) kv_gather_kernel(const GatherParams p) {
    constexpr bool COPY = std::is_void<T>::value;
    constexpr int B = NE * (COPY ? ES : 1);
    pdl_launch_dependents();
    const GatherSide& S = p.side[blockIdx.y];
    const int64_t base = (int64_t)blockIdx.x * (kGatherThreads * kGatherU);
    if (base >= S.total) return;
    // the CTA's first vector: one 64-bit division; from there 32 bits suffice
    const int64_t token0 = base / S.token.d;
    const uint32_t first = (uint32_t)(base - token0 * S.token.d);
    int64_t from[kGatherU], to[kGatherU];
    pdl_wait();
#pragma unroll
    for (int u = 0; u < kGatherU; ++u) {
        const uint32_t k = u * kGatherThreads + threadIdx.x;
        from[u] = to[u] = -1;
        if (base + k < S.total) {
            const uint32_t q = fast_quot(first + k, S.token);
            const uint32_t c = first + k - q * S.token.d;
            const uint32_t h = fast_quot(c, S.head);
            const int64_t j = (int64_t)(c - h * S.head.d) * NE;
            const int64_t slot = ld_id(p.slots, token0 + q, p.itype);
            to[u] = (token0 + q) * S.ot + h * S.oh + j;
            if (slot >= 0 && slot < p.nslots) {
                const uint32_t g = fast_quot((uint32_t)slot, p.page);
                from[u] = g * S.cp + (int64_t)((uint32_t)slot - g * p.page.d) * S.cs + h * S.ch + j;
            }
        }
    }
    Raw<B> r[kGatherU];
#pragma unroll
    for (int u = 0; u < kGatherU; ++u) {
        r[u] = Raw<B>{};
        if (from[u] >= 0) r[u] = ld_bytes<B>((const char*)S.cache + from[u] * (COPY ? ES : 1));
    }
#pragma unroll
    for (int u = 0; u < kGatherU; ++u) {
        if (to[u] < 0) continue;
        if constexpr (COPY)
            st_raw<B>((char*)S.out + to[u] * ES, r[u]);
        else
            store_from_e4m3<T, NE>((T*)S.out + to[u], r[u], from[u] >= 0 ? S.scale : 0.f);
    }
}

namespace {
template <typename T, int NE, int ES>
cudaError_t gather_run(const GatherParams& p, cudaStream_t s) {
    const int64_t most = p.side[0].total > p.side[1].total ? p.side[0].total : p.side[1].total;
    const int64_t per = kGatherThreads * kGatherU;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((most + per - 1) / per), 2);
    cfg.blockDim = dim3(kGatherThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_gather_kernel<T, NE, ES>, p);
}
template <typename T>
cudaError_t gather_e4m3(int ne, const GatherParams& p, cudaStream_t s) {
    switch (ne) {
        case 8: return gather_run<T, 8, 1>(p, s);
        case 4: return gather_run<T, 4, 1>(p, s);
        case 2: return gather_run<T, 2, 1>(p, s);
        default: return gather_run<T, 1, 1>(p, s);
    }
}
}  // namespace

cudaError_t kv_gather_launch(int cache_dtype, int dtype, int ne, const GatherParams& p,
                             cudaStream_t s) {
    if (cache_dtype == DT_E4M3) {
        switch (dtype) {
            case DT_BF16: return gather_e4m3<__nv_bfloat16>(ne, p, s);
            case DT_F16: return gather_e4m3<__half>(ne, p, s);
            default: return gather_e4m3<float>(ne, p, s);
        }
    }
    if (dtype == DT_F32) {
        switch (ne) {
            case 4: return gather_run<void, 4, 4>(p, s);
            case 2: return gather_run<void, 2, 4>(p, s);
            default: return gather_run<void, 1, 4>(p, s);
        }
    }
    switch (ne) {
        case 8: return gather_run<void, 8, 2>(p, s);
        case 4: return gather_run<void, 4, 2>(p, s);
        case 2: return gather_run<void, 2, 2>(p, s);
        default: return gather_run<void, 1, 2>(p, s);
    }
}

}  // namespace rn
