// rn_tokens.cuh -- device helpers of the token operators: ids, vectors of 1 to
// 8 elements of any storage type, and the exponential.
#pragma once

#include "rn_device.cuh"
#include "rn_tokens.h"

namespace rn {

__device__ __forceinline__ uint32_t fast_quot(uint32_t n, FastDiv f) {
    return (__umulhi(f.m, n) + n) >> f.s;
}

// The id at position i as 64 bits. Coherent load (see rn_device.cuh).
__device__ __forceinline__ int64_t ld_id(const void* p, int64_t i, int itype) {
    if (itype == IT_I64) {
        long long v;
        asm volatile("ld.global.b64 %0, [%1];" : "=l"(v) : "l"((const long long*)p + i));
        return v;
    }
    int v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"((const int*)p + i));
    return v;
}
__device__ __forceinline__ uint32_t ld_u32(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// B bytes (2, 4, 8 or 16) as 32-bit words.
template <int B>
struct Raw {
    uint32_t w[B <= 4 ? 1 : B / 4];
};
template <int B>
__device__ __forceinline__ Raw<B> ld_raw(const void* p) {
    Raw<B> r;
    if constexpr (B == 16)
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                     : "l"(p));
    else if constexpr (B == 8)
        asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];"
                     : "=r"(r.w[0]), "=r"(r.w[1])
                     : "l"(p));
    else if constexpr (B == 4)
        asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(r.w[0]) : "l"(p));
    else {
        uint16_t h;
        asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(h) : "l"(p));
        r.w[0] = h;
    }
    return r;
}
// (Written once and not read again by the kernel: streaming hint. It leaves the L2 to the rows that
// are read again; embedding rows 32768 x 8192 BF16 took 137 us without it, 122 us with it.)
template <int B>
__device__ __forceinline__ void st_raw(void* p, const Raw<B>& r) {
    if constexpr (B == 16)
        asm volatile("st.global.cs.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]),
                     "r"(r.w[2]), "r"(r.w[3])
                     : "memory");
    else if constexpr (B == 8)
        asm volatile("st.global.cs.v2.b32 [%0], {%1,%2};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1])
                     : "memory");
    else if constexpr (B == 4)
        asm volatile("st.global.cs.b32 [%0], %1;" ::"l"(p), "r"(r.w[0]) : "memory");
    else
        asm volatile("st.global.cs.u16 [%0], %1;" ::"l"(p), "h"((uint16_t)r.w[0]) : "memory");
}

// 16 bytes from global to this CTA's shared memory, without waiting; the copies up to a commit are
// a group, and copy_wait<N> returns when all but this thread's newest N groups have arrived.
__device__ __forceinline__ void copy_async(void* smem, const void* p) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(smem)),
                 "l"(p)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// NE elements of T between raw words and FP32.
template <typename T, int NE>
__device__ __forceinline__ void unpack(float* v, const Raw<NE * (int)sizeof(T)>& r) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < NE; ++k) v[k] = __uint_as_float(r.w[k]);
    } else if constexpr (NE == 1) {
        v[0] = half_to_f((uint16_t)r.w[0], (T*)nullptr);
    } else {
#pragma unroll
        for (int k = 0; k < NE / 2; ++k) unpack2(r.w[k], v[2 * k], v[2 * k + 1], (T*)nullptr);
    }
}
template <typename T, int NE>
__device__ __forceinline__ Raw<NE * (int)sizeof(T)> pack(const float* v) {
    Raw<NE * (int)sizeof(T)> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < NE; ++k) r.w[k] = __float_as_uint(v[k]);
    } else if constexpr (NE == 1) {
        r.w[0] = f_to_half(v[0], (T*)nullptr);
    } else {
#pragma unroll
        for (int k = 0; k < NE / 2; ++k) r.w[k] = pack2(v[2 * k], v[2 * k + 1], (T*)nullptr);
    }
    return r;
}
// NE elements at p, in accesses of at most 16 bytes.
template <typename T, int NE>
__device__ __forceinline__ void ld_elems(float* v, const T* p) {
    constexpr int B = NE * (int)sizeof(T);
    if constexpr (B <= 16) {
        unpack<T, NE>(v, ld_raw<B>(p));
    } else {
        ld_elems<T, NE / 2>(v, p);
        ld_elems<T, NE / 2>(v + NE / 2, p + NE / 2);
    }
}
template <typename T, int NE>
__device__ __forceinline__ void st_elems(T* p, const float* v) {
    constexpr int B = NE * (int)sizeof(T);
    if constexpr (B <= 16) {
        st_raw<B>(p, pack<T, NE>(v));
    } else {
        st_elems<T, NE / 2>(p, v);
        st_elems<T, NE / 2>(p + NE / 2, v + NE / 2);
    }
}

// 2^x by the special-function unit; subnormal results are zero.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// scale * (x - m) for x <= m and scale > 0. The difference may be beyond FP32's range where its
// product with a small scale is not; halves are exact for numbers that large.
__device__ __forceinline__ float scaled_diff(float x, float m, float scale) {
    const float d = x - m;
    if (d == -INFINITY && x > -INFINITY) return (0.5f * x - 0.5f * m) * scale * 2.f;
    return d * scale;
}

// ---- thread-block clusters --------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared variable in the CTA of rank r of the cluster.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t r) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(r));
    return a;
}
__device__ __forceinline__ uint32_t peer_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void peer_store(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t a, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

}  // namespace rn
