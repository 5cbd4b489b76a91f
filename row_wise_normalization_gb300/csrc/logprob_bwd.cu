// logprob_bwd.cu -- gradient of log probabilities and entropies:
//   p_j = e^{x_j - lse},  x_j = scale * logit_j,
//   dlogit_j = scale * (g (d_jt - p_j) - h p_j (log p_j + H))
// with g the gradient of log p_t and h that of the entropy H.
//
// Element by element, each logit read once and each gradient written once:
// bytes bound it. A CTA takes a tile of one row, so that the row's five
// numbers are read once a thread, and every thread has its loads in flight together.
// Written as e^z (a + b z), z = log p_j, a pair of elements takes three packed instructions beside
// the exponentials, and the target's own term is added in the one vector that holds its column:
// 8192 x 128000 BF16 with entropies 597 us, 1.04 of the measured copy's rate over its
// 4.2 GB (1373 us with scalar arithmetic and a comparison an element).
// Rows with g = h = 0 (padding) are written as zeros without being read. p_j = 0
// makes both terms zero: e^-128 is below the smallest FP32 number the exponential
// gives, so log p_j is held above -128 and 0 * -inf cannot arise. dlogits may be logits itself: a
// thread writes only what it, or its CTA, has read.
//
// lse is rounded to 24 bits, and every p_j of a row is off by what that leaves off: half a step,
// 2^-24 |lse| at most, so 2^-13 just below 4096 (and below the half step of 16-bit gradients
// everywhere). Where |lse| >= 4096 (logits far from zero; a mask of the type's lowest value on every
// column, beyond FP32's range even at a scale above 1; or nothing but -inf) the first CTA of the
// row takes m and log S from the logits again and does the whole row, and the row's other CTAs
// leave: 2048 x 128000 BF16 of such rows 690 us, of nothing but -inf 166, ordinary ones 151.
// Rows of logits and gradient in different 16-byte phases are done an element an access: 2048 x
// 50001 BF16 at a stride of 50048 into a contiguous gradient 139 us, into one of that stride 61.
#include "rn_tokens.cuh"

namespace rn {

constexpr int kLpbThreads = 256;
constexpr int kLpbU = 4;
constexpr float kLpbFar = 4096.f;

// (m, log S) of a row: its largest logit, and the logarithm of the sum of
// e^{scale (x_j - m)}. All threads of the CTA.
template <typename T, int VEC>
__device__ float2 row_sums(const T* X, int V, float scale) {
    __shared__ float red[kLpbThreads / 32];
    const int t = threadIdx.x;
    auto meet = [&](float v, bool sum) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float w = __shfl_xor_sync(0xffffffffu, v, o);
            v = sum ? v + w : fmaxf(v, w);
        }
        __syncthreads();
        if ((t & 31) == 0) red[t >> 5] = v;
        __syncthreads();
        v = red[0];
        for (int k = 1; k < kLpbThreads / 32; ++k) v = sum ? v + red[k] : fmaxf(v, red[k]);
        return v;
    };
    float m = -INFINITY;
    const int head = VEC > 1 ? head_peel_t(X, V) : 0, nv = (V - head) / VEC, tail0 = head + nv * VEC;
    constexpr int U = 2;   // (8 CTAs of ordinary rows an SM leave registers for no more)
    for (int v = t; v < nv; v += kLpbThreads * U) {
        Raw<VEC * (int)sizeof(T)> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)   // (past the end: the first again)
            r[u] = ld_raw<VEC * (int)sizeof(T)>(
                X + head + (int64_t)(v + u * kLpbThreads < nv ? v + u * kLpbThreads : v) * VEC);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[VEC];
            unpack<T, VEC>(x, r[u]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) m = fmaxf(m, x[i]);
        }
    }
    if (t < head + (V - tail0)) m = fmaxf(m, ldt_x1(X + (t < head ? t : tail0 + t - head)));
    m = meet(m, false);
    if (m == -INFINITY) return make_float2(m, m);
    float s = 0.f;
    for (int c = t; c < V; c += kLpbThreads) s += ex2((ldt_x1(X + c) - m) * scale * kLog2e);
    return make_float2(m, logf(meet(s, true)));
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kLpbThreads, 8) logprob_bwd_kernel(const LogprobBwdParams p) {
    pdl_launch_dependents();
    const int t = threadIdx.x, V = p.vocab;
    const uint32_t row = fast_quot(blockIdx.x, p.tiles);
    const int tile = (int)(blockIdx.x - row * p.tiles.d);
    const T* const X = (const T*)p.logits + row * p.ld;
    T* const D = (T*)p.dlogits + row * p.ldd;
    const int head = VEC > 1 ? head_peel_t(X, V) : 0;
    const int nv = (V - head) / VEC;
    const int tail0 = head + nv * VEC;
    const int v0 = tile * (kLpbThreads * kLpbU) + t;
    pdl_wait();
    const int64_t id64 = p.targets ? ld_id(p.targets, row, p.itype) : -1;
    const int id = id64 >= 0 && id64 < V ? (int)id64 : -1;
    const float lse = ld_p1(p.lse + row);
    float g = p.dlogp && id >= 0 ? ld_p1(p.dlogp + row) : 0.f;
    float h = p.dentropy ? ld_p1(p.dentropy + row) : 0.f;
    const float H = p.dentropy ? ld_p1(p.entropy + row) : 0.f;
    const Raw<VEC * (int)sizeof(T)> z = {};
    if (g == 0.f && h == 0.f) {
#pragma unroll
        for (int u = 0; u < kLpbU; ++u) {
            const int v = v0 + u * kLpbThreads;
            if (v < nv) st_raw(D + head + (int64_t)v * VEC, z);
        }
        if (tile == 0 && t < head + (V - tail0)) {
            const float o[1] = {0.f};
            st_elems<T, 1>(D + (t < head ? t : tail0 + t - head), o);
        }
        return;
    }
    // dlogit = e^z (a + b z) with z = log p, and gs more for the target
    const float gs = g * p.scale, b = -h * p.scale, a = fmaf(b, H, -gs);
    auto grad = [&](float z, int c) {
        return ex2(z * kLog2e) * fmaf(b, fmaxf(z, -128.f), a) + (c == id ? gs : 0.f);
    };
    if (fabsf(lse) >= kLpbFar) {
        if (tile == 0) {
            const float2 ms = row_sums<T, VEC>(X, V, p.scale);
            if (ms.x == -INFINITY) {   // nothing but -inf: no probability depends on a logit
                for (int v = t; v < nv; v += kLpbThreads) st_raw(D + head + (int64_t)v * VEC, z);
                if (t < head + (V - tail0)) {
                    const float o[1] = {0.f};
                    st_elems<T, 1>(D + (t < head ? t : tail0 + t - head), o);
                }
                return;
            }
            for (int c = t; c < V; c += kLpbThreads) {
                const float o[1] = {grad((ldt_x1(X + c) - ms.x) * p.scale - ms.y, c)};
                st_elems<T, 1>(D + c, o);
            }
        }
        return;
    }
    Raw<VEC * (int)sizeof(T)> r[kLpbU];
#pragma unroll
    for (int u = 0; u < kLpbU; ++u) {
        const int v = v0 + u * kLpbThreads;
        if (v < nv) r[u] = ld_raw<VEC * (int)sizeof(T)>(X + head + (int64_t)v * VEC);
    }
#pragma unroll
    for (int u = 0; u < kLpbU; ++u) {
        const int v = v0 + u * kLpbThreads;
        if (v < nv) {
            const int c = head + v * VEC;
            float x[VEC];
            unpack<T, VEC>(x, r[u]);
            if constexpr (VEC == 1) {
                x[0] = grad(fmaf(x[0], p.scale, -lse), c);
            } else {
                const F2 s2 = f2s(p.scale), l2 = f2s(-lse), k2 = f2s(kLog2e);
                const F2 a2 = f2s(a), b2 = f2s(b);
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    F2 z = fma2(f2(x[i], x[i + 1]), s2, l2);
                    float z0, z1;
                    f2_get(mul2(z, k2), z0, z1);
                    const F2 e = f2(ex2(z0), ex2(z1));
                    F2 q = a2;
                    if (b != 0.f) {   // the row's, so the CTA's
                        f2_get(z, z0, z1);
                        q = fma2(b2, f2(fmaxf(z0, -128.f), fmaxf(z1, -128.f)), a2);
                    }
                    f2_get(mul2(e, q), x[i], x[i + 1]);
                }
                if ((unsigned)(id - c) < (unsigned)VEC) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) x[i] += c + i == id ? gs : 0.f;
                }
            }
            st_elems<T, VEC>(D + c, x);
        }
    }
    // the row's head and tail, by its first tile
    if (tile == 0 && t < head + (V - tail0)) {
        const int c = t < head ? t : tail0 + t - head;
        const float o[1] = {grad(fmaf(ldt_x1(X + c), p.scale, -lse), c)};
        st_elems<T, 1>(D + c, o);
    }
}

static int64_t logprob_bwd_tiles(int vocab, int vec) {
    const int64_t nv = ((int64_t)vocab + vec - 1) / vec, per = kLpbThreads * kLpbU;
    return (nv + per - 1) / per;
}

template <typename T, int VEC>
static cudaError_t logprob_bwd_go(const LogprobBwdParams& q, cudaStream_t s) {
    LogprobBwdParams p = q;
    const int64_t tiles = logprob_bwd_tiles(p.vocab, VEC);
    // (a matrix of that many tiles would not fit any memory)
    if (p.rows * tiles > 0x7fffffff) return cudaErrorInvalidConfiguration;
    p.tiles = fast_div((uint32_t)tiles);
    return launch_pdl(logprob_bwd_kernel<T, VEC>, (unsigned)(p.rows * tiles), kLpbThreads, 0, s, p);
}

cudaError_t logprob_bwd_launch(int dtype, bool vec, const LogprobBwdParams& p, cudaStream_t s) {
    switch (dtype) {
        case DT_BF16:
            return vec ? logprob_bwd_go<__nv_bfloat16, 8>(p, s)
                       : logprob_bwd_go<__nv_bfloat16, 1>(p, s);
        case DT_F16:
            return vec ? logprob_bwd_go<__half, 8>(p, s) : logprob_bwd_go<__half, 1>(p, s);
        default:
            return vec ? logprob_bwd_go<float, 4>(p, s) : logprob_bwd_go<float, 1>(p, s);
    }
}

}  // namespace rn
