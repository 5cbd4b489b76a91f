// logprob_bwd.cu -- gradient of log probabilities and entropies:
//   p_j = e^{x_j - lse},  x_j = scale * logit_j,
//   dlogit_j = scale * (g (d_jt - p_j) - h p_j (log p_j + H))
// with g the gradient of log p_t and h that of the entropy H.
//
// Element by element, each logit read once and each gradient written once:
// bytes bound it. A CTA takes a tile of one row, so that the row's five
// numbers are read once a thread, and every thread has its loads in flight together.
// Rows with g = h = 0 (padding) are written as zeros without being read. p_j = 0
// makes both terms zero: e^-128 is below the smallest FP32 number the exponential
// gives, so log p_j is held above -128 and 0 * -inf cannot arise. dlogits may be logits itself: a thread writes only what
// it has read.
#include "rn_tokens.cuh"

namespace rn {

constexpr int kLpbThreads = 256;
constexpr int kLpbU = 4;

constexpr float kLpbFar = 4096.f;

// (m, log S) of a row: its largest logit, and the logarithm of the sum of
// e^{scale (x_j - m)}. All threads of the CTA.
template <typename T>
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
    for (int c = t; c < V; c += kLpbThreads) m = fmaxf(m, ldt_x1(X + c));
    m = meet(m, false);
    float s = 0.f;
    for (int c = t; c < V; c += kLpbThreads) s += ex2((ldt_x1(X + c) - m) * scale * kLog2e);
    return make_float2(m, logf(meet(s, true)));
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kLpbThreads) logprob_bwd_kernel(const LogprobBwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int t = threadIdx.x, V = p.vocab;
    for (int64_t b = blockIdx.x; b < p.total; b += gridDim.x) {
        const int64_t row = b / p.tiles;
        const int tile = (int)(b - row * p.tiles);
        const T* const X = (const T*)p.logits + row * p.ld;
        T* const D = (T*)p.dlogits + row * p.ldd;
        const int64_t id = p.targets ? ld_id(p.targets, row, p.itype) : -1;
        const bool there = id >= 0 && id < V;
        const float lse = ld_p1(p.lse + row);
        float g = p.dlogp && there ? ld_p1(p.dlogp + row) : 0.f;
        float h = p.dentropy ? ld_p1(p.dentropy + row) : 0.f;
        const float H = p.dentropy ? ld_p1(p.entropy + row) : 0.f;
        // a row of -inf: no probability depends on a logit
        if (lse == -INFINITY) g = h = 0.f;
        const bool zero = g == 0.f && h == 0.f;
        const float gs = g * p.scale, hs = h * p.scale;
        const int head = VEC > 1 ? head_peel_t(X, V) : 0;
        const int nv = (V - head) / VEC;
        const int tail0 = head + nv * VEC;
        auto grad = [&](float z, int64_t c) {   // z = log p_c
            const float e = ex2(z * kLog2e);
            const float u = fmaf(hs, fmaxf(z, -128.f) + H, gs);
            const float d = -e * u;
            return (c == id ? gs : 0.f) + d;
        };
        if (!zero && fabsf(lse) >= kLpbFar) {
            if (tile == 0) {
                const float2 ms = row_sums<T>(X, V, p.scale);
                for (int c = t; c < V; c += kLpbThreads) {
                    float v[1] = {grad((ldt_x1(X + c) - ms.x) * p.scale - ms.y, c)};
                    st_elems<T, 1>(D + c, v);
                }
            }
            continue;
        }
        const int64_t v0 = (int64_t)tile * (kLpbThreads * kLpbU) + t;
        float x[kLpbU][VEC];
        if (!zero) {
#pragma unroll
            for (int u = 0; u < kLpbU; ++u) {
                const int64_t v = v0 + u * kLpbThreads;
                if (v < nv) ld_elems<T, VEC>(x[u], X + head + v * VEC);
            }
        }
#pragma unroll
        for (int u = 0; u < kLpbU; ++u) {
            const int64_t v = v0 + u * kLpbThreads;
            if (v < nv) {
                const int64_t c = head + v * VEC;
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    x[u][i] = zero ? 0.f : grad(fmaf(x[u][i], p.scale, -lse), c + i);
                st_elems<T, VEC>(D + c, x[u]);
            }
        }
        // the row's head and tail, by its first tile
        if (tile == 0 && t < head + (V - tail0)) {
            const int c = t < head ? t : tail0 + t - head;
            float v[1] = {zero ? 0.f : grad(fmaf(ldt_x1(X + c), p.scale, -lse), c)};
            st_elems<T, 1>(D + c, v);
        }
    }
}

template <typename T, int VEC>
static cudaError_t logprob_bwd_go(const LogprobBwdParams& q, cudaStream_t s) {
    LogprobBwdParams p = q;
    const int64_t nv = ((int64_t)p.vocab + VEC - 1) / VEC, per = kLpbThreads * kLpbU;
    p.tiles = (nv + per - 1) / per;
    p.total = p.rows * p.tiles;
    const int64_t grid = p.total < (1 << 30) ? p.total : (1 << 30);
    return launch_pdl(logprob_bwd_kernel<T, VEC>, (unsigned)grid, kLpbThreads, 0, s, p);
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
