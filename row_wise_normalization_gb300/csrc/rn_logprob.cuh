// rn_logprob.cuh -- log probabilities over rows of logits.
//
// With x_j = scale * logit_j, m = max_j x_j, z_j = x_j - m, S = sum_j e^{z_j}
// and W = sum_j e^{z_j} z_j:
//     lse = m + log S,   log p_t = x_t - lse,   H = log S - W / S
// (both terms of H are >= 0: nothing cancels). One pass: every thread keeps
// its own running (m, S, W) over the batches of 16 or 32 elements it reads. A
// batch that raises m from m0 to m1 rescales, with r = m0 - m1 <= 0,
//     S <- S e^r,  W <- e^r (W + r S).
// Exponents are kept in units of log 2 (one instruction an exponential), and W
// with them. A masked element (-inf) gives e = 0 and 0 * -inf = NaN in W: a
// batch whose W comes out NaN is summed again with that product left out, so
// that rows without a mask do not pay for the test.
//
// Alternatives: the `top` largest logits, the lowest index first among equal
// ones, found in the same pass. A candidate is a 64-bit key: the value's bits in
// an order-preserving form above the complement of its index, so that keys
// differ and compare as wanted. The CTA holds up to kTopCap candidates and the
// key `thr` that a new one has to exceed. In the first batch the threshold comes
// from the maxima of 64 groups of threads: at least `top` elements reach the
// top-th largest of them. When the buffer is full the `top` best of it are
// kept, thr becomes the least of them, and the threads that still hold
// candidates of the batch go on. Which slot a candidate takes depends on the
// order of atomics; which keys are kept does not.
#pragma once

#include <type_traits>

#include "rn_tokens.cuh"

namespace rn {

constexpr int kTopCap = 512;
constexpr int kTopGroups = 64;

// Bits of x in an order that compares as unsigned integers do: -inf lowest, both zeros
// equal, any NaN highest.
__device__ __forceinline__ uint32_t order_bits(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    if (x != x) return 0xffffffffu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t o) {
    if (o == 0xffffffffu) return __uint_as_float(0x7fffffffu);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ unsigned long long top_key(float x, uint32_t idx) {
    return ((unsigned long long)order_bits(x) << 32) | (uint32_t)~idx;
}

// Running (m, S, W) of one thread; k = scale * log2(e).
template <bool ENT>
struct Soft {
    float m, s, w;   // m: raw logit
    __device__ __forceinline__ void init() {
        m = -INFINITY;
        s = 0.f;
        w = 0.f;
    }
    // the reference of the exponents: m, or 0 while nothing above -inf was seen
    static __device__ __forceinline__ float ref(float m) { return m == -INFINITY ? 0.f : m; }
    __device__ __forceinline__ void raise(float m1, float k) {
        const float r = m == -INFINITY ? 0.f : (m - m1) * k;   // S is 0 then
        const float f = ex2(r);
        // (r may be -inf where f is 0)
        if constexpr (ENT) w = f == 0.f ? 0.f : f * fmaf(r, s, w);
        s *= f;
        m = m1;
    }
    template <int N>
    __device__ __forceinline__ void add(const float* x, float k) {
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) mx = fmaxf(mx, x[i]);
        if (mx > m) raise(mx, k);
        const float c = ref(m);
        float sb = 0.f, wb = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float z = (x[i] - c) * k;
            const float e = ex2(z);
            sb += e;
            if constexpr (ENT) wb = fmaf(e, z, wb);
        }
        if constexpr (ENT) {
            if (wb != wb) {
                wb = 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float z = (x[i] - c) * k;
                    const float e = ex2(z);
                    if (e != 0.f) wb = fmaf(e, z, wb);
                }
            }
            w += wb;
        }
        s += sb;
    }
    __device__ __forceinline__ void merge(float m2, float s2, float w2, float k) {
        const float m1 = fmaxf(m, m2);
        const float r1 = m == -INFINITY ? 0.f : (m - m1) * k;
        const float r2 = m2 == -INFINITY ? 0.f : (m2 - m1) * k;
        const float f1 = ex2(r1), f2 = ex2(r2);
        if constexpr (ENT) {
            // (r is -inf only where f is 0; S is finite there)
            const float a = f1 == 0.f ? 0.f : f1 * fmaf(r1, s, w);
            const float b = f2 == 0.f ? 0.f : f2 * fmaf(r2, s2, w2);
            w = a + b;
        }
        s = f1 * s + f2 * s2;
        m = m1;
    }
};

// Shared state of a row's candidates.
struct TopState {
    unsigned long long cand[kTopCap];
    unsigned long long best[kMaxTop];
    unsigned long long thr;
    float group[kTopGroups];
    int count;
};

// The `top` largest of st.cand[0..n), largest first, into st.best (fewer if n is
// less). A key's place is the number of larger keys. All threads; ends without a barrier.
template <int NT>
__device__ __forceinline__ void top_rank(TopState& st, int n, int top) {
    for (int i = threadIdx.x; i < n; i += NT) {
        const unsigned long long me = st.cand[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += st.cand[j] > me;
        if (r < top) st.best[r] = me;
    }
}

// A full buffer: keep the best, raise the threshold. All threads; ends with a barrier.
template <int NT>
__device__ __forceinline__ void top_compact(TopState& st, int top) {
    top_rank<NT>(st, kTopCap, top);
    __syncthreads();
    if (threadIdx.x < (unsigned)top) st.cand[threadIdx.x] = st.best[threadIdx.x];
    if (threadIdx.x == 0) {
        st.count = top;
        st.thr = st.best[top - 1];
    }
    __syncthreads();
}

template <typename T, int NT, int VEC, bool ENT, bool TOP>
__global__ void __launch_bounds__(NT) logprob_fwd_kernel(const LogprobParams p) {
    constexpr int U = 4;              // vectors a thread holds of a batch
    constexpr int NB = U * VEC;       // elements, at most 32
    constexpr int NW = NT / 32;
    __shared__ float red[NW][3];
    __shared__ TopState st;
    pdl_launch_dependents();
    const int t = threadIdx.x, w = t >> 5, lane = t & 31;
    const float k = p.scale * kLog2e;
    const int V = p.vocab;
    pdl_wait();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* const X = (const T*)p.logits + row * p.ld;
        // elements before the first 16-byte boundary, and after the last vector
        const int head = VEC > 1 ? head_peel_t(X, V) : 0;
        const int nv = (V - head) / VEC;
        const int tail0 = head + nv * VEC;
        Soft<ENT> a;
        a.init();
        if constexpr (TOP) {
            if (t == 0) {
                st.thr = 0;
                st.count = 0;
            }
            __syncthreads();
        }
        bool first = true;
        // one batch: x[i] at column col(i), `have` of them
        auto batch = [&](const float* x, auto col, auto in, auto n_const) {
            constexpr int N = decltype(n_const)::value;
            a.template add<N>(x, k);
            if constexpr (TOP) {
                if (first) {
                    // the top-th largest of the maxima of 64 groups of threads
                    constexpr int G = NT / kTopGroups;
                    float mx = x[0];
#pragma unroll
                    for (int i = 1; i < N; ++i) mx = fmaxf(mx, x[i]);
#pragma unroll
                    for (int o = 1; o < G; o <<= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    if (t % G == 0) st.group[t / G] = mx;
                    __syncthreads();
                    if (t < kTopGroups) {
                        const float me = st.group[t];
                        int r = 0;
                        for (int j = 0; j < kTopGroups; ++j)
                            r += st.group[j] > me || (st.group[j] == me && j < t);
                        // (every element at this value is above a key without an index)
                        if (r == p.top - 1 && me > -INFINITY)
                            st.thr = (unsigned long long)order_bits(me) << 32;
                    }
                    __syncthreads();
                    first = false;
                }
                const float lo = order_value((uint32_t)(st.thr >> 32));
                const bool any = st.thr == 0;
                uint32_t pend = 0;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (in(i) && (any || !(x[i] < lo))) pend |= 1u << i;
                while (true) {
                    const unsigned long long thr = st.thr;
                    if (pend) {
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            if ((pend >> i & 1u) && top_key(x[i], col(i)) <= thr)
                                pend &= ~(1u << i);
                        const int n = __popc(pend);
                        int at = n ? atomicAdd(&st.count, n) : kTopCap;
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            if (pend >> i & 1u) {
                                if (at < kTopCap) {
                                    st.cand[at] = top_key(x[i], col(i));
                                    pend &= ~(1u << i);
                                }
                                ++at;
                            }
                    }
                    if (!__syncthreads_or(pend != 0)) break;
                    top_compact<NT>(st, p.top);
                }
            }
        };
        using One = std::integral_constant<int, 1>;
        using All = std::integral_constant<int, NB>;
        const int step = NT * U;
        for (int v0 = 0; v0 < nv; v0 += step) {
            float x[NB];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int v = v0 + u * NT + t;
                if (v < nv) {
                    ld_elems<T, VEC>(x + u * VEC, X + head + (int64_t)v * VEC);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) x[u * VEC + i] = -INFINITY;
                }
            }
            batch(
                x, [&](int i) { return (uint32_t)(head + (v0 + i / VEC * NT + t) * VEC + i % VEC); },
                [&](int i) { return v0 + i / VEC * NT + t < nv; }, All{});
        }
        // head and tail: fewer than 2 * VEC elements, one a thread
        if (head + (V - tail0) > 0) {
            const bool in = t < head + (V - tail0);
            const int c = t < head ? t : tail0 + t - head;
            float x = -INFINITY;
            if (in) x = ldt_x1(X + c);
            batch(&x, [&](int) { return (uint32_t)c; }, [&](int) { return in; }, One{});
        }
        // meet
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, a.m, o);
            const float s2 = __shfl_xor_sync(0xffffffffu, a.s, o);
            const float w2 = __shfl_xor_sync(0xffffffffu, a.w, o);
            a.merge(m2, s2, w2, k);
        }
        if (lane == 0) {
            red[w][0] = a.m;
            red[w][1] = a.s;
            red[w][2] = a.w;
        }
        __syncthreads();
        a.init();
        for (int i = 0; i < NW; ++i) a.merge(red[i][0], red[i][1], red[i][2], k);
        const bool none = a.m == -INFINITY && a.s == 0.f;   // every logit is -inf
        const float ls = logf(a.s);
        const float mx = a.m * p.scale;
        // a row with a NaN or a +inf has none of its values
        const float lse = a.s != a.s ? a.s : none ? -INFINITY : mx + ls;
        if (t == 0) {
            if (p.lse) p.lse[row] = lse;
            if (ENT && p.entropy)
                p.entropy[row] = a.s != a.s ? a.s : none ? 0.f : ls - a.w / a.s * kLn2;
            if (p.logp) {
                const int64_t id = ld_id(p.targets, row, p.itype);
                float lp = 0.f;
                if (id >= 0 && id < V) {
                    const float x = ldt_x1(X + id);
                    lp = lse != lse ? lse : none ? -INFINITY : (x - a.m) * p.scale - ls;
                }
                p.logp[row] = lp;
            }
        }
        if constexpr (TOP) {
            const int n = min(st.count, kTopCap);
            top_rank<NT>(st, n, p.top);
            __syncthreads();
            if (t < p.top) {
                const unsigned long long key = st.best[t];
                const uint32_t idx = ~(uint32_t)key;
                if (p.top_ids) {
                    if (p.itype == IT_I64)
                        ((int64_t*)p.top_ids)[row * p.top + t] = idx;
                    else
                        ((int32_t*)p.top_ids)[row * p.top + t] = (int32_t)idx;
                }
                if (p.top_logp) {
                    const float x = order_value((uint32_t)(key >> 32));
                    p.top_logp[row * p.top + t] =
                        lse != lse ? lse : x == -INFINITY ? x : (x - a.m) * p.scale - ls;
                }
            }
        }
        __syncthreads();   // the next row reuses the shared state
    }
}

template <typename T, int VEC, bool ENT, bool TOP>
static cudaError_t logprob_fwd_go(const LogprobParams& p, cudaStream_t s) {
    constexpr int NT = 512;
    const int64_t grid = p.rows < (1 << 30) ? p.rows : (1 << 30);
    return launch_pdl(logprob_fwd_kernel<T, NT, VEC, ENT, TOP>, (unsigned)grid, NT, 0, s, p);
}

template <typename T>
cudaError_t logprob_fwd_t(const LogprobParams& p, cudaStream_t s) {
    constexpr int VEC = Elem<T>::kVec;
    const bool ent = p.entropy != nullptr;
    if (p.top > 0)
        return ent ? logprob_fwd_go<T, VEC, true, true>(p, s)
                   : logprob_fwd_go<T, VEC, false, true>(p, s);
    return ent ? logprob_fwd_go<T, VEC, true, false>(p, s)
               : logprob_fwd_go<T, VEC, false, false>(p, s);
}

}  // namespace rn
