// rn_heads.cuh -- norms of queries and keys for each head with the position
// rotation, and the same on the way into a paged cache.
//
// A row is one head of one token, d values. With norm:
//   n_j = x_j r w_j,  r = (mean_j x_j^2 + eps)^-1/2,  else n = x;
// the first `rot` of them are turned by the token's position, pair i (values i
// and i + rot/2, or 2i and 2i + 1) by the angle whose cosine c_i and sine s_i
// the table holds:
//   y_a = n_a c_i - n_b s_i,   y_b = n_b c_i + n_a s_i,
// the others pass.
//
// Bytes bound it: every row is read and written once, while cosines, sines and
// weights are shared by a token's heads. LPR lanes hold a row, so that 32 / LPR
// rows fill a warp, and a lane holds whole pairs, its vector of first values and
// its vector of second ones: the rotation then needs no exchange, and the only
// one left is the row's sum, log2(LPR) shuffles. A warp takes one token and
// U * 32 / LPR of its heads: cosines, sines and weights are read once for U rows.
// Arithmetic is FP32, each value is rounded once, to its storage type.
#pragma once

#include <cuda_fp8.h>

#include "rn_heads.h"
#include "rn_tokens.cuh"

namespace rn {

// Where a lane's pair p of vectors lies in its row: first and second vector. Behind the
// rotated pairs (rp of them) the vectors are plain neighbours, as they are wherever pairs are
// (`interleaved`).
template <int V>
__device__ __forceinline__ void pair_at(int p, int rp, bool interleaved, int& lo, int& hi) {
    if (p < rp && !interleaved) {
        lo = p * V;
        hi = lo + rp * V;
    } else {
        lo = 2 * p * V;
        hi = lo + V;
    }
}

// V floats of the table.
template <int V>
__device__ __forceinline__ void ld_table(float* v, const float* p) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const float4 t = ld_p4(p + k);
            v[k] = t.x;
            v[k + 1] = t.y;
            v[k + 2] = t.z;
            v[k + 3] = t.w;
        }
    } else if constexpr (V == 2) {
        asm volatile("ld.global.v2.f32 {%0,%1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p));
    } else {
        v[0] = ld_p1(p);
    }
}

// A lane's cosines and sines for its pairs; 1 and 0 where nothing is turned.
template <int V, int CH, int LPR>
__device__ __forceinline__ void ld_turn(float (&c)[CH][V], float (&s)[CH][V], const float* row,
                                        int l, int rp, bool back) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const int p = l + k * LPR;
        if (p < rp) {
            ld_table<V>(c[k], row + p * V);
            ld_table<V>(s[k], row + (rp + p) * V);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                c[k][i] = 1.f;
                s[k][i] = 0.f;
            }
        }
        if (back) {
#pragma unroll
            for (int i = 0; i < V; ++i) s[k][i] = -s[k][i];
        }
    }
}

// The rotation of one lane's vectors a (first values) and b (second ones).
template <int V>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float (&c)[V],
                                     const float (&s)[V], bool interleaved) {
    if (V == 1 || !interleaved) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float t = a[i];
            a[i] = t * c[i] - b[i] * s[i];
            b[i] = b[i] * c[i] + t * s[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float t = a[2 * i], u = b[2 * i];
            a[2 * i] = t * c[i] - a[2 * i + 1] * s[i];
            a[2 * i + 1] = a[2 * i + 1] * c[i] + t * s[i];
            b[2 * i] = u * c[V / 2 + i] - b[2 * i + 1] * s[V / 2 + i];
            b[2 * i + 1] = b[2 * i + 1] * c[V / 2 + i] + u * s[V / 2 + i];
        }
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Weights at a row's vectors; ones without any.
template <typename T, int V>
__device__ __forceinline__ void ld_weight(float* v, const T* w, int at) {
    if (w) {
        const Raw<V * (int)sizeof(T)> r = ld_raw<V * (int)sizeof(T)>(w + at);
        unpack<T, V>(v, r);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 1.f;
    }
}

// V values as e4m3, to nearest even, those beyond its largest to that.
template <int V>
__device__ __forceinline__ void st_e4m3(uint8_t* p, const float* v) {
    if constexpr (V == 1) {
        *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[(V + 3) / 4] = {};
#pragma unroll
        for (int k = 0; k < V; k += 2)
            w[k / 4] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[k], v[k + 1]),
                                                           __NV_SATFINITE, __NV_E4M3)
                        << (8 * (k % 4));
        Raw<V> r;
#pragma unroll
        for (int k = 0; k < (V + 3) / 4; ++k) r.w[k] = w[k];
        st_raw<V>(p, r);
    }
}

// The unit of a warp: a token, a segment and its first head. False beyond the last unit.
struct HeadUnit {
    int64_t token;
    int seg, head;
};
__device__ __forceinline__ HeadUnit head_unit(const HeadsParams& p, uint32_t unit, int rows) {
    const uint32_t t = fast_quot(unit, p.units);
    int g = (int)(unit - t * p.units.d), seg = 0;
    if (g >= p.seg[0].groups) {
        g -= p.seg[0].groups;
        seg = 1;
        if (g >= p.seg[1].groups) {
            g -= p.seg[1].groups;
            seg = 2;
        }
    }
    return {(int64_t)t, seg, g * rows};
}

// APPEND: keys and values (segments 1 and 2) go into the cache, at the token's slot.
template <typename T, int V, int LPR, int CH, int U, bool APPEND, bool E4M3>
__global__ void __launch_bounds__(kHeadsThreads) heads_fwd_kernel(const HeadsParams p) {
    constexpr int SG = 32 / LPR, B = V * (int)sizeof(T);
    pdl_launch_dependents();
    const uint32_t unit = blockIdx.x * kHeadsWarps + (threadIdx.x >> 5);
    if (unit >= p.total) return;
    const int lane = threadIdx.x & 31, l = lane % LPR, sg = lane / LPR;
    const HeadUnit u0 = head_unit(p, unit, SG * U);
    const HeadSeg& S = p.seg[u0.seg];
    const bool value = APPEND && u0.seg == 2;
    const int d = p.d[u0.seg], rp = value ? 0 : p.rot / 2 / V;
    const uint32_t b = fast_quot((uint32_t)u0.token, p.len);
    const int64_t t = u0.token - (int64_t)b * p.len.d;
    pdl_wait();
    Raw<B> xa[U][CH], xb[U][CH];
    const T* const X = (const T*)S.x + b * S.xb + t * S.xt;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = u0.head + u * SG + sg;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int q = l + k * LPR;
            xa[u][k] = xb[u][k] = Raw<B>{};
            if (h < S.heads && 2 * q * V < d) {
                int lo, hi;
                pair_at<V>(q, rp, p.interleaved, lo, hi);
                xa[u][k] = ld_raw<B>(X + h * S.xh + lo);
                xb[u][k] = ld_raw<B>(X + h * S.xh + hi);
            }
        }
    }
    char* Y = (char*)S.y;
    int64_t ybase = b * S.yb + t * S.yt;
    if (APPEND && u0.seg > 0) {
        const int64_t slot = ld_id(p.slots, u0.token, p.itype);
        if (slot < 0 || slot >= p.nslots) return;     // (the whole warp: one token)
        const uint32_t page = fast_quot((uint32_t)slot, p.page);
        ybase = page * S.yb + (int64_t)((uint32_t)slot - page * p.page.d) * S.yt;
    }
    float c[CH][V], s[CH][V];
    bool there = true;
    if (rp > 0) {
        const int64_t pos = ld_id(p.positions, u0.token, p.itype);
        there = pos >= 0 && pos < p.table_rows;
        ld_turn<V, CH, LPR>(c, s, p.table + (there ? pos : 0) * p.ldt, l, rp, p.back);
    }
    float wa[CH][V], wb[CH][V];
    const bool norm = p.norm && !value;
    if (norm) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int q = l + k * LPR;
            if (2 * q * V < d) {
                int lo, hi;
                pair_at<V>(q, rp, p.interleaved, lo, hi);
                ld_weight<T, V>(wa[k], (const T*)S.w, lo);
                ld_weight<T, V>(wb[k], (const T*)S.w, hi);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float a[CH][V], e[CH][V];
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            unpack<T, V>(a[k], xa[u][k]);
            unpack<T, V>(e[k], xb[u][k]);
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(a[k][i], a[k][i], fmaf(e[k][i], e[k][i], ss));
        }
        if (norm) {
            const float r = rsqrtf(row_sum<LPR>(ss) / (float)d + p.eps);
#pragma unroll
            for (int k = 0; k < CH; ++k) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    a[k][i] = a[k][i] * r * wa[k][i];
                    e[k][i] = e[k][i] * r * wb[k][i];
                }
            }
        }
        const int h = u0.head + u * SG + sg;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int q = l + k * LPR;
            if (h < S.heads && 2 * q * V < d) {
                int lo, hi;
                pair_at<V>(q, rp, p.interleaved, lo, hi);
                if (rp > 0) {
                    turn<V>(a[k], e[k], c[k], s[k], p.interleaved);
                    if (!there) {
#pragma unroll
                        for (int i = 0; i < V; ++i) a[k][i] = e[k][i] = 0.f;
                    }
                }
                const int64_t at = ybase + h * S.yh;
                if (E4M3 && u0.seg > 0) {
                    const float f = p.store[u0.seg];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        a[k][i] *= f;
                        e[k][i] *= f;
                    }
                    st_e4m3<V>((uint8_t*)Y + at + lo, a[k]);
                    st_e4m3<V>((uint8_t*)Y + at + hi, e[k]);
                } else {
                    st_elems<T, V>((T*)Y + at + lo, a[k]);
                    st_elems<T, V>((T*)Y + at + hi, e[k]);
                }
            }
        }
    }
}

// The gradient. With g the transposed rotation of dy (sines negated) and r the row's, taken
// again from x:
//   dx_j = r (w_j g_j - x_j r^2 mean_k(w_k g_k x_k)),   dw_j = sum over rows of g_j x_j r.
// A lane meets the same columns in every row, so its shares of dw stay in registers over all the
// rows of a warp; the CTA joins its warps' and writes one row of p.part, which the column
// reduction adds in order: no atomics, the same bits for the same sizes and grid.
template <typename T, int V, int LPR, int CH, int U>
__global__ void __launch_bounds__(kHeadsThreads, 2) heads_bwd_kernel(const HeadsParams p) {
    constexpr int SG = 32 / LPR, B = V * (int)sizeof(T);
    __shared__ float sums[kHeadsWarps][2 * V * LPR * CH];
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sg = lane / LPR;
    const int d = p.d[0], rp = p.rot / 2 / V;
    const float inv = 1.f / (float)d;
    pdl_wait();
    for (int seg = 0; seg < 2; ++seg) {
        const HeadSeg& S = p.seg[seg];
        float da[CH][V], db[CH][V], wa[CH][V], wb[CH][V];
        int lo[CH], hi[CH];
        bool in[CH];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int q = l + k * LPR;
            in[k] = 2 * q * V < d;
            pair_at<V>(q, rp, p.interleaved, lo[k], hi[k]);
#pragma unroll
            for (int i = 0; i < V; ++i) da[k][i] = db[k][i] = wa[k][i] = wb[k][i] = 0.f;
            if (in[k]) {
                ld_weight<T, V>(wa[k], (const T*)S.w, lo[k]);
                ld_weight<T, V>(wb[k], (const T*)S.w, hi[k]);
            }
        }
        const uint32_t total = (uint32_t)(p.tokens * S.groups);
        for (uint32_t unit = blockIdx.x * kHeadsWarps + warp; unit < total;
             unit += gridDim.x * kHeadsWarps) {
            const uint32_t token = fast_quot(unit, S.per);
            const int head = (int)(unit - token * S.per.d) * (SG * U);
            const uint32_t b = fast_quot(token, p.len);
            const int64_t t = token - b * p.len.d;
            const T* const X = (const T*)S.x + b * S.xb + t * S.xt;
            const T* const G = (const T*)S.dy + b * S.gb + t * S.gt;
            T* const Y = (T*)S.y + b * S.yb + t * S.yt;
            Raw<B> xa[U][CH], xb[U][CH], ga[U][CH], gb[U][CH];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = head + u * SG + sg;
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    xa[u][k] = xb[u][k] = ga[u][k] = gb[u][k] = Raw<B>{};
                    if (h < S.heads && in[k]) {
                        xa[u][k] = ld_raw<B>(X + h * S.xh + lo[k]);
                        xb[u][k] = ld_raw<B>(X + h * S.xh + hi[k]);
                        ga[u][k] = ld_raw<B>(G + h * S.gh + lo[k]);
                        gb[u][k] = ld_raw<B>(G + h * S.gh + hi[k]);
                    }
                }
            }
            float c[CH][V], s[CH][V];
            bool there = true;
            if (rp > 0) {
                const int64_t pos = ld_id(p.positions, token, p.itype);
                there = pos >= 0 && pos < p.table_rows;
                ld_turn<V, CH, LPR>(c, s, p.table + (there ? pos : 0) * p.ldt, l, rp, true);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = head + u * SG + sg;
                float x1[CH][V], x2[CH][V], g1[CH][V], g2[CH][V];
                float ss = 0.f, dot = 0.f;
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    unpack<T, V>(x1[k], xa[u][k]);
                    unpack<T, V>(x2[k], xb[u][k]);
                    unpack<T, V>(g1[k], ga[u][k]);
                    unpack<T, V>(g2[k], gb[u][k]);
                    if (rp > 0) turn<V>(g1[k], g2[k], c[k], s[k], p.interleaved);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        ss = fmaf(x1[k][i], x1[k][i], fmaf(x2[k][i], x2[k][i], ss));
                        dot = fmaf(wa[k][i] * g1[k][i], x1[k][i],
                                   fmaf(wb[k][i] * g2[k][i], x2[k][i], dot));
                    }
                }
                ss = row_sum<LPR>(ss);
                dot = row_sum<LPR>(dot);
                const float r = rsqrtf(ss * inv + p.eps);
                const float m = dot * inv * r * r;
                if (h < S.heads) {
#pragma unroll
                    for (int k = 0; k < CH; ++k) {
                        if (!in[k]) continue;
                        float y1[V], y2[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            y1[i] = there ? r * (wa[k][i] * g1[k][i] - x1[k][i] * m) : 0.f;
                            y2[i] = there ? r * (wb[k][i] * g2[k][i] - x2[k][i] * m) : 0.f;
                            if (there) {
                                da[k][i] = fmaf(g1[k][i], x1[k][i] * r, da[k][i]);
                                db[k][i] = fmaf(g2[k][i], x2[k][i] * r, db[k][i]);
                            }
                        }
                        st_elems<T, V>(Y + h * S.yh + lo[k], y1);
                        st_elems<T, V>(Y + h * S.yh + hi[k], y2);
                    }
                }
            }
        }
        if (p.part) {
            // the warp's row groups, then the CTA's warps in order
#pragma unroll
            for (int k = 0; k < CH; ++k) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
#pragma unroll
                    for (int o = LPR; o < 32; o <<= 1) {
                        da[k][i] += __shfl_xor_sync(0xffffffffu, da[k][i], o);
                        db[k][i] += __shfl_xor_sync(0xffffffffu, db[k][i], o);
                    }
                    if (sg == 0 && in[k]) {
                        sums[warp][lo[k] + i] = da[k][i];
                        sums[warp][hi[k] + i] = db[k][i];
                    }
                }
            }
            __syncthreads();
            for (int j = threadIdx.x; j < d; j += kHeadsThreads) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kHeadsWarps; ++w) v += sums[w][j];
                p.part[((int64_t)blockIdx.x * 2 + seg) * d + j] = v;
            }
            __syncthreads();
        }
    }
}

// ---- instances -----------------------------------------------------------------
// Calls f.template operator()<V, LPR, CH>() for a shape.
template <typename T, typename F>
cudaError_t for_shape(HeadShape sh, F f) {
    constexpr int V = Elem<T>::kVec;
    if (sh.v == V) {
        switch (sh.lpr) {
            case 4: return f.template run<V, 4, 1>();
            case 8: return f.template run<V, 8, 1>();
            case 16: return f.template run<V, 16, 1>();
            default:
                if constexpr (sizeof(T) == 4)
                    if (sh.ch == 2) return f.template run<V, 32, 2>();
                return f.template run<V, 32, 1>();
        }
    }
    if (sh.v == 2) return sh.ch == 1 ? f.template run<2, 32, 1>() : f.template run<2, 32, 4>();
    return sh.ch == 2 ? f.template run<1, 32, 2>() : f.template run<1, 32, 8>();
}

template <typename T, bool APPEND, bool E4M3>
struct FwdRun {
    const HeadsParams& p;
    cudaStream_t s;
    template <int V, int LPR, int CH>
    cudaError_t run() {
        constexpr int U = heads_fwd_rows(CH);
        return launch_pdl(heads_fwd_kernel<T, V, LPR, CH, U, APPEND, E4M3>,
                          (p.total + kHeadsWarps - 1) / kHeadsWarps, kHeadsThreads, 0, s, p);
    }
};
template <typename T>
struct BwdRun {
    const HeadsParams& p;
    int ctas;
    cudaStream_t s;
    template <int V, int LPR, int CH>
    cudaError_t run() {
        constexpr int U = heads_bwd_rows(CH);
        return launch_pdl(heads_bwd_kernel<T, V, LPR, CH, U>, (unsigned)ctas, kHeadsThreads, 0, s,
                          p);
    }
};

template <typename T>
cudaError_t heads_fwd_t(bool append, bool e4m3, HeadShape sh, const HeadsParams& p,
                        cudaStream_t s) {
    if (!append) return for_shape<T>(sh, FwdRun<T, false, false>{p, s});
    if (e4m3) return for_shape<T>(sh, FwdRun<T, true, true>{p, s});
    return for_shape<T>(sh, FwdRun<T, true, false>{p, s});
}
template <typename T>
cudaError_t heads_bwd_t(HeadShape sh, const HeadsParams& p, int ctas, cudaStream_t s) {
    return for_shape<T>(sh, BwdRun<T>{p, ctas, s});
}

}  // namespace rn
