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
// one left is the row's sum, log2(LPR) shuffles. A warp takes one token and up to
// kHeadsLoops * 32 / LPR of its heads, for which cosines, sines and weights are
// read once (where tokens have few heads: several tokens, a lane group's each).
// Arithmetic is FP32 (packed in pairs), each value is rounded once, to its
// storage type.
#pragma once

#include <type_traits>

#include <cuda_fp8.h>

#include "rn_heads.h"
#include "rn_tokens.cuh"

namespace rn {

// Where a lane's pair p of vectors lies in a row of d: in the halves of what is turned (rp pairs), then
// in the halves of the rest, so that neighbouring lanes' vectors are neighbours, however values are
// paired (32768 tokens of 16 + 16 heads of 128 BF16, neighbours turned: 86 us; with a lane's two
// vectors side by side, which left half of every sector to the other access, 119). Single values of
// pairs of neighbours are such.
template <int V>
__device__ __forceinline__ void pair_at(int p, int rp, int d, bool interleaved, int& lo, int& hi) {
    if (V == 1 && interleaved && p < rp) {
        lo = 2 * p;
        hi = lo + 1;
    } else {
        lo = (p < rp ? p : rp + p) * V;
        hi = p < rp ? lo + rp * V : p * V + d / 2;
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

// A lane's cosines and sines for its pairs; 1 and 0 where nothing is turned. Neighbours are paired
// within each of its vectors: half of the angles are the first vector's.
template <int V, int CH, int LPR>
__device__ __forceinline__ void ld_turn(float (&c)[CH][V], float (&s)[CH][V], const float* row,
                                        int l, int rp, bool interleaved) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const int p = l + k * LPR;
        if (p < rp && (V == 1 || !interleaved)) {
            ld_table<V>(c[k], row + p * V);
            ld_table<V>(s[k], row + (rp + p) * V);
        } else if (p < rp) {
            constexpr int H = V > 1 ? V / 2 : 1;
            const float* const at = row + p * H;
            ld_table<H>(c[k], at);
            ld_table<H>(c[k] + V / 2, at + rp * H);
            ld_table<H>(s[k], at + rp * V);
            ld_table<H>(s[k] + V / 2, at + rp * (V + H));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                c[k][i] = 1.f;
                s[k][i] = 0.f;
            }
        }
    }
}

// The transposed rotation of one lane's vectors a (first values) and b (second ones).
template <int V>
__device__ __forceinline__ void turn_back(float (&a)[V], float (&b)[V], const float (&c)[V],
                                          const float (&s)[V], bool interleaved) {
    if constexpr (V == 1) {
        const float t = a[0];
        a[0] = fmaf(b[0], s[0], t * c[0]);
        b[0] = fmaf(-t, s[0], b[0] * c[0]);
    } else if (!interleaved) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const F2 u = f2(a[i], a[i + 1]), v = f2(b[i], b[i + 1]), c2 = f2(c[i], c[i + 1]);
            const F2 s2 = f2(s[i], s[i + 1]);
            f2_get(fma2(v, s2, mul2(u, c2)), a[i], a[i + 1]);
            f2_get(sub2(mul2(v, c2), mul2(u, s2)), b[i], b[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const F2 u = f2(a[2 * i], a[2 * i + 1]), v = f2(b[2 * i], b[2 * i + 1]);
            const float cu = c[i], su = s[i], cv = c[V / 2 + i], sv = s[V / 2 + i];
            f2_get(fma2(f2(a[2 * i + 1], a[2 * i]), f2(su, -su), mul2(u, f2s(cu))), a[2 * i],
                   a[2 * i + 1]);
            f2_get(fma2(f2(b[2 * i + 1], b[2 * i]), f2(sv, -sv), mul2(v, f2s(cv))), b[2 * i],
                   b[2 * i + 1]);
        }
    }
}

// A lane's share of a row's sum of w g x.
template <int V>
__device__ __forceinline__ float dots(const float (&x1)[V], const float (&x2)[V],
                                      const float (&g1)[V], const float (&g2)[V],
                                      const float (&w1)[V], const float (&w2)[V]) {
    if constexpr (V == 1) {
        return fmaf(w1[0] * g1[0], x1[0], w2[0] * g2[0] * x2[0]);
    } else {
        F2 t = f2s(0.f);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            t = fma2(mul2(f2(g1[i], g1[i + 1]), f2(w1[i], w1[i + 1])), f2(x1[i], x1[i + 1]), t);
            t = fma2(mul2(f2(g2[i], g2[i + 1]), f2(w2[i], w2[i + 1])), f2(x2[i], x2[i + 1]), t);
        }
        float lo, hi;
        f2_get(t, lo, hi);
        return lo + hi;
    }
}

// dw += g x r, x := r (w g + x m).
template <int V>
__device__ __forceinline__ void grads(float (&x)[V], const float (&g)[V], const float (&w)[V],
                                      float (&dw)[V], float r, float m) {
    if constexpr (V == 1) {
        dw[0] = fmaf(g[0], x[0] * r, dw[0]);
        x[0] = r * fmaf(x[0], m, w[0] * g[0]);
    } else {
        const F2 r2 = f2s(r), m2 = f2s(m);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const F2 xx = f2(x[i], x[i + 1]), gg = f2(g[i], g[i + 1]);
            f2_get(fma2(mul2(xx, r2), gg, f2(dw[i], dw[i + 1])), dw[i], dw[i + 1]);
            f2_get(mul2(fma2(xx, m2, mul2(gg, f2(w[i], w[i + 1]))), r2), x[i], x[i + 1]);
        }
    }
}

// The sum over a row's LPR lanes, in each of them. Of a number that is no power of two: each lane adds
// the sums of 1, 2 and 4 lanes from its own on, around the row, to those of the lanes that are left.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, int lane) {
    if constexpr ((LPR & (LPR - 1)) == 0) {
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    } else {
        const int l = lane % LPR;
        auto from = [&](float x, int o) {
            return __shfl_sync(0xffffffffu, x, lane + (l + o < LPR ? o : o - LPR));
        };
        const float two = v + from(v, 1), four = two + from(two, 2);
        if constexpr (LPR == 5) return four + from(v, 4);
        if constexpr (LPR == 6) return four + from(two, 4);
        static_assert(LPR == 5 || LPR == 6 || LPR == 10 || (LPR & (LPR - 1)) == 0, "lanes of a row");
        const float eight = four + from(four, 4);
        return eight + from(two, 8);
    }
}

// V values over a scale as e4m3: their FP32 quotients to nearest even, those beyond the largest to
// that. A product with 1 / scale rounded once goes to the wrong side of ties (0.1708984375 / 7 is one),
// so the reciprocal is two numbers, hi <= 1 / scale and the rest: RN(a hi + RN(a lo)) is RN(x (1 + h))
// of the quotient x, |h| < 9 2^-49 (each part is off by 2^-24 of itself at most, lo < 2^-23 hi). That is
// x where x is an FP32 number, as all ties of e4m3 are; any other x is on the same side of a tie unless
// it is that close to the middle between the tie and an FP32 number beside it, as quotients of few
// numbers are: tests/test_heads_rules.py tries them all. Both parts are positive, so that infinities
// stay infinite. (32768 tokens' 8 keys and values of 128 BF16: 45 us, 43 by the product alone, 47 by a
// product corrected by its remainder, 70 by __fdiv_rn.)
// (Scales come last: the rotation of values near FP32's largest stays finite.)
template <int V>
__device__ __forceinline__ void st_e4m3(uint8_t* p, const float* a, const E4m3Scale& e) {
    if constexpr (V == 1) {
        *p = __nv_cvt_float_to_fp8(fmaf(a[0], e.hi, a[0] * e.lo), __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[(V + 3) / 4] = {};
        const F2 hi = f2s(e.hi), lo = f2s(e.lo);
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const F2 t = f2(a[k], a[k + 1]);
            float2 q;
            f2_get(fma2(t, hi, mul2(t, lo)), q.x, q.y);
            w[k / 4] |= (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3)
                        << (8 * (k % 4));
        }
        Raw<V> r;
#pragma unroll
        for (int k = 0; k < (V + 3) / 4; ++k) r.w[k] = w[k];
        st_raw<V>(p, r);
    }
}
// The same of V values as they are stored, which take the scale's power first. (FP16 ones need none:
// over scales that have one they are zero with or without it.)
template <typename T, int V>
__device__ __forceinline__ void st_e4m3_of(uint8_t* p, const Raw<V * (int)sizeof(T)>& r,
                                           const E4m3Scale& e) {
    float v[V];
    unpack<T, V>(v, r);
    if constexpr (!std::is_same<T, __half>::value) {
        if constexpr (V == 1) {
            v[0] *= e.power;
        } else {
#pragma unroll
            for (int k = 0; k < V; k += 2)
                f2_get(mul2(f2(v[k], v[k + 1]), f2s(e.power)), v[k], v[k + 1]);
        }
    }
    st_e4m3<V>(p, v, e);
}

// The unit of a warp: a token, a segment and its first head. Units of one segment lie together, so
// that the warps of a CTA take about the same time: token by token they left a CTA's place half
// empty beside its last warps (queries of 64 heads beside keys of 8).
struct HeadUnit {
    uint32_t token;
    int seg, head;
};
__device__ __forceinline__ HeadUnit head_unit(const HeadsParams& p, uint32_t unit) {
    // (a loop, though only two segments have units: from a choice of two the compiler selects every
    // field of theirs, which cost 32768 tokens' keys and values 5 us of 45)
    int seg = 0;
    while (seg < 2 && unit >= p.seg[seg].units) {
        unit -= p.seg[seg].units;
        ++seg;
    }
    const uint32_t t = fast_quot(unit, p.seg[seg].per);
    return {t, seg, (int)(unit - t * p.seg[seg].per.d) * p.per};
}

// A row's rotation and weights as two factors a value: y_j = r x_j A_j + r x_partner B_j, where the
// partner is the other value of j's pair: A = w c, B = -+ w_partner s. They are a token's, so that a
// row costs three packed products for two values. Values that are not turned have A alone. (r comes
// first, as in rms_fwd: r x stays within sqrt(d) whatever x and w.)
template <int V>
struct Factors {
    F2 a1[(V + 1) / 2], b1[(V + 1) / 2], a2[(V + 1) / 2], b2[(V + 1) / 2];   // first, second vector
};

__device__ __forceinline__ F2 swap2(F2 v) {
    float a, b;
    f2_get(v, a, b);
    return f2(b, a);
}

// Factors of a lane's pair of vectors, from weights w1, w2 and, where it is turned, the table's
// cosines c and sines s.
template <int V>
__device__ __forceinline__ void set_factors(Factors<V>& f, const float (&w1)[V], const float (&w2)[V],
                                            const float (&c)[V], const float (&s)[V], bool turned,
                                            bool interleaved) {
    if constexpr (V == 1) {
        f.a1[0] = f2(turned ? w1[0] * c[0] : w1[0], turned ? w2[0] * c[0] : w2[0]);
        f.b1[0] = f2(-(w2[0] * s[0]), w1[0] * s[0]);
        return;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const F2 u = f2(w1[2 * i], w1[2 * i + 1]), v = f2(w2[2 * i], w2[2 * i + 1]);
        if (!turned) {
            f.a1[i] = u;
            f.a2[i] = v;
        } else if (!interleaved) {
            const F2 cc = f2(c[2 * i], c[2 * i + 1]);
            f.a1[i] = mul2(u, cc);
            f.a2[i] = mul2(v, cc);
            f.b1[i] = mul2(v, f2(-s[2 * i], -s[2 * i + 1]));
            f.b2[i] = mul2(u, f2(s[2 * i], s[2 * i + 1]));
        } else {
            const float su = s[i], sv = s[V / 2 + i];
            f.a1[i] = mul2(u, f2s(c[i]));
            f.a2[i] = mul2(v, f2s(c[V / 2 + i]));
            f.b1[i] = mul2(f2(w1[2 * i + 1], w1[2 * i]), f2(-su, su));
            f.b2[i] = mul2(f2(w2[2 * i + 1], w2[2 * i]), f2(-sv, sv));
        }
    }
}

// x1, x2 := (r x) A + (r partner) B, or (r x) A where nothing is turned.
template <int V>
__device__ __forceinline__ void apply_factors(float (&x1)[V], float (&x2)[V], const Factors<V>& f,
                                              float r, bool turned, bool interleaved) {
    if constexpr (V == 1) {
        float a1, a2, b1, b2;
        f2_get(f.a1[0], a1, a2);
        f2_get(f.b1[0], b1, b2);
        const float t = r * x1[0], u = r * x2[0];
        x1[0] = turned ? t * a1 + u * b1 : t * a1;
        x2[0] = turned ? u * a2 + t * b2 : u * a2;
    } else {
        const F2 r2 = f2s(r);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const F2 u = mul2(f2(x1[i], x1[i + 1]), r2), v = mul2(f2(x2[i], x2[i + 1]), r2);
            F2 a = mul2(u, f.a1[i / 2]), b = mul2(v, f.a2[i / 2]);
            if (turned) {
                a = fma2(interleaved ? swap2(u) : v, f.b1[i / 2], a);
                b = fma2(interleaved ? swap2(v) : u, f.b2[i / 2], b);
            }
            f2_get(a, x1[i], x1[i + 1]);
            f2_get(b, x2[i], x2[i + 1]);
        }
    }
}

// A lane's share of a row's sum of squares.
template <int V, int CH>
__device__ __forceinline__ float squares(const float (&x1)[CH][V], const float (&x2)[CH][V]) {
    if constexpr (V == 1) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < CH; ++k) ss = fmaf(x1[k][0], x1[k][0], fmaf(x2[k][0], x2[k][0], ss));
        return ss;
    } else {
        F2 t = f2s(0.f);
#pragma unroll
        for (int k = 0; k < CH; ++k) {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const F2 u = f2(x1[k][i], x1[k][i + 1]), v = f2(x2[k][i], x2[k][i + 1]);
                t = fma2(u, u, t);
                t = fma2(v, v, t);
            }
        }
        float lo, hi;
        f2_get(t, lo, hi);
        return lo + hi;
    }
}

// Row groups that a warp copies ahead, in shared memory, where each lane reads what it copied
// itself (32768 tokens of 64 + 8 heads of 128 BF16: 182 us; rows loaded into registers 226): four,
// as deep as that gains anything; two where a lane holds more than 16 bytes of either half of a row
// (wide FP32 rows); one, in registers, where accesses are of 2 bytes (asynchronous copies take no fewer
// than 4). The append, whose groups are twice as large, copies three ahead at most.
template <typename T, int V, int CH>
constexpr int heads_ring() {
    return V * (int)sizeof(T) < 4 ? 1 : V * (int)sizeof(T) * CH <= 16 ? 4 : 2;
}

template <int B>
__device__ __forceinline__ Raw<B> ld_ring(const Raw<B>* p) {
    Raw<B> r;
    if constexpr (B == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        r.w[0] = v.x;
        r.w[1] = v.y;
        r.w[2] = v.z;
        r.w[3] = v.w;
    } else if constexpr (B == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r.w[0] = v.x;
        r.w[1] = v.y;
    } else {
        r.w[0] = p->w[0];
    }
    return r;
}
// B bytes (4, 8 or 16) to shared memory, without waiting.
template <int B>
__device__ __forceinline__ void copy_raw(Raw<B>* smem, const void* p) {
    if constexpr (B == 16)
        copy_async(smem, p);
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(smem)),
                     "l"(p), "n"(B)
                     : "memory");
}

// CTAs an SM holds at least: twelve, which spills 4 to 16 bytes in the append's kernels of 16-byte
// vectors of 16-bit rows and is the faster all the same (16384 tokens of 64 + 8 heads of 128 BF16 into
// 8 bits 102 us, 103 by ten without a spill); ten where the append's lanes hold two chunks of four
// values (8192 tokens of 16 + 4 heads of 512 FP32 126 us, 146 by twelve, which spill 36 to 60 bytes);
// eight where lanes hold more chunks.
template <int V, int CH, bool APPEND>
constexpr int heads_ctas() {
    return CH > 2 ? 8 : APPEND && CH == 2 && V == 4 ? 10 : 12;
}

// APPEND: keys (segment 1) go into the cache, at the token's slot, and with each the value of the same
// head (segment 2, which has no units of its own: 32768 tokens of 8 heads of 128, BF16 into 8 bits,
// without queries went from 52 us to 45 by that, with three groups ahead, 46 with four; 43 by later
// steps, 45 with quotients by the scales in place of products by their reciprocals). A warp
// takes p.per heads of its token, a row for each lane group at a time, with the next rows under way.
template <typename T, int V, int LPR, int CH, bool APPEND, bool E4M3>
__global__ void __launch_bounds__(kHeadsThreads, heads_ctas<V, CH, APPEND>())
    heads_fwd_kernel(const HeadsParams p) {
    constexpr int SG = 32 / LPR, B = V * (int)sizeof(T);
    constexpr int DEEP = heads_ring<T, V, CH>(), RING = APPEND && DEEP > 3 ? 3 : DEEP;
    constexpr int SIDES = APPEND ? 4 : 2;      // vectors of a group: a key's two, its value's two
    __shared__ __align__(16) Raw<B> ring[RING > 1 ? kHeadsWarps : 1][RING > 1 ? RING : 1]
                                        [RING > 1 ? SIDES * CH : 1][32];
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const uint32_t unit = blockIdx.x * kHeadsWarps + warp;
    if (unit >= p.total) return;
    const int lane = threadIdx.x & 31, l = lane % LPR, sg = lane / LPR;
    const HeadUnit u0 = head_unit(p, unit);
    const HeadSeg& S = p.seg[u0.seg];
    const bool key = APPEND && u0.seg == 1;
    const HeadSeg& W = p.seg[2];               // the values beside keys
    const int d = p.d[0], rp = p.rot / 2 / V;
    const int end = S.heads < u0.head + p.per ? S.heads : u0.head + p.per;
    // the lane group's token and head: where a token has few heads, a warp holds several tokens
    uint32_t token = u0.token, off = 0;
    int h = u0.head + sg;
    if (S.pack > 1) {
        off = fast_quot(sg, S.few);
        h = sg - off * S.few.d;
        token = u0.token * S.pack + off;
    }
    // (lanes behind the last row stand aside)
    const bool side = sg < SG && off < (uint32_t)S.pack && token < (uint32_t)p.tokens;
    if (!side) token = u0.token * S.pack;
    const uint32_t b = fast_quot(token, p.len), t = token - b * p.len.d;
    int lo[CH], hi[CH];
    bool in[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const int q = l + k * LPR;
        in[k] = 2 * q * V < d && side;
        pair_at<V>(q, rp, d, p.interleaved, lo[k], hi[k]);
    }
    const T* X = (const T*)S.x + b * S.xb + t * S.xt + h * S.xh;
    const T* Z = key ? (const T*)W.x + b * W.xb + t * W.xt + h * W.xh : nullptr;
    // the lane group's next row (and value): into the ring, or registers
    Raw<B> n1[CH], n2[CH], z1[CH], z2[CH];
    int ahead = h, put = 0, get = 0;
    auto load = [&]() {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const bool there = ahead < end && in[k];
            if (APPEND && key) {
                const int q = (l + k * LPR) * V, half = p.d[2] / 2;
                const bool beside = ahead < end && q < half && side;
                if constexpr (RING > 1) {
                    if (beside) {
                        copy_raw<B>(&ring[warp][put][SIDES * k + 2][lane], Z + q);
                        copy_raw<B>(&ring[warp][put][SIDES * k + 3][lane], Z + q + half);
                    }
                } else {
                    z1[k] = z2[k] = Raw<B>{};
                    if (beside) {
                        z1[k] = ld_raw<B>(Z + q);
                        z2[k] = ld_raw<B>(Z + q + half);
                    }
                }
            }
            if constexpr (RING > 1) {
                if (there) {
                    copy_raw<B>(&ring[warp][put][SIDES * k][lane], X + lo[k]);
                    copy_raw<B>(&ring[warp][put][SIDES * k + 1][lane], X + hi[k]);
                }
            } else {
                n1[k] = n2[k] = Raw<B>{};
                if (there) {
                    n1[k] = ld_raw<B>(X + lo[k]);
                    n2[k] = ld_raw<B>(X + hi[k]);
                }
            }
        }
        if constexpr (RING > 1) {
            copy_commit();
            put = put + 1 == RING ? 0 : put + 1;
        }
        ahead += SG;
        X += SG * S.xh;
        if (APPEND && key) Z += SG * W.xh;
    };
    pdl_wait();
    // All that does not wait for anything is under way before the first wait, the position's, for
    // the table's row.
    const bool norm = p.norm, eight = E4M3 && key;
    int64_t pos = 0, slot = 0;
    if (rp > 0) pos = ld_id(p.positions, token, p.itype);
    if (key) slot = ld_id(p.slots, token, p.itype);
#pragma unroll
    for (int k = 0; k < (RING > 1 ? RING - 1 : 1); ++k) load();
    Raw<B> wa[CH], wb[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        wa[k] = wb[k] = Raw<B>{};
        if (norm && S.w && in[k]) {
            wa[k] = ld_raw<B>((const T*)S.w + lo[k]);
            wb[k] = ld_raw<B>((const T*)S.w + hi[k]);
        }
    }
    bool there = true;
    Factors<V> f[CH];
    {
        const float* row = nullptr;
        if (rp > 0) {
            there = pos >= 0 && pos < p.table_rows;
            row = p.table + (there ? pos : 0) * p.ldt;
        }
        float c[CH][V], s[CH][V];
        ld_turn<V, CH, LPR>(c, s, row, l, rp, p.interleaved);
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            float w1[V], w2[V];
            unpack<T, V>(w1, wa[k]);
            unpack<T, V>(w2, wb[k]);
            if (!norm || !S.w) {
#pragma unroll
                for (int i = 0; i < V; ++i) w1[i] = w2[i] = 1.f;
            }
            if (p.back) {
#pragma unroll
                for (int i = 0; i < V; ++i) s[k][i] = -s[k][i];
            }
            set_factors<V>(f[k], w1, w2, c[k], s[k], l + k * LPR < rp, p.interleaved);
        }
    }
    int64_t at = b * S.yb + t * S.yt + h * S.yh, zat = 0;
    bool kept = true;
    if (key) {
        kept = slot >= 0 && slot < p.nslots;
        const uint32_t page = fast_quot((uint32_t)slot, p.page);
        const int64_t i = (uint32_t)slot - page * p.page.d;
        at = page * S.yb + i * S.yt + h * S.yh;
        zat = page * W.yb + i * W.yt + h * W.yh;
    }
    const float inv = 1.f / (float)d;
    for (int first = u0.head; first < end; first += SG, h += SG) {
        if constexpr (RING > 1) {
            load();
            copy_wait<RING - 1>();
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                n1[k] = n2[k] = Raw<B>{};
                if (h < end && in[k]) {       // (a lane reads what it copied itself)
                    n1[k] = ld_ring(&ring[warp][get][SIDES * k][lane]);
                    n2[k] = ld_ring(&ring[warp][get][SIDES * k + 1][lane]);
                }
            }
        }
        float a[CH][V], e[CH][V];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            unpack<T, V>(a[k], n1[k]);
            unpack<T, V>(e[k], n2[k]);
        }
        if (key && h < end && kept) {
            // the value, as it is or in 8 bits
            char* const Y = (char*)W.y + zat * (E4M3 ? 1 : (int)sizeof(T));
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const int q = (l + k * LPR) * V, half = p.d[2] / 2;
                if (q >= half || !side) continue;
                if constexpr (RING > 1) {
                    z1[k] = ld_ring(&ring[warp][get][SIDES * k + 2][lane]);
                    z2[k] = ld_ring(&ring[warp][get][SIDES * k + 3][lane]);
                }
                if constexpr (E4M3) {
                    st_e4m3_of<T, V>((uint8_t*)Y + q, z1[k], p.scale[2]);
                    st_e4m3_of<T, V>((uint8_t*)Y + q + half, z2[k], p.scale[2]);
                } else {
                    st_raw<B>((T*)Y + q, z1[k]);
                    st_raw<B>((T*)Y + q + half, z2[k]);
                }
            }
            zat += SG * W.yh;
        }
        if constexpr (RING == 1)
            load();
        else
            get = get + 1 == RING ? 0 : get + 1;
        float r = 1.f;
        if (norm) r = rsqrtf(fmaf(row_sum<LPR>(squares<V, CH>(a, e), lane), inv, p.eps));
        if (eight) r *= p.scale[1].power;
        if (h < end && kept) {
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                if (!in[k]) continue;
                const bool turned = l + k * LPR < rp;
                if (p.interleaved)
                    apply_factors<V>(a[k], e[k], f[k], r, turned, true);
                else
                    apply_factors<V>(a[k], e[k], f[k], r, turned, false);
                if (!there) {
#pragma unroll
                    for (int i = 0; i < V; ++i) a[k][i] = e[k][i] = 0.f;
                }
                if (eight) {
                    st_e4m3<V>((uint8_t*)S.y + at + lo[k], a[k], p.scale[1]);
                    st_e4m3<V>((uint8_t*)S.y + at + hi[k], e[k], p.scale[1]);
                } else {
                    st_elems<T, V>((T*)S.y + at + lo[k], a[k]);
                    st_elems<T, V>((T*)S.y + at + hi[k], e[k]);
                }
            }
        }
        at += SG * S.yh;
    }
    if constexpr (RING > 1) copy_wait<0>();
}

// The gradient. With g the transposed rotation of dy (sines negated) and r the row's, taken
// again from x:
//   dx_j = r (w_j g_j - x_j r^2 mean_k(w_k g_k x_k)),   dw_j = sum over rows of g_j x_j r.
// A lane meets the same columns in every row, so its shares of dw stay in registers over all the
// rows of a warp. A CTA works on one segment and writes one row of p.part, and heads_join_kernel
// adds those in a fixed order: no atomics, the same bits for the same sizes and grid. A warp goes
// through its units in turn, and its copies run ahead over their borders. (The forward kernel's warps
// have one unit each: with several, 32768 tokens of 64 + 8 heads of 128 BF16 took 187 us and not 184,
// since fewer of them even out less.)
template <typename T, int V, int CH>
constexpr int heads_bwd_smem(int d) {
    constexpr int WARPS = heads_bwd_warps(V, CH);
    const int ring = heads_ring<T, V, CH>() > 1
                         ? WARPS * heads_ring<T, V, CH>() * 4 * CH * 32 * V * (int)sizeof(T)
                         : 0;
    const int sums = WARPS * d * 4;
    return ring > sums ? ring : sums;
}

// PACK: a segment's units may be of several tokens, as the forward kernel's (15293 tokens of 2 + 2
// heads of 32 FP16: 10 us, 34 a token at a time). A form of its own, since what it keeps for that
// costs the others (32768 tokens of 32 + 8 heads of 80 BF16, 20 turned: 190 us with it, 176 without).
template <typename T, int V, int LPR, int CH, bool INTER, bool PACK>
__global__ void __launch_bounds__(heads_bwd_warps(V, CH) * 32, kHeadsBwdPerSm)
    heads_bwd_kernel(const HeadsParams p) {
    constexpr int SG = 32 / LPR, B = V * (int)sizeof(T), RING = heads_ring<T, V, CH>();
    constexpr int WARPS = heads_bwd_warps(V, CH);
    extern __shared__ uint4 shared[];      // the warps' rings; at the end their sums
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sg = lane / LPR;
    const int seg = (int)blockIdx.x >= p.first_k ? 1 : 0;
    const HeadSeg& S = p.seg[seg];
    const int d = p.d[0], rp = p.rot / 2 / V;
    const float inv = 1.f / (float)d;
    const uint32_t stride = (seg ? gridDim.x - p.first_k : p.first_k) * WARPS;
    uint32_t unit = (blockIdx.x - (seg ? p.first_k : 0)) * WARPS + warp;
    // the lane group's token of a unit and head of it, as in the forward kernel
    uint32_t off = 0;
    int mine = sg;
    if (PACK && S.pack > 1) {
        off = fast_quot(sg, S.few);
        mine = sg - off * S.few.d;
    }
    const bool side = sg < SG && (!PACK || off < (uint32_t)S.pack);
    auto token_of = [&](uint32_t unit) {
        if (!PACK) return fast_quot(unit, S.per);
        const uint32_t t = fast_quot(unit, S.per) * S.pack;
        return side && t + off < (uint32_t)p.tokens ? t + off : t;
    };
    auto live = [&](uint32_t unit) {
        return !PACK || (side && fast_quot(unit, S.per) * S.pack + off < (uint32_t)p.tokens);
    };
    int lo[CH], hi[CH];
    bool in[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const int q = l + k * LPR;
        in[k] = 2 * q * V < d && side;         // (lanes behind the last row stand aside)
        pair_at<V>(q, rp, d, INTER, lo[k], hi[k]);
    }
    Raw<B>* const ring = reinterpret_cast<Raw<B>*>(shared) + warp * (RING * 4 * CH * 32) + lane;
    // what is loaded next: its unit, the lane group's row, heads that are left
    uint32_t next = unit;
    const T *X = nullptr, *G = nullptr;
    int left = 0, put = 0, get = 0;
    bool held = true;                      // the lane group has a token of it
    Raw<B> x1[CH], x2[CH], g1[CH], g2[CH];
    auto enter = [&]() {
        const uint32_t token = token_of(next);
        const int head = (int)(next - fast_quot(next, S.per) * S.per.d) * p.per;
        const uint32_t b = fast_quot(token, p.len), t = token - b * p.len.d;
        left = S.heads - head < p.per ? S.heads - head : p.per;
        held = live(next);
        X = (const T*)S.x + b * S.xb + t * S.xt + (head + mine) * S.xh;
        G = (const T*)S.dy + b * S.gb + t * S.gt + (head + mine) * S.gh;
    };
    auto load = [&]() {
        const bool more = next < S.units;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const bool there = more && held && mine < left && in[k];
            if constexpr (RING > 1) {
                if (there) {
                    Raw<B>* const at = ring + (put * CH + k) * 128;
                    copy_raw<B>(at, X + lo[k]);
                    copy_raw<B>(at + 32, X + hi[k]);
                    copy_raw<B>(at + 64, G + lo[k]);
                    copy_raw<B>(at + 96, G + hi[k]);
                }
            } else {
                x1[k] = x2[k] = g1[k] = g2[k] = Raw<B>{};
                if (there) {
                    x1[k] = ld_raw<B>(X + lo[k]);
                    x2[k] = ld_raw<B>(X + hi[k]);
                    g1[k] = ld_raw<B>(G + lo[k]);
                    g2[k] = ld_raw<B>(G + hi[k]);
                }
            }
        }
        if constexpr (RING > 1) {
            copy_commit();
            put = put + 1 == RING ? 0 : put + 1;
        }
        X += SG * S.xh;
        G += SG * S.gh;
        left -= SG;
        if (left <= 0 && more) {
            next += stride;
            if (next < S.units) enter();
        }
    };
    pdl_wait();
    if (next < S.units) enter();
#pragma unroll
    for (int k = 0; k < (RING > 1 ? RING - 1 : 1); ++k) load();
    float da[CH][V], db[CH][V];
    Raw<B> wa[CH], wb[CH];      // (as they are stored: registers)
#pragma unroll
    for (int k = 0; k < CH; ++k) {
#pragma unroll
        for (int i = 0; i < V; ++i) da[k][i] = db[k][i] = 0.f;
        wa[k] = wb[k] = Raw<B>{};
        if (in[k] && S.w) {
            wa[k] = ld_raw<B>((const T*)S.w + lo[k]);
            wb[k] = ld_raw<B>((const T*)S.w + hi[k]);
        } else if (in[k]) {
            float ones[V];
#pragma unroll
            for (int i = 0; i < V; ++i) ones[i] = 1.f;
            wa[k] = wb[k] = pack<T, V>(ones);
        }
    }
    uint32_t token = token_of(unit);
    int64_t pos = rp > 0 && unit < S.units ? ld_id(p.positions, token, p.itype) : 0;
    while (unit < S.units) {
        const uint32_t group = PACK ? fast_quot(unit, S.per) : token;
        const int head = (int)(unit - group * S.per.d) * p.per;
        const bool holds = live(unit);
        const uint32_t b = fast_quot(token, p.len), t = token - b * p.len.d;
        const int rows = S.heads - head < p.per ? S.heads - head : p.per;
        int64_t at = b * S.yb + t * S.yt + (head + mine) * S.yh;
        const bool there = rp == 0 || (pos >= 0 && pos < p.table_rows);
        float c[CH][V], s[CH][V];
        ld_turn<V, CH, LPR>(c, s, p.table + (there ? pos : 0) * p.ldt, l, rp, INTER);
        unit += stride;
        token = token_of(unit);
        if (rp > 0 && unit < S.units) pos = ld_id(p.positions, token, p.itype);
        for (int h = mine; h - mine < rows; h += SG) {
            if constexpr (RING > 1) {
                load();
                copy_wait<RING - 1>();
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    x1[k] = x2[k] = g1[k] = g2[k] = Raw<B>{};
                    if (h < rows && holds && in[k]) {       // (a lane reads what it copied itself)
                        const Raw<B>* const at = ring + (get * CH + k) * 128;
                        x1[k] = ld_ring(at);
                        x2[k] = ld_ring(at + 32);
                        g1[k] = ld_ring(at + 64);
                        g2[k] = ld_ring(at + 96);
                    }
                }
                get = get + 1 == RING ? 0 : get + 1;
            }
            float u1[CH][V], u2[CH][V], v1[CH][V], v2[CH][V];     // x and g
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                unpack<T, V>(u1[k], x1[k]);
                unpack<T, V>(u2[k], x2[k]);
                unpack<T, V>(v1[k], g1[k]);
                unpack<T, V>(v2[k], g2[k]);
                if (l + k * LPR < rp) turn_back<V>(v1[k], v2[k], c[k], s[k], INTER);
            }
            if constexpr (RING == 1) load();
            const float ss = row_sum<LPR>(squares<V, CH>(u1, u2), lane);
            float dot = 0.f;
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                float w1[V], w2[V];
                unpack<T, V>(w1, wa[k]);
                unpack<T, V>(w2, wb[k]);
                dot += dots<V>(u1[k], u2[k], v1[k], v2[k], w1, w2);
            }
            dot = row_sum<LPR>(dot, lane);
            const float r = rsqrtf(ss * inv + p.eps);
            const float m = -(dot * inv * r * r);
            if (h < rows && holds) {
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    if (!in[k]) continue;
                    if (there) {
                        float w1[V], w2[V];
                        unpack<T, V>(w1, wa[k]);
                        unpack<T, V>(w2, wb[k]);
                        grads<V>(u1[k], v1[k], w1, da[k], r, m);
                        grads<V>(u2[k], v2[k], w2, db[k], r, m);
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) u1[k][i] = u2[k][i] = 0.f;
                    }
                    st_elems<T, V>((T*)S.y + at + lo[k], u1[k]);
                    st_elems<T, V>((T*)S.y + at + hi[k], u2[k]);
                }
            }
            at += SG * S.yh;
        }
    }
    if constexpr (RING > 1) copy_wait<0>();
    if (!p.part) return;
    // the warp's row groups, then the CTA's warps in order
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(shared);
    if constexpr ((LPR & (LPR - 1)) == 0) {
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
                    sums[warp * d + lo[k] + i] = da[k][i];
                    sums[warp * d + hi[k] + i] = db[k][i];
                }
            }
        }
    } else {
        static_assert(CH == 1, "rows of one chunk a lane");
        for (int g = 0; g < SG; ++g) {
            if (sg == g && in[0]) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float* const u = sums + warp * d + lo[0] + i;
                    float* const v = sums + warp * d + hi[0] + i;
                    *u = g ? *u + da[0][i] : da[0][i];
                    *v = g ? *v + db[0][i] : db[0][i];
                }
            }
            __syncwarp();
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < d; j += WARPS * 32) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += sums[w * d + j];
        p.part[(int64_t)blockIdx.x * d + j] = v;
    }
}

// The CTAs' rows into the weights' gradients: columns of queries from the first first_k rows, of
// keys from the others. Latency bounds it: 8 columns a CTA and 128 rows of them at a time, so that
// a thread has at most 19 rows, in two batches whose loads do not wait for one another; then the
// warp's four rows, then the warps in order.
constexpr int kJoinThreads = 1024;
constexpr int kJoinCols = 8;
constexpr int kJoinBatch = 10;     // rows a thread loads together
template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
    heads_join_kernel(const float* part, int d, int first_k, int ctas, T* dwq, T* dwk) {
    __shared__ float sums[kJoinThreads / 32][kJoinCols];
    const int per = (d + kJoinCols - 1) / kJoinCols;
    const bool key = (int)blockIdx.x >= per;
    const int col = ((int)blockIdx.x - (key ? per : 0)) * kJoinCols + threadIdx.x % kJoinCols;
    const int begin = key ? first_k : 0, end = key ? ctas : first_k;
    T* const out = key ? dwk : dwq;
    pdl_wait();
    if (!out) return;
    float v = 0.f;
    if (col < d) {
        constexpr int ROWS = kJoinThreads / kJoinCols;
        for (int r = begin + threadIdx.x / kJoinCols; r < end; r += kJoinBatch * ROWS) {
            float x[kJoinBatch];
#pragma unroll
            for (int u = 0; u < kJoinBatch; ++u)
                x[u] = r + u * ROWS < end ? __ldcg(part + (int64_t)(r + u * ROWS) * d + col) : 0.f;
#pragma unroll
            for (int u = 0; u < kJoinBatch; ++u) v += x[u];
        }
    }
#pragma unroll
    for (int o = kJoinCols; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int lane = threadIdx.x & 31;
    if (lane < kJoinCols) sums[threadIdx.x >> 5][lane] = v;
    __syncthreads();
    if (threadIdx.x < kJoinCols && col < d) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) t += sums[w][threadIdx.x];
        stt_y1(out + col, t);
    }
}

// ---- instances -----------------------------------------------------------------
// Calls f.run<V, LPR, CH>() for a shape, of those that head_shape gives for the direction.
template <typename T, bool BWD, typename F>
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
    if constexpr (V == 8) {
        if (sh.v == 4) {
            switch (sh.lpr) {
                case 4: return f.template run<4, 4, 1>();
                case 5: return f.template run<4, 5, 1>();
                case 6: return f.template run<4, 6, 1>();
                case 8: return f.template run<4, 8, 1>();
                case 10: return f.template run<4, 10, 1>();
                case 16: return f.template run<4, 16, 1>();
                default:
                    return sh.ch == 2 ? f.template run<4, 32, 2>() : f.template run<4, 32, 1>();
            }
        }
    }
    if (sh.v == 2) {
        if constexpr (BWD) {
            if (sh.lpr == 8) return f.template run<2, 8, 4>();
        } else {
            if (sh.ch == 1) return f.template run<2, 32, 1>();
        }
        return sh.lpr == 16 ? f.template run<2, 16, 4>() : f.template run<2, 32, 4>();
    }
    if constexpr (BWD) {
        if (sh.lpr == 16) return f.template run<1, 16, 4>();
        if (sh.ch == 4) return f.template run<1, 32, 4>();
    } else {
        if (sh.lpr == 16) return f.template run<1, 16, 8>();
        if (sh.ch == 2) return f.template run<1, 32, 2>();
    }
    return f.template run<1, 32, 8>();
}

template <typename T, bool APPEND, bool E4M3>
struct FwdRun {
    const HeadsParams& p;
    cudaStream_t s;
    template <int V, int LPR, int CH>
    cudaError_t run() {
        return launch_pdl(heads_fwd_kernel<T, V, LPR, CH, APPEND, E4M3>,
                          (p.total + kHeadsWarps - 1) / kHeadsWarps, kHeadsThreads, 0, s, p);
    }
};
template <typename T>
struct BwdRun {
    const HeadsParams& p;
    int ctas;
    cudaStream_t s;
    template <int V, int LPR, int CH, bool INTER, bool PACK>
    cudaError_t launch() {
        const auto kernel = heads_bwd_kernel<T, V, LPR, CH, INTER, PACK>;
        const int smem = heads_bwd_smem<T, V, CH>(p.d[0]);
        constexpr int MOST = heads_bwd_smem<T, V, CH>((int)kMaxHeadDim);
        if constexpr (MOST > 48 * 1024) {
            // (an attribute of the function in a context)
            static thread_local unsigned long long done = 0;
            unsigned long long ctx = 0;
            cudaError_t err = current_context_id(&ctx);
            if (err == cudaSuccess)
                err = once_in_context(ctx, done, [&] {
                    return cudaFuncSetAttribute(
                        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
                });
            if (err != cudaSuccess) return err;
        }
        return launch_pdl(kernel, (unsigned)ctas, heads_bwd_warps(V, CH) * 32, smem, s, p);
    }
    template <int V, int LPR, int CH>
    cudaError_t run() {
        if constexpr (LPR <= 16)           // (a warp holds several rows)
            if (p.seg[0].pack > 1 || p.seg[1].pack > 1)
                return p.interleaved ? launch<V, LPR, CH, true, true>()
                                     : launch<V, LPR, CH, false, true>();
        return p.interleaved ? launch<V, LPR, CH, true, false>()
                             : launch<V, LPR, CH, false, false>();
    }
};

template <typename T, bool APPEND, bool E4M3>
cudaError_t heads_fwd_t(HeadShape sh, const HeadsParams& p, cudaStream_t s) {
    return for_shape<T, false>(sh, FwdRun<T, APPEND, E4M3>{p, s});
}
template <typename T>
cudaError_t heads_bwd_t(HeadShape sh, const HeadsParams& p, int ctas, void* dwq, void* dwk,
                        cudaStream_t s) {
    const cudaError_t err = for_shape<T, true>(sh, BwdRun<T>{p, ctas, s});
    if (err != cudaSuccess || !p.part) return err;
    return launch_pdl(heads_join_kernel<T>, 2 * ((p.d[0] + kJoinCols - 1) / kJoinCols),
                      kJoinThreads, 0, s, (const float*)p.part, p.d[0], p.first_k, ctas, (T*)dwq,
                      (T*)dwk);
}

}  // namespace rn
