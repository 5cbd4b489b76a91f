// rn_logprob.cuh -- log probabilities over rows of logits.
//
// With x_j = scale * logit_j and any reference c,
//     S = sum_j e^{x_j - c},  W = sum_j e^{x_j - c} (x_j - c):
//     lse = c + log S,   log p_t = (x_t - c) - log S,   H = log S - W / S.
// One pass: every thread keeps a running (c, S, W) over the batches of 16 or 32
// elements it reads, c near the largest element it has seen (both terms of H are
// then >= 0 and nothing cancels). A batch that raises c from c0 to c1 rescales,
// with r = c0 - c1 <= 0,
//     S <- S e^r,  W <- e^r (W + r S).
// Exponents are kept in units of log 2: z = logit * (scale * log2 e) - c is one
// fused multiply-add, whose constant c need not equal the largest element's product
// exactly (it is a reference, and the same in every term), and e^z one
// special-function instruction. Pairs of elements go through the packed FP32
// pipe: 4 instructions a pair beside the two exponentials, so that the pass
// stays below the time its bytes take even for 16-bit logits: 8192 x 128000 BF16 with
// entropies 296 us, a little above the measured copy's rate over its 2.1 GB (608 us with scalar
// arithmetic, a test of every element for -inf and two CTAs of 512 threads an SM; four of 256 let
// one row's end overlap another's reading).
//
// Where there is more to do than sums, a thread keeps the next two batches under way into shared
// memory, 32 KB a CTA, so that the memory does not wait for a row's barriers and alternatives: a
// thread copies its own vectors and needs no barrier for them. 2048 x 128000 BF16 with entropies
// 86 us by loads into registers, this way 82; with 8 alternatives too 108, 91 (with what is
// below). Sums alone are better off without: 700 x 128000 30 us, this way 37. (CTAs that go on to
// further rows, with the next one's batches under way: 2048 x 128000 with 8 alternatives 111 us,
// where one row each took 106: rows are handed out more evenly.)
//
// A masked element (-inf) gives e = 0, and 0 * -inf would be NaN in W: where entropies are
// wanted, elements are held at -1e30 or above (NaN passes), where e is 0 as well: one packed
// instruction a pair of BF16 (summing masked batches twice instead: 2048 x 128000 BF16, a fifth
// masked, 20 alternatives 157 us, this way 124 us). A row whose largest product is beyond 2^24
// (every column at a mask's lowest value, say) cannot be referred to c in FP32: it is
// summed again, from differences of logits (row_again), by one CTA and an element an access: 2048 x
// 128000 BF16 of the lowest value 281 us, where ordinary rows take 81; one such row among them 119.
//
// A row is split over the CTAs of a cluster where there are few rows; the
// CTAs' results meet in the first one's shared memory (one row of 128000 FP32 3.0 us, of
// which the launch is about 2, 6.6 with 20 alternatives; 64 x 50001 BF16 5.3 and 9.8 us).
//
// Alternatives: the `top` largest logits, the lowest index first among equal
// ones, found in the same pass. A candidate is a 64-bit key: the value's bits in
// an order-preserving form above the complement of its index, so that keys
// differ and compare as wanted. Each warp keeps its newest candidates in shared
// memory and, past 31 of them, its 32 best, sorted, in its lanes, and a new one has to exceed the
// threshold `thr`, below which the row's `top` best cannot lie. It comes from groups of
// threads: the top-th largest of the groups' maxima so far, since at least `top` elements
// reach it. It is taken after the first two batches, before either is looked at, then each time
// the columns read have doubled, so that about `top` candidates are met between two of them (with
// the first threshold alone 2048 x 128000 BF16 with 8 alternatives took 139 us where it then took
// 101; the first one after one batch: 94 us, not 91, with 32 alternatives 130, not 117). Past the
// first, no barrier is needed: maxima only grow, and a stale one is a lower bound too. So is the
// top-th of what a warp keeps. A batch without a candidate costs a comparison of its maximum, which
// is there anyway; in one with a candidate, the warp looks at the elements of the lane that has it,
// an element a lane, where they lie in shared memory. At the end the keys that reach the last
// threshold, of all warps, go into one list: mostly one or two warps' sorts (every warp sorting and
// keeping 32, then merging 8 lists: 8 alternatives 106 us, this way 95 at the time). The order in
// which warps run changes which keys are tried, not which are kept.
// What alternatives cost now is instructions: a row of 128000 BF16 takes 28000 warp instructions
// with its entropy, 38000 with 8 alternatives as well and 51000 with 32 (82, 91, 117 us for 2048).
// Rows in which most elements equal the largest are the slowest, since every one of those is a
// candidate until its column decides: 2048 x 128000 BF16 of one value 538 us with 8.
#pragma once

#include <type_traits>

#include "rn_tokens.cuh"

namespace rn {

constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpStages = 2;         // batches a thread has under way
constexpr int kTopCap = 64;          // candidates a warp holds unsorted: 31 and 32 more
constexpr int kTopGroups = 64;
constexpr float kRef = 16777216.f;  // references stay within 2^24: their rounding is below 1
constexpr float kHeld = -1e30f;      // logits are held at this or above where entropies are wanted
static_assert(kMaxTop == 32, "a lane for each alternative");

// Bits of x in an order that compares as unsigned integers do: -inf lowest, both
// zeros equal, any NaN highest.
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

// The largest of the N elements held in raw vectors of T (NaN left out). 16-bit
// elements are compared in pairs before they are widened.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __nv_bfloat16*) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __half*) {
    const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&a),
                              *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}
template <typename T>
__device__ __forceinline__ float raw_max(const Raw<16>* r) {
    if constexpr (sizeof(T) == 4) {
        float m = __uint_as_float(r[0].w[0]);
#pragma unroll
        for (int u = 0; u < kLpU; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, __uint_as_float(r[u].w[i]));
        return m;
    } else {
        uint32_t m = r[0].w[0];
#pragma unroll
        for (int u = 0; u < kLpU; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max2(m, r[u].w[i], (T*)nullptr);
        float a, b;
        unpack2(m, a, b, (T*)nullptr);
        return fmaxf(a, b);
    }
}
template <typename T>
constexpr uint32_t raw_low() {   // -inf in every element
    return sizeof(T) == 4 ? 0xff800000u
                          : (std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u);
}

// Logits held at -1e30 or above, NaN kept: a pair of BF16, or an FP32 value.
__device__ __forceinline__ uint32_t hold2(uint32_t w) {
    uint32_t o;   // 0xf14a is BF16's -1e30
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(w), "r"(0xf14af14au));
    return o;
}
__device__ __forceinline__ float hold1(float x) {
    float o;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(x), "f"(kHeld));
    return o;
}

// Pair i of the raw vectors.
template <typename T, bool HOLD>
__device__ __forceinline__ F2 raw_pair(const Raw<16>* r, int i) {
    float a, b;
    if constexpr (sizeof(T) == 4) {
        a = __uint_as_float(r[i / 2].w[i % 2 * 2]);
        b = __uint_as_float(r[i / 2].w[i % 2 * 2 + 1]);
    } else {
        uint32_t w = r[i / 4].w[i % 4];
        if constexpr (HOLD && std::is_same<T, __nv_bfloat16>::value) w = hold2(w);
        unpack2(w, a, b, (T*)nullptr);
    }
    // (FP16's own lowest value is an ordinary logit: held as FP32)
    if constexpr (HOLD && !std::is_same<T, __nv_bfloat16>::value) {
        a = hold1(a);
        b = hold1(b);
    }
    return f2(a, b);
}

// Running (c, S, W) with the largest logit m; k = scale * log2(e).
template <bool ENT>
struct Soft {
    float m, c, s, w;
    __device__ __forceinline__ void init() {
        m = -INFINITY;
        c = -kRef;
        s = 0.f;
        w = 0.f;
    }
    __device__ __forceinline__ void rescale(float c1) {
        const float r = c - c1, f = ex2(r);
        if constexpr (ENT) w = f * fmaf(r, s, w);
        s *= f;
        c = c1;
    }
    __device__ __forceinline__ void reach(float mx, float k) {
        if (mx > m) {
            m = mx;
            rescale(fminf(fmaxf(mx * k, -kRef), kRef));
        }
    }
    // one element
    __device__ __forceinline__ void add(float x, float k) {
        reach(x, k);
        const float z = fmaf(x, k, -c), e = ex2(z);
        s += e;
        if constexpr (ENT) w += e != 0.f ? e * z : 0.f;
    }
    // a batch of raw vectors of T whose maximum is mx
    template <typename T>
    __device__ __forceinline__ void add(const Raw<16>* r, float mx, float k) {
        constexpr int NP = kLpU * Elem<T>::kVec / 2;
        reach(mx, k);
        F2 s2 = f2s(0.f), w2 = f2s(0.f);
        // (nothing above -inf yet: any reference but -kRef, above which a tiny scale might
        // lift held values)
        const F2 k2 = f2s(k), c2 = f2s(m == -INFINITY ? 0.f : -c);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const F2 z = fma2(raw_pair<T, ENT>(r, i), k2, c2);
            float z0, z1;
            f2_get(z, z0, z1);
            const F2 e = f2(ex2(z0), ex2(z1));
            s2 = add2(s2, e);
            if constexpr (ENT) w2 = fma2(e, z, w2);
        }
        float a, b;
        f2_get(s2, a, b);
        s += a + b;
        if constexpr (ENT) {
            f2_get(w2, a, b);
            w += a + b;
        }
    }
    __device__ __forceinline__ void merge(float m2, float c2, float s2, float w2) {
        m = fmaxf(m, m2);
        const float c1 = fmaxf(c, c2);
        const float r1 = c - c1, r2 = c2 - c1, f1 = ex2(r1), f2 = ex2(r2);
        if constexpr (ENT) w = f1 * fmaf(r1, s, w) + f2 * fmaf(r2, s2, w2);
        s = f1 * s + f2 * s2;
        c = c1;
    }
};

// Candidates of a CTA.
struct TopState {
    unsigned long long cand[kLpWarps][kTopCap];
    unsigned long long list[kLpMaxCluster][32];   // sorted lists of 32: the warps', the CTAs'
    unsigned long long thr;
    float group[kTopGroups];
    int found;                       // keys in `list`, before it is sorted
};
static_assert(kLpWarps * (kTopCap - 1) <= kLpMaxCluster * 32, "TopState::list");

// Sorting networks over a warp's lanes, largest first, a value a lane: the last stage
// orders a bitonic sequence, and all of them any sequence. Two sorted lists a and b
// become the sorted 32 best of both by max(a[i], b[31 - i]) and a last stage.
template <typename K>
__device__ __forceinline__ K sort_stage(K v, int n, int lane) {
#pragma unroll
    for (int o = n / 2; o > 0; o >>= 1) {
        const K h = __shfl_xor_sync(0xffffffffu, v, o);
        const bool larger = ((lane & o) == 0) == ((lane & n) == 0);
        v = (h > v) == larger ? h : v;
    }
    return v;
}
template <typename K>
__device__ __forceinline__ K warp_sort(K v, int lane) {
#pragma unroll
    for (int n = 2; n <= 32; n <<= 1) v = sort_stage(v, n, lane);
    return v;
}
template <typename K>
__device__ __forceinline__ K warp_merge(K a, K b, int lane) {
    const K r = __shfl_sync(0xffffffffu, b, 31 - lane);
    return sort_stage(r > a ? r : a, 32, lane);
}

// The n (a power of two, at most twice the warps) lists of st.list, merged into the first.
// All threads; the lists are written and a barrier passed before.
__device__ __forceinline__ void merge_lists(TopState& st, int n, int w, int lane) {
    for (int h = n / 2; h > 0; h /= 2) {
        if (w < h) st.list[w][lane] = warp_merge(st.list[w][lane], st.list[w + h][lane], lane);
        __syncthreads();
    }
}

// The values of a row that FP32 products cannot be referred to (see above), from
// differences of logits: (log S, W / S in units of log 2). All threads. (By the scale first: log2 e
// times a scale above 2.36e38 is infinite, and 0 times that would be NaN.)
template <typename T>
__device__ void row_again(const T* X, int V, float scale, float m, float (*red)[4], float* ls,
                          float* ws) {
    const int t = threadIdx.x, w = t >> 5, lane = t & 31;
    float s = 0.f, q = 0.f;
    for (int i = t; i < V; i += kLpThreads) {
        const float z = scaled_diff(ldt_x1(X + i), m, scale) * kLog2e, e = ex2(z);
        s += e;
        if (e != 0.f) q = fmaf(e, z, q);
    }
    s = warp_sum(s);
    q = warp_sum(q);
    __syncthreads();
    if (lane == 0) {
        red[w][0] = s;
        red[w][1] = q;
    }
    __syncthreads();
    s = q = 0.f;
    for (int i = 0; i < kLpWarps; ++i) {
        s += red[i][0];
        q += red[i][1];
    }
    *ls = logf(s);
    *ws = q / s;
}

template <typename T, bool ENT, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 4) logprob_fwd_kernel(const LogprobParams p) {
    constexpr int VEC = Elem<T>::kVec;
    constexpr int NB = kLpU * VEC;    // elements of a batch, at most 32
    __shared__ float red[kLpWarps][4];
    __shared__ float parts[kLpMaxCluster][4];     // in a row's first CTA: every CTA's sums
    __shared__ unsigned long long tops[TOP ? kLpMaxCluster : 1][kMaxTop];   // and candidates
    __shared__ TopState st;
    // batches under way: a thread copies vectors for itself (and, of a batch with a candidate, the
    // warp reads the lane's)
    constexpr bool RING = ENT || TOP;
    __shared__ __align__(16) uint4 ring[RING ? kLpStages : 1][kLpU][RING ? kLpThreads : 1];
    pdl_launch_dependents();
    if (p.split > 1) cluster_arrive();            // (the peers write here: see below)
    const int t = threadIdx.x, w = t >> 5, lane = t & 31;
    const float k = p.scale * kLog2e;
    const int V = p.vocab;
    const int64_t row = blockIdx.x / (unsigned)p.split;
    const int rank = (int)(blockIdx.x - (unsigned)row * p.split);
    // this CTA's share of the row: vectors [va, vb), and the first also the
    // elements before the first 16-byte boundary and after the last vector
    const T* const X = (const T*)p.logits + row * p.ld;
    const int head = head_peel_t(X, V);
    const int nv = (V - head) / VEC;
    const int tail0 = head + nv * VEC;
    const int share = (nv + p.split - 1) / p.split;
    const int va = min(nv, rank * share), vb = min(nv, va + share);
    const T* const XV = X + head;
    const int extra = rank == 0 ? head + (V - tail0) : 0;
    Soft<ENT> a;
    a.init();
    int cnt = 0;                       // this warp's candidates
    if constexpr (TOP) {
        if (t == 0) {
            st.thr = 0;
            st.found = 0;
        }
    }
    pdl_wait();
    unsigned long long thr = 0;
    float lo = order_value(0);            // thr's value when last looked at
    unsigned long long kept = 0;          // this warp's 32 best so far, a lane each
    // The first 32 of the warp's candidates (fewer: the rest are 0) into `kept`.
    auto keep = [&]() {
        __syncwarp();
        const unsigned long long v = lane < cnt ? st.cand[w][lane] : 0;
        kept = warp_merge(kept, warp_sort(v, lane), lane);
        // (0 while there are fewer than `top`)
        thr = max(thr, __shfl_sync(0xffffffffu, kept, p.top - 1));
        const unsigned long long rest = 32 + lane < cnt ? st.cand[w][32 + lane] : 0;
        __syncwarp();
        st.cand[w][lane] = rest;
        cnt = cnt > 32 ? cnt - 32 : 0;
    };
    // Keys of this warp's lanes, where they exceed the threshold.
    auto append = [&](bool ok, float x, uint32_t col) {
        const unsigned long long key = ok ? top_key(x, col) : 0;
        const bool put = key > thr;
        const unsigned who = __ballot_sync(0xffffffffu, put);
        if (put) st.cand[w][cnt + __popc(who & ((1u << lane) - 1))] = key;
        cnt += __popc(who);
        if (cnt >= 32) {
            keep();
            if (lane == 0) atomicMax(&st.thr, thr);
        }
    };
    // This thread's maximum so far, to its group's.
    constexpr int kGroup = kLpThreads / kTopGroups;
    volatile float* const groups = st.group;
    auto tell = [&]() {
        float g = a.m;
#pragma unroll
        for (int o = 1; o < kGroup; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
        if (t % kGroup == 0) groups[t / kGroup] = g;
    };
    // The threshold from the groups' maxima: a warp sorts them. (32 groups twice the size do
    // for few alternatives; for 32 the least of 32 maxima would let 130 elements a
    // doubling pass, that of 64 lets 44.) A key without an index: every element of this
    // value is above it.
    auto raise = [&]() {
        float g = groups[lane];
        const float h = groups[32 + lane];
        if (p.top > 16)
            g = warp_merge(warp_sort(g, lane), warp_sort(h, lane), lane);
        else
            g = warp_sort(fmaxf(g, h), lane);
        g = __shfl_sync(0xffffffffu, g, p.top - 1);
        if (g > -INFINITY) thr = max(thr, (unsigned long long)order_bits(g) << 32);
        lo = order_value((uint32_t)(thr >> 32));
    };
    constexpr int kStep = kLpThreads * kLpU;
    int turn = 0;                         // batches read
    // The batch at v0, by this thread; all but a row's last are whole, and done without tests.
    const T* const mine = XV + (int64_t)t * VEC;
    auto ask = [&](int to, int v0) {
        uint4* const q = &ring[to][0][t];
        const T* const x = mine + (int64_t)v0 * VEC;
        if (v0 + kStep <= vb) {
#pragma unroll
            for (int u = 0; u < kLpU; ++u) copy_async(q + u * kLpThreads, x + u * kLpThreads * VEC);
        } else {
#pragma unroll
            for (int u = 0; u < kLpU; ++u)
                if (v0 + u * kLpThreads + t < vb)
                    copy_async(q + u * kLpThreads, x + u * kLpThreads * VEC);
        }
        copy_commit();
    };
    auto vector = [&](int v0, int u, int from) {
        if constexpr (RING) {
            const uint4 q = ring[from][u][t];
            return Raw<16>{{q.x, q.y, q.z, q.w}};
        } else {
            return ld_raw<16>(mine + (int64_t)(v0 + u * kLpThreads) * VEC);
        }
    };
    // The sums of the batch at v0 (in slot `from`), which gives its maximum.
    Raw<16> r[kLpU];
    auto sum = [&](int v0, int from) {
        if (RING && v0 + kStep <= vb) {
#pragma unroll
            for (int u = 0; u < kLpU; ++u) r[u] = vector(v0, u, from);
        } else {
#pragma unroll
            for (int u = 0; u < kLpU; ++u) {
                constexpr uint32_t low = raw_low<T>();
                r[u] = v0 + u * kLpThreads + t < vb ? vector(v0, u, from)
                                                    : Raw<16>{{low, low, low, low}};
            }
        }
        const float mx = raw_max<T>(r);
        a.template add<T>(r, mx, k);
        return mx;
    };
    // Candidates of the batch at v0 in slot `from`, whose maxima are mx.
    auto look = [&](float mx, int v0, int from) {
        // (equal values may be wanted, a NaN always is; a threshold of 0 is a NaN)
        const bool odd = a.s != a.s;
        unsigned lanes = __ballot_sync(0xffffffffu, !(mx < lo) || odd);
        if (!lanes) return;
        // with the other warps' threshold?
        thr = max(thr, *(volatile unsigned long long*)&st.thr);
        lo = order_value((uint32_t)(thr >> 32));
        lanes = __ballot_sync(0xffffffffu, !(mx < lo) || odd);
        if (!lanes) return;
        __syncwarp();                             // (every lane's copies have arrived)
        // this lane's element of the first lane's batch, and its vector
        const T* const e = (const T*)&ring[from][lane % NB / VEC][w * 32] + lane % VEC;
        const int v = v0 + lane % NB / VEC * kLpThreads + w * 32;
        const int end = lane < NB ? vb - v : 0;
        const uint32_t col = (uint32_t)(head + v * VEC + lane % VEC);
        do {
            const int at = __ffs(lanes) - 1;
            lanes &= lanes - 1;
            append(at < end, lds_f(e + at * VEC), col + (uint32_t)at * VEC);
        } while (lanes);
        __syncwarp();
    };
    int v0 = va, slot = 0;
    if constexpr (RING) {
        static_assert(kLpStages == 2, "the loop below");
        ask(0, va);
        ask(1, va + kStep);
    }
    if constexpr (TOP) {
        // the first threshold is that of two batches, which are looked at after it
        if (va < vb) {
            copy_wait<1>();
            const float m0 = sum(va, 0);
            copy_wait<0>();
            const float m1 = sum(va + kStep, 1);
            tell();
            __syncthreads();                      // (and st.thr and st.found are set)
            raise();
            look(m0, va, 0);
            ask(0, va + 2 * kStep);
            look(m1, va + kStep, 1);
            ask(1, va + 3 * kStep);
            turn = 2;
            v0 = va + 2 * kStep;
        }
    }
    for (; v0 < vb; v0 += kStep) {
        if constexpr (RING) copy_wait<1>();
        const float mx = sum(v0, slot);
        if constexpr (TOP) {
            if ((turn & (turn + 1)) == 0) {       // 4, 8, ... batches read
                tell();
                if (w == (turn & (kLpWarps - 1))) {
                    raise();
                    if (lane == 0) atomicMax(&st.thr, thr);
                }
            }
            ++turn;
            look(mx, v0, slot);
        }
        if constexpr (RING) {
            ask(slot, v0 + 2 * kStep);
            slot ^= 1;
        }
    }
    // head and tail: fewer than 2 * VEC elements, one a thread
    if (t / 32 * 32 < extra) {
        const bool in = t < extra;
        const int c = t < head ? t : tail0 + t - head;
        float x = -INFINITY;
        if (in) x = ldt_x1(X + c);
        a.add(x, k);
        if constexpr (TOP) append(in, x, (uint32_t)c);
    }
    // meet: lanes, warps, the CTAs of the cluster
    auto meet = [&](int lanes) {
        for (int o = lanes / 2; o > 0; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, a.m, o);
            const float c2 = __shfl_xor_sync(0xffffffffu, a.c, o);
            const float s2 = __shfl_xor_sync(0xffffffffu, a.s, o);
            const float w2 = __shfl_xor_sync(0xffffffffu, a.w, o);
            a.merge(m2, c2, s2, w2);
        }
    };
    auto take = [&](const float* v) {
        a.m = v[0];
        a.c = v[1];
        a.s = v[2];
        a.w = v[3];
    };
    meet(32);
    if (lane == 0) {
        red[w][0] = a.m;
        red[w][1] = a.c;
        red[w][2] = a.s;
        red[w][3] = a.w;
    }
    if constexpr (TOP) {
        // the keys that are left, of all warps, into one list
        if (turn == 0) __syncthreads();           // (st.found is set)
        __syncwarp();
        const unsigned long long least = max(thr, *(volatile unsigned long long*)&st.thr);
        const unsigned long long fresh = lane < cnt ? st.cand[w][lane] : 0;
        const bool put1 = fresh != 0 && fresh >= least, put2 = kept != 0 && kept >= least;
        const unsigned who1 = __ballot_sync(0xffffffffu, put1);
        const unsigned who2 = __ballot_sync(0xffffffffu, put2);
        int at = 0;
        if (lane == 0) at = atomicAdd(&st.found, __popc(who1) + __popc(who2));
        at = __shfl_sync(0xffffffffu, at, 0);
        const unsigned below = (1u << lane) - 1;
        unsigned long long* const all = st.list[0];
        if (put1) all[at + __popc(who1 & below)] = fresh;
        if (put2) all[at + __popc(who1) + __popc(who2 & below)] = kept;
    }
    __syncthreads();
    take(red[lane % kLpWarps]);
    meet(kLpWarps);
    if constexpr (TOP) {
        // 32 at a time are sorted, and the lists merged
        const int found = st.found;
        int lists = 1;
        while (lists * 32 < found) lists *= 2;
        for (int q = w; q < lists; q += kLpWarps) {
            const int i = q * 32 + lane;
            const unsigned long long v = warp_sort(i < found ? st.list[q][lane] : 0ull, lane);
            st.list[q][lane] = v;
        }
        __syncthreads();
        merge_lists(st, lists, w, lane);
    }
    if (p.split > 1) {
        // every CTA leaves its results in the first one's shared memory, once that has started
        cluster_wait();
        if (t < 4) peer_store(peer_addr(&parts[rank][t], 0), t == 0   ? a.m
                                                             : t == 1 ? a.c
                                                             : t == 2 ? a.s
                                                                      : a.w);
        if constexpr (TOP) {
            // (a CTA with fewer columns leaves keys of 0)
            if (t < 32) peer_store(peer_addr(&tops[rank][t], 0), st.list[0][t]);
        }
        cluster_arrive();
        if (rank != 0) return;
        cluster_wait();
        take(parts[lane % p.split]);
        meet(p.split);
        if constexpr (TOP) {
            for (int q = w; q < p.split; q += kLpWarps) st.list[q][lane] = tops[q][lane];
            __syncthreads();
            merge_lists(st, p.split, w, lane);
        }
    }
    // (a scale with which kHeld is not far below every other product, or beyond FP32's
    // range: the sums say nothing, and the row is summed again)
    const bool odd = !(k > 1e-20f && k < 1e8f) && a.m > -INFINITY;
    bool nan = a.s != a.s && !odd;                  // (odd: row_again's own sum says)
    const bool none = a.m == -INFINITY && !nan;     // every logit is -inf
    const float ref = a.m * p.scale;
    float ls = logf(a.s), ws = a.w / a.s;
    const bool far = !nan && !none && fabsf(a.m) < INFINITY &&
                     (odd || !(fabsf(a.m * k) < kRef && fabsf(a.m) < -0.1f * kHeld));
    if (far) {
        row_again<T>(X, V, p.scale, a.m, red, &ls, &ws);
        nan = ls != ls;
    }
    // log p of a logit
    auto logp = [&](float x) {
        if (nan || a.m == INFINITY) return __uint_as_float(0x7fffffffu);
        if (none || x == -INFINITY) return -INFINITY;
        if (far) return scaled_diff(x, a.m, p.scale) - ls;
        // (a mask's lowest value, times k, may be beyond FP32's range)
        return (fabsf(x * k) < kRef ? fmaf(x, k, -a.c) * kLn2 : x * p.scale - ref) - ls;
    };
    if (t == 0) {
        const float bad = __uint_as_float(0x7fffffffu);
        const bool spoilt = nan || a.m == INFINITY;
        if (p.lse) {
            // The largest product with what its rounding left off, and log S referred to it rather
            // than to c, which is m k rounded: one rounding of a large number in all. (c ln 2 + log S
            // has two more, and was off by 2.8e-4 at 3900, where half a step is 1.2e-4.)
            const float left = fmaf(a.m, p.scale, -ref);
            const float log_s = far ? ls : ls - fmaf(a.m, k, -a.c) * kLn2;
            const float lse = fabsf(ref) < INFINITY ? ref + (log_s + left) : ref;
            p.lse[row] = spoilt ? bad : none ? -INFINITY : lse;
        }
        if (ENT) p.entropy[row] = spoilt ? bad : none ? 0.f : ls - ws * kLn2;
        if (p.logp) {
            const int64_t id = ld_id(p.targets, row, p.itype);
            p.logp[row] = id >= 0 && id < V ? logp(ldt_x1(X + id)) : 0.f;
        }
    }
    if constexpr (TOP) {
        if (t < p.top) {
            const unsigned long long key = st.list[0][t];
            const uint32_t idx = ~(uint32_t)key;
            if (p.top_ids) {
                if (p.itype == IT_I64)
                    ((int64_t*)p.top_ids)[row * p.top + t] = idx;
                else
                    ((int32_t*)p.top_ids)[row * p.top + t] = (int32_t)idx;
            }
            if (p.top_logp) p.top_logp[row * p.top + t] = logp(order_value((uint32_t)(key >> 32)));
        }
    }
}

template <typename T, bool ENT, bool TOP>
static cudaError_t logprob_fwd_go(const LogprobParams& q, cudaStream_t s) {
    LogprobParams p = q;
    auto* kernel = logprob_fwd_kernel<T, ENT, TOP>;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    p.split = logprob_split(p.rows, p.vocab, Elem<T>::kVec, sms, kLpMaxCluster);
    if (p.split > 1) {
        // clusters of more than 8 CTAs have to be asked for, and may not fit: once in each context,
        // by each thread
        static thread_local unsigned long long prepared = 0;
        static thread_local int most = 1;
        unsigned long long ctx = 0;
        err = current_context_id(&ctx);
        if (err == cudaSuccess)
            err = once_in_context(ctx, prepared, [&] {
                const cudaError_t e =
                    cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
                if (e == cudaSuccess)
                    most = placeable_cluster(kLpMaxCluster, [&](int c) {
                        return resident_clusters((const void*)kernel, c, kLpThreads, 0);
                    });
                return e;
            });
        if (err != cudaSuccess) return err;
        p.split = logprob_split(p.rows, p.vocab, Elem<T>::kVec, sms, most);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.rows * p.split), 1, 1);
    cfg.blockDim = dim3(kLpThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T>
cudaError_t logprob_fwd_t(const LogprobParams& p, cudaStream_t s) {
    const bool ent = p.entropy != nullptr;
    if (p.top > 0)
        return ent ? logprob_fwd_go<T, true, true>(p, s) : logprob_fwd_go<T, false, true>(p, s);
    return ent ? logprob_fwd_go<T, true, false>(p, s) : logprob_fwd_go<T, false, false>(p, s);
}

}  // namespace rn
