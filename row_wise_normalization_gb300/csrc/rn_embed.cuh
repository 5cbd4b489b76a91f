// rn_embed.cuh -- device parts of the embedding gradient: the sort of the ids in a
// cluster's shared memory, the rows of zeros, the sums of the sorted rows, and the joining of
// sums that run over several chunks. embed_sort.cu and embed_bwd.cuh make kernels of them.
#pragma once

#include "rn_async.cuh"
#include "rn_tokens.cuh"

namespace rn {

// ---- sort -------------------------------------------------------------------
// The sort key of the id at position i.
__device__ __forceinline__ uint32_t id_key(const SortParams& p, int64_t i) {
    const int64_t id = ld_id(p.tokens, i, p.itype);
    return (uint32_t)((id >= 0 && id < p.vocab) ? id : p.vocab);
}

// Sum of v over the threads before this one (all kSortThreads of them call it).
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t* wsum) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t q = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += q;
    }
    if (lane == 31) wsum[w] = incl;
    __syncthreads();
    uint32_t run = incl - v;
    for (int k = 0; k < w; ++k) run += wsum[k];
    return run;
}

// The lanes of the warp that hold an id with this lane's digit: a ballot a bit.
__device__ __forceinline__ unsigned same_digit(uint32_t dg, bool in) {
    unsigned same = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int b = 0; b < kSortBits; ++b) {
        const unsigned one = __ballot_sync(0xffffffffu, dg >> b & 1u);
        same &= dg >> b & 1u ? one : ~one;
    }
    return same;
}
// The number of this lane's digit among the warp's ids so far (cnt: the warp's table,
// advanced). All lanes; `in` false: no id.
__device__ __forceinline__ uint32_t warp_rank(uint32_t* cnt, uint32_t dg, unsigned same, bool in,
                                              int lane) {
    const uint32_t r = in ? cnt[dg] : 0;
    const unsigned below = same & ((1u << lane) - 1);
    __syncwarp();
    if (in && below == 0) cnt[dg] = r + __popc(same);
    __syncwarp();
    return r + __popc(below);
}

constexpr int cluster_fixed_bytes() { return kSortWarps * kSortBins * 4 + kSortBins * 4; }
constexpr int cluster_bytes(int share, int passes) {
    return cluster_fixed_bytes() + (passes > 1 ? 2 : 1) * share * 8 + share * 2;
}

// The sort of at most p.cluster * p.share ids by the CTAs of a cluster, of which this is number
// `me`. smem: cluster_bytes(p.share, p.passes) bytes, in the same place in every CTA. Ends with
// a barrier of the cluster.
__device__ __forceinline__ void cluster_sort(const SortParams& p, unsigned char* smem,
                                             uint32_t* wsum, int me) {
    static_assert(kSortThreads == kSortBins, "one thread for each digit");
    static_assert(kSortMaxShare <= 65536 && cluster_bytes(kSortMaxShare, 2) <= 232448 - 1024,
                  "16-bit ranks; the shared memory of a CTA");
    uint32_t(*cnt)[kSortBins] = (uint32_t(*)[kSortBins])smem;
    uint32_t* const tots = (uint32_t*)smem + kSortWarps * kSortBins;
    unsigned long long* const buf = (unsigned long long*)(smem + cluster_fixed_bytes());
    uint16_t* const rank = (uint16_t*)(buf + (p.passes > 1 ? 2 : 1) * p.share);
    const int t = threadIdx.x, w = t >> 5, lane = t & 31;
    const uint32_t mask = (1u << p.bits) - 1;
    const int64_t base = (int64_t)me * p.share;
    // this CTA's ids, and this warp's of them: [w0, w1)
    const int mine = (int)max((int64_t)0, min((int64_t)p.share, p.n - base));
    const int per = p.share / kSortWarps;
    const int w0 = min(mine, w * per), w1 = min(mine, w0 + per);
    if (me == 0 && t == 0) *p.zeroed = 0;
    for (int i = w0 + lane; i < w1; i += 32)
        buf[i] = ((unsigned long long)id_key(p, base + i) << 32) | (uint32_t)(base + i);
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.bits;
        unsigned long long* const src = buf + (pass & 1) * p.share;
        unsigned long long* const dst = buf + ((pass & 1) ^ 1) * p.share;
        for (int k = 0; k < kSortWarps; ++k) cnt[k][t] = 0;
        __syncthreads();
        // (the ballots of 4 steps are independent of each other; the counts are not)
        constexpr int U = 4;
        for (int i0 = w0; i0 < w1; i0 += 32 * U) {
            uint32_t dg[U];
            unsigned same[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * 32 + lane;
                dg[u] = i < w1 ? (uint32_t)(src[i] >> (32 + shift)) & mask : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * 32 < w1) same[u] = same_digit(dg[u], i0 + u * 32 + lane < w1);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * 32 + lane;
                if (i0 + u * 32 >= w1) break;
                const uint32_t r = warp_rank(cnt[w], dg[u], same[u], i < w1, lane);
                if (i < w1) rank[i] = (uint16_t)r;
            }
        }
        __syncthreads();
        uint32_t sum = 0;
        for (int k = 0; k < kSortWarps; ++k) sum += cnt[k][t];
        tots[t] = sum;
        cluster_sync();
        // (all loads in flight: one after another they took half of the sort's time)
        uint32_t c[kSortMaxCluster], before = 0, total = 0;
#pragma unroll
        for (int q = 0; q < kSortMaxCluster; ++q)
            c[q] = q < p.cluster ? peer_u32(peer_addr(tots + t, q)) : 0;
#pragma unroll
        for (int q = 0; q < kSortMaxCluster; ++q) {
            before += q < me ? c[q] : 0;
            total += c[q];
        }
        uint32_t run = before + sum_before(total, wsum);
        for (int k = 0; k < kSortWarps; ++k) {
            const uint32_t c = cnt[k][t];
            cnt[k][t] = run;
            run += c;
        }
        __syncthreads();
        const bool last = pass == p.passes - 1;
#pragma unroll 4
        for (int i = w0 + lane; i < w1; i += 32) {
            const unsigned long long v = src[i];
            const uint32_t at = cnt[w][(uint32_t)(v >> (32 + shift)) & mask] + rank[i];
            if (last) {
                p.key[0][at] = (uint32_t)(v >> 32);
                p.pos[0][at] = (int32_t)v;
            } else {
                const uint32_t q = fast_quot(at, p.owner);
                peer_store(peer_addr(dst + (at - q * (uint32_t)p.share), q), v);
            }
        }
        // the peers' ids have arrived, and they are past their reads of tots
        cluster_sync();
    }
}

// ---- rows of zeros ----------------------------------------------------------
constexpr int kZeroRange = 32768;   // ids a CTA marks at a time (4 KB of bits)
// Zeros by the bulk-copy engine (one instruction a row, from zeros in shared memory) or by the
// threads' stores. Measured on GB300 with the sums in other CTAs of the launch (embed_few_kernel):
// 512 x 768 FP32 into 32000 rows 18.7 us, by stores 22.3; 512 x 1024 BF16 13.1, 15.7; 300 x 771
// FP16 into FP32 19.5, 20.5; 16 x 512 FP32 into 50000 rows 18.6, 17.8; rows of 512 bytes 10.0,
// 13.1. Copies of 8 KB: 1 us more. Beside the sort and long sums there is no gain, and the registers
// cost: 16383 x 771 FP16 49.9, by stores 48.8, 65536 x 4096 BF16 291, 277 (embed_bwd_kernel).
constexpr int kZeroBytes = 4096;    // of a copy
constexpr int kClearWords = kZeroRange / 32 + kZeroBytes / 4;   // shared memory of a CTA that clears

// Ids, from L2: a CTA that clears does not wait for the kernel ahead itself (embed_bwd_kernel), so
// nothing else keeps it from an older copy in its SM's L1.
__device__ __forceinline__ Raw<16> ld_ids(const void* p) {
    Raw<16> r;
    asm volatile("ld.relaxed.gpu.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ int64_t ld_id_l2(const void* p, int64_t i, int itype) {
    if (itype == IT_I64) {
        long long v;
        asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];"
                     : "=l"(v)
                     : "l"((const long long*)p + i)
                     : "memory");
        return v;
    }
    int v;
    asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"((const int*)p + i) : "memory");
    return v;
}

__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
                 "r"(bytes)
                 : "memory");
}
// Ends when this thread's copies have been written.
__device__ __forceinline__ void bulk_s2g_wait() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Clears `bytes` (a multiple of 2) at p by `lanes` threads, of which this is number l. zeros: the
// address of kZeroBytes of zeros in shared memory, from which the first thread has the bulk-copy
// engine write the row's 16-byte vectors (0: the threads store them).
__device__ __forceinline__ void clear_row(char* p, int64_t bytes, int l, int lanes,
                                          uint32_t zeros) {
    const int64_t head = min((int64_t)((0u - (unsigned)(uintptr_t)p) & 15u), bytes);
    const int64_t nv = (bytes - head) / 16, tail = head + nv * 16;
    const Raw<16> z = {};
    if (!zeros) {
        for (int64_t v = l; v < nv; v += lanes) st_raw(p + head + v * 16, z);
    } else if (l == 0) {
        for (int64_t b = head; b < tail; b += kZeroBytes)
            bulk_s2g(p + b, zeros, (uint32_t)min((int64_t)kZeroBytes, tail - b));
    }
    const Raw<2> h = {};
    for (int64_t b = 2 * l; b < head; b += 2 * lanes) st_raw(p + b, h);
    for (int64_t b = tail + 2 * l; b < bytes; b += 2 * lanes) st_raw(p + b, h);
}

// Clears the rows of the absent ids of part `part` of the vocabulary, of `parts`, by a CTA of NT
// threads. BULK: long rows by the bulk-copy engine. mem: kClearWords words of shared memory, 16-byte
// aligned.
template <int NT, bool BULK>
__device__ __forceinline__ void clear_absent(const SortParams& p, int part, int parts,
                                             uint32_t* mem) {
    uint32_t* const bits = mem + kZeroBytes / 4;
    const int t = threadIdx.x;
    // (whole groups of 32 rows, where that leaves every CTA rows: 16383 x 771 FP16 into FP32 took
    // 69 us without, 57 us with; 64 x 4096 BF16 into 2000 rows 11.7 us with, 6.8 us without)
    int64_t whole = 32;
    while (whole > 1 && whole * parts > p.vocab) whole /= 2;
    const int64_t share = ((p.vocab + parts - 1) / parts + whole - 1) / whole * whole;
    const int64_t end = min(p.vocab, (int64_t)(part + 1) * share);
    // the ids as 16-byte vectors, and fewer than two vectors' before and after
    const int64_t per = 16 / index_size(p.itype);
    const int64_t head = min(p.n, (int64_t)((0u - (unsigned)(uintptr_t)p.tokens) & 15u) /
                                      index_size(p.itype));
    const int64_t nv = (p.n - head) / per;
    const char* const body = (const char*)p.tokens + head * index_size(p.itype);
    // threads of a row: as many 16-byte stores as it has, up to a warp's; one where copies do all
    const bool bulk = BULK && p.bulk;
    int lanes = 32;
    if (bulk) {
        if ((((uint64_t)(uintptr_t)p.zero | (uint64_t)p.zero_pitch | (uint64_t)p.zero_bytes) & 15) == 0)
            lanes = 1;
        for (int k = t; k < kZeroBytes / 4; k += NT) mem[k] = 0;
        fence_proxy_async_smem();
    } else {
        while (lanes > 1 && (lanes / 2) * 16 >= p.zero_bytes) lanes /= 2;
    }
    const uint32_t zeros = bulk ? smem_addr(mem) : 0;
    for (int64_t lo = (int64_t)part * share; lo < end; lo += kZeroRange) {
        const int cnt = (int)min((int64_t)kZeroRange, end - lo);
        __syncthreads();
        for (int w = t; w < (cnt + 31) / 32; w += NT) bits[w] = 0;
        __syncthreads();
        auto mark = [&](int64_t id) {
            const uint64_t k = (uint64_t)id - (uint64_t)lo;
            if (k < (uint64_t)cnt) atomicOr(&bits[k >> 5], 1u << (k & 31));
        };
        // Many loads in flight: once the first CTAs store, a load waits behind their stores
        // (8-byte loads, twice as many rounds: some CTAs read 65536 ids for 98 us).
        constexpr int U = 8;
        for (int64_t v = t; v < nv; v += NT * U) {
            Raw<16> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v + u * NT < nv) r[u] = ld_ids(body + (v + u * NT) * 16);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (v + u * NT < nv) {
                    if (p.itype == IT_I64) {
                        mark((int64_t)((uint64_t)r[u].w[1] << 32 | r[u].w[0]));
                        mark((int64_t)((uint64_t)r[u].w[3] << 32 | r[u].w[2]));
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mark((int32_t)r[u].w[k]);
                    }
                }
            }
        }
        if (t < p.n - nv * per) mark(ld_id_l2(p.tokens, t < head ? t : nv * per + t, p.itype));
        __syncthreads();
        for (int r = t / lanes; r < cnt; r += NT / lanes)
            if (!((bits[r >> 5] >> (r & 31)) & 1u))
                clear_row(p.zero + (lo + r) * p.zero_pitch, p.zero_bytes, t % lanes, lanes, zeros);
    }
    if (bulk) bulk_s2g_wait();
}

// ---- sums -------------------------------------------------------------------
constexpr int kSegThreads = 256;
constexpr int kSegU = 8;            // rows in flight

// Vectors of NE elements a thread has of a row: 16 bytes, at most 4.
template <typename T, int NE>
constexpr int seg_vectors() {
    return 16 / (NE * (int)sizeof(T)) < 4 ? 16 / (NE * (int)sizeof(T)) : 4;
}

// Sums chunk c's rows in the columns of a slice, by p.tx threads of which this is number tx: whole
// warps, which do not wait for each other.
template <typename T, typename G, int NE>
__device__ __forceinline__ void sum_chunk(const EmbedBwdParams& p, int64_t c, int slice, int tx) {
    constexpr int M = seg_vectors<T, NE>();
    constexpr int B = NE * (int)sizeof(T);
    G* const DG = (G*)p.dtable;
    const int lane = tx & 31;
    // this thread's vectors: every 32nd of its warp's, from column j0 on
    const int64_t j0 = (((int64_t)slice * p.tx + (tx - lane)) * M + lane) * NE;
    constexpr int step = 32 * NE;
    if (j0 - lane * NE >= p.d) return;     // a warp past the row's end
    const int cols = (int)max((int64_t)-1, min((int64_t)(M * step), p.d - j0));   // of them in the row
    const T* const X = (const T*)p.dout + j0;
    const int64_t i0 = c * p.chunk;
    const int len = (int)min((int64_t)p.chunk, p.n - i0);
    const uint32_t prev = i0 > 0 ? ld_u32(p.key + i0 - 1) : 0xffffffffu;
    const uint32_t next = i0 + len < p.n ? ld_u32(p.key + i0 + len) : 0xffffffffu;
    uint32_t my_key = 0xffffffffu;
    int32_t my_pos = 0;
    if (lane < len) {
        my_key = ld_u32(p.key + i0 + lane);
        my_pos = (int32_t)ld_u32((const uint32_t*)p.pos + i0 + lane);
    }
    // positions of ids outside the vocabulary come last: cnt without them
    const int cnt = __popc(__ballot_sync(0xffffffffu, my_key < (uint32_t)p.vocab));
    if (cnt == 0) return;
    // bit i: position i begins an id; `open`: the chunk's first began in an earlier chunk
    const uint32_t left = __shfl_up_sync(0xffffffffu, my_key, 1);
    const unsigned heads = __ballot_sync(0xffffffffu, lane > 0 && my_key != left);
    bool open = prev == __shfl_sync(0xffffffffu, my_key, 0);
    constexpr int E = M * NE;           // elements of this thread, in pairs
    F2 acc[E / 2];
    auto clear = [&]() {
#pragma unroll
        for (int k = 0; k < E / 2; ++k) acc[k] = f2s(0.f);
    };
    clear();
    // The sum of the id of position i, complete as far as this chunk goes; `on`: it goes on in
    // the next.
    auto put = [&](int i, bool on) {
        const uint32_t id = __shfl_sync(0xffffffffu, my_key, i);
        float* const w = p.part + (2 * c + (open ? 0 : 1)) * p.dpad + j0;
        G* const g = DG + (int64_t)id * p.ldg + j0;
        float s[E];
#pragma unroll
        for (int k = 0; k < E / 2; ++k) f2_get(acc[k], s[2 * k], s[2 * k + 1]);
        float o[E];
        if (M > 1 && p.accumulate && !open && !on) {   // together: 16383 x 771 47 us, not 61
#pragma unroll
            for (int m = 0; m < M; ++m)
                if (m * step < cols) ld_elems<G, NE>(o + m * NE, g + m * step);
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
            if (m * step < cols) {
                if (open || on) {
                    st_elems<float, NE>(w + m * step, s + m * NE);
                } else {
                    if (M == 1 && p.accumulate) ld_elems<G, NE>(o, g);
#pragma unroll
                    for (int k = m * NE; k < (m + 1) * NE; ++k)
                        o[k] = p.accumulate ? fmaf(p.scale, s[k], o[k]) : p.scale * s[k];
                    st_elems<G, NE>(g + m * step, o + m * NE);
                }
            }
        }
        open = false;
    };
    auto add = [&](const Raw<B>(&r)[M]) {
        float v[E];
#pragma unroll
        for (int m = 0; m < M; ++m) unpack<T, NE>(v + m * NE, r[m]);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) acc[k] = add2(acc[k], f2(v[2 * k], v[2 * k + 1]));
    };
    for (int i = 0; i < cnt; i += kSegU) {
        Raw<B> r[kSegU][M];
#pragma unroll
        for (int u = 0; u < kSegU; ++u) {
            const int64_t at = __shfl_sync(0xffffffffu, my_pos, (i + u) & 31);
            if (i + u < cnt) {
#pragma unroll
                for (int m = 0; m < M; ++m)
                    if (m * step < cols) r[u][m] = ld_raw<B>(X + at * p.lddo + m * step);
            }
        }
        const unsigned h = heads >> i;
        if (p.accumulate) {
            // the gradient's rows that these are added to, so that put() finds them in L2: 65536 x
            // 4096 BF16 into 128000 rows 186 us without, 179 with (260, 244 where the ids are
            // uniform, so that more rows occur); 16383 x 771 FP16 into FP32 48, 43
#pragma unroll
            for (int u = 0; u < kSegU; ++u) {
                const uint32_t id = __shfl_sync(0xffffffffu, my_key, (i + u) & 31);
                if (i + u < cnt && (h >> u & 1u || i + u == 0)) {
#pragma unroll
                    for (int m = 0; m < M; ++m)
                        if (m * step < cols) prefetch_l2(DG + (int64_t)id * p.ldg + j0 + m * step);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kSegU; ++u) {
            if (i + u < cnt) {
                if (h >> u & 1u) {
                    put(i + u - 1, false);
                    clear();
                }
                add(r[u]);
            }
        }
    }
    put(cnt - 1, next == __shfl_sync(0xffffffffu, my_key, cnt - 1));
}

// The ids whose positions run over a chunk's edge. Each warp of a CTA looks at one chunk and, if
// such an id begins in it and ends within kJoinWarps chunks, adds the id's
// sums of the chunks in order, kJoinCols blocks of 128 columns at a time so that enough
// loads are in flight. A longer id is left to the whole CTA, whose warps take its sums in turn;
// the warps' sums are added in order. The CTA takes every ny-th block of columns.
// In long batches an id may have thousands of sums, and it takes two launches: the
// first also adds the kJoinWarps sums of every CTA whose chunks lie within one id, and lists the
// long ids; the second does those, in any order, with the CTAs' sums.
// (The sums lie in rows of their own, 16-byte aligned whatever the gradient's rows are;
// `vec` says whether those are.)
constexpr int kJoinWarps = 8;       // warps, and chunks, of a CTA
constexpr int kJoinCols = 4;
constexpr int kJoinBlock = 128;
// Chunks up to which one launch does: 1500 ids (188 chunks) 15.9 us in two launches, 14.4 in one;
// 3000 ids, more than half of them one id (375 chunks), 18.3 and 18.9, and the host saves 2.5 us.
constexpr int kJoinOnce = 512;
struct alignas(16) LongId {          // its first and last chunk
    uint32_t first, last, id, pad;
};

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

// A block's 128 columns of row q of the sums, 4 a lane.
__device__ __forceinline__ void join_load(const EmbedBwdParams& p, float* v, int64_t q, int64_t b,
                                          int lane) {
    const int64_t j = b * kJoinBlock + lane * 4;
    if (j < p.d) {
        ld_elems<float, 4>(v, p.part + q * p.dpad + j);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = 0.f;
    }
}

// The sum of a long id, by a CTA: its sums are the first chunk's second row, the chunks up to
// the next CTA's, the CTAs' that lie within it (`grouped`), and the chunks that remain.
template <typename G>
__device__ __forceinline__ void join_long(const EmbedBwdParams& p, bool vec, bool grouped,
                                          const LongId& id, float (*sum)[kJoinBlock], int y,
                                          int ny) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = id.first, end = id.last;
    const int64_t ga = grouped ? first / kJoinWarps + 1 : 0;
    const int64_t gb = grouped ? end / kJoinWarps : 0;   // (ga <= gb: it spans kJoinWarps chunks more)
    const int64_t head = grouped ? ga * kJoinWarps - first : end + 1 - first;
    const int64_t terms = grouped ? head + (gb - ga) + (end + 1 - gb * kJoinWarps) : head;
    auto row = [&](int64_t t) {
        if (t == 0) return 2 * first + 1;
        if (t < head) return 2 * (first + t);
        if (t < head + (gb - ga)) return 2 * (ga + t - head) * kJoinWarps;
        return 2 * (gb * kJoinWarps + t - head - (gb - ga));
    };
    const int64_t blocks = (p.d + kJoinBlock - 1) / kJoinBlock;
    for (int64_t b = y; b < blocks; b += ny) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int64_t t = w; t < terms; t += 8 * kJoinWarps) {
            float v[8][4];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (t + u * kJoinWarps < terms) {
                    join_load(p, v[u], row(t + u * kJoinWarps), b, lane);
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
            join_put<G>(p, vec, id.id, j, acc);
        }
    }
}

// The ids that begin in chunks c0 .. c0 + kJoinWarps - 1, by a CTA, in the blocks of columns y,
// y + ny, ... `once`: the long ones as well (else they are listed).
struct JoinState {
    LongId longid;           // a long id that begins here (there is one at most)
    bool any;
};
template <typename G>
__device__ __forceinline__ void join_chunks(const EmbedBwdParams& p, bool vec, bool once, int64_t c0,
                                            int y, int ny, JoinState& st,
                                            float (*sum)[kJoinBlock]) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = c0 + w;
    const int64_t i0 = c * p.chunk, i1 = i0 + p.chunk;
    const int64_t blocks = (p.d + kJoinBlock - 1) / kJoinBlock;
    if (threadIdx.x == 0) st.any = false;
    int64_t last = -1;
    uint32_t cur = 0xffffffffu;
    bool within = false;                // the CTA's chunks lie within one id
    if (i1 < p.n) {
        // (loads together: most chunks need no more)
        const uint32_t before = i0 > 0 ? ld_u32(p.key + i0 - 1) : 0xffffffffu;
        const uint32_t begin = ld_u32(p.key + i0), after = ld_u32(p.key + i1);
        const int64_t e = min(i1 + p.chunk, p.n) - 1;
        const uint32_t far = ld_u32(p.key + e);
        cur = ld_u32(p.key + i1 - 1);
        if (!once) {
            const int64_t g0 = c0 * p.chunk, g1 = g0 + (int64_t)kJoinWarps * p.chunk;
            within = g0 > 0 && g1 < p.n && ld_u32(p.key + g0 - 1) == cur &&
                     ld_u32(p.key + g1) == cur && cur < (uint32_t)p.vocab;
        }
        if (cur < (uint32_t)p.vocab && after == cur && !(begin == cur && before == cur)) {
            last = c + 1;
            if (far == cur && e + 1 < p.n) {
                // the first position after the id's, in [lo, hi]: 32 places at a time
                int64_t lo = e + 1, hi = p.n;
                while (lo < hi) {
                    const int64_t w32 = (hi - lo + 31) / 32;
                    const int64_t at = min(lo + (lane + 1) * w32, hi) - 1;
                    const unsigned same = __ballot_sync(0xffffffffu, ld_u32(p.key + at) == cur);
                    const int k = __popc(same);      // the first k places are the id's
                    const int64_t from = lo + k * w32;
                    lo = k == 32 ? hi : from;
                    if (k < 32) hi = min(from + w32, hi) - 1;
                }
                last = (lo - 1) / p.chunk;
            }
        }
    }
    const bool many = last - c >= kJoinWarps;
    __syncthreads();
    if (many && lane == 0) {
        st.any = true;
        st.longid = LongId{(uint32_t)c, (uint32_t)last, cur, 0};
        if (!once && y == 0)
            ((LongId*)(p.longs + 4))[atomicAdd(p.longs, 1u)] = st.longid;
    }
    if (last >= 0 && !many) {
        for (int64_t b0 = y; b0 < blocks; b0 += (int64_t)ny * kJoinCols) {
            float acc[kJoinCols][4], two[kJoinCols][4];
            // (the first two chunks, which every such id has, in one go)
#pragma unroll
            for (int u = 0; u < kJoinCols; ++u)
                join_load(p, acc[u], 2 * c + 1, b0 + u * ny, lane);
#pragma unroll
            for (int u = 0; u < kJoinCols; ++u)
                join_load(p, two[u], 2 * (c + 1), b0 + u * ny, lane);
            for (int64_t q = c + 2;; ++q) {
#pragma unroll
                for (int u = 0; u < kJoinCols; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[u][k] += two[u][k];
                if (q > last) break;
#pragma unroll
                for (int u = 0; u < kJoinCols; ++u)
                    join_load(p, two[u], 2 * q, b0 + u * ny, lane);
            }
#pragma unroll
            for (int u = 0; u < kJoinCols; ++u) {
                const int64_t j = (b0 + u * ny) * kJoinBlock + lane * 4;
                if (j < p.d) join_put<G>(p, vec, cur, j, acc[u]);
            }
        }
    }
    if (within) {
        // the sum of the CTA's chunks, in the place of the first one's
        for (int64_t b = y + (int64_t)w * ny; b < blocks;
             b += (int64_t)kJoinWarps * ny) {
            float v[kJoinWarps][4];
#pragma unroll
            for (int u = 0; u < kJoinWarps; ++u) join_load(p, v[u], 2 * (c0 + u), b, lane);
#pragma unroll
            for (int u = 1; u < kJoinWarps; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[0][k] += v[u][k];
            const int64_t j = b * kJoinBlock + lane * 4;
            if (j < p.d) st_elems<float, 4>(p.part + 2 * c0 * p.dpad + j, v[0]);
        }
    }
    if (!once) return;
    __syncthreads();
    if (st.any) join_long<G>(p, vec, false, st.longid, sum, y, ny);
}

}  // namespace rn
