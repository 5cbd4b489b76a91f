// rn_heads.h -- kernel arguments of the head operators (norms of queries and
// keys with the position rotation, their gradient, the paged cache of keys and
// values), shared by the C-ABI unit and the kernel units.
#pragma once

#include <cmath>

#include "rn_tokens.h"

namespace rn {

constexpr int DT_E4M3 = 3;         // 8-bit floating point, caches only
constexpr int64_t kMaxHeadDim = 512;
// Warps of a CTA of the forward kernel: few, since a CTA's place is free again when its last warp
// ends, and warps take different times (32768 tokens' 8 keys and values of 128, into an 8-bit cache:
// two warps a CTA 52 us, eight 56, while keys and values had units of their own).
constexpr int kHeadsWarps = 2;
constexpr int kHeadsThreads = kHeadsWarps * 32;
// Warps of a CTA of the gradient's kernel, of which an SM holds two: a lane that holds 16 values of a
// row takes about 150 registers (six warps; with eight at 128 registers, some of them in memory,
// 32768 tokens of 64 + 8 heads of 128 BF16 took 282 us, not 273).
constexpr int heads_bwd_warps(int v, int ch) { return v * ch >= 8 ? 6 : 8; }
constexpr int kHeadsBwdPerSm = 2;

// Rows of one kind (queries, keys, values): one for each head of each token.
struct HeadSeg {
    const void* x;
    const void* dy;            // the gradient's kernel: what reaches the rows' outputs
    void* y;
    const void* w;             // may be NULL: ones
    int64_t xb, xt, xh;        // strides in elements: batch, token, head
    int64_t gb, gt, gh;        // of dy
    int64_t yb, yt, yh;        // of y; into a cache: page, slot, head
    int heads;
    FastDiv per;               // warps' units that a token's rows take
    int pack;                  // tokens of a unit, whose heads (few) lane groups share
    FastDiv few;               // division by those
    uint32_t units;            // of all tokens
};

// The scale of an 8-bit cache: 1 / (scale power) = hi + lo, both positive (see st_e4m3). power is 1, or
// 2^-64 for scales above 2^96, so that lo keeps its bits: of values times that, only those lose any
// that are far below e4m3's smallest.
struct E4m3Scale {
    float hi, lo, power;
};
inline E4m3Scale e4m3_scale(float scale) {
    const float power = scale > 0x1p96f ? 0x1p-64f : 1.f;
    const double s = (double)scale * power;
    float hi = (float)(1. / s);
    if (hi * s > 1.) hi = std::nextafter(hi, 0.f);      // (24 bits each: exact)
    const float lo = (float)((1. - hi * s) / s);
    return {hi, lo > 0.f ? lo : 0x1p-149f, power};
}

// How a warp holds rows: lpr lanes each, every lane ch pairs of vectors of v elements.
struct HeadShape {
    int v, lpr, ch;
};

struct HeadsParams {
    HeadSeg seg[3];            // queries, keys; append: the values beside keys
    FastDiv len;               // tokens of a sequence of the batch
    uint32_t total;            // units in all
    int per;                   // heads of a unit
    int64_t tokens;
    const void* positions;
    const float* table;        // [table_rows][ldt]: rot / 2 cosines, rot / 2 sines
    int64_t table_rows, ldt;
    const void* slots;         // append
    int64_t nslots;
    FastDiv page;
    float* part;               // gradient: [CTAs][d] sums for the weights, or NULL
    int first_k;               // gradient: the first CTA of the keys
    float eps;
    E4m3Scale scale[3];        // of what an 8-bit cache holds of keys (1) and values (2)
    int d[3];                  // width of each segment's rows
    int rot, itype;
    bool norm, interleaved, back;   // back: the transposed rotation
};

// Pairs of vectors of v elements that fill a row of d, and the lanes that hold them: vectors of 16
// bytes (vec elements); of 8 bytes where 16 do not divide a 16-bit row's rotation (32768 tokens of 32
// + 8 heads of 80, 40 values of each turned, BF16 89 us, 140 by two elements); else 2 or 1 elements.
// Lanes of a row: a power of two, or with 8-byte vectors 5, 6 or 10 too, of which more rows fit a warp
// (that case 89 us, 105 by 16 lanes; with 16-byte vectors nothing gained: heads of 96 by 6 lanes 98 us,
// by 8 98, their gradient 154 and 151). With narrow accesses fewer lanes spread a row's own cost over
// fewer of its values, but split its sectors: what was faster, by width and direction (gradients by two
// elements, 80 wide: 176 us by 8 lanes, 223 by 32; by one, 8192 tokens of 16 + 4 heads of 78 FP16: 53
// by 16, 76 by 32; forward by one, 5836 tokens appended at 256 wide: 54 by 16, 62 by 32, but 9990
// tokens of 16 + 16 heads of 78 51 by 32, 82 by 8).
constexpr HeadShape head_shape(int v, int vec, int64_t d, bool bwd) {
    const int64_t pairs = (d / 2 + v - 1) / v;
    if (v >= 4) {
        for (int lpr : {4, 5, 6, 8, 10, 16})
            if (pairs <= lpr && (v != vec || (lpr & (lpr - 1)) == 0)) return {v, lpr, 1};
        return {v, 32, pairs > 32 ? 2 : 1};
    }
    if (v == 2) {
        if (pairs <= 32) return bwd ? HeadShape{2, 8, 4} : HeadShape{2, 32, 1};
        return {2, pairs <= 64 ? 16 : 32, 4};
    }
    if (pairs <= 64) return bwd ? HeadShape{1, 16, 4} : HeadShape{1, 32, 2};
    if (pairs <= 128) return bwd ? HeadShape{1, 32, 4} : HeadShape{1, 16, 8};
    return {1, 32, 8};
}

// Heads of a unit, one token's: what a warp holds at once (32 / lpr rows), kHeadsLoops times, so
// that a token's factors serve many rows (16 times 182 us for 32768 tokens of 64 + 8 heads of 128 BF16,
// four times 198); fewer where that leaves an SM fewer than `least` units. In the forward kernel 16 (512
// tokens of 32 + 8 heads of 128 BF16 with 4 5.8 us, 16 4.3, 48 4.9; 2048 of them with 12 9.7, 16 8.6),
// 12 where accesses are narrow (332 tokens of 20 + 5 heads of 128 FP16, 106 values turned: 8.3, with 16
// 11.1); in the gradient's, whose warps take several, 4 (511 tokens of 12 + 12 heads of 64 FP32 4.4,
// with 16 5.4).
constexpr int kHeadsLoops = 16;
constexpr int kBwdUnits = 4;
constexpr int fwd_units(int v) { return v < 4 ? 12 : 16; }
constexpr int heads_per_unit(int lpr, int64_t heads, int64_t tokens, int least) {
    const int at_once = 32 / lpr;
    int loops = kHeadsLoops;
    while (loops > 1 &&
           tokens * ((heads + at_once * loops - 1) / (at_once * loops)) < 152 * least)
        loops /= 2;
    return loops * at_once;
}

// cache_dtype: -1 without a cache.
cudaError_t heads_fwd_launch(int dtype, int cache_dtype, HeadShape shape, const HeadsParams& p,
                             cudaStream_t s);
// ctas: rows of p.part.
cudaError_t heads_bwd_launch(int dtype, HeadShape shape, const HeadsParams& p, int ctas, void* dwq,
                             void* dwk, cudaStream_t s);
// CTAs of the gradient's kernel, and rows of its workspace, at most: eight rounds of what a GB300
// holds, since CTAs take different times (32768 tokens of 64 + 8 heads of 128 BF16: one round 365 us,
// four 309, eight 289, sixteen 290).
constexpr int kHeadsBwdCtas = 2432;

struct SlotsParams {
    const void* page_table;    // [seqs][ld]
    const void* starts;        // [seqs]
    const void* offsets;       // [seqs + 1]
    void* slots;               // [n]
    void* positions;           // [n], may be NULL
    int64_t n, ld, width, pages;
    int seqs;
    int64_t page;
    int itype;
};
cudaError_t kv_slots_launch(const SlotsParams& p, cudaStream_t s);

// The first of entries 1 .. seqs beyond t, seqs + 1 if none is, by bisection: at(i) are entries that
// do not fall. (seqs is up to 2^30, so that lo + hi passes 32 bits.)
template <typename At>
#ifdef __CUDACC__
__device__ __forceinline__
#else
inline
#endif
int first_beyond(At at, int seqs, int64_t t) {
    int lo = 1, hi = seqs + 1;
    while (lo < hi) {
        const int mid = lo + ((hi - lo) >> 1);
        if (at(mid) > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

struct GatherSide {
    const void* cache;
    void* out;
    int64_t cp, cs, ch;        // page, slot, head strides of the cache
    int64_t ot, oh;            // token, head strides of out
    int64_t total;             // n * heads * vectors of a head's row
    FastDiv token, head;       // vectors of a token, of a head
    float scale;
};
struct GatherParams {
    GatherSide side[2];
    const void* slots;
    int64_t nslots;
    FastDiv page;
    int itype;
};
// ne: elements of an access, one for both sides.
cudaError_t kv_gather_launch(int cache_dtype, int dtype, int ne, const GatherParams& p,
                             cudaStream_t s);

}  // namespace rn
