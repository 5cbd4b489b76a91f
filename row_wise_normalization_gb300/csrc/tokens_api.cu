// tokens_api.cu -- the C ABI of the token operators (include/rownorm.h):
// argument validation, the choice of access width, workspace layout and launch.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "rownorm.h"
#include "rn_tokens.h"

namespace rn {
cudaError_t logprob_fwd_f32(const LogprobParams& p, cudaStream_t s);
cudaError_t logprob_fwd_bf16(const LogprobParams& p, cudaStream_t s);
cudaError_t logprob_fwd_f16(const LogprobParams& p, cudaStream_t s);

cudaError_t embed_bwd_f32(int, int, bool, const SortParams&, int, const EmbedBwdParams&,
                          cudaStream_t);
cudaError_t embed_bwd_bf16(int, int, bool, const SortParams&, int, const EmbedBwdParams&,
                          cudaStream_t);
cudaError_t embed_bwd_f16(int, int, bool, const SortParams&, int, const EmbedBwdParams&,
                          cudaStream_t);

// Few ids: one launch. Else the sort, the sums with the rows of zeros beside both, the joins.
cudaError_t embed_bwd_launch(int dtype, int gtype, int ne, const SortParams& sp,
                             const EmbedBwdParams& q, cudaStream_t s) {
    EmbedBwdParams p = q;
    const int bytes = ne * dtype_size(dtype);
    const int m = 16 / bytes < 4 ? 16 / bytes : 4;      // seg_vectors
    const int64_t vpt = (p.d / ne + m - 1) / m;         // threads a row could use
    p.tx = 32;
    while (p.tx < 256 && p.tx < vpt) p.tx *= 2;
    p.ty = 256 / p.tx;
    p.slices = (int)((vpt + p.tx - 1) / p.tx);
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const bool few = embed_few(p.n, p.d, dtype_size(dtype));
    if (err == cudaSuccess && !few) err = embed_sort_launch(sp, s);
    if (err != cudaSuccess) return err;
    switch (dtype) {
        case DT_BF16: return embed_bwd_bf16(gtype, ne, few, sp, sms, p, s);
        case DT_F16: return embed_bwd_f16(gtype, ne, few, sp, sms, p, s);
        default: return embed_bwd_f32(gtype, ne, few, sp, sms, p, s);
    }
}

cudaError_t logprob_fwd_launch(int dtype, const LogprobParams& p, cudaStream_t s) {
    switch (dtype) {
        case DT_BF16: return logprob_fwd_bf16(p, s);
        case DT_F16: return logprob_fwd_f16(p, s);
        default: return logprob_fwd_f32(p, s);
    }
}
}  // namespace rn

namespace {

using namespace rn;

constexpr int64_t kMaxElems = (int64_t)1 << 61;
constexpr int64_t kMaxVocab = (int64_t)1 << 30;   // columns are 32-bit numbers
constexpr int64_t kMaxWidth = (int64_t)1 << 30;
constexpr int64_t kMaxCount = ((int64_t)1 << 31) - 1;

uintptr_t addr(const void* p) { return (uintptr_t)p; }
bool known_dtype(int d) { return d == DT_F32 || d == DT_BF16 || d == DT_F16; }
bool known_index(int t) { return t == IT_I32 || t == IT_I64; }
bool misaligned(const void* p, int64_t a) { return (addr(p) & (uintptr_t)(a - 1)) != 0; }

// A byte range [p, p + n); nothing where p is NULL.
struct Range {
    const void* p;
    int64_t n;
};
bool overlaps(Range a, Range b) {
    if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
    return addr(a.p) < addr(b.p) + (uintptr_t)b.n && addr(b.p) < addr(a.p) + (uintptr_t)a.n;
}
template <int NO, int NI>
bool aliased(const Range (&outs)[NO], const Range (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlaps(outs[i], ins[j])) return true;
        for (int j = i + 1; j < NO; ++j)
            if (overlaps(outs[i], outs[j])) return true;
    }
    return false;
}
// Whether a [rows][d] matrix with row stride ld stays within the element limit.
bool fits(int64_t rows, int64_t d, int64_t ld) {
    return rows <= 0 || (rows - 1) <= (kMaxElems - d) / ld;
}
int64_t span(int64_t rows, int64_t d, int64_t ld) { return rows > 0 ? (rows - 1) * ld + d : 0; }

int done(cudaError_t err) { return err == cudaSuccess ? RN_OK : record_cuda_error(err); }

// The widest access, in elements of a power of two up to 16 bytes of storage type
// `es`, that divides the width and both strides and is aligned at both bases.
int access_elems(int64_t d, const void* a, int es_a, int64_t lda, const void* b, int es_b,
                 int64_t ldb) {
    for (int ne = 16 / es_a; ne > 1; ne /= 2) {
        const int wb = ne * es_b < 16 ? ne * es_b : 16;
        if (d % ne == 0 && lda % ne == 0 && ldb % ne == 0 && !misaligned(a, ne * es_a) &&
            !misaligned(b, wb))
            return ne;
    }
    return 1;
}

// ---- workspace of embed_bwd -------------------------------------------------
struct EmbedWorkspace {
    int64_t key[2], pos[2], hist, longs, part, total;   // byte offsets
    int64_t tiles, chunks, dpad;
};
EmbedWorkspace embed_workspace(int64_t n, int64_t d) {
    EmbedWorkspace w;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    w.tiles = (n + kSortTile - 1) / kSortTile;
    w.chunks = (n + embed_chunk(n, d) - 1) / embed_chunk(n, d);
    w.dpad = (d + 7) / 8 * 8;
    const bool global = sort_may_use_memory(n);   // the sort's second arrays and its counts
    for (int k = 0; k < 2; ++k) {
        w.key[k] = take(k == 0 || global ? n * 4 : 0);
        w.pos[k] = take(k == 0 || global ? n * 4 : 0);
    }
    w.hist = take(global ? w.tiles * kSortBins * 4 : 0);
    w.longs = take((w.chunks / 8 + 2) * 16);   // a long id fills at least 8 chunks
    w.part = take(2 * w.chunks * w.dpad * 4);
    w.total = at;
    return w;
}

bool embed_bwd_sizes_ok(int64_t n, int64_t vocab, int64_t d) {
    if (n < 0 || n > kMaxCount || vocab <= 0 || vocab > kMaxVocab || d <= 0 || d > kMaxWidth)
        return false;
    // (chunks x slices of the widest grid: 32 scalars a slice)
    return (n / embed_chunk(n, d) + 1) * (d / 32 + 1) < kMaxCount;
}

bool host_resident(const void* p) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    return a.type == cudaMemoryTypeHost || a.type == cudaMemoryTypeUnregistered;
}

}  // namespace

extern "C" {

int embed_fwd(int dtype, int itype, const void* tokens, const void* table, int64_t ldt, void* out,
              int64_t ldo, int64_t n, int64_t vocab, int64_t d, float scale, void* stream) {
    if (!known_dtype(dtype) || !known_index(itype)) return RN_ERR_DTYPE;
    if (n < 0 || vocab <= 0 || vocab > kMaxVocab || d <= 0 || d > kMaxWidth || ldt < d ||
        ldo < d || !fits(n, d, ldo) || !fits(vocab, d, ldt) || n > kMaxCount / (d / 512 + 1))
        return RN_ERR_SIZE;   // (the last: one launch's grid, a warp for 512 elements of a row)
    if (!std::isfinite(scale)) return RN_ERR_SCALE;
    if (n == 0) return RN_OK;
    if (!tokens || !table || !out) return RN_ERR_NULL;
    const int es = dtype_size(dtype), is = index_size(itype);
    if (misaligned(tokens, is) || misaligned(table, es) || misaligned(out, es))
        return RN_ERR_ALIGN;
    const Range outs[] = {{out, span(n, d, ldo) * es}};
    const Range ins[] = {{tokens, n * is}, {table, span(vocab, d, ldt) * es}};
    if (aliased(outs, ins)) return RN_ERR_ALIAS;
    const int ne = access_elems(d, table, es, ldt, out, es, ldo);
    EmbedParams p;
    p.tokens = tokens;
    p.table = table;
    p.out = out;
    p.n = n;
    p.vocab = vocab;
    p.ldt = ldt;
    p.ldo = ldo;
    p.vpr = fast_div((uint32_t)(d / ne));
    p.total = n * (d / ne);
    p.scale = scale;
    return done(embed_fwd_launch(dtype, itype, ne, d, p, (cudaStream_t)stream));
}

int embed_bwd_workspace_size(int64_t n, int64_t vocab, int64_t d, size_t* bytes) {
    if (!bytes) return RN_ERR_NULL;
    *bytes = 0;
    if (!embed_bwd_sizes_ok(n, vocab, d)) return RN_ERR_SIZE;
    if (n > 0) *bytes = (size_t)embed_workspace(n, d).total;
    return RN_OK;
}

int embed_bwd(int dtype, int gtype, int itype, const void* dout, int64_t lddo, const void* tokens,
              void* dtable, int64_t ldg, int64_t n, int64_t vocab, int64_t d, float scale,
              int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
    if (!known_dtype(dtype) || !known_index(itype) || (gtype != dtype && gtype != DT_F32))
        return RN_ERR_DTYPE;
    if (!embed_bwd_sizes_ok(n, vocab, d) || lddo < d || ldg < d || !fits(n, d, lddo) ||
        !fits(vocab, d, ldg))
        return RN_ERR_SIZE;
    if (!std::isfinite(scale)) return RN_ERR_SCALE;
    const int es = dtype_size(dtype), gs = dtype_size(gtype), is = index_size(itype);
    const cudaStream_t s = (cudaStream_t)stream;
    if (n == 0) {
        // an empty batch still defines the gradient: zero (all-zero bits in every type)
        if (accumulate) return RN_OK;
        if (!dtable) return RN_ERR_NULL;
        if (misaligned(dtable, gs)) return RN_ERR_ALIGN;
        if (ldg == d) return done(cudaMemsetAsync(dtable, 0, (size_t)(vocab * d * gs), s));
        return done(cudaMemset2DAsync(dtable, (size_t)(ldg * gs), 0, (size_t)(d * gs),
                                      (size_t)vocab, s));
    }
    if (!dout || !tokens || !dtable || !workspace) return RN_ERR_NULL;
    if (misaligned(dout, es) || misaligned(tokens, is) || misaligned(dtable, gs) ||
        misaligned(workspace, 16))
        return RN_ERR_ALIGN;
    const EmbedWorkspace w = embed_workspace(n, d);
    if (workspace_bytes < (size_t)w.total) return RN_ERR_SIZE;
    const Range outs[] = {{dtable, span(vocab, d, ldg) * gs}, {workspace, w.total}};
    const Range ins[] = {{dout, span(n, d, lddo) * es}, {tokens, n * is}};
    if (aliased(outs, ins)) return RN_ERR_ALIAS;
    if (host_resident(workspace)) return RN_ERR_HOSTMEM;
    char* const base = (char*)workspace;
    SortParams sp = {};
    sp.tokens = tokens;
    sp.n = n;
    sp.vocab = vocab;
    for (int k = 0; k < 2; ++k) {
        sp.key[k] = (uint32_t*)(base + w.key[k]);
        sp.pos[k] = (int32_t*)(base + w.pos[k]);
    }
    sp.hist = (uint32_t*)(base + w.hist);
    sp.zeroed = (uint32_t*)(base + w.longs);
    sp.tiles = (int)w.tiles;
    sp.itype = itype;
    if (!accumulate) {
        sp.zero = (char*)dtable;
        sp.zero_pitch = ldg * gs;
        sp.zero_bytes = d * gs;
        // (the bulk-copy engine is given device memory only)
        sp.bulk = embed_few(n, d, es) && sp.zero_bytes >= kZeroBulk && !host_resident(dtable);
    }
    EmbedBwdParams p = {};
    p.dout = dout;
    p.dtable = dtable;
    p.key = sp.key[0];
    p.pos = sp.pos[0];
    p.part = (float*)(base + w.part);
    p.longs = sp.zeroed;
    p.n = n;
    p.vocab = vocab;
    p.d = d;
    p.dpad = w.dpad;
    p.lddo = lddo;
    p.ldg = ldg;
    p.chunks = w.chunks;
    p.chunk = embed_chunk(n, d);
    p.scale = scale;
    p.accumulate = accumulate != 0;
    const int ne = access_elems(d, dout, es, lddo, dtable, gs, ldg);
    return done(embed_bwd_launch(dtype, gtype, ne, sp, p, s));
}

int logprob_fwd(int dtype, int itype, const void* logits, int64_t ldl, const void* targets,
                float* logp, float* entropy, float* lse, void* top_ids, float* top_logp,
                int64_t rows, int64_t vocab, int top, float scale, void* stream) {
    if (!known_dtype(dtype) || !known_index(itype)) return RN_ERR_DTYPE;
    if (rows < 0 || rows > kMaxCount || vocab <= 0 || vocab > kMaxVocab || ldl < vocab ||
        !fits(rows, vocab, ldl) || top < 0 || top > RN_LOGPROB_MAX_TOP || top > vocab)
        return RN_ERR_SIZE;
    if (!std::isfinite(scale) || scale <= 0.f) return RN_ERR_SCALE;
    if (rows == 0) return RN_OK;
    if (!logits || (logp && !targets)) return RN_ERR_NULL;
    if (top == 0) {
        top_ids = nullptr;
        top_logp = nullptr;
    } else if (!top_ids && !top_logp) {
        return RN_ERR_NULL;
    }
    if (!logp && !entropy && !lse && top == 0) return RN_ERR_NULL;
    const int es = dtype_size(dtype), is = index_size(itype);
    if (misaligned(logits, es) || misaligned(targets, is) || misaligned(logp, 4) ||
        misaligned(entropy, 4) || misaligned(lse, 4) || misaligned(top_ids, is) ||
        misaligned(top_logp, 4))
        return RN_ERR_ALIGN;
    const Range outs[] = {{logp, rows * 4},
                          {entropy, rows * 4},
                          {lse, rows * 4},
                          {top_ids, rows * top * is},
                          {top_logp, rows * top * 4}};
    const Range ins[] = {{logits, span(rows, vocab, ldl) * es}, {targets, rows * is}};
    if (aliased(outs, ins)) return RN_ERR_ALIAS;
    LogprobParams p;
    p.logits = logits;
    p.targets = targets;
    p.logp = logp;
    p.entropy = entropy;
    p.lse = lse;
    p.top_ids = top_ids;
    p.top_logp = top_logp;
    p.rows = rows;
    p.ld = ldl;
    p.vocab = (int)vocab;
    p.top = top;
    p.itype = itype;
    p.scale = scale;
    return done(logprob_fwd_launch(dtype, p, (cudaStream_t)stream));
}

int logprob_bwd(int dtype, int itype, const float* dlogp, const float* dentropy,
                const void* logits, int64_t ldl, const void* targets, const float* lse,
                const float* entropy, void* dlogits, int64_t ldd, int64_t rows, int64_t vocab,
                float scale, void* stream) {
    if (!known_dtype(dtype) || !known_index(itype)) return RN_ERR_DTYPE;
    if (rows < 0 || rows > kMaxCount || vocab <= 0 || vocab > kMaxVocab || ldl < vocab ||
        ldd < vocab || !fits(rows, vocab, ldl) || !fits(rows, vocab, ldd))
        return RN_ERR_SIZE;
    if (!std::isfinite(scale) || scale <= 0.f) return RN_ERR_SCALE;
    if (rows == 0) return RN_OK;
    if (!logits || !lse || !dlogits || (!dlogp && !dentropy) || (dlogp && !targets) ||
        (dentropy && !entropy))
        return RN_ERR_NULL;
    if (!dlogp) targets = nullptr;
    if (!dentropy) entropy = nullptr;
    const int es = dtype_size(dtype), is = index_size(itype);
    if (misaligned(logits, es) || misaligned(dlogits, es) || misaligned(targets, is) ||
        misaligned(dlogp, 4) || misaligned(dentropy, 4) || misaligned(lse, 4) ||
        misaligned(entropy, 4))
        return RN_ERR_ALIGN;
    const Range outs[] = {{dlogits, span(rows, vocab, ldd) * es}};
    // the one overlap that is allowed: the gradient in place of the logits
    const bool in_place = dlogits == logits && ldd == ldl;
    const Range ins[] = {{in_place ? nullptr : logits, span(rows, vocab, ldl) * es},
                         {targets, rows * is},
                         {dlogp, rows * 4},
                         {dentropy, rows * 4},
                         {lse, rows * 4},
                         {entropy, rows * 4}};
    if (aliased(outs, ins)) return RN_ERR_ALIAS;
    LogprobBwdParams p = {};
    p.dlogp = dlogp;
    p.dentropy = dentropy;
    p.logits = logits;
    p.targets = targets;
    p.lse = lse;
    p.entropy = entropy;
    p.dlogits = dlogits;
    p.rows = rows;
    p.ld = ldl;
    p.ldd = ldd;
    p.vocab = (int)vocab;
    p.itype = itype;
    p.scale = scale;
    const bool vec = ((addr(logits) ^ addr(dlogits)) & 15u) == 0 && ((ldl - ldd) * es) % 16 == 0;
    return done(logprob_bwd_launch(dtype, vec, p, (cudaStream_t)stream));
}

}  // extern "C"
