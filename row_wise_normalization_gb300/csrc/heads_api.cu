// heads_api.cu -- the C ABI of the head operators (include/rownorm.h): argument
// validation, the choice of access width and lanes, and launch.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "rownorm.h"
#include "rn_boxes.h"
#include "rn_heads.h"

namespace rn {
cudaError_t heads_fwd_f32(HeadShape, const HeadsParams&, cudaStream_t);
cudaError_t heads_fwd_bf16(HeadShape, const HeadsParams&, cudaStream_t);
cudaError_t heads_fwd_f16(HeadShape, const HeadsParams&, cudaStream_t);
cudaError_t heads_append_f32(HeadShape, const HeadsParams&, cudaStream_t);
cudaError_t heads_append_bf16(HeadShape, const HeadsParams&, cudaStream_t);
cudaError_t heads_append_f16(HeadShape, const HeadsParams&, cudaStream_t);
cudaError_t heads_append8_f32(HeadShape, const HeadsParams&, cudaStream_t);
cudaError_t heads_append8_bf16(HeadShape, const HeadsParams&, cudaStream_t);
cudaError_t heads_append8_f16(HeadShape, const HeadsParams&, cudaStream_t);
cudaError_t heads_bwd_f32(HeadShape, const HeadsParams&, int, void*, void*, cudaStream_t);
cudaError_t heads_bwd_bf16(HeadShape, const HeadsParams&, int, void*, void*, cudaStream_t);
cudaError_t heads_bwd_f16(HeadShape, const HeadsParams&, int, void*, void*, cudaStream_t);

cudaError_t heads_fwd_launch(int dtype, int cache_dtype, HeadShape sh, const HeadsParams& p,
                             cudaStream_t s) {
    const int kind = cache_dtype < 0 ? 0 : cache_dtype != DT_E4M3 ? 1 : 2;
    using Run = cudaError_t (*)(HeadShape, const HeadsParams&, cudaStream_t);
    static const Run runs[3][3] = {{heads_fwd_f32, heads_fwd_bf16, heads_fwd_f16},
                                   {heads_append_f32, heads_append_bf16, heads_append_f16},
                                   {heads_append8_f32, heads_append8_bf16, heads_append8_f16}};
    return runs[kind][dtype](sh, p, s);        // (DT_F32, DT_BF16, DT_F16: 0, 1, 2)
}
cudaError_t heads_bwd_launch(int dtype, HeadShape sh, const HeadsParams& p, int ctas, void* dwq,
                             void* dwk, cudaStream_t s) {
    switch (dtype) {
        case DT_BF16: return heads_bwd_bf16(sh, p, ctas, dwq, dwk, s);
        case DT_F16: return heads_bwd_f16(sh, p, ctas, dwq, dwk, s);
        default: return heads_bwd_f32(sh, p, ctas, dwq, dwk, s);
    }
}
}  // namespace rn

namespace {

using namespace rn;

constexpr int64_t kMaxCount = ((int64_t)1 << 31) - 1;

bool known_dtype(int d) { return d == DT_F32 || d == DT_BF16 || d == DT_F16; }
bool known_index(int t) { return t == IT_I32 || t == IT_I64; }
int elem_size(int dtype) { return dtype == DT_E4M3 ? 1 : dtype_size(dtype); }
bool misaligned(const void* p, int64_t a) { return ((uintptr_t)p & (uintptr_t)(a - 1)) != 0; }
int done(cudaError_t err) { return err == cudaSuccess ? RN_OK : record_cuda_error(err); }

Box box(const rn_heads& h, int64_t batch, int64_t len, int64_t d, int es) {
    return {h.heads > 0 ? h.data : nullptr,
            {batch, len, h.heads},
            {h.batch_stride * es, h.token_stride * es, h.head_stride * es},
            d * es};
}
// Strides whose bytes still fit, and heads, and an address of the elements' alignment.
int check_heads(const rn_heads& h, int64_t batch, int64_t len, int64_t d, int es, bool data) {
    if (h.heads < 0 || h.heads > RN_MAX_HEADS) return RN_ERR_SIZE;
    if (h.heads == 0) return RN_OK;
    for (int64_t st : {h.batch_stride, h.token_stride, h.head_stride})
        if (st < 0 || st > kMaxElems / 4) return RN_ERR_SIZE;
    if (!fits(box(h, batch, len, d, es))) return RN_ERR_SIZE;
    if (!data) return RN_OK;
    if (!h.data) return RN_ERR_NULL;
    return misaligned(h.data, es) ? RN_ERR_ALIGN : RN_OK;
}
// Whether accesses of v elements of es bytes suit the rows of h.
bool suits(const rn_heads& h, int64_t batch, int64_t len, int v, int es) {
    return h.heads == 0 || (!misaligned(h.data, v * es) && (batch <= 1 || h.batch_stride % v == 0) &&
                            (len <= 1 || h.token_stride % v == 0) &&
                            (h.heads <= 1 || h.head_stride % v == 0));
}
bool same_rows(const rn_heads& a, const rn_heads& b, int64_t batch, int64_t len) {
    return a.data == b.data && (batch <= 1 || a.batch_stride == b.batch_stride) &&
           (len <= 1 || a.token_stride == b.token_stride) &&
           (a.heads <= 1 || a.head_stride == b.head_stride);
}

// What every call on queries and keys checks first. `rows`: their data is read.
int check_qk(const rn_qk* in, bool rows, int* es) {
    if (!in) return RN_ERR_NULL;
    if (!known_dtype(in->dtype) || (in->rot != 0 && !known_index(in->itype))) return RN_ERR_DTYPE;
    *es = dtype_size(in->dtype);
    if (in->batch < 0 || in->len < 0 || in->d < 2 || in->d > kMaxHeadDim || in->d % 2 ||
        in->rot < 0 || in->rot > in->d || in->rot % 2)
        return RN_ERR_SIZE;
    if (in->batch > kMaxCount || in->len > kMaxCount || in->batch * in->len > kMaxCount)
        return RN_ERR_SIZE;
    if (in->rot > 0 && (in->table_rows <= 0 || in->table_stride < in->rot ||
                        in->table_stride > kMaxElems / 4 || in->table_rows > kMaxElems / 4 ||
                        (in->table_rows - 1) > (kMaxElems / 4 - in->rot) / in->table_stride))
        return RN_ERR_SIZE;
    if (in->norm && (!(in->eps >= 0.f) || std::isinf(in->eps))) return RN_ERR_EPS;
    if (in->q.heads + in->k.heads <= 0) return RN_ERR_SIZE;
    if (in->batch * in->len == 0) return RN_OK;
    int st = check_heads(in->q, in->batch, in->len, in->d, *es, rows);
    if (st == RN_OK) st = check_heads(in->k, in->batch, in->len, in->d, *es, rows);
    if (st != RN_OK) return st;
    if (in->rot > 0) {
        if (!in->positions || !in->table) return RN_ERR_NULL;
        if (misaligned(in->positions, index_size(in->itype)) || misaligned(in->table, 4))
            return RN_ERR_ALIGN;
    }
    if (in->norm && (misaligned(in->wq, *es) || misaligned(in->wk, *es))) return RN_ERR_ALIGN;
    return RN_OK;
}
// An output's rows, of `heads` heads.
int check_out(const rn_heads* h, int64_t heads, int64_t batch, int64_t len, int64_t d, int es) {
    if (!h) return heads > 0 ? RN_ERR_NULL : RN_OK;
    if (h->heads != heads) return RN_ERR_SIZE;
    return check_heads(*h, batch, len, d, es, true);
}

// Side inputs that outputs must not touch.
struct Sides {
    Box w[2], positions, table;
};
Sides sides(const rn_qk& in, int es) {
    const int64_t n = in.batch * in.len;
    const bool rot = in.rot > 0;
    return {{flat(in.norm ? in.wq : nullptr, in.d * es), flat(in.norm ? in.wk : nullptr, in.d * es)},
            flat(rot ? in.positions : nullptr, n * index_size(in.itype)),
            flat(rot ? in.table : nullptr,
                 rot ? ((in.table_rows - 1) * in.table_stride + in.rot) * 4 : 0)};
}

// Whether accesses of v elements suit the table, the weights, and pairs of vectors the row.
bool row_suits(const rn_qk& in, int v, int es) {
    if (in.rot % (2 * v) || in.d % (2 * v)) return false;
    if (in.rot > 0) {
        const int floats = v < 4 ? v : 4;
        if (misaligned(in.table, 4 * floats) || in.table_stride % floats) return false;
    }
    return !in.norm || (!misaligned(in.wq, v * es) && !misaligned(in.wk, v * es));
}

// The parameters that calls on queries and keys share; least: units an SM should have.
HeadsParams qk_params(const rn_qk& in, const HeadShape& sh, int least) {
    HeadsParams p = {};
    p.len = fast_div((uint32_t)in.len);
    p.tokens = in.batch * in.len;
    p.positions = in.positions;
    p.table = in.table;
    p.table_rows = in.table_rows;
    p.ldt = in.table_stride;
    p.eps = in.eps;
    p.rot = (int)in.rot;
    p.itype = in.itype;
    p.norm = in.norm != 0;
    p.interleaved = in.interleaved != 0;
    p.page = fast_div(1);
    const rn_heads* const x[2] = {&in.q, &in.k};
    for (int i = 0; i < 2; ++i) {
        HeadSeg& g = p.seg[i];
        g.x = x[i]->data;
        g.w = !in.norm ? nullptr : i == 0 ? in.wq : in.wk;
        g.xb = x[i]->batch_stride;
        g.xt = x[i]->token_stride;
        g.xh = x[i]->head_stride;
        g.heads = (int)x[i]->heads;
        p.d[i] = (int)in.d;
    }
    p.per = heads_per_unit(sh.lpr, in.q.heads + in.k.heads, p.tokens, least);
    return p;
}
void set_y(HeadSeg& g, const rn_heads* h) {
    if (!h || h->heads == 0) return;
    g.y = h->data;
    g.yb = h->batch_stride;
    g.yt = h->token_stride;
    g.yh = h->head_stride;
}
// The units of every segment; false where they are too many for one launch. at_once: rows that a
// warp holds; it takes those of several tokens where a token has at most half as many
// (12265 tokens of 8 queries, 2 keys and values of 64 BF16 appended: 12 us, 18 a token at a time),
// as long as that leaves an SM `least` units.
bool set_units(HeadsParams& p, int at_once, int least) {
    int64_t total = 0;
    for (int i = 0; i < 2; ++i) {           // (values go with their keys)
        HeadSeg& g = p.seg[i];
        const int64_t groups = (g.heads + p.per - 1) / p.per;
        g.per = fast_div((uint32_t)(groups > 0 ? groups : 1));
        g.pack = 1;
        if (groups == 1)
            for (g.pack = at_once / g.heads; g.pack > 1 && p.tokens / g.pack < 152 * least;)
                g.pack /= 2;
        if (g.pack < 1) g.pack = 1;
        g.few = fast_div((uint32_t)(g.heads > 0 ? g.heads : 1));
        const int64_t units = groups * ((p.tokens + g.pack - 1) / g.pack);
        total += units;
        if (total > kMaxCount) return false;
        g.units = (uint32_t)units;
    }
    p.total = (uint32_t)total;
    return true;
}

// CTAs of the gradient's kernel: kBwdGroups row groups (what a warp holds at once) a warp, so that a
// CTA's start and its sums weigh little, at most kHeadsBwdCtas (several rounds of what the GPU holds
// at once, which evens out CTAs that take longer) and no more than there are units. They are shared
// in proportion to the segments' work, in which a unit's start counts as much as two groups (32768
// tokens of 32 + 8 heads of 96 BF16: 147 us, 151 by groups alone).
struct BwdCtas {
    int q, k;
};
constexpr int kBwdGroups = 16;
constexpr int kBwdStart = 2;
BwdCtas bwd_ctas(const HeadsParams& p, int at_once, int warps) {
    int64_t most[2], groups[2], work[2];
    for (int i = 0; i < 2; ++i) {
        most[i] = ((int64_t)p.seg[i].units + warps - 1) / warps;
        groups[i] = p.seg[i].pack > 1 ? (int64_t)p.seg[i].units
                                      : (p.seg[i].heads + at_once - 1) / at_once * p.tokens;
        work[i] = groups[i] + kBwdStart * (int64_t)p.seg[i].units;
    }
    int64_t ctas = (groups[0] + groups[1]) / (warps * kBwdGroups);
    if (ctas < 152 * kHeadsBwdPerSm) ctas = 152 * kHeadsBwdPerSm;
    if (ctas > kHeadsBwdCtas) ctas = kHeadsBwdCtas;
    const int64_t all = work[0] + work[1];
    int64_t q = (ctas * work[0] + all / 2) / all;
    if (q > ctas - 1 && work[1] > 0) q = ctas - 1;
    if (q < 1 && work[0] > 0) q = 1;
    int64_t k = ctas - q;
    if (q > most[0]) q = most[0];
    if (k > most[1]) k = most[1];
    return {(int)q, (int)k};
}

// The widest access, of the vector (16 bytes of rows), 4, 2 or 1 elements, that `ok` accepts.
template <typename F>
int widest(int vec, F ok) {
    return ok(vec) ? vec : vec > 4 && ok(4) ? 4 : ok(2) ? 2 : 1;
}

int check_cache(const rn_cache* c, int64_t heads, int64_t d, int dtype, int* cs, Box* k, Box* v) {
    if (!c) return RN_ERR_NULL;
    if (c->dtype != DT_E4M3 && c->dtype != dtype) return RN_ERR_DTYPE;
    *cs = elem_size(c->dtype);
    if (c->pages < 0 || c->page_size <= 0 || c->page_size > kMaxCount || c->pages > kMaxCount ||
        c->pages * c->page_size > kMaxCount || c->d_v < 2 || c->d_v > kMaxHeadDim || c->d_v % 2)
        return RN_ERR_SIZE;
    for (int64_t st : {c->k_page_stride, c->k_slot_stride, c->k_head_stride, c->v_page_stride,
                       c->v_slot_stride, c->v_head_stride})
        if (st < 0 || st > kMaxElems / 4) return RN_ERR_SIZE;
    if (c->dtype == DT_E4M3) {
        for (float s : {c->k_scale, c->v_scale})
            if (!std::isfinite(s) || !(s > 0.f) || !std::isfinite(1.f / s)) return RN_ERR_SCALE;
    } else if (c->k_scale != 1.f || c->v_scale != 1.f) {
        return RN_ERR_SCALE;
    }
    *k = {c->k, {c->pages, c->page_size, heads},
          {c->k_page_stride * *cs, c->k_slot_stride * *cs, c->k_head_stride * *cs}, d * *cs};
    *v = {c->v, {c->pages, c->page_size, heads},
          {c->v_page_stride * *cs, c->v_slot_stride * *cs, c->v_head_stride * *cs}, c->d_v * *cs};
    if (!fits(*k) || !fits(*v)) return RN_ERR_SIZE;
    if (c->pages > 0 && (!c->k || !c->v)) return RN_ERR_NULL;
    if (misaligned(c->k, *cs) || misaligned(c->v, *cs)) return RN_ERR_ALIGN;
    return RN_OK;
}
bool cache_suits(const Box& b, int v, int cs) {
    if (b.count[0] <= 0) return true;
    for (int i = 0; i < 3; ++i)
        if (b.count[i] > 1 && b.stride[i] % (v * cs)) return false;
    return !misaligned(b.p, v * cs);
}

}  // namespace

extern "C" {

int qk_rope_fwd(const rn_qk* in, const rn_heads* q_out, const rn_heads* k_out, void* stream) {
    int es = 0;
    int st = check_qk(in, true, &es);
    if (st != RN_OK) return st;
    const int64_t batch = in->batch, len = in->len, d = in->d;
    if (batch * len == 0) return RN_OK;
    st = check_out(q_out, in->q.heads, batch, len, d, es);
    if (st == RN_OK) st = check_out(k_out, in->k.heads, batch, len, d, es);
    if (st != RN_OK) return st;
    const rn_heads none = {};
    if (!q_out) q_out = &none;
    if (!k_out) k_out = &none;
    const Sides sd = sides(*in, es);
    const Box oq = box(*q_out, batch, len, d, es), ok = box(*k_out, batch, len, d, es);
    const Box iq = box(in->q, batch, len, d, es), ik = box(in->k, batch, len, d, es);
    // the one overlap that is allowed: an output in its input's place
    const bool q_in = same_rows(*q_out, in->q, batch, len),
               k_in = same_rows(*k_out, in->k, batch, len);
    const Box outs[] = {oq, ok};
    const Box ins[] = {sd.w[0], sd.w[1], sd.positions, sd.table};
    if (aliased(outs, ins) || !apart(oq, ik) || !apart(ok, iq) || (!q_in && !apart(oq, iq)) ||
        (!k_in && !apart(ok, ik)))
        return RN_ERR_ALIAS;
    const int vec = 16 / es;
    const int v = widest(vec, [&](int w) {
        return row_suits(*in, w, es) && suits(in->q, batch, len, w, es) &&
               suits(in->k, batch, len, w, es) && suits(*q_out, batch, len, w, es) &&
               suits(*k_out, batch, len, w, es);
    });
    const HeadShape sh = head_shape(v, vec, d, false);
    HeadsParams p = qk_params(*in, sh, fwd_units(sh.v));
    set_y(p.seg[0], q_out);
    set_y(p.seg[1], k_out);
    if (!set_units(p, 32 / sh.lpr, fwd_units(sh.v))) return RN_ERR_SIZE;
    return done(heads_fwd_launch(in->dtype, -1, sh, p, (cudaStream_t)stream));
}

int qk_rope_bwd_workspace_size(int64_t d, size_t* bytes) {
    if (!bytes) return RN_ERR_NULL;
    *bytes = 0;
    if (d < 2 || d > kMaxHeadDim || d % 2) return RN_ERR_SIZE;
    *bytes = (size_t)(kHeadsBwdCtas * d * 4);
    return RN_OK;
}

int qk_rope_bwd(const rn_qk* in, const rn_heads* dq_out, const rn_heads* dk_out,
                const rn_heads* dq, const rn_heads* dk, void* dwq, void* dwk, void* workspace,
                size_t workspace_bytes, void* stream) {
    int es = 0;
    int st = check_qk(in, in && in->norm, &es);
    if (st != RN_OK) return st;
    const int64_t batch = in->batch, len = in->len, d = in->d;
    const bool params = dwq || dwk;
    if ((dwq && !(in->norm && in->wq)) || (dwk && !(in->norm && in->wk))) return RN_ERR_NULL;
    if (misaligned(dwq, es) || misaligned(dwk, es)) return RN_ERR_ALIGN;
    const cudaStream_t s = (cudaStream_t)stream;
    if (batch * len == 0) {
        // an empty batch still defines the weights' gradients: zero (all-zero bits in every type)
        cudaError_t err = cudaSuccess;
        if (dwq) err = cudaMemsetAsync(dwq, 0, (size_t)(d * es), s);
        if (dwk && err == cudaSuccess) err = cudaMemsetAsync(dwk, 0, (size_t)(d * es), s);
        return done(err);
    }
    const rn_heads none = {};
    for (const rn_heads** h : {&dq_out, &dk_out, &dq, &dk}) {
        const int64_t heads = h == &dq_out || h == &dq ? in->q.heads : in->k.heads;
        st = check_out(*h, heads, batch, len, d, es);
        if (st != RN_OK) return st;
        if (!*h) *h = &none;
    }
    const size_t need = (size_t)(kHeadsBwdCtas * d * 4);
    if (params) {
        if (!workspace) return RN_ERR_NULL;
        if (misaligned(workspace, 16)) return RN_ERR_ALIGN;
        if (workspace_bytes < need) return RN_ERR_SIZE;
    }
    const Sides sd = sides(*in, es);
    const Box oq = box(*dq, batch, len, d, es), ok = box(*dk, batch, len, d, es);
    const Box gq = box(*dq_out, batch, len, d, es), gk = box(*dk_out, batch, len, d, es);
    const Box iq = in->norm ? box(in->q, batch, len, d, es) : Box{};
    const Box ik = in->norm ? box(in->k, batch, len, d, es) : Box{};
    const Box outs[] = {oq, ok, flat(dwq, d * es), flat(dwk, d * es),
                        flat(params ? workspace : nullptr, (int64_t)need)};
    const Box ins[] = {sd.w[0], sd.w[1], sd.positions, sd.table};
    if (aliased(outs, ins)) return RN_ERR_ALIAS;
    for (int i = 2; i < 5; ++i)
        for (const Box* b : {&iq, &ik, &gq, &gk})
            if (!apart(outs[i], *b)) return RN_ERR_ALIAS;
    // the overlaps that are allowed: an output in the place of either of its inputs
    if (!apart(oq, ik) || !apart(oq, gk) || !apart(ok, iq) || !apart(ok, gq) ||
        (!apart(oq, iq) && !same_rows(*dq, in->q, batch, len)) ||
        (!apart(oq, gq) && !same_rows(*dq, *dq_out, batch, len)) ||
        (!apart(ok, ik) && !same_rows(*dk, in->k, batch, len)) ||
        (!apart(ok, gk) && !same_rows(*dk, *dk_out, batch, len)))
        return RN_ERR_ALIAS;
    const int vec = 16 / es;
    const int v = widest(vec, [&](int w) {
        if (in->norm && !(suits(in->q, batch, len, w, es) && suits(in->k, batch, len, w, es)))
            return false;
        return row_suits(*in, w, es) && suits(*dq_out, batch, len, w, es) &&
               suits(*dk_out, batch, len, w, es) && suits(*dq, batch, len, w, es) &&
               suits(*dk, batch, len, w, es);
    });
    const HeadShape sh = head_shape(v, vec, d, in->norm != 0);
    const bool plain = !in->norm;      // a rotation alone: the forward kernel, turned back
    rn_qk at = *in;
    if (plain) {
        at.q = *dq_out;
        at.k = *dk_out;
    }
    HeadsParams p = qk_params(at, sh, plain ? fwd_units(sh.v) : kBwdUnits);
    set_y(p.seg[0], dq);
    set_y(p.seg[1], dk);
    p.back = true;
    if (!set_units(p, 32 / sh.lpr, fwd_units(sh.v))) return RN_ERR_SIZE;
    if (plain) return done(heads_fwd_launch(in->dtype, -1, sh, p, s));
    const rn_heads* const g[2] = {dq_out, dk_out};
    for (int i = 0; i < 2; ++i) {
        p.seg[i].dy = g[i]->data;
        p.seg[i].gb = g[i]->batch_stride;
        p.seg[i].gt = g[i]->token_stride;
        p.seg[i].gh = g[i]->head_stride;
    }
    p.part = params ? (float*)workspace : nullptr;
    const BwdCtas c = bwd_ctas(p, 32 / sh.lpr, heads_bwd_warps(sh.v, sh.ch));
    p.first_k = c.q;
    const int ctas = c.q + c.k;
    return done(heads_bwd_launch(in->dtype, sh, p, ctas, dwq, dwk, s));
}

int kv_append(const rn_qk* in, const rn_heads* q_out, const rn_heads* v, const rn_cache* cache,
              const void* slots, void* stream) {
    int es = 0;
    int st = check_qk(in, true, &es);
    if (st != RN_OK) return st;
    if (!v || !cache) return RN_ERR_NULL;
    if (!known_index(in->itype)) return RN_ERR_DTYPE;
    const int64_t batch = in->batch, len = in->len, d = in->d, n = batch * len;
    int cs = 0;
    Box bk, bv;
    st = check_cache(cache, in->k.heads, d, in->dtype, &cs, &bk, &bv);
    if (st != RN_OK) return st;
    if (in->k.heads <= 0 || v->heads != in->k.heads) return RN_ERR_SIZE;
    if (n == 0) return RN_OK;
    st = check_heads(*v, batch, len, cache->d_v, es, true);
    if (st == RN_OK) st = check_out(q_out, in->q.heads, batch, len, d, es);
    if (st != RN_OK) return st;
    if (!slots) return RN_ERR_NULL;
    if (misaligned(slots, index_size(in->itype))) return RN_ERR_ALIGN;
    const rn_heads none = {};
    if (!q_out) q_out = &none;
    const Sides sd = sides(*in, es);
    const Box oq = box(*q_out, batch, len, d, es), iq = box(in->q, batch, len, d, es);
    const Box outs[] = {oq, bk, bv};
    const Box ins[] = {sd.w[0], sd.w[1], sd.positions, sd.table,
                       flat(slots, n * index_size(in->itype)), box(in->k, batch, len, d, es),
                       box(*v, batch, len, cache->d_v, es)};
    // the one overlap that is allowed: the queries in their own place
    if (aliased(outs, ins) || !apart(bk, iq) || !apart(bv, iq) ||
        (!apart(oq, iq) && !same_rows(*q_out, in->q, batch, len)))
        return RN_ERR_ALIAS;
    const int vec = 16 / es;
    const int w = widest(vec, [&](int e) {
        return row_suits(*in, e, es) && cache->d_v % (2 * e) == 0 &&
               suits(in->q, batch, len, e, es) && suits(in->k, batch, len, e, es) &&
               suits(*v, batch, len, e, es) && suits(*q_out, batch, len, e, es) &&
               cache_suits(bk, e, cs) && cache_suits(bv, e, cs);
    });
    const HeadShape sh = head_shape(w, vec, d > cache->d_v ? d : cache->d_v, false);
    HeadsParams p = qk_params(*in, sh, fwd_units(sh.v));
    set_y(p.seg[0], q_out);
    HeadSeg& k = p.seg[1];
    k.y = cache->k;
    k.yb = cache->k_page_stride;
    k.yt = cache->k_slot_stride;
    k.yh = cache->k_head_stride;
    HeadSeg& g = p.seg[2];
    g.x = v->data;
    g.xb = v->batch_stride;
    g.xt = v->token_stride;
    g.xh = v->head_stride;
    g.y = cache->v;
    g.yb = cache->v_page_stride;
    g.yt = cache->v_slot_stride;
    g.yh = cache->v_head_stride;
    g.heads = (int)v->heads;
    p.d[2] = (int)cache->d_v;
    p.scale[1] = e4m3_scale(cache->k_scale);
    p.scale[2] = e4m3_scale(cache->v_scale);
    p.slots = slots;
    p.nslots = cache->pages * cache->page_size;
    p.page = fast_div((uint32_t)cache->page_size);
    if (!set_units(p, 32 / sh.lpr, fwd_units(sh.v))) return RN_ERR_SIZE;
    return done(heads_fwd_launch(in->dtype, cache->dtype, sh, p, (cudaStream_t)stream));
}

int kv_gather(const rn_cache* cache, int64_t d, const void* slots, int itype, int64_t n,
              int dtype, const rn_heads* k_out, const rn_heads* v_out, void* stream) {
    if (!cache || !k_out || !v_out) return RN_ERR_NULL;
    if (!known_dtype(dtype) || !known_index(itype)) return RN_ERR_DTYPE;
    const int64_t heads = k_out->heads;
    if (n < 0 || n > kMaxCount || d < 2 || d > kMaxHeadDim || d % 2 || heads <= 0 ||
        heads > RN_MAX_HEADS || v_out->heads != heads)
        return RN_ERR_SIZE;
    const int es = dtype_size(dtype);
    int cs = 0;
    Box bk, bv;
    int st = check_cache(cache, heads, d, dtype, &cs, &bk, &bv);
    if (st != RN_OK) return st;
    if (n == 0) return RN_OK;
    st = check_heads(*k_out, 1, n, d, es, true);
    if (st == RN_OK) st = check_heads(*v_out, 1, n, cache->d_v, es, true);
    if (st != RN_OK) return st;
    if (!slots) return RN_ERR_NULL;
    if (misaligned(slots, index_size(itype))) return RN_ERR_ALIGN;
    const Box outs[] = {box(*k_out, 1, n, d, es), box(*v_out, 1, n, cache->d_v, es)};
    const Box ins[] = {bk, bv, flat(slots, n * index_size(itype))};
    if (aliased(outs, ins)) return RN_ERR_ALIAS;
    // an access: 16 bytes of rows that are copied, 8 of an 8-bit cache's
    const int vec = cache->dtype == DT_E4M3 ? 8 : 16 / es;
    const int ne = widest(vec, [&](int w) {
        const int out = w * es < 16 ? w : 16 / es;     // elements of an output's access
        return d % w == 0 && cache->d_v % w == 0 && cache_suits(bk, w, cs) &&
               cache_suits(bv, w, cs) && suits(*k_out, 1, n, out, es) &&
               suits(*v_out, 1, n, out, es);
    });
    GatherParams p = {};
    p.slots = slots;
    p.nslots = cache->pages * cache->page_size;
    p.page = fast_div((uint32_t)cache->page_size);
    p.itype = itype;
    for (int i = 0; i < 2; ++i) {
        GatherSide& g = p.side[i];
        const rn_heads& o = i == 0 ? *k_out : *v_out;
        const int64_t per = (i == 0 ? d : cache->d_v) / ne;
        g.cache = i == 0 ? cache->k : cache->v;
        g.out = o.data;
        g.cp = i == 0 ? cache->k_page_stride : cache->v_page_stride;
        g.cs = i == 0 ? cache->k_slot_stride : cache->v_slot_stride;
        g.ch = i == 0 ? cache->k_head_stride : cache->v_head_stride;
        g.ot = o.token_stride;
        g.oh = o.head_stride;
        g.total = n * heads * per;
        g.token = fast_div((uint32_t)(heads * per));
        g.head = fast_div((uint32_t)per);
        g.scale = i == 0 ? cache->k_scale : cache->v_scale;
        if (g.total / 1024 >= kMaxCount) return RN_ERR_SIZE;     // (the grid of one launch)
    }
    return done(kv_gather_launch(cache->dtype, dtype, ne, p, (cudaStream_t)stream));
}

int kv_slots(int itype, const void* page_table, int64_t ld, int64_t width, const void* starts,
             const void* offsets, int64_t seqs, int64_t page_size, void* slots, void* positions,
             int64_t n, void* stream) {
    if (!known_index(itype)) return RN_ERR_DTYPE;
    if (n < 0 || n > kMaxCount || seqs < 0 || seqs > (1 << 30) || width < 0 || width > kMaxCount ||
        ld < width || ld > kMaxElems / 8 || page_size <= 0 || page_size > kMaxCount)
        return RN_ERR_SIZE;
    const int is = index_size(itype);
    const Box table = {width > 0 ? page_table : nullptr, {1, 1, seqs}, {0, 0, ld * is}, width * is};
    if (!fits(table)) return RN_ERR_SIZE;
    if (n == 0) return RN_OK;
    if (!slots || !offsets || (seqs > 0 && (!starts || (width > 0 && !page_table))))
        return RN_ERR_NULL;
    if (misaligned(page_table, is) || misaligned(starts, is) || misaligned(offsets, is) ||
        misaligned(slots, is) || misaligned(positions, is))
        return RN_ERR_ALIGN;
    const Box outs[] = {flat(slots, n * is), flat(positions, n * is)};
    const Box ins[] = {table, flat(starts, seqs * is), flat(offsets, (seqs + 1) * is)};
    if (aliased(outs, ins)) return RN_ERR_ALIAS;
    SlotsParams p = {};
    p.page_table = page_table;
    p.starts = starts;
    p.offsets = offsets;
    p.slots = slots;
    p.positions = positions;
    p.n = n;
    p.ld = ld;
    p.width = width;
    p.pages = kMaxCount / page_size;
    p.seqs = (int)seqs;
    p.page = page_size;
    p.itype = itype;
    return done(kv_slots_launch(p, (cudaStream_t)stream));
}

}  // extern "C"
