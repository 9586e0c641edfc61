// abi_softmax.cpp — the C ABI of softmax attention, its paged cache and the position rotation: argument validation, launch
// planning, scratch, dispatch. See include/ssm_scan.h for the contract of every entry point.
#include "ssm_scan.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <tuple>

#include "host_util.h"
#include "launch_attn.h"
#include "launch_softmax.h"

namespace {

using ssm::KvAppendLaunch;
using ssm::launchable;
using ssm::mul_ok;
using ssm::overlaps;
using ssm::SoftmaxLaunch;
using ssm::SoftmaxStepLaunch;
using ssm::Span;
using ssm::valid_dtype;

constexpr int64_t kMost = INT64_C(1) << 40;      // elements of any tensor, and reach of any stride
constexpr int64_t kMostStep = INT64_C(1) << 24;  // between tokens: 64 rows are addressed with 32-bit byte offsets
constexpr int64_t kMostTokens = INT64_C(1) << 30;  // of a sequence

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int NO, int NI> bool any_overlap(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (const Span &in : ins)
            if (overlaps(outs[i], in)) return true;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], outs[j])) return true;
    }
    return false;
}

// The caller's workspace, or scratch from the pool that is returned at the end of the call.
struct Scratch {
    void *p = nullptr;
    bool own = false;
    ssm_status_t take(void *workspace, int64_t given, int64_t need, hipStream_t stream) {
        if (need == 0) return SSM_OK;
        if (workspace) {
            if (given < need) return SSM_ERR_SCRATCH;
            if (!aligned16(workspace)) return SSM_ERR_UNSUPPORTED;
            p = workspace;
            return SSM_OK;
        }
        if (ssm::scratch_alloc(&p, (size_t)need, stream) != hipSuccess) return SSM_ERR_HIP;
        own = true;
        return SSM_OK;
    }
    ssm_status_t done(hipError_t e, hipStream_t stream) {
        if (own && hipFreeAsync(p, stream) != hipSuccess) return SSM_ERR_HIP;
        return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    }
};

// A strided tensor [b][t][heads][D] (b is 1 where tokens are packed).
struct View {
    int64_t b, t, heads, D;
    int64_t sb, st, sh;
    // strides as given or dense; false where one is negative or reaches too far. An axis of one element has no stride of its own.
    bool set(bool given, int64_t gb, int64_t gt, int64_t gh) {
        if (!given) {
            sh = D;
            st = heads * D;
            sb = t * st;
            return true;
        }
        const int64_t n[3] = {b, t, heads}, s[3] = {gb, gt, gh};
        int64_t use[3];
        for (int i = 0; i < 3; ++i) {
            int64_t reach = 0;
            if (s[i] < 0 || !mul_ok(s[i], n[i] > 0 ? n[i] : 1, &reach) || reach > kMost) return false;
            use[i] = n[i] > 1 ? s[i] : 0;
        }
        if (use[1] > kMostStep) return false;
        sb = use[0];
        st = t > 1 ? use[1] : D;  // as if more rows followed
        sh = use[2];
        return true;
    }
    Span span(const void *p, int64_t es) const {
        return {p, b < 1 || t < 1 ? 0 : ((b - 1) * sb + (t - 1) * st + (heads - 1) * sh + D) * es};
    }
    // every row of D elements takes 16-byte accesses, and lies past the end of a buffer that ends with the row before
    bool vec(const void *p, int64_t es) const {
        const int64_t v = 16 / es;
        return aligned16(p) && D % v == 0 && st >= D && sb % v == 0 && st % v == 0 && sh % v == 0;
    }
};

ssm_status_t check_heads(int64_t H, int64_t G, int64_t D, ssm_dtype_t dtype, float scale) {
    if (!valid_dtype(dtype)) return SSM_ERR_UNSUPPORTED;
    if (H < 1 || G < 1 || D < 1 || H % G != 0) return SSM_ERR_SHAPE;
    if (D > SSM_ATTN_MAX_D || !std::isfinite(scale)) return SSM_ERR_UNSUPPORTED;
    if (H > kMostStep / D) return SSM_ERR_SHAPE;
    return SSM_OK;
}

ssm::AttnRows attn_rows(const ssm_attn_rows_t &r) {
    return {r.cu_q, r.cu_k, r.len_q, r.len_k, r.b, r.Lq, r.Lk, r.tokens_q, r.tokens_k};
}

// Tokens of queries and keys; checks the rows.
ssm_status_t check_rows(const ssm_attn_rows_t *r, int64_t H, int64_t G, int64_t *tokens_q, int64_t *tokens_k) {
    if (!r) return SSM_ERR_NULL;
    if (r->b < 1 || r->Lq < 0 || r->Lk < 0 || r->Lq > kMostTokens || r->Lk > kMostTokens) return SSM_ERR_SHAPE;
    if ((r->cu_q == nullptr) != (r->cu_k == nullptr)) return SSM_ERR_NULL;
    if (r->cu_q) {
        if (r->tokens_q < 0 || r->tokens_k < 0) return SSM_ERR_SHAPE;
        // offsets are 32-bit
        if (r->tokens_q > INT32_MAX || r->tokens_k > INT32_MAX || r->b >= INT32_MAX) return SSM_ERR_SHAPE;
        *tokens_q = r->tokens_q;
        *tokens_k = r->tokens_k;
    } else if (!mul_ok(r->b, r->Lq, tokens_q) || !mul_ok(r->b, r->Lk, tokens_k)) {
        return SSM_ERR_SHAPE;
    }
    if (*tokens_q > kMost / SSM_ATTN_MAX_D / H || *tokens_k > kMost / SSM_ATTN_MAX_D / G) return SSM_ERR_SHAPE;
    if (r->b > kMost / H) return SSM_ERR_SHAPE;
    // No plan is made of sizes whose blocks alone are more than a launch takes.
    for (const auto &[L, tokens, heads] : {std::tuple(r->Lq, *tokens_q, H), std::tuple(r->Lk, *tokens_k, G)}) {
        int64_t n = 0;
        if (!mul_ok(r->b, ceil_div(L, ssm::kSoftmaxBlock), &n)) return SSM_ERR_SHAPE;
        const int64_t slots = tokens / ssm::kSoftmaxBlock + r->b;
        if (!mul_ok(r->cu_q && slots < n ? slots : n, heads, &n) || !launchable(n, 2 * ssm::kSoftmaxThreads)) return SSM_ERR_SHAPE;
    }
    const ssm::AttnRows z = attn_rows(*r);
    for (const ssm::SoftmaxWork &w : {ssm::softmax_fwd_work(z, H, G, true), ssm::softmax_fwd_work(z, H, G, false),
                                      ssm::softmax_dq_work(z, H, G), ssm::softmax_dkv_work(z, H, G)}) {
        int64_t n = 0;
        if (!mul_ok((w.units + 7) / 8 * 8, w.each, &n) || !launchable(n, 2 * ssm::kSoftmaxThreads)) return SSM_ERR_SHAPE;
        if (w.splits > 1 && !launchable(ssm::softmax_groups(ssm::softmax_join_work(w)), ssm::kSoftmaxThreads)) return SSM_ERR_SHAPE;
    }
    return SSM_OK;
}

struct Prompt {
    View q, k, v, dout;
    SoftmaxLaunch p{};
    ssm_status_t set(const ssm_attn_rows_t &r, int64_t tq, int64_t tk, int64_t H, int64_t G, int64_t D, ssm_dtype_t dtype,
                     const ssm_attn_strides_t *s) {
        const bool packed = r.cu_q != nullptr;
        const int64_t b = packed ? 1 : r.b, lq = packed ? tq : r.Lq, lk = packed ? tk : r.Lk;
        q = {b, lq, H, D, 0, 0, 0};
        k = v = {b, lk, G, D, 0, 0, 0};
        dout = q;
        const ssm_attn_strides_t z{}, &u = s ? *s : z;
        if (!q.set(s, u.q_b, u.q_t, u.q_h) || !k.set(s, u.k_b, u.k_t, u.k_h) || !v.set(s, u.v_b, u.v_t, u.v_h) ||
            !dout.set(s, u.do_b, u.do_t, u.do_h))
            return SSM_ERR_SHAPE;
        p.rows = attn_rows(r);
        p.H = (int)H; p.G = (int)G; p.D = (int)D;
        p.bf16 = dtype == SSM_BF16;
        p.q_b = packed ? 0 : q.sb; p.q_t = q.st; p.q_h = q.sh;
        p.k_b = packed ? 0 : k.sb; p.k_t = k.st; p.k_h = k.sh;
        p.v_b = packed ? 0 : v.sb; p.v_t = v.st; p.v_h = v.sh;
        p.do_b = packed ? 0 : dout.sb; p.do_t = dout.st; p.do_h = dout.sh;
        return SSM_OK;
    }
};

int64_t offsets_bytes(const ssm_attn_rows_t &r, const int32_t *p) { return p ? (r.b + (r.cu_q ? 1 : 0)) * 4 : 0; }

// Bytes of the pieces of a forward call's walks; of a gradient's stats and pieces, which the queries' gradient and the keys' hold
// one after the other.
int64_t fwd_bytes(const ssm_attn_rows_t &r, int64_t tq, int64_t H, int64_t G, int64_t D, ssm_dtype_t dtype) {
    const int64_t n = ssm::softmax_fwd_work(attn_rows(r), H, G, dtype == SSM_BF16).splits;
    return n > 1 ? n * tq * H * (D + 2) * 4 : 0;
}
int64_t stats_bytes(const ssm_attn_rows_t &r, int64_t tq, int64_t H, int64_t G) {
    return ceil_div((2 + ssm::softmax_dq_work(attn_rows(r), H, G).splits) * tq * H * 4, 256) * 256;
}
int64_t bwd_bytes(const ssm_attn_rows_t &r, int64_t tq, int64_t tk, int64_t H, int64_t G, int64_t D) {
    const int64_t nq = ssm::softmax_dq_work(attn_rows(r), H, G).splits, nk = ssm::softmax_dkv_work(attn_rows(r), H, G).splits;
    const int64_t q = nq > 1 ? nq * tq * H * D * 4 : 0, k = nk > 1 ? 2 * nk * tk * G * D * 4 : 0;
    return stats_bytes(r, tq, H, G) + (q > k ? q : k);
}

// ---- the paged cache ---------------------------------------------------------------------------------------------

ssm_status_t check_pages(const ssm_pages_t *g, int64_t G, int64_t D) {
    if (!g) return SSM_ERR_NULL;
    if (g->pages < 1 || g->page_size < 1 || g->max_pages < 1 || g->page_size > (INT64_C(1) << 20) ||
        g->max_pages > kMostTokens / g->page_size || g->pages > INT32_MAX)
        return SSM_ERR_SHAPE;
    const int64_t dense = g->page_size * G * D;
    for (const int64_t s : {g->k_page, g->v_page}) {
        int64_t reach = 0;
        if (s < 0 || (s > 0 && s < dense && g->pages > 1)) return SSM_ERR_SHAPE;
        if (!mul_ok(s > 0 ? s : dense, g->pages, &reach) || reach > kMost) return SSM_ERR_SHAPE;
    }
    return SSM_OK;
}

int64_t page_stride(const ssm_pages_t &g, int64_t given, int64_t G, int64_t D) {
    return given > 0 ? given : g.page_size * G * D;
}
Span cache_span(const ssm_pages_t &g, const void *p, int64_t stride, int64_t G, int64_t D, int64_t es) {
    return {p, ((g.pages - 1) * stride + g.page_size * G * D) * es};
}
// Whether no page of one cache overlaps a page of the other (both may lie in one pool, page about).
bool caches_apart(const ssm_pages_t &g, const Span &k, const Span &v, int64_t ks, int64_t vs, int64_t G, int64_t D, int64_t es) {
    if (!overlaps(k, v)) return true;
    if (ks != vs) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(k.p), b = reinterpret_cast<uintptr_t>(v.p);
    const int64_t step = ks * es, gap = (int64_t)((a < b ? b - a : a - b) % (uintptr_t)step), page = g.page_size * G * D * es;
    return gap >= page && step - gap >= page;
}

constexpr int kLeast = 256;         // tokens of a piece: one tile for each wavefront
constexpr int64_t kGroups = 512;    // workgroups that fill the device (two on each of 256 compute units)
// Tokens of a piece, so that one long row among short ones is spread too. Pieces of 2048, 4096 and 8192, us (bf16, 32 heads on 8 key
// heads of 128): 64 rows of up to 8192: 237, 260, 293; one of 8192 among 63 short ones 70, 79, 124; 64 of up to 16384 437, 437,
// 488, one among short ones 103, 96, 137; 256 of up to 8192 790, 807, 846, one among short ones 176, 115, 146.
constexpr int64_t kLongest = 4096;

// Pieces that the longest row is cut into.
int64_t step_splits(int64_t b, int64_t H, int64_t G, int64_t max_len) {
    const int64_t groups = b * G * ceil_div(H / G, 16), most = ceil_div(max_len, kLeast);
    int64_t n = ceil_div(kGroups, groups);
    if (n < ceil_div(max_len, kLongest)) n = ceil_div(max_len, kLongest);
    return n < 1 || most < 1 ? 1 : (n > most ? most : n);
}

ssm_status_t plan_step(int64_t b, int64_t H, int64_t G, int64_t D, const ssm_pages_t *g, int64_t max_len, int64_t *splits,
                       int64_t *bytes) {
    if (b < 1 || b > kMost / SSM_ATTN_MAX_D || max_len < 0) return SSM_ERR_SHAPE;
    const ssm_status_t st = check_pages(g, G, D);
    if (st != SSM_OK) return st;
    int64_t bh = 0, n = 0;
    if (!mul_ok(b, H, &bh) || bh > kMost / SSM_ATTN_MAX_D || !launchable(bh, ssm::kSoftmaxThreads)) return SSM_ERR_SHAPE;
    const int64_t table = g->max_pages * g->page_size;
    *splits = step_splits(b, H, G, max_len > 0 && max_len < table ? max_len : table);
    if (!mul_ok(b * G * ceil_div(H / G, 16), *splits, &n) || !launchable(n, ssm::kSoftmaxThreads)) return SSM_ERR_SHAPE;
    *bytes = *splits > 1 ? bh * *splits * (D + 2) * 4 : 0;
    return SSM_OK;
}

// ---- new tokens ----------------------------------------------------------------------------------------------------

ssm_status_t check_tokens(const ssm_tokens_t *t) {
    if (!t) return SSM_ERR_NULL;
    int64_t n = 0;
    if (t->b < 1 || t->b >= INT32_MAX || t->T < 0 || !launchable(t->T, ssm::kAppendThreads)) return SSM_ERR_SHAPE;
    if (!t->cu && (t->L < 0 || !mul_ok(t->b, t->L, &n) || n != t->T)) return SSM_ERR_SHAPE;
    return SSM_OK;
}
ssm_status_t check_rotation(const double *freq, int64_t rotary, int64_t D) {
    return freq && (rotary < 2 || rotary % 2 != 0 || rotary > D) ? SSM_ERR_SHAPE : SSM_OK;
}
// Whether `out` may take x's place: all of it, dense.
bool in_place(const View &x, const void *p, const void *out) {
    View d = x;
    (void)d.set(false, 0, 0, 0);
    return p == out && (x.heads == 1 || x.sh == d.sh) && (x.t <= 1 || x.st == d.st) && (x.b <= 1 || x.sb == d.sb);
}
void set_tokens(const ssm_tokens_t &t, const double *freq, int64_t rotary, int32_t interleaved, ssm_dtype_t dtype,
                KvAppendLaunch *p) {
    p->tokens = {t.cu, t.new_lengths, t.b, t.L, t.T};
    p->freq = freq;
    p->rotary = freq ? (int)rotary : 0;
    p->interleaved = interleaved != 0;
    p->bf16 = dtype == SSM_BF16;
}
// Whether the rotated part of a head falls into 16-byte pieces: of both halves, or of pairs in turn.
bool vec_rotation(const KvAppendLaunch &p, int64_t es) { return p.rotary % (2 * (16 / es)) == 0; }

}  // namespace

extern "C" {

ssm_status_t ssm_attn_fwd_workspace(const ssm_attn_rows_t *rows, int64_t H, int64_t G, int64_t D, ssm_dtype_t dtype,
                                    int64_t *bytes) {
    if (!bytes) return SSM_ERR_NULL;
    ssm_status_t st = check_heads(H, G, D, dtype, 1.0f);
    if (st != SSM_OK) return st;
    int64_t tq = 0, tk = 0;
    if ((st = check_rows(rows, H, G, &tq, &tk)) != SSM_OK) return st;
    *bytes = fwd_bytes(*rows, tq, H, G, D, dtype);
    return SSM_OK;
}

ssm_status_t ssm_attn_fwd(const void *q, const void *k, const void *v, float scale, int32_t causal, const ssm_attn_rows_t *rows,
                          void *o, float *lse, int64_t H, int64_t G, int64_t D, ssm_dtype_t dtype,
                          const ssm_attn_strides_t *strides, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    ssm_status_t st = check_heads(H, G, D, dtype, scale);
    if (st != SSM_OK) return st;
    int64_t tq = 0, tk = 0;
    if ((st = check_rows(rows, H, G, &tq, &tk)) != SSM_OK) return st;
    Prompt c;
    if ((st = c.set(*rows, tq, tk, H, G, D, dtype, strides)) != SSM_OK) return st;
    if ((tq > 0 && (!q || !o)) || (tk > 0 && (!k || !v))) return SSM_ERR_NULL;
    const int64_t es = dtype == SSM_BF16 ? 2 : 4, need = fwd_bytes(*rows, tq, H, G, D, dtype);
    const Span outs[] = {{o, tq * H * D * es}, {lse, tq * H * 4}, {workspace, need}};
    const Span ins[] = {c.q.span(q, es), c.k.span(k, es), c.v.span(v, es), {rows->cu_q, offsets_bytes(*rows, rows->cu_q)},
                        {rows->cu_k, offsets_bytes(*rows, rows->cu_k)}, {rows->len_q, offsets_bytes(*rows, rows->len_q)},
                        {rows->len_k, offsets_bytes(*rows, rows->len_k)}};
    if (any_overlap(outs, ins)) return SSM_ERR_ALIAS;
    if (tq == 0 || rows->Lq == 0) return SSM_OK;
    Scratch scratch;
    if ((st = scratch.take(workspace, workspace_bytes, need, stream)) != SSM_OK) return st;
    SoftmaxLaunch &p = c.p;
    p.part = static_cast<float *>(scratch.p);
    p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse;
    p.scale = scale;
    p.causal = causal != 0;
    p.vec = c.q.vec(q, es) && c.k.vec(k, es) && c.v.vec(v, es) && aligned16(o);
    return scratch.done(ssm::launch_softmax_fwd(p, stream), stream);
}

ssm_status_t ssm_attn_bwd_workspace(const ssm_attn_rows_t *rows, int64_t H, int64_t G, int64_t D, int64_t *bytes) {
    if (!bytes) return SSM_ERR_NULL;
    ssm_status_t st = check_heads(H, G, D, SSM_F32, 1.0f);
    if (st != SSM_OK) return st;
    int64_t tq = 0, tk = 0;
    if ((st = check_rows(rows, H, G, &tq, &tk)) != SSM_OK) return st;
    *bytes = bwd_bytes(*rows, tq, tk, H, G, D);
    return SSM_OK;
}

ssm_status_t ssm_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *do_,
                          float scale, int32_t causal, const ssm_attn_rows_t *rows, void *dq, void *dk, void *dv, int64_t H,
                          int64_t G, int64_t D, ssm_dtype_t dtype, const ssm_attn_strides_t *strides, void *workspace,
                          int64_t workspace_bytes, hipStream_t stream) {
    ssm_status_t st = check_heads(H, G, D, dtype, scale);
    if (st != SSM_OK) return st;
    int64_t tq = 0, tk = 0;
    if ((st = check_rows(rows, H, G, &tq, &tk)) != SSM_OK) return st;
    Prompt c;
    if ((st = c.set(*rows, tq, tk, H, G, D, dtype, strides)) != SSM_OK) return st;
    if ((tq > 0 && (!q || !o || !lse || !do_ || !dq)) || (tk > 0 && (!k || !v || !dk || !dv))) return SSM_ERR_NULL;
    const int64_t es = dtype == SSM_BF16 ? 2 : 4, need = bwd_bytes(*rows, tq, tk, H, G, D);
    const Span outs[] = {{dq, tq * H * D * es}, {dk, tk * G * D * es}, {dv, tk * G * D * es}, {workspace, need}};
    const Span ins[] = {c.q.span(q, es), c.k.span(k, es), c.v.span(v, es), c.dout.span(do_, es), {o, tq * H * D * es},
                        {lse, tq * H * 4}, {rows->cu_q, offsets_bytes(*rows, rows->cu_q)},
                        {rows->cu_k, offsets_bytes(*rows, rows->cu_k)}, {rows->len_q, offsets_bytes(*rows, rows->len_q)},
                        {rows->len_k, offsets_bytes(*rows, rows->len_k)}};
    if (any_overlap(outs, ins)) return SSM_ERR_ALIAS;
    Scratch scratch;
    if ((st = scratch.take(workspace, workspace_bytes, need, stream)) != SSM_OK) return st;
    SoftmaxLaunch &p = c.p;
    p.q = q; p.k = k; p.v = v; p.o_in = o; p.lse_in = lse; p.dout = do_;
    p.dq = dq; p.dk = dk; p.dv = dv;
    p.stats = static_cast<float *>(scratch.p);
    p.rest = p.stats + 2 * tq * H;
    p.part = p.stats + stats_bytes(*rows, tq, H, G) / 4;
    p.scale = scale;
    p.causal = causal != 0;
    p.vec = c.q.vec(q, es) && c.k.vec(k, es) && c.v.vec(v, es) && c.dout.vec(do_, es) && aligned16(o) && aligned16(dq) &&
            aligned16(dk) && aligned16(dv);
    return scratch.done(ssm::launch_softmax_bwd(p, stream), stream);
}

ssm_status_t ssm_attn_step_workspace(int64_t b, int64_t H, int64_t G, int64_t D, const ssm_pages_t *pages, int64_t max_len,
                                     int64_t *bytes) {
    if (!bytes) return SSM_ERR_NULL;
    const ssm_status_t st = check_heads(H, G, D, SSM_F32, 1.0f);
    if (st != SSM_OK) return st;
    int64_t splits = 0;
    return plan_step(b, H, G, D, pages, max_len, &splits, bytes);
}

ssm_status_t ssm_attn_step(const void *q, const void *k_cache, const void *v_cache, const ssm_pages_t *pages,
                           const int32_t *lengths, float scale, void *o, float *lse, int64_t b, int64_t H, int64_t G, int64_t D,
                           int64_t q_b, int64_t q_h, int64_t max_len, ssm_dtype_t dtype, void *workspace,
                           int64_t workspace_bytes, hipStream_t stream) {
    ssm_status_t st = check_heads(H, G, D, dtype, scale);
    if (st != SSM_OK) return st;
    int64_t splits = 0, need = 0;
    if ((st = plan_step(b, H, G, D, pages, max_len, &splits, &need)) != SSM_OK) return st;
    View qv{1, b, H, D, 0, 0, 0};
    if (!qv.set(q_b != 0 || q_h != 0, 0, q_b, q_h)) return SSM_ERR_SHAPE;
    if (!q || !k_cache || !v_cache || !lengths || !pages->page_table || !o) return SSM_ERR_NULL;
    const int64_t es = dtype == SSM_BF16 ? 2 : 4;
    SoftmaxStepLaunch p{};
    p.k_page = page_stride(*pages, pages->k_page, G, D);
    p.v_page = page_stride(*pages, pages->v_page, G, D);
    const Span outs[] = {{o, b * H * D * es}, {lse, b * H * 4}, {workspace, need}};
    const Span ins[] = {qv.span(q, es), cache_span(*pages, k_cache, p.k_page, G, D, es),
                        cache_span(*pages, v_cache, p.v_page, G, D, es), {pages->page_table, b * pages->max_pages * 4},
                        {lengths, b * 4}};
    if (any_overlap(outs, ins)) return SSM_ERR_ALIAS;
    Scratch scratch;
    if ((st = scratch.take(workspace, workspace_bytes, need, stream)) != SSM_OK) return st;
    p.q = q; p.k_cache = k_cache; p.v_cache = v_cache;
    p.pages = {pages->page_table, pages->max_pages, pages->pages, (int32_t)pages->page_size};
    p.lengths = lengths;
    p.scale = scale;
    p.bf16 = dtype == SSM_BF16;
    p.b = b; p.H = (int)H; p.G = (int)G; p.D = (int)D;
    p.q_b = qv.st; p.q_h = qv.sh;
    p.o = o; p.lse = lse;
    p.splits = (int)splits;
    p.least = kLeast;
    p.part = static_cast<float *>(scratch.p);
    const int64_t vl = 16 / es;
    p.vec = qv.vec(q, es) && aligned16(k_cache) && aligned16(v_cache) && p.k_page % vl == 0 && p.v_page % vl == 0;
    return scratch.done(ssm::launch_softmax_step(p, stream), stream);
}

ssm_status_t ssm_kv_append(const void *q, const void *k, const void *v, void *q_out, void *k_out, void *k_cache, void *v_cache,
                           const ssm_pages_t *pages, const int32_t *lengths, const ssm_tokens_t *tokens, const double *freq,
                           int64_t rotary, int32_t interleaved, int64_t H, int64_t G, int64_t D, ssm_dtype_t dtype,
                           const ssm_attn_strides_t *strides, hipStream_t stream) {
    ssm_status_t st = check_heads(H, G, D, dtype, 1.0f);
    if (st != SSM_OK) return st;
    if ((st = check_pages(pages, G, D)) != SSM_OK) return st;
    if ((st = check_tokens(tokens)) != SSM_OK) return st;
    if ((st = check_rotation(freq, rotary, D)) != SSM_OK) return st;
    const bool packed = tokens->cu != nullptr;
    const int64_t vb = packed ? 1 : tokens->b, vt = packed ? tokens->T : tokens->L;
    View qv{vb, vt, H, D, 0, 0, 0}, kv{vb, vt, G, D, 0, 0, 0}, vv = kv;
    const ssm_attn_strides_t z{}, &u = strides ? *strides : z;
    if (!qv.set(strides, u.q_b, u.q_t, u.q_h) || !kv.set(strides, u.k_b, u.k_t, u.k_h) || !vv.set(strides, u.v_b, u.v_t, u.v_h))
        return SSM_ERR_SHAPE;
    if ((q == nullptr) != (q_out == nullptr) || !k_cache || !v_cache || !pages->page_table || !lengths) return SSM_ERR_NULL;
    if (tokens->T > 0 && (!k || !v)) return SSM_ERR_NULL;
    const int64_t es = dtype == SSM_BF16 ? 2 : 4;
    KvAppendLaunch p{};
    p.k_page = page_stride(*pages, pages->k_page, G, D);
    p.v_page = page_stride(*pages, pages->v_page, G, D);
    const Span kc = cache_span(*pages, k_cache, p.k_page, G, D, es), vc = cache_span(*pages, v_cache, p.v_page, G, D, es);
    if (!caches_apart(*pages, kc, vc, p.k_page, p.v_page, G, D, es)) return SSM_ERR_ALIAS;
    const Span qo{q_out, tokens->T * H * D * es}, ko{k_out, tokens->T * G * D * es};
    const Span qs = in_place(qv, q, q_out) ? Span{nullptr, 0} : qv.span(q, es);
    const Span ks = in_place(kv, k, k_out) ? Span{nullptr, 0} : kv.span(k, es);
    const Span rest[] = {vv.span(v, es), {pages->page_table, tokens->b * pages->max_pages * 4}, {lengths, tokens->b * 4},
                         {tokens->cu, packed ? (tokens->b + 1) * 4 : 0},
                         {tokens->new_lengths, packed ? 0 : tokens->b * 4}, {freq, freq ? rotary / 2 * 8 : 0}};
    for (const Span &out : {qo, ko, kc, vc}) {
        for (const Span &in : rest)
            if (overlaps(out, in)) return SSM_ERR_ALIAS;
        if (overlaps(out, qs) || overlaps(out, ks)) return SSM_ERR_ALIAS;
    }
    if (overlaps(qo, ko) || overlaps(qo, kc) || overlaps(qo, vc) || overlaps(ko, kc) || overlaps(ko, vc)) return SSM_ERR_ALIAS;
    if (tokens->T == 0) return SSM_OK;
    p.q = q; p.k = k; p.v = v;
    p.q_out = q_out; p.k_out = k_out; p.k_cache = k_cache; p.v_cache = v_cache;
    p.pages = {pages->page_table, pages->max_pages, pages->pages, (int32_t)pages->page_size};
    p.lengths = lengths;
    set_tokens(*tokens, freq, rotary, interleaved, dtype, &p);
    p.H = (int)H; p.G = (int)G; p.D = (int)D;
    p.q_b = qv.sb; p.q_t = qv.st; p.q_h = qv.sh;
    p.k_b = kv.sb; p.k_t = kv.st; p.k_h = kv.sh;
    p.v_b = vv.sb; p.v_t = vv.st; p.v_h = vv.sh;
    const int64_t vl = 16 / es;
    p.vec = (!q || qv.vec(q, es)) && kv.vec(k, es) && vv.vec(v, es) && aligned16(q_out) && aligned16(k_out) &&
            aligned16(k_cache) && aligned16(v_cache) && p.k_page % vl == 0 && p.v_page % vl == 0 && vec_rotation(p, es);
    return ssm::launch_kv_append(p, stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

ssm_status_t ssm_rope(const void *x, void *out, const int32_t *lengths, const ssm_tokens_t *tokens, const double *freq,
                      int64_t rotary, int32_t interleaved, int32_t inverse, int64_t H, int64_t D, int64_t x_b, int64_t x_t,
                      int64_t x_h, ssm_dtype_t dtype, hipStream_t stream) {
    ssm_status_t st = check_heads(H, 1, D, dtype, 1.0f);
    if (st != SSM_OK) return st;
    if ((st = check_tokens(tokens)) != SSM_OK) return st;
    if (!freq) return SSM_ERR_NULL;
    if ((st = check_rotation(freq, rotary, D)) != SSM_OK) return st;
    const bool packed = tokens->cu != nullptr;
    View xv{packed ? 1 : tokens->b, packed ? tokens->T : tokens->L, H, D, 0, 0, 0};
    if (!xv.set(x_b != 0 || x_t != 0 || x_h != 0, x_b, x_t, x_h)) return SSM_ERR_SHAPE;
    if (tokens->T > 0 && (!x || !out)) return SSM_ERR_NULL;
    const int64_t es = dtype == SSM_BF16 ? 2 : 4;
    const Span outs[] = {{out, tokens->T * H * D * es}};
    const Span ins[] = {in_place(xv, x, out) ? Span{nullptr, 0} : xv.span(x, es), {lengths, tokens->b * 4},
                        {tokens->cu, packed ? (tokens->b + 1) * 4 : 0},
                        {tokens->new_lengths, packed ? 0 : tokens->b * 4}, {freq, rotary / 2 * 8}};
    if (any_overlap(outs, ins)) return SSM_ERR_ALIAS;
    if (tokens->T == 0) return SSM_OK;
    KvAppendLaunch p{};
    p.q = x;
    p.q_out = out;
    p.lengths = lengths;
    set_tokens(*tokens, freq, rotary, interleaved, dtype, &p);
    p.inverse = inverse != 0;
    p.H = (int)H; p.G = 1; p.D = (int)D;
    p.q_b = xv.sb; p.q_t = xv.st; p.q_h = xv.sh;
    p.vec = xv.vec(x, es) && aligned16(out) && vec_rotation(p, es);
    return ssm::launch_kv_append(p, stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
