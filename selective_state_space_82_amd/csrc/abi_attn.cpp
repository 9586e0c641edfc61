// abi_attn.cpp — the C ABI of linear attention and layer norm: argument validation, launch planning, scratch,
// dispatch. See include/ssm_scan.h for the contract of every entry point.
#include "ssm_scan.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "host_util.h"
#include "launch.h"

namespace {

using ssm::LinAttnLaunch;
using ssm::NormLaunch;
using ssm::Span;
using ssm::mul_ok;
using ssm::overlaps;
using ssm::scratch_alloc;
using ssm::valid_dtype;

constexpr int64_t kMost = INT64_C(1) << 40;  // elements of any tensor, and reach of any stride
// A chunk's rows are addressed with 32-bit byte offsets: 64 rows of 2^24 fp32 elements.
constexpr int64_t kMostStep = INT64_C(1) << 24;
constexpr int64_t kChunk = 64, kBlockP = 64;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

// ---- scratch: the caller's workspace, or the pool's ---------------------------------------------------------------

struct Scratch {
    void *p = nullptr;
    bool own = false;
    hipStream_t stream = nullptr;
    ssm_status_t take(void *workspace, int64_t given, int64_t need, hipStream_t s) {
        stream = s;
        if (need == 0) return SSM_OK;
        if (workspace) {
            if (given < need) return SSM_ERR_SCRATCH;
            if (!aligned(workspace, 16)) return SSM_ERR_UNSUPPORTED;
            p = workspace;
            return SSM_OK;
        }
        if (scratch_alloc(&p, (size_t)need, s) != hipSuccess) return SSM_ERR_HIP;
        own = true;
        return SSM_OK;
    }
    ssm_status_t done(hipError_t e) {
        if (own && hipFreeAsync(p, stream) != hipSuccess) return SSM_ERR_HIP;
        return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    }
};

// Hands out pieces of the scratch, 256 bytes apart.
struct Pieces {
    uintptr_t base;
    int64_t at = 0;
    template <typename T> T *next(int64_t n) {
        T *r = reinterpret_cast<T *>(base + (uintptr_t)at);
        at += ceil_div(n * (int64_t)sizeof(T), 256) * 256;
        return r;
    }
};

// ---- linear attention ----------------------------------------------------------------------------------------------

struct AttnSizes {
    int64_t b, L, H, G, N, P;
};

ssm_status_t check_sizes(const AttnSizes &z, ssm_dtype_t dtype) {
    if (!valid_dtype(dtype)) return SSM_ERR_UNSUPPORTED;
    if (z.b < 1 || z.L < 0 || z.H < 1 || z.G < 1 || z.N < 1 || z.P < 1) return SSM_ERR_SHAPE;
    if (z.H % z.G != 0) return SSM_ERR_SHAPE;
    if (z.N > SSM_LINATTN_MAX_N || z.P > SSM_LINATTN_MAX_P) return SSM_ERR_UNSUPPORTED;
    int64_t bl = 0, bh = 0, n = 0;
    const int64_t L = z.L > 0 ? z.L : 1;
    if (!mul_ok(z.b, L, &bl) || !mul_ok(z.b, z.H, &bh) || bl > kMost || bh > kMost) return SSM_ERR_SHAPE;
    // the padded widths bound every tensor and the states of all chunks
    const int64_t width = ceil_div(z.P, kBlockP) * kBlockP;
    if (z.H > kMostStep / (width > 128 ? width : 128)) return SSM_ERR_SHAPE;
    if (!mul_ok(bl, z.H * (width > 128 ? width : 128), &n) || n > kMost) return SSM_ERR_SHAPE;
    if (!mul_ok(bh, ceil_div(L, kChunk) * (width / kBlockP) * 32, &n) || n >= (INT64_C(1) << 31)) return SSM_ERR_SHAPE;
    return SSM_OK;
}

// How the steps are cut into segments. One workgroup walks a segment's chunks in order; the gradient's chunks run
// independently of each other. The forward call takes the number of segments that a count of its time in chunks makes
// least: the rounds in which the device takes its workgroups (two on a compute unit, or one where fp32 tiles of N > 32
// fill its LDS), each of a segment's chunks and half a chunk to start and end; and with more than one segment the walk
// over the segments' own states, 0.4 of a chunk each with four workgroups on a compute unit, and 1.5 for two more
// launches. (fp32, 72 blocks of 16 chunks: 4 segments, 288 workgroups in two rounds, took 71 us.) Planned, as the scan is,
// for 256 compute units, and for at most 64 segments, which the carry steps over one after the other.
void plan(const AttnSizes &z, bool gradient, LinAttnLaunch *p) {
    const int64_t chunks = ceil_div(z.L, kChunk);
    p->seg_chunks = chunks;
    if (gradient) {
        p->seg_chunks = 1;
    } else {
        const int64_t groups = z.b * z.H * ceil_div(z.P, kBlockP);
        const int64_t at_once = 256 * (!p->bf16 && z.N > 32 ? 1 : 2);
        double least = 0.0;
        for (int64_t s = 1; s <= chunks && s <= 64; ++s) {
            const int64_t each = ceil_div(chunks, s), n = ceil_div(chunks, each);
            double t = (double)ceil_div(groups * n, at_once) * ((double)each + 0.5);
            if (n > 1) t += (double)ceil_div(groups * (n - 1), 1024) * (double)each * 0.4 + 1.5;
            if (s == 1 || t < least) {
                least = t;
                p->seg_chunks = each;
            }
        }
    }
    p->n_seg = p->seg_chunks > 0 ? ceil_div(chunks, p->seg_chunks) : 0;
}

// Whether HIP takes every launch of the planned call (launchable() in launch_attn.h).
bool launches(const AttnSizes &z, bool gradient, const LinAttnLaunch &p) {
    if (p.n_seg == 0) return true;
    const int64_t bh = z.b * z.H, blocks = ceil_div(z.P, kBlockP), cols = ssm::linattn_cols(z.P);
    const int64_t walks = gradient ? 2 * p.n_seg - 1 : p.n_seg - 1;  // over the segments' own states and adjoints
    const int64_t carries = bh * (blocks * kBlockP * ssm::linattn_nt(z.N) / (4 * ssm::kLinAttnThreads)) * (gradient ? 2 : 1);
    if (!ssm::launchable(bh * walks * ceil_div(z.P, cols), 4 * cols)) return false;
    if ((gradient || p.n_seg > 1) && !ssm::launchable(carries, ssm::kLinAttnThreads)) return false;
    return gradient ? ssm::launchable(bh * p.n_seg, ssm::kLinAttnThreads)
                    : ssm::launchable(bh * p.n_seg * blocks, ssm::kLinAttnOutThreads);
}

// Cuts the scratch at `base` (which may be null: for the size alone) into the call's pieces.
int64_t layout(const AttnSizes &z, bool gradient, bool g_per_step, void *base, LinAttnLaunch *p) {
    Pieces s{reinterpret_cast<uintptr_t>(base)};
    const int64_t state = ceil_div(z.P, kBlockP) * kBlockP * ssm::linattn_nt(z.N), n = z.b * z.H * p->n_seg;
    if (p->n_seg == 0 || (!gradient && p->n_seg == 1)) return 0;
    p->S = s.next<float>(n * state);
    p->gsum = s.next<double>(n);
    // a segment of one chunk has no chunks that the walk over its own state could leave out
    if (!gradient && p->seg_chunks > 1) p->bad = s.next<uint32_t>(n * ceil_div(z.P, kBlockP) * 8);
    if (gradient) {
        p->E = s.next<float>(n * state);
        if (!g_per_step) p->dg_steps = s.next<float>(z.b * z.L * z.H);
        if (z.G < z.H) {
            p->dq_part = s.next<float>(z.b * z.L * z.H * z.N);
            p->dk_part = s.next<float>(z.b * z.L * z.H * z.N);
        }
    }
    return s.at;
}

// Strides as given or dense; false where one is negative or reaches too far.
bool set_strides(const AttnSizes &z, const ssm_linattn_strides_t *st, bool step, LinAttnLaunch *p) {
    const int64_t L = step ? 1 : z.L, qt = z.G * z.N, vt = z.H * z.P;
    const ssm_linattn_strides_t dense{L * qt, qt, z.N, L * qt, qt, z.N, L * vt, vt, z.P, L * vt, vt, z.P};
    const ssm_linattn_strides_t &s = st ? *st : dense;
    const int64_t all[12] = {s.q_b, s.q_t, s.q_h, s.k_b, s.k_t, s.k_h, s.v_b, s.v_t, s.v_h, s.do_b, s.do_t, s.do_h};
    const int64_t n[3] = {z.b, L > 0 ? L : 1, 0};
    // an axis of one element has no stride of its own; one step's is the row's width, as if more rows followed
    const int64_t width[4] = {z.N, z.N, z.P, z.P};
    int64_t use[12] = {0};
    for (int i = 0; i < 12; ++i) {
        if (step && (i % 3 == 1 || i >= 9)) continue;
        const int64_t count = i % 3 < 2 ? n[i % 3] : (i < 6 ? z.G : z.H);
        int64_t reach = 0;
        if (all[i] < 0 || !mul_ok(all[i], count, &reach) || reach > kMost) return false;
        if (i % 3 == 1 && count > 1 && all[i] > kMostStep) return false;
        use[i] = count > 1 ? all[i] : i % 3 == 1 ? width[i / 3] : 0;
    }
    p->q_b = use[0]; p->q_t = use[1]; p->q_h = use[2];
    p->k_b = use[3]; p->k_t = use[4]; p->k_h = use[5];
    p->v_b = use[6]; p->v_t = use[7]; p->v_h = use[8];
    p->do_b = use[9]; p->do_t = use[10]; p->do_h = use[11];
    return true;
}

// Bytes from the first to one past the last element of a strided input.
int64_t extent(int64_t b, int64_t t, int64_t h, int64_t width, int64_t sb, int64_t st, int64_t sh, int64_t es) {
    return ((b - 1) * sb + (t - 1) * st + (h - 1) * sh + width) * es;
}

// Whether rows of `width` elements at these strides take 16-byte loads, and steps lie at least a row apart.
bool loads16(const void *p, int64_t width, int64_t sb, int64_t st, int64_t sh, int64_t es) {
    const int64_t v = 16 / es;
    return aligned(p, 16) && width % v == 0 && st >= width && sb % v == 0 && st % v == 0 && sh % v == 0;
}

void set_common(const AttnSizes &z, ssm_dtype_t dtype, LinAttnLaunch *p) {
    p->b = z.b; p->L = z.L;
    p->H = (int)z.H; p->G = (int)z.G; p->N = (int)z.N; p->P = (int)z.P;
    p->bf16 = dtype == SSM_BF16;
    const int64_t es = p->bf16 ? 2 : 4;
    const int64_t v = 16 / es;
    p->vec = z.N % v == 0 && z.P % v == 0 && loads16(p->q, z.N, p->q_b, p->q_t, p->q_h, es) &&
             loads16(p->k, z.N, p->k_b, p->k_t, p->k_h, es) && loads16(p->v, z.P, p->v_b, p->v_t, p->v_h, es) &&
             (!p->dout || loads16(p->dout, z.P, p->do_b, p->do_t, p->do_h, es)) && aligned(p->o, 16) &&
             aligned(p->dq, 16) && aligned(p->dk, 16) && aligned(p->dv, 16);
}

ssm_status_t fill_state(const float *src, float *dst, int64_t n, hipStream_t stream) {
    if (!dst) return SSM_OK;
    hipError_t e = src ? hipMemcpyAsync(dst, src, (size_t)n * 4, hipMemcpyDeviceToDevice, stream) : hipSuccess;
    constexpr int64_t kPiece = INT64_C(1) << 31;  // of the threads that HIP takes to a launch
    for (int64_t i = 0; !src && i < n && e == hipSuccess; i += kPiece)
        e = ssm::launch_fill_zero(dst + i, n - i < kPiece ? n - i : kPiece, stream);
    return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

template <int NO, int NI> bool any_overlap(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (const Span &in : ins)
            if (overlaps(outs[i], in)) return true;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], outs[j])) return true;
    }
    return false;
}

}  // namespace

extern "C" {

ssm_status_t ssm_linattn_workspace(int32_t gradient, int64_t b, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P,
                                   ssm_dtype_t dtype, int32_t g_per_step, int64_t *bytes) {
    const AttnSizes z{b, L, H, G, N, P};
    if (!bytes) return SSM_ERR_NULL;
    const ssm_status_t st = check_sizes(z, dtype);
    if (st != SSM_OK) return st;
    LinAttnLaunch p{};
    p.bf16 = dtype == SSM_BF16;
    plan(z, gradient != 0, &p);
    if (!launches(z, gradient != 0, p)) return SSM_ERR_SHAPE;
    *bytes = layout(z, gradient != 0, g_per_step != 0, nullptr, &p);
    return SSM_OK;
}

ssm_status_t ssm_linattn_fwd(const void *q, const void *k, const void *v, const float *g, int32_t g_per_step, float scale,
                             const float *initial_state, const int32_t *lengths, void *o, float *final_state, int64_t b,
                             int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, ssm_dtype_t dtype,
                             const ssm_linattn_strides_t *strides, void *workspace, int64_t workspace_bytes,
                             hipStream_t stream) {
    const AttnSizes z{b, L, H, G, N, P};
    ssm_status_t st = check_sizes(z, dtype);
    if (st != SSM_OK) return st;
    LinAttnLaunch p{};
    p.bf16 = dtype == SSM_BF16;
    plan(z, false, &p);
    if (!launches(z, false, p) || !set_strides(z, strides, false, &p)) return SSM_ERR_SHAPE;
    if (L > 0 && (!q || !k || !v || !g || !o)) return SSM_ERR_NULL;
    const int64_t es = dtype == SSM_BF16 ? 2 : 4, state = b * H * P * N;
    const int64_t need = layout(z, false, g_per_step != 0, nullptr, &p);
    const Span outs[] = {{L > 0 ? o : nullptr, b * L * H * P * es}, {final_state, state * 4}, {workspace, need}};
    const Span ins[] = {{L > 0 ? q : nullptr, extent(b, L, G, N, p.q_b, p.q_t, p.q_h, es)},
                        {L > 0 ? k : nullptr, extent(b, L, G, N, p.k_b, p.k_t, p.k_h, es)},
                        {L > 0 ? v : nullptr, extent(b, L, H, P, p.v_b, p.v_t, p.v_h, es)},
                        {L > 0 ? g : nullptr, (g_per_step ? b * L : 1) * H * 4},
                        {initial_state, state * 4},
                        {lengths, b * 4}};
    if (any_overlap(outs, ins)) return SSM_ERR_ALIAS;
    if (L == 0) return fill_state(initial_state, final_state, state, stream);
    Scratch scratch;
    if ((st = scratch.take(workspace, workspace_bytes, need, stream)) != SSM_OK) return st;
    layout(z, false, g_per_step != 0, scratch.p, &p);
    p.q = q; p.k = k; p.v = v; p.g = g;
    p.g_per_step = g_per_step != 0;
    p.scale = scale;
    p.initial_state = initial_state; p.lengths = lengths; p.o = o; p.final_state = final_state;
    set_common(z, dtype, &p);
    return scratch.done(ssm::launch_linattn_fwd(p, stream));
}

ssm_status_t ssm_linattn_step(float *state, const void *q, const void *k, const void *v, const float *g,
                              int32_t g_per_step, float scale, void *o, int64_t b, int64_t H, int64_t G, int64_t N,
                              int64_t P, ssm_dtype_t dtype, const ssm_linattn_strides_t *strides, hipStream_t stream) {
    const AttnSizes z{b, 1, H, G, N, P};
    const ssm_status_t st = check_sizes(z, dtype);
    if (st != SSM_OK) return st;
    LinAttnLaunch p{};
    if (!ssm::launchable(b * H * ceil_div(P, kBlockP), ssm::kLinAttnThreads)) return SSM_ERR_SHAPE;
    if (!set_strides(z, strides, true, &p)) return SSM_ERR_SHAPE;
    if (!state || !q || !k || !v || !g || !o) return SSM_ERR_NULL;
    const int64_t es = dtype == SSM_BF16 ? 2 : 4;
    const Span outs[] = {{o, b * H * P * es}, {state, b * H * P * N * 4}};
    const Span ins[] = {{q, extent(b, 1, G, N, p.q_b, 0, p.q_h, es)},
                        {k, extent(b, 1, G, N, p.k_b, 0, p.k_h, es)},
                        {v, extent(b, 1, H, P, p.v_b, 0, p.v_h, es)},
                        {g, (g_per_step ? b : 1) * H * 4}};
    if (any_overlap(outs, ins)) return SSM_ERR_ALIAS;
    p.q = q; p.k = k; p.v = v; p.g = g; p.o = o;
    p.g_per_step = g_per_step != 0;
    p.scale = scale;
    set_common(z, dtype, &p);
    return ssm::launch_linattn_step(state, p, stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

ssm_status_t ssm_linattn_bwd(const void *q, const void *k, const void *v, const float *g, int32_t g_per_step, float scale,
                             const float *initial_state, const int32_t *lengths, const void *do_,
                             const float *d_final_state, void *dq, void *dk, void *dv, float *dg, float *d_initial_state,
                             int64_t b, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, ssm_dtype_t dtype,
                             const ssm_linattn_strides_t *strides, void *workspace, int64_t workspace_bytes,
                             hipStream_t stream) {
    const AttnSizes z{b, L, H, G, N, P};
    ssm_status_t st = check_sizes(z, dtype);
    if (st != SSM_OK) return st;
    LinAttnLaunch p{};
    plan(z, true, &p);
    if (!launches(z, true, p) || !set_strides(z, strides, false, &p)) return SSM_ERR_SHAPE;
    if (L > 0 && (!q || !k || !v || !g || !do_ || !dq || !dk || !dv || !dg)) return SSM_ERR_NULL;
    if (L == 0 && !g_per_step && !dg) return SSM_ERR_NULL;
    const int64_t es = dtype == SSM_BF16 ? 2 : 4, state = b * H * P * N;
    const int64_t need = layout(z, true, g_per_step != 0, nullptr, &p);
    const bool some = L > 0;
    const Span outs[] = {{some ? dq : nullptr, b * L * G * N * es}, {some ? dk : nullptr, b * L * G * N * es},
                         {some ? dv : nullptr, b * L * H * P * es}, {dg, (g_per_step ? b * L : 1) * H * 4},
                         {d_initial_state, state * 4}, {workspace, need}};
    const Span ins[] = {{some ? q : nullptr, extent(b, L, G, N, p.q_b, p.q_t, p.q_h, es)},
                        {some ? k : nullptr, extent(b, L, G, N, p.k_b, p.k_t, p.k_h, es)},
                        {some ? v : nullptr, extent(b, L, H, P, p.v_b, p.v_t, p.v_h, es)},
                        {some ? do_ : nullptr, extent(b, L, H, P, p.do_b, p.do_t, p.do_h, es)},
                        {some ? g : nullptr, (g_per_step ? b * L : 1) * H * 4},
                        {initial_state, state * 4},
                        {d_final_state, state * 4},
                        {lengths, b * 4}};
    if (any_overlap(outs, ins)) return SSM_ERR_ALIAS;
    if (L == 0) {
        if (!g_per_step && ssm::launch_fill_zero(dg, H, stream) != hipSuccess) return SSM_ERR_HIP;
        return fill_state(d_final_state, d_initial_state, state, stream);
    }
    Scratch scratch;
    if ((st = scratch.take(workspace, workspace_bytes, need, stream)) != SSM_OK) return st;
    layout(z, true, g_per_step != 0, scratch.p, &p);
    p.q = q; p.k = k; p.v = v; p.g = g; p.dout = do_;
    p.g_per_step = g_per_step != 0;
    p.scale = scale;
    p.initial_state = initial_state; p.d_final_state = d_final_state; p.lengths = lengths;
    p.dq = dq; p.dk = dk; p.dv = dv; p.dg = dg; p.d_initial_state = d_initial_state;
    set_common(z, dtype, &p);
    return scratch.done(ssm::launch_linattn_bwd(p, stream));
}

// ---- layer norm ----------------------------------------------------------------------------------------------------

static ssm_status_t check_norm(int64_t rows, int64_t d, int64_t w_rows, int64_t *stride, ssm_dtype_t dtype) {
    int64_t n = 0;
    if (!valid_dtype(dtype)) return SSM_ERR_UNSUPPORTED;
    if (rows < 0 || d < 1 || w_rows < 1 || rows % w_rows != 0) return SSM_ERR_SHAPE;
    if (d > SSM_LAYERNORM_MAX_D) return SSM_ERR_UNSUPPORTED;
    if (!ssm::launchable(w_rows, ssm::layernorm_threads(d))) return SSM_ERR_SHAPE;
    if (*stride == 0) *stride = d;
    if (*stride < d || !mul_ok(rows, *stride, &n) || n > kMost) return SSM_ERR_SHAPE;
    return SSM_OK;
}

ssm_status_t ssm_layernorm_fwd(const void *x, const float *w, const float *bias, void *y, float *mean, float *rstd,
                               int64_t rows, int64_t d, int64_t w_rows, int64_t x_stride, float eps, ssm_dtype_t dtype,
                               hipStream_t stream) {
    const ssm_status_t st = check_norm(rows, d, w_rows, &x_stride, dtype);
    if (st != SSM_OK) return st;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return SSM_ERR_UNSUPPORTED;
    if (rows == 0) return SSM_OK;
    if (!x || !y) return SSM_ERR_NULL;
    const int64_t es = dtype == SSM_BF16 ? 2 : 4;
    const bool in_place = y == x && x_stride == d;
    const Span outs[] = {{y, rows * d * es}, {mean, rows * 4}, {rstd, rows * 4}};
    const Span ins[] = {{in_place ? nullptr : x, ((rows - 1) * x_stride + d) * es}, {w, w_rows * d * 4},
                        {bias, w_rows * d * 4}};
    if (any_overlap(outs, ins)) return SSM_ERR_ALIAS;
    NormLaunch p{};
    p.x = x; p.w = w; p.bias = bias; p.y = y; p.mean = mean; p.rstd = rstd;
    p.rows = rows; p.d = d; p.w_rows = w_rows; p.x_stride = x_stride;
    p.eps = eps;
    p.bf16 = dtype == SSM_BF16;
    const int64_t v = 16 / es;
    p.vec = d % v == 0 && x_stride % v == 0 && aligned(x, 16) && aligned(y, 16);
    return ssm::launch_layernorm_fwd(p, stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

ssm_status_t ssm_layernorm_bwd_workspace(int64_t rows, int64_t d, int64_t w_rows, int64_t *bytes) {
    int64_t stride = 0;
    if (!bytes) return SSM_ERR_NULL;
    const ssm_status_t st = check_norm(rows, d, w_rows, &stride, SSM_F32);
    if (st != SSM_OK) return st;
    *bytes = rows == 0 ? 0 : ssm::layernorm_part_floats(rows, d, w_rows) * 4;
    return SSM_OK;
}

ssm_status_t ssm_layernorm_bwd(const void *x, const float *w, const void *dy, const float *mean, const float *rstd,
                               void *dx, float *dw, float *dbias, int64_t rows, int64_t d, int64_t w_rows,
                               int64_t x_stride, int64_t dy_stride, ssm_dtype_t dtype, void *workspace,
                               int64_t workspace_bytes, hipStream_t stream) {
    ssm_status_t st = check_norm(rows, d, w_rows, &x_stride, dtype);
    if (st == SSM_OK) st = check_norm(rows, d, w_rows, &dy_stride, dtype);
    if (st != SSM_OK) return st;
    if (rows > 0 && (!x || !dy || !mean || !rstd || !dx)) return SSM_ERR_NULL;
    const int64_t es = dtype == SSM_BF16 ? 2 : 4;
    const int64_t need = rows > 0 && (dw || dbias) ? ssm::layernorm_part_floats(rows, d, w_rows) * 4 : 0;
    const bool on_x = dx == x && x_stride == d, on_dy = dx == dy && dy_stride == d;
    const Span outs[] = {{rows > 0 ? dx : nullptr, rows * d * es}, {dw, w_rows * d * 4}, {dbias, w_rows * d * 4},
                         {workspace, need}};
    const Span ins[] = {{w, w_rows * d * 4}, {mean, rows * 4}, {rstd, rows * 4}};
    if (any_overlap(outs, ins)) return SSM_ERR_ALIAS;
    const Span big[] = {{x, ((rows - 1) * x_stride + d) * es}, {dy, ((rows - 1) * dy_stride + d) * es}};
    for (int i = 0; i < 4 && rows > 0; ++i) {
        if (!(i == 0 && on_x) && overlaps(outs[i], big[0])) return SSM_ERR_ALIAS;
        if (!(i == 0 && on_dy) && overlaps(outs[i], big[1])) return SSM_ERR_ALIAS;
    }
    if (rows == 0 && !dw && !dbias) return SSM_OK;
    Scratch scratch;
    if ((st = scratch.take(workspace, workspace_bytes, need, stream)) != SSM_OK) return st;
    NormLaunch p{};
    p.x = x; p.dy = dy; p.w = w; p.mean_in = mean; p.rstd_in = rstd;
    p.y = dx; p.dw = dw; p.dbias = dbias;
    p.rows = rows; p.d = d; p.w_rows = w_rows; p.x_stride = x_stride; p.dy_stride = dy_stride;
    p.bf16 = dtype == SSM_BF16;
    p.part = static_cast<float *>(scratch.p);
    const int64_t v = 16 / es;
    p.vec = d % v == 0 && x_stride % v == 0 && dy_stride % v == 0 && aligned(x, 16) && aligned(dy, 16) && aligned(dx, 16);
    return scratch.done(ssm::launch_layernorm_bwd(p, stream));
}

}  // extern "C"
