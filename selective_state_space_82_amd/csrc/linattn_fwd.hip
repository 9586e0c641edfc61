// linattn_fwd.hip — linear attention with a per-head decay, forward: chunk by chunk as matrix products.
//
// Page "State Space Models（SSM）とMamba" §4.6 (state space duality) with the unrolled recurrence of page
// "Mambaとは？Transformer以外の系列モデル", section Mambaの核心は入力依存のDelta、B、C. With c_t the running sum of
// the log-decays in a chunk of 64 steps and S the state entering it,
//     o_t   = scale·( Σ_{s<=t} e^{c_t − c_s} (q_t·k_s) v_s + e^{c_t} S q_t ),
//     S_out = e^{c_end} S + Σ_s e^{c_end − c_s} v_s k_sᵀ.
#include "linattn_common.h"

namespace ssm {
namespace la {
namespace {

struct Work {
    int64_t ib, seg, bh;
    int h, grp, p0;  // p0: first value column
};
template <int NW> __device__ __forceinline__ Work work_of(const LinAttnLaunch &a, int64_t n_seg) {
    int64_t id = work_index(blockIdx.x, gridDim.x);
    const int npb = (a.P + 16 * NW - 1) / (16 * NW);
    Work w;
    w.p0 = 16 * NW * (int)(id % npb);
    id /= npb;
    w.h = (int)(id % a.H);
    id /= a.H;
    w.seg = id % n_seg;
    w.ib = id / n_seg;
    w.grp = w.h / (a.H / a.G);
    w.bh = w.ib * a.H + w.h;
    return w;
}

__device__ __forceinline__ const float *decays_of(const LinAttnLaunch &a, const Work &w, int64_t *stride) {
    *stride = a.g_per_step ? a.H : 0;
    return a.g_per_step ? a.g + w.ib * a.L * a.H + w.h : a.g + w.h;
}

// A lane's part of the state, four values of N at row p, as result tiles; zeros outside [P][N].
template <int NT>
__device__ __forceinline__ void load_state(f4 (&S)[NT / 16], const float *src, int64_t p, int P, int N) {
    const int g4 = 4 * ((threadIdx.x & 63) >> 4);
#pragma unroll
    for (int i = 0; i < NT / 16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int n = 16 * i + g4 + r;
            S[i][r] = p < P && n < N ? src[p * N + n] : 0.0f;
        }
}

// ---- outputs: one workgroup walks the chunks of (row, head, 16·NW value columns, segment) in order ---------------
//
// Wavefront w keeps the state's value columns 16w .. 16w+15 (all N of them) in its result tiles. Per chunk the NW of
// them share the 10 lower-triangular 16×16 tiles of the decayed scores through LDS; the rest (outputs of its own
// columns, the state's update) each wavefront does from its own state and its own columns of V, which are scaled
// and cut into bf16 parts once and used for every tile of N. The next chunk's rows are fetched into registers, and its
// decays formed by the last wavefront (which has the fewest tiles), while this one is computed.
template <typename T, int NT, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2))) void la_out_kernel(LinAttnLaunch a) {
    constexpr int THREADS = 64 * NW, PB = 16 * NW;
    constexpr int SN = NT + kPad<T>, SP = kC + kPad<T>, SV = PB + kPad<T>;
    constexpr int PARTS = sizeof(T) == 2 ? 2 : 1;
    __shared__ __align__(16) T s_q[kC * SN];
    __shared__ __align__(16) T s_k[kC * SN];
    __shared__ __align__(16) T s_v[kC * SV];
    __shared__ __align__(16) T s_p[PARTS][kC * SP];  // decayed scores [t][s]
    __shared__ Decays s_g[2];

    const Work wk = work_of<NW>(a, a.n_seg);
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, col = l & 15, g4 = 4 * (l >> 4);
    const int64_t len = row_length(a.lengths, wk.ib, a.L);
    int64_t g_stride;
    const float *gp = decays_of(a, wk, &g_stride);
    const T *qp = static_cast<const T *>(a.q) + wk.ib * a.q_b + wk.grp * a.q_h;
    const T *kp = static_cast<const T *>(a.k) + wk.ib * a.k_b + wk.grp * a.k_h;
    const T *vp = static_cast<const T *>(a.v) + wk.ib * a.v_b + wk.h * a.v_h;
    T *op = static_cast<T *>(a.o) + (wk.ib * a.L * a.H + wk.h) * a.P;
    const uint32_t o_t = (uint32_t)a.H * a.P;  // elements between steps of o
    const int p0 = wk.p0, p_wave = p0 + 16 * w;

    f4 S[NT / 16];
    const int64_t p_lane = p_wave + col, Pp = (a.P + kPB - 1) / kPB * kPB;
    if (a.n_seg > 1 && p_lane < Pp) {
        const float *src = a.S + ((wk.bh * a.n_seg + wk.seg) * Pp + p_lane) * NT + g4;
#pragma unroll
        for (int i = 0; i < NT / 16; ++i) S[i] = *reinterpret_cast<const f4 *>(src + 16 * i);
    } else if (a.n_seg == 1 && a.initial_state) {
        load_state<NT>(S, a.initial_state + wk.bh * a.P * a.N, p_lane, a.P, a.N);
    } else {
#pragma unroll
        for (int i = 0; i < NT / 16; ++i) S[i] = f4{0, 0, 0, 0};
    }

    // the tiles right of the diagonal that a 32-step contraction touches stay zero
    for (int i = tid; i < 2 * 16 * 16; i += THREADS) {
        const int t = 32 * (i >> 8) + ((i >> 4) & 15), s = 32 * (i >> 8) + 16 + (i & 15);
#pragma unroll
        for (int e = 0; e < PARTS; ++e) s_p[e][t * SP + s] = (T)0;
    }

    const int64_t n_chunks = (a.L + kC - 1) / kC, live = (len + kC - 1) / kC;
    const int64_t ch0 = wk.seg * a.seg_chunks, ch1 = ch0 + a.seg_chunks < n_chunks ? ch0 + a.seg_chunks : n_chunks;
    const int64_t chl = ch1 < live ? ch1 : live;  // chunks with any step of the row
    Stage<T, NT, THREADS, VEC> rq, rk;
    Stage<T, PB, THREADS, VEC> rv;
    float g_next = 0.0f;
    auto fetch = [&](int64_t t0) {
        const int rows = rows_of(t0, len);
        rq.load(qp + t0 * a.q_t, (uint32_t)a.q_t, rows, 0, a.N);
        rk.load(kp + t0 * a.k_t, (uint32_t)a.k_t, rows, 0, a.N);
        rv.load(vp + t0 * a.v_t, (uint32_t)a.v_t, rows, p0, a.P);
    };
    auto fetch_g = [&](int64_t t0) { return load_g(gp + t0 * g_stride, (uint32_t)g_stride, rows_of(t0, len)); };
    if (ch0 < chl) {
        if (VEC) fetch(ch0 * kC);
        if (w == NW - 1) {
            s_g[0].set(log_decay(fetch_g(ch0 * kC)), a.scale);
            g_next = fetch_g((ch0 + 1) * kC);
        }
    }
    for (int64_t ch = ch0; ch < chl; ++ch) {
        const int64_t t0 = ch * kC;
        const Decays &dec = s_g[(ch - ch0) & 1];
        const int all = rows_of(t0, a.L), some = rows_of(t0, len);
        const Buffer out = rows_buffer(op + t0 * o_t, o_t, all, a.P);
        if (!VEC) fetch(t0);
        rq.store(s_q);
        rk.store(s_k);
        rv.store(s_v);
        lds_barrier();
        if (VEC) fetch(t0 + kC);  // past the last chunk: nothing

        // decayed scores, tile (tb, sb): D[s][t] = k_s·q_t
        for (int i = w; i < 10; i += NW) {
            const int tb = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3;
            const int sb = i - tb * (tb + 1) / 2;
            f4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int n = 0; n < NT; n += 32) mma(acc, row_frag(s_k, SN, 16 * sb, n), row_frag(s_q, SN, 16 * tb, n));
            const int t = 16 * tb + col, s = 16 * sb + g4;
            const float th = dec.c.hi[t], tl = dec.c.lo[t];
            const f4 sh = *reinterpret_cast<const f4 *>(&dec.c.hi[s]), sl = *reinterpret_cast<const f4 *>(&dec.c.lo[s]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = a.scale * exp2_fast((th - sh[r]) + (tl - sl[r]));
                acc[r] = s + r <= t ? acc[r] * d : 0.0f;
            }
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int e = 0; e < PARTS; ++e) {
                    const bf4 v = __builtin_convertvector(acc, bf4);
                    *reinterpret_cast<bf4 *>(&s_p[e][t * SP + s]) = v;
                    acc -= __builtin_convertvector(v, f4);
                }
            } else {
                *reinterpret_cast<f4 *>(&s_p[0][t * SP + s]) = acc;
            }
        }
        if (w == NW - 1) {
            s_g[(ch + 1 - ch0) & 1].set(log_decay(g_next), a.scale);
            g_next = fetch_g(t0 + 2 * kC);
        }
        lds_barrier();

        Frag<T> vf[2];
        f8 vw[2];
        float probe = 0.0f;
#pragma unroll
        for (int sp = 0; sp < 2; ++sp) {
            vf[sp] = col_frag(s_v, SV, 32 * sp, 16 * w);
            vw[sp] = wide(vf[sp]);
#pragma unroll
            for (int j = 0; j < 8; ++j) probe = __builtin_fmaf(vw[sp][j], 0.0f, probe);
        }
        // A NaN or Inf in V would reach earlier steps through the zero scores of the later ones.
        const bool finite = !__any(probe != 0.0f);
        f4 acc[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) acc[tb] = f4{0, 0, 0, 0};
#pragma unroll
        for (int n = 0; n < NT / 32; ++n) {
            const Split<T, 2> sv(join(S[2 * n], S[2 * n + 1]));
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) mma(acc[tb], sv, row_frag(s_q, SN, 16 * tb, 32 * n));
        }
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const int tl = 16 * tb + col;
            acc[tb] *= dec.in[tl];
            if (finite) {
#pragma unroll
                for (int sp = 0; sp <= tb / 2; ++sp)
#pragma unroll
                    for (int e = 0; e < PARTS; ++e) mma(acc[tb], vf[sp], row_frag(s_p[e], SP, 16 * tb, 32 * sp));
            } else {
                for (int s = 0; s <= tl; ++s) {
                    float pr = 0.0f;
#pragma unroll
                    for (int e = 0; e < PARTS; ++e) pr += widen(s_p[e][tl * SP + s]);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[tb][r] = __builtin_fmaf(pr, widen(s_v[s * SV + 16 * w + g4 + r]), acc[tb][r]);
                }
            }
            if (tl >= some) acc[tb] = f4{0, 0, 0, 0};
            store4<T, VEC>(out, o_t, tl, p_wave + g4, a.P, acc[tb]);
        }

        // the state's update: V's columns scaled, three parts (the state is an fp32 result)
        const float end = dec.end;
#pragma unroll
        for (int i = 0; i < NT / 16; ++i) S[i] *= end;
#pragma unroll
        for (int sp = 0; sp < 2; ++sp) {
            const f4 u = *reinterpret_cast<const f4 *>(&dec.out[32 * sp + g4]);
            const f4 v = *reinterpret_cast<const f4 *>(&dec.out[32 * sp + 16 + g4]);
            const Split<T, 3> vs(vw[sp] * join(u, v));
#pragma unroll
            for (int i = 0; i < NT / 16; ++i) mma(S[i], col_frag(s_k, SN, 32 * sp, 16 * i), vs);
        }
        lds_barrier();
    }

    // past the row's end: outputs are zero, the state stays
    for (int64_t ch = chl > ch0 ? chl : ch0; ch < ch1; ++ch) {
        const Buffer out = rows_buffer(op + ch * kC * o_t, o_t, rows_of(ch * kC, a.L), a.P);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) store4<T, VEC>(out, o_t, 16 * tb + col, p_wave + g4, a.P, f4{0, 0, 0, 0});
    }

    if (a.final_state && wk.seg == a.n_seg - 1 && p_lane < a.P) {
        float *dst = a.final_state + (wk.bh * a.P + p_lane) * a.N;
#pragma unroll
        for (int i = 0; i < NT / 16; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (16 * i + g4 + r < a.N) dst[16 * i + g4 + r] = S[i][r];
    }
}

// ---- a segment's own state, or its own adjoint -------------------------------------------------------------------
//
// Forward: S = Σ_s e^{c_end − c_s} v_s k_sᵀ over the segment. Adjoint (REV): the gradient reaching the state that
// enters the segment from its own outputs, E = Σ_u scale·e^{c_u} do_u q_uᵀ. Workgroup (row, head, 16·NW value columns,
// segment) as above. Both walk the chunks from the far end of the decay to the near one, S from the last chunk back
// and E from the first on, so that each chunk's weights carry the decay of all chunks walked before it. The walk ends
// where that decay is below e^-200: what the rest would add is it times a state (adjoint) of the recurrence, which as
// an fp32 number is at most e^88.8, and the product is 0 in fp32 (smallest positive value e^-103.3).
template <typename T, int NT, int NW, bool VEC, bool REV>
__global__ __launch_bounds__(64 * NW) void la_states_kernel(LinAttnLaunch a, int64_t first_seg, int64_t n_own) {
    constexpr int THREADS = 64 * NW, PB = 16 * NW;
    constexpr int SN = NT + kPad<T>, SV = PB + kPad<T>;
    __shared__ __align__(16) T s_k[kC * SN];
    __shared__ __align__(16) T s_v[kC * SV];
    __shared__ Decays s_g;

    Work wk = work_of<NW>(a, n_own);
    wk.seg += first_seg;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, col = l & 15, g4 = 4 * (l >> 4);
    const int64_t len = row_length(a.lengths, wk.ib, a.L);
    int64_t g_stride;
    const float *gp = decays_of(a, wk, &g_stride);
    const int64_t kt = REV ? a.q_t : a.k_t, vt = REV ? a.do_t : a.v_t;
    const T *kp = REV ? static_cast<const T *>(a.q) + wk.ib * a.q_b + wk.grp * a.q_h
                      : static_cast<const T *>(a.k) + wk.ib * a.k_b + wk.grp * a.k_h;
    const T *vp = REV ? static_cast<const T *>(a.dout) + wk.ib * a.do_b + wk.h * a.do_h
                      : static_cast<const T *>(a.v) + wk.ib * a.v_b + wk.h * a.v_h;
    const int p0 = wk.p0;

    f4 S[NT / 16];
#pragma unroll
    for (int i = 0; i < NT / 16; ++i) S[i] = f4{0, 0, 0, 0};
    const int64_t n_chunks = (a.L + kC - 1) / kC, live = (len + kC - 1) / kC;
    const int64_t ch0 = wk.seg * a.seg_chunks, ch1 = ch0 + a.seg_chunks < n_chunks ? ch0 + a.seg_chunks : n_chunks;
    const int64_t chl = ch1 < live ? ch1 : live;
    Stage<T, NT, THREADS, VEC> rk;
    Stage<T, PB, THREADS, VEC> rv;
    double passed = 0.0;  // in every wavefront: the sum of g over the chunks walked
    float g_next = 0.0f;
    const int64_t n = chl - ch0;
    auto start = [&](int64_t j) { return (REV ? ch0 + j : chl - 1 - j) * kC; };
    auto fetch = [&](int64_t t0) {
        const int rows = rows_of(t0, len);
        rk.load(kp + t0 * kt, (uint32_t)kt, rows, 0, a.N);
        rv.load(vp + t0 * vt, (uint32_t)vt, rows, p0, a.P);
    };
    auto fetch_g = [&](int64_t t0) { return load_g(gp + t0 * g_stride, (uint32_t)g_stride, rows_of(t0, len)); };
    if (n > 0) {
        if (VEC) fetch(start(0));
        g_next = fetch_g(start(0));
    }
    for (int64_t j = 0; j < n && !(passed <= -200.0); ++j) {
        if (!VEC) fetch(start(j));
        rk.store(s_k);
        rv.store(s_v);
        const double sum = wave_running_sum(log_decay(g_next)), total = lane_value(sum, 63);
        // the weight of the lane's step, from all chunks walked and from this one
        const float wt = (REV ? a.scale : 1.0f) * exp_of((float)(passed + (REV ? sum : total - sum)));
        if (w == 0) s_g.out[l] = wt;
        passed += total;
        lds_barrier();
        if (j + 1 < n) {
            if (VEC) fetch(start(j + 1));
            g_next = fetch_g(start(j + 1));
        }
#pragma unroll
        for (int sp = 0; sp < 2; ++sp) {
            const f4 u = *reinterpret_cast<const f4 *>(&s_g.out[32 * sp + g4]);
            const f4 v = *reinterpret_cast<const f4 *>(&s_g.out[32 * sp + 16 + g4]);
            const Split<T, 3> vs(wide(col_frag(s_v, SV, 32 * sp, 16 * w)) * join(u, v));
#pragma unroll
            for (int i = 0; i < NT / 16; ++i) mma(S[i], col_frag(s_k, SN, 32 * sp, 16 * i), vs);
        }
        lds_barrier();
    }
    const int64_t Pp = (a.P + kPB - 1) / kPB * kPB, at = wk.bh * a.n_seg + wk.seg, p = p0 + 16 * w + col;
    if (p < Pp) {
        float *dst = (REV ? a.E : a.S) + (at * Pp + p) * NT + g4;
#pragma unroll
        for (int i = 0; i < NT / 16; ++i) *reinterpret_cast<f4 *>(dst + 16 * i) = S[i];
    }
    if (tid == 0 && p0 == 0) a.gsum[at] = passed;
}

// ---- from the segments' own states to those entering them (adjoints: leaving them), in place ---------------------
//
// One thread per four state elements steps over the segments; four loads are kept in flight.
template <bool REV>
__global__ __launch_bounds__(kThreads) void la_carry_kernel(LinAttnLaunch a, int NT) {
    const int64_t Pp = (a.P + kPB - 1) / kPB * kPB;
    const int64_t per = Pp * NT / 4;                       // four-element groups of one state: a multiple of 256
    const int64_t bh = blockIdx.x / (per / kThreads);
    const int64_t e = blockIdx.x % (per / kThreads) * kThreads + threadIdx.x;
    const int64_t p = 4 * e / NT, n = 4 * e % NT;
    f4 *base = reinterpret_cast<f4 *>(REV ? a.E : a.S) + bh * a.n_seg * per + e;
    const double *gs = a.gsum + bh * a.n_seg;
    const float *first = REV ? a.d_final_state : a.initial_state;
    f4 carry = {0, 0, 0, 0};
    if (first && p < a.P)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < a.N) carry[r] = first[(bh * a.P + p) * a.N + n + r];
    constexpr int U = 4;
    for (int64_t j0 = 0; j0 < a.n_seg; j0 += U) {
        f4 own[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // the last own state (adjoint: the first, unless asked for) is not needed and may not be there
            const int64_t j = j0 + u, s = REV ? a.n_seg - 1 - j : j;
            const bool need = j < a.n_seg && (j + 1 < a.n_seg || (REV && a.d_initial_state));
            own[u] = need ? base[s * per] : f4{0, 0, 0, 0};
            d[u] = need ? exp_of((float)gs[s]) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t j = j0 + u, s = REV ? a.n_seg - 1 - j : j;
            if (j < a.n_seg) {
                base[s * per] = carry;
                carry = carry * d[u] + own[u];
            }
        }
    }
    if (REV && a.d_initial_state && p < a.P)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < a.N) a.d_initial_state[(bh * a.P + p) * a.N + n + r] = carry[r];
}

// f(NT, NW, VEC): the padded width of N, wavefronts per workgroup, and whether all rows take 16-byte accesses. Eight
// wavefronts share the scores, queries and keys of 128 value columns where P is that wide.
template <typename F> hipError_t by_width(const LinAttnLaunch &p, F f) {
    const int nt = linattn_nt(p.N);
    auto with = [&](auto nw, auto vec) {
        return nt == 32 ? f(std::integral_constant<int, 32>{}, nw, vec)
               : nt == 64 ? f(std::integral_constant<int, 64>{}, nw, vec)
                          : f(std::integral_constant<int, 128>{}, nw, vec);
    };
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 8> eight;
    if (linattn_cols(p.P) == 64) return p.vec ? with(four, std::true_type{}) : with(four, std::false_type{});
    return p.vec ? with(eight, std::true_type{}) : with(eight, std::false_type{});
}
unsigned value_blocks(const LinAttnLaunch &p) {
    const int cols = (int)linattn_cols(p.P);
    return (unsigned)((p.P + cols - 1) / cols);
}

template <typename T>
hipError_t states(const LinAttnLaunch &p, bool adjoint, int64_t first, int64_t n, hipStream_t stream) {
    const dim3 grid((unsigned)(p.b * p.H * n) * value_blocks(p));
    return by_width(p, [&](auto nt, auto nw, auto vec) {
        constexpr int NT = decltype(nt)::value, NW = decltype(nw)::value;
        constexpr bool VEC = decltype(vec)::value;
        if (adjoint) la_states_kernel<T, NT, NW, VEC, true><<<grid, 64 * NW, 0, stream>>>(p, first, n);
        else la_states_kernel<T, NT, NW, VEC, false><<<grid, 64 * NW, 0, stream>>>(p, first, n);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t outputs(const LinAttnLaunch &p, hipStream_t stream) {
    const dim3 grid((unsigned)(p.b * p.H * p.n_seg) * value_blocks(p));
    return by_width(p, [&](auto nt, auto nw, auto vec) {
        constexpr int NT = decltype(nt)::value, NW = decltype(nw)::value;
        constexpr bool VEC = decltype(vec)::value;
        la_out_kernel<T, NT, NW, VEC><<<grid, 64 * NW, 0, stream>>>(p);
        return hipGetLastError();
    });
}

}  // namespace
}  // namespace la

hipError_t launch_linattn_states(const LinAttnLaunch &p, bool adjoint, int64_t first, int64_t n, hipStream_t stream) {
    return p.bf16 ? la::states<uint16_t>(p, adjoint, first, n, stream) : la::states<float>(p, adjoint, first, n, stream);
}

hipError_t launch_linattn_carry(const LinAttnLaunch &p, bool adjoint, hipStream_t stream) {
    const int nt = linattn_nt(p.N);
    const int64_t per = (p.P + la::kPB - 1) / la::kPB * la::kPB * nt / 4 / la::kThreads;
    const dim3 grid((unsigned)(p.b * p.H * per));
    if (adjoint) la::la_carry_kernel<true><<<grid, la::kThreads, 0, stream>>>(p, nt);
    else la::la_carry_kernel<false><<<grid, la::kThreads, 0, stream>>>(p, nt);
    return hipGetLastError();
}

hipError_t launch_linattn_fwd(const LinAttnLaunch &p, hipStream_t stream) {
    if (p.n_seg > 1) {
        hipError_t e = launch_linattn_states(p, false, 0, p.n_seg - 1, stream);
        if (e == hipSuccess) e = launch_linattn_carry(p, false, stream);
        if (e != hipSuccess) return e;
    }
    return p.bf16 ? la::outputs<uint16_t>(p, stream) : la::outputs<float>(p, stream);
}

}  // namespace ssm
