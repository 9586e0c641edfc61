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
    int h, grp, pb;
};
__device__ __forceinline__ Work work_of(const LinAttnLaunch &a, int64_t n_seg) {
    int64_t id = work_index(blockIdx.x, gridDim.x);
    const int npb = (a.P + kPB - 1) / kPB;
    Work w;
    w.pb = (int)(id % npb);
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

// ---- outputs: one workgroup walks the chunks of (row, head, 64 value columns, segment) in order ----------------
//
// Wavefront w keeps the state's value columns 16w .. 16w+15 (all N of them) in its result tiles. Per chunk the four
// share the 10 lower-triangular 16×16 tiles of the decayed scores through LDS; the rest (outputs of its own
// columns, the state's update) each wavefront does from its own state and its own columns of V, which are scaled
// and cut into bf16 parts once and used for every tile of N.
template <typename T, int NT>
__global__ __launch_bounds__(kThreads) void la_out_kernel(LinAttnLaunch a) {
    constexpr int SN = NT + kPad<T>, SP = kC + kPad<T>, SV = kPB + kPad<T>;
    constexpr int PARTS = sizeof(T) == 2 ? 2 : 1;
    __shared__ __align__(16) T s_q[kC * SN];
    __shared__ __align__(16) T s_k[kC * SN];
    __shared__ __align__(16) T s_v[kC * SV];
    __shared__ __align__(16) T s_p[PARTS][kC * SP];  // decayed scores [t][s]
    __shared__ Sums s_c;
    __shared__ __align__(16) float s_in[kC], s_out[kC];  // scale·e^{c_t}, e^{c_end − c_s}
    __shared__ float s_end;

    const Work wk = work_of(a, a.n_seg);
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, col = l & 15, g4 = 4 * (l >> 4);
    const int64_t len = row_length(a.lengths, wk.ib, a.L);
    int64_t g_stride;
    const float *gp = decays_of(a, wk, &g_stride);
    const T *qp = static_cast<const T *>(a.q) + wk.ib * a.q_b + wk.grp * a.q_h;
    const T *kp = static_cast<const T *>(a.k) + wk.ib * a.k_b + wk.grp * a.k_h;
    const T *vp = static_cast<const T *>(a.v) + wk.ib * a.v_b + wk.h * a.v_h;
    T *op = static_cast<T *>(a.o) + (wk.ib * a.L * a.H + wk.h) * a.P;
    const int64_t o_t = (int64_t)a.H * a.P;
    const int p0 = kPB * wk.pb;

    f4 S[NT / 16];
    const int64_t p_lane = p0 + 16 * w + col;
    if (a.n_seg > 1) {
        const int64_t Pp = (a.P + kPB - 1) / kPB * kPB;
        const float *src = a.S + ((wk.bh * a.n_seg + wk.seg) * Pp + p_lane) * NT + g4;
#pragma unroll
        for (int i = 0; i < NT / 16; ++i) S[i] = *reinterpret_cast<const f4 *>(src + 16 * i);
    } else if (a.initial_state) {
        load_state<NT>(S, a.initial_state + wk.bh * a.P * a.N, p_lane, a.P, a.N);
    } else {
#pragma unroll
        for (int i = 0; i < NT / 16; ++i) S[i] = f4{0, 0, 0, 0};
    }

    // the tiles right of the diagonal that a 32-step contraction touches stay zero
    for (int i = tid; i < 2 * 16 * 16; i += kThreads) {
        const int t = 32 * (i >> 8) + ((i >> 4) & 15), s = 32 * (i >> 8) + 16 + (i & 15);
#pragma unroll
        for (int e = 0; e < PARTS; ++e) s_p[e][t * SP + s] = (T)0;
    }

    const int64_t n_chunks = (a.L + kC - 1) / kC;
    const int64_t ch0 = wk.seg * a.seg_chunks, ch1 = ch0 + a.seg_chunks < n_chunks ? ch0 + a.seg_chunks : n_chunks;
    for (int64_t ch = ch0; ch < ch1; ++ch) {
        const int64_t t0 = ch * kC;
        if (t0 >= len) {  // past the row's end: outputs are zero, the state stays
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                const int64_t t = t0 + 16 * tb + col;
                if (t < a.L) store4<T>(op + t * o_t, p0 + 16 * w + g4, a.P, a.vec_p, f4{0, 0, 0, 0});
            }
            continue;
        }
        stage<T, NT>(s_q, qp, a.q_t, t0, len, 0, a.N, a.vec_q);
        stage<T, NT>(s_k, kp, a.k_t, t0, len, 0, a.N, a.vec_k);
        stage<T, kPB>(s_v, vp, a.v_t, t0, len, p0, a.P, a.vec_v);
        if (w == 0) {
            const double c = wave_running_sum(log_decay(gp, g_stride, t0 + l, len));
            const double end = __shfl(c, 63);
            s_c.set(l, c);
            s_in[l] = a.scale * exp_of((float)c);
            s_out[l] = exp_of((float)(end - c));
            if (l == 63) s_end = exp_of((float)c);
        }
        __syncthreads();

        // decayed scores, tile (tb, sb): D[s][t] = k_s·q_t
        for (int i = w; i < 10; i += 4) {
            const int tb = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3;
            const int sb = i - tb * (tb + 1) / 2;
            f4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int n = 0; n < NT; n += 32) mma(acc, row_frag(s_k, SN, 16 * sb, n), row_frag(s_q, SN, 16 * tb, n));
            const int t = 16 * tb + col, s = 16 * sb + g4;
            const float th = s_c.hi[t], tl = s_c.lo[t];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = (th - s_c.hi[s + r]) + (tl - s_c.lo[s + r]);
                acc[r] = s + r <= t ? acc[r] * (a.scale * exp_of(d)) : 0.0f;
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
        __syncthreads();

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
            acc[tb] *= s_in[tl];
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
            const int64_t t = t0 + tl;
            if (t < a.L) {
                if (t >= len) acc[tb] = f4{0, 0, 0, 0};
                store4<T>(op + t * o_t, p0 + 16 * w + g4, a.P, a.vec_p, acc[tb]);
            }
        }

        // the state's update: V's columns scaled, three parts (the state is an fp32 result)
        const float end = s_end;
#pragma unroll
        for (int i = 0; i < NT / 16; ++i) S[i] *= end;
#pragma unroll
        for (int sp = 0; sp < 2; ++sp) {
            const f4 u = *reinterpret_cast<const f4 *>(&s_out[32 * sp + g4]);
            const f4 v = *reinterpret_cast<const f4 *>(&s_out[32 * sp + 16 + g4]);
            const Split<T, 3> vs(vw[sp] * join(u, v));
#pragma unroll
            for (int i = 0; i < NT / 16; ++i) mma(S[i], col_frag(s_k, SN, 32 * sp, 16 * i), vs);
        }
        __syncthreads();
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
// Forward: S = Σ_s e^{c_end − c_s} v_s k_sᵀ over the segment. Adjoint (REV, chunks in reverse order): the gradient
// reaching the state that enters the segment from its own outputs, E = Σ_u scale·e^{c_u} do_u q_uᵀ. Workgroup (row,
// head, 64 value columns, segment) as above.
template <typename T, int NT, bool REV>
__global__ __launch_bounds__(kThreads) void la_states_kernel(LinAttnLaunch a, int64_t first_seg, int64_t n_own) {
    constexpr int SN = NT + kPad<T>, SV = kPB + kPad<T>;
    __shared__ __align__(16) T s_k[kC * SN];
    __shared__ __align__(16) T s_v[kC * SV];
    __shared__ __align__(16) float s_w[kC];
    __shared__ float s_end;

    Work wk = work_of(a, n_own);
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
    const bool vec_k = REV ? a.vec_q : a.vec_k, vec_v = REV ? a.vec_do : a.vec_v;
    const int p0 = kPB * wk.pb;

    f4 S[NT / 16];
#pragma unroll
    for (int i = 0; i < NT / 16; ++i) S[i] = f4{0, 0, 0, 0};
    const int64_t n_chunks = (a.L + kC - 1) / kC;
    const int64_t ch0 = wk.seg * a.seg_chunks;
    const int64_t ch1 = ch0 + a.seg_chunks < n_chunks ? ch0 + a.seg_chunks : n_chunks;
    double total = 0.0;
    for (int64_t j = ch0; j < ch1; ++j) {
        const int64_t ch = REV ? ch1 - 1 - (j - ch0) : j;
        const int64_t t0 = ch * kC;
        if (t0 >= len) continue;
        stage<T, NT>(s_k, kp, kt, t0, len, 0, a.N, vec_k);
        stage<T, kPB>(s_v, vp, vt, t0, len, p0, a.P, vec_v);
        if (w == 0) {
            const double c = wave_running_sum(log_decay(gp, g_stride, t0 + l, len));
            const double end = __shfl(c, 63);
            s_w[l] = REV ? a.scale * exp_of((float)c) : exp_of((float)(end - c));
            if (l == 63) s_end = exp_of((float)c);
            total += end;
        }
        __syncthreads();
        const float end = s_end;
#pragma unroll
        for (int i = 0; i < NT / 16; ++i) S[i] *= end;
#pragma unroll
        for (int sp = 0; sp < 2; ++sp) {
            const f4 u = *reinterpret_cast<const f4 *>(&s_w[32 * sp + g4]);
            const f4 v = *reinterpret_cast<const f4 *>(&s_w[32 * sp + 16 + g4]);
            const Split<T, 3> vs(wide(col_frag(s_v, SV, 32 * sp, 16 * w)) * join(u, v));
#pragma unroll
            for (int i = 0; i < NT / 16; ++i) mma(S[i], col_frag(s_k, SN, 32 * sp, 16 * i), vs);
        }
        __syncthreads();
    }
    const int64_t Pp = (a.P + kPB - 1) / kPB * kPB, at = wk.bh * a.n_seg + wk.seg;
    float *dst = (REV ? a.E : a.S) + (at * Pp + p0 + 16 * w + col) * NT + g4;
#pragma unroll
    for (int i = 0; i < NT / 16; ++i) *reinterpret_cast<f4 *>(dst + 16 * i) = S[i];
    if (tid == 0 && wk.pb == 0) a.gsum[at] = total;
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

template <typename T>
hipError_t states(const LinAttnLaunch &p, bool adjoint, int64_t first, int64_t n, hipStream_t stream) {
    const int nt = linattn_nt(p.N);
    const dim3 grid((unsigned)(p.b * p.H * n * ((p.P + kPB - 1) / kPB)));
    if (nt == 32) {
        if (adjoint) la_states_kernel<T, 32, true><<<grid, kThreads, 0, stream>>>(p, first, n);
        else la_states_kernel<T, 32, false><<<grid, kThreads, 0, stream>>>(p, first, n);
    } else if (nt == 64) {
        if (adjoint) la_states_kernel<T, 64, true><<<grid, kThreads, 0, stream>>>(p, first, n);
        else la_states_kernel<T, 64, false><<<grid, kThreads, 0, stream>>>(p, first, n);
    } else {
        if (adjoint) la_states_kernel<T, 128, true><<<grid, kThreads, 0, stream>>>(p, first, n);
        else la_states_kernel<T, 128, false><<<grid, kThreads, 0, stream>>>(p, first, n);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t outputs(const LinAttnLaunch &p, hipStream_t stream) {
    const int nt = linattn_nt(p.N);
    const dim3 grid((unsigned)(p.b * p.H * p.n_seg * ((p.P + kPB - 1) / kPB)));
    if (nt == 32) la_out_kernel<T, 32><<<grid, kThreads, 0, stream>>>(p);
    else if (nt == 64) la_out_kernel<T, 64><<<grid, kThreads, 0, stream>>>(p);
    else la_out_kernel<T, 128><<<grid, kThreads, 0, stream>>>(p);
    return hipGetLastError();
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
