// linattn_bwd.hip — gradients of linear attention with a per-head decay.
//
// By the chain rule on o_t = scale·S_t q_t, S_t = e^{g_t} S_{t−1} + v_t k_tᵀ (page "Mambaとは？Transformer以外の系列
// モデル", section 状態空間モデルを一つの式から理解する): with E_t = scale·do_t q_tᵀ + e^{g_{t+1}} E_{t+1} the adjoint
// of S_t,
//     dq_t = scale·S_tᵀ do_t,  dk_t = E_tᵀ v_t,  dv_t = E_t k_t,  dg_t = e^{g_t}·<S_{t−1}, E_t>.
// In a chunk with running sums c, the state S entering it and the adjoint E leaving it (of the state after its last
// step), A1_ts = scale·e^{c_t − c_s} q_t·k_s and A2_ts = scale·e^{c_t − c_s} do_t·v_s for s <= t:
//     dq_t = Σ_s A2_ts k_s + scale·e^{c_t} Sᵀdo_t,      dk_s = Σ_t A2_ts q_t + e^{c_end − c_s} Eᵀv_s,
//     dv_s = Σ_t A1_ts do_t + e^{c_end − c_s} E k_s,
//     dg_t = Σ_{u>=t} (Σ_{s<u} W_us − Σ_{s>u} W_su + X_u) + Σ_{s<t} Y_s + e^{c_end}<S, E>
// with W_us = A1_us·(do_u·v_s), X_u = q_u·(scale·e^{c_u} Sᵀdo_u), Y_s = v_s·(e^{c_end − c_s} E k_s): the paths from a
// step before t to one at or after it, by whether either end lies outside the chunk. The pairs that do not span t cancel
// between the sums over rows and over columns: both are of the same fp32 terms and taken in fp64, so that 2^-53 of them is
// left, and no sum runs past the chunk.
#include "linattn_common.h"

namespace ssm {
namespace la {
namespace {

// Sum over the four 16-lane groups of a wavefront (same column), for every lane: the rows of 16 lanes swapped pairwise.
__device__ __forceinline__ float sum_groups(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
// Sum over the 16 lanes of a group, for every lane: rotations within the row.
template <int N> __device__ __forceinline__ float row_rotate(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x120 + N, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum_cols(float v) {
    v += row_rotate<8>(v);
    v += row_rotate<4>(v);
    v += row_rotate<2>(v);
    return v + row_rotate<1>(v);
}

// The same for fp64 values, word by word.
__device__ __forceinline__ double of_words(uint32_t lo, uint32_t hi) {
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double sum_groups(double v) {
    uint64_t u = __builtin_bit_cast(uint64_t, v);
    const auto a = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
    u = __builtin_bit_cast(uint64_t, of_words(a[0], b[0]) + of_words(a[1], b[1]));
    const auto c = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
    const auto d = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
    return of_words(c[0], d[0]) + of_words(c[1], d[1]);
}
template <int N> __device__ __forceinline__ double row_rotate(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return of_words(__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, 0x120 + N, 0xf, 0xf, false),
                    __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), 0x120 + N, 0xf, 0xf, false));
}
__device__ __forceinline__ double sum_cols(double v) {
    v += row_rotate<8>(v);
    v += row_rotate<4>(v);
    v += row_rotate<2>(v);
    return v + row_rotate<1>(v);
}

// ---- one workgroup per (row, head, chunk), all value columns -----------------------------------------------------
//
// The four wavefronts share the lower-triangular tiles of both score matrices through LDS; wavefront w takes the value
// columns 16w .. of dv, and 16-column jobs of dq and dk, whose parts through state and adjoint come first: V is free then
// and A1 takes its place, which leaves room for three workgroups on a compute unit. Bound: memory and its latency. b 4,
// L 2048, 24 heads, N = P = 64 in bf16 takes 67 us for 0.30 GB (4.4 TB/s); eight wavefronts to a workgroup took 13 us more.
// PARTS: bf16 parts of the scores A1 and A2 (E, as it enters dv, takes as many; S and E in dq and dk take three, because dg's
// terms come from them). Two leave 2^-16 of each product, and dq, dk and dv as far off as rounding them to bf16 alone; one
// leaves them 1.4 times as far off, twice where a group's heads are summed. The second parts wait in registers and take
// A2's place one after the other, four barriers more: the call above takes 131 us, with one part 128, with all four tiles
// in LDS, which leave room for two workgroups, 141.
template <typename T, int NT, bool VEC>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(sizeof(T) == 2 && NT < 128 ? 3 : 1)))
void la_grad_kernel(LinAttnLaunch a) {
    constexpr int PARTS = sizeof(T) == 2 ? 2 : 1;
    constexpr int SN = NT + kPad<T>, SP = kC + kPad<T>, SV = kPB + kPad<T>;
    constexpr int TILES = NT / 16, JOBS = 2 * TILES / 4;
    __shared__ __align__(16) T s_q[kC * SN];
    __shared__ __align__(16) T s_k[kC * SN];
    static_assert(SP == SV, "A1 takes V's place");
    __shared__ __align__(16) T s_v[kC * SV];
    __shared__ __align__(16) T s_d[kC * SV];
    // A2 [t][s], then the second parts of A2 and of A1; the terms of dg are taken before any is rounded
    __shared__ __align__(16) T s_a2[kC * SP];
    T *const s_a1 = s_v;
    __shared__ Decays s_g;
    __shared__ double s_row[4][kC], s_col[4][kC];
    __shared__ float s_x[TILES][kC], s_y[TILES][kC], s_z[4];

    int64_t id = work_index(blockIdx.x, gridDim.x);
    const int h = (int)(id % a.H);
    id /= a.H;
    const int64_t ch = id % a.n_seg, ib = id / a.n_seg;
    const int ratio = a.H / a.G, grp = h / ratio;
    const int64_t bh = ib * a.H + h;
    const int tid = threadIdx.x, w = wave_id(), l = tid & 63, col = l & 15, g4 = 4 * (l >> 4);
    const int64_t len = row_length(a.lengths, ib, a.L);
    const int64_t t0 = ch * kC;
    const int64_t rows = a.L - t0 < kC ? a.L - t0 : kC;
    const int some = rows_of(t0, len);  // steps of the row in this chunk
    const int npb = (a.P + kPB - 1) / kPB;

    float *dgp = (a.g_per_step ? a.dg : a.dg_steps) + (ib * a.L + t0) * a.H + h;
    T *dvp = static_cast<T *>(a.dv) + ((ib * a.L + t0) * a.H + h) * a.P;
    const int64_t dv_t = (int64_t)a.H * a.P;
    // dq and dk: straight to the outputs, or this head's share in fp32
    const bool part = ratio > 1;
    const int64_t n_t = (int64_t)(part ? a.H : a.G) * a.N, n_off = (ib * a.L + t0) * n_t + (int64_t)(part ? h : grp) * a.N;

    if (t0 >= len) {
        for (int64_t i = tid; i < rows * a.P; i += kThreads) dvp[i / a.P * dv_t + i % a.P] = (T)0;
        for (int64_t i = tid; i < rows * a.N; i += kThreads) {
            const int64_t at = n_off + i / a.N * n_t + i % a.N;
            if (part) {
                a.dq_part[at] = 0.0f;
                a.dk_part[at] = 0.0f;
            } else {
                static_cast<T *>(a.dq)[at] = (T)0;
                static_cast<T *>(a.dk)[at] = (T)0;
            }
        }
        for (int64_t i = tid; i < rows; i += kThreads) dgp[i * a.H] = 0.0f;
        return;
    }

    const Buffer dv_buf = rows_buffer(dvp, (uint32_t)dv_t, (int)rows, a.P);
    const Buffer dq_buf = part ? rows_buffer(a.dq_part + n_off, (uint32_t)n_t, (int)rows, a.N)
                               : rows_buffer(static_cast<T *>(a.dq) + n_off, (uint32_t)n_t, (int)rows, a.N);
    const Buffer dk_buf = part ? rows_buffer(a.dk_part + n_off, (uint32_t)n_t, (int)rows, a.N)
                               : rows_buffer(static_cast<T *>(a.dk) + n_off, (uint32_t)n_t, (int)rows, a.N);
    const int64_t g_stride = a.g_per_step ? a.H : 0;
    const float *gp = a.g_per_step ? a.g + ib * a.L * a.H + h : a.g + h;
    const T *qp = static_cast<const T *>(a.q) + ib * a.q_b + grp * a.q_h;
    const T *kp = static_cast<const T *>(a.k) + ib * a.k_b + grp * a.k_h;
    const T *vp = static_cast<const T *>(a.v) + ib * a.v_b + h * a.v_h;
    const T *dp = static_cast<const T *>(a.dout) + ib * a.do_b + h * a.do_h;

    {
        Stage<T, NT, kThreads, VEC> q((uint32_t)a.q_t, 0, a.N), k((uint32_t)a.k_t, 0, a.N);
        q.load(qp + t0 * a.q_t, rows_of(t0, len));
        k.load(kp + t0 * a.k_t, rows_of(t0, len));
        if (w == 0) s_g.set<false>(log_decay(load_g(gp + t0 * g_stride, (uint32_t)g_stride, rows_of(t0, len))), a.scale);
        q.store(s_q);
        k.store(s_k);
    }
    // The wavefront's parts of the entering state S and the leaving adjoint E: eight values along P at its columns of N.
    const int64_t Pp = (int64_t)npb * kPB;
    const float *Sp = a.S + (bh * a.n_seg + ch) * Pp * NT;
    const float *Ep = a.E + (bh * a.n_seg + ch) * Pp * NT;
    f8 x[JOBS][2];
    auto fetch_states = [&](int pb) {
#pragma unroll
        for (int j = 0; j < JOBS; ++j) {
            const int job = w + 4 * j;
            const bool is_q = job < TILES;
            const float *src = (is_q ? Sp : Ep) + (pb * kPB + 2 * g4) * NT + 16 * (is_q ? job : job - TILES) + col;
#pragma unroll
            for (int pp = 0; pp < 2; ++pp)
#pragma unroll
                for (int r = 0; r < 8; ++r) x[j][pp][r] = src[(32 * pp + r) * NT];
        }
    };

    // Over the value columns: the scores' tiles (tb, sb), D[s][t] of q·k and do·v, and the parts of dq and dk that come
    // through the state and the adjoint (in three bf16 parts: dg's terms X and Y are taken from them).
    f4 aq[3], ad[3], acc[JOBS][4];
#pragma unroll
    for (int j = 0; j < 3; ++j) aq[j] = ad[j] = f4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < JOBS; ++j)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[j][b] = f4{0, 0, 0, 0};
    float z = 0.0f;
    for (int pb = 0; pb < npb; ++pb) {
        Stage<T, kPB, kThreads, VEC> v((uint32_t)a.v_t, pb * kPB, a.P), d((uint32_t)a.do_t, pb * kPB, a.P);
        v.load(vp + t0 * a.v_t, rows_of(t0, len));
        d.load(dp + t0 * a.do_t, rows_of(t0, len));
        fetch_states(pb);
        if (pb) lds_barrier();
        v.store(s_v);
        d.store(s_d);
        lds_barrier();
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int i = w + 4 * j;
            if (i < 10) {
                const int tb = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3, sb = i - tb * (tb + 1) / 2;
                if (pb == 0)
#pragma unroll
                    for (int n = 0; n < NT; n += 32) mma(aq[j], row_frag(s_k, SN, 16 * sb, n), row_frag(s_q, SN, 16 * tb, n));
#pragma unroll
                for (int n = 0; n < kPB; n += 32) mma(ad[j], row_frag(s_v, SV, 16 * sb, n), row_frag(s_d, SV, 16 * tb, n));
            }
        }
#pragma unroll
        for (int j = 0; j < JOBS; ++j) {
            const T *tile = w + 4 * j < TILES ? s_d : s_v;
#pragma unroll
            for (int pp = 0; pp < 2; ++pp) {
                const Split<T, 3> xs(x[j][pp]);
#pragma unroll
                for (int b = 0; b < 4; ++b) mma(acc[j][b], xs, row_frag(tile, SV, 16 * b, 32 * pp));
            }
        }
        // <S, E>
        if (JOBS == 1) {  // a wavefront has dq's state or dk's adjoint, not both
            const int64_t at = (int64_t)(pb * kPB + 16 * w + col) * NT + g4;
#pragma unroll
            for (int i = 0; i < NT / 16; ++i) {
                const f4 u = *reinterpret_cast<const f4 *>(Sp + at + 16 * i), v4 = *reinterpret_cast<const f4 *>(Ep + at + 16 * i);
                z += (u[0] * v4[0] + u[1] * v4[1]) + (u[2] * v4[2] + u[3] * v4[3]);
            }
        } else {  // the same columns of N in its job of dq and in that of dk
#pragma unroll
            for (int j = 0; j < JOBS / 2; ++j)
#pragma unroll
                for (int pp = 0; pp < 2; ++pp)
#pragma unroll
                    for (int r = 0; r < 8; ++r) z = __builtin_fmaf(x[j][pp][r], x[j + JOBS / 2][pp][r], z);
        }
    }
#pragma unroll
    for (int j = 0; j < JOBS; ++j) {
        const int job = w + 4 * j;
        const bool is_q = job < TILES;
        const int tile = is_q ? job : job - TILES;
        const T *rows_n = is_q ? s_q : s_k;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int t = 16 * b + col;
            f4 &v = acc[j][b];
            v *= is_q ? s_g.in[t] : s_g.out[t];
            const T *r = rows_n + t * SN + 16 * tile + g4;
            const float xy = sum_groups((v[0] * widen(r[0]) + v[1] * widen(r[1])) + (v[2] * widen(r[2]) + v[3] * widen(r[3])));
            if (l < 16) (is_q ? s_x : s_y)[tile][t] = xy;
        }
    }
    z = sum_groups(sum_cols(z));
    if (l == 0) s_z[w] = z;

    // E once more, eight values along N at the wavefront's value columns (for dv), on their way while the scores are weighted
    f8 e[NT / 32];
    auto fetch_adjoint = [&](int pb) {
        const float *src = Ep + (int64_t)(pb * kPB + 16 * w + col) * NT + 2 * g4;
#pragma unroll
        for (int n = 0; n < NT / 32; ++n)
            e[n] = join(*reinterpret_cast<const f4 *>(src + 32 * n), *reinterpret_cast<const f4 *>(src + 32 * n + 4));
    };
    fetch_adjoint(0);
    lds_barrier();  // V's tile is free: A1 takes its place

    // the tiles right of the diagonal that a 32-step contraction touches
    for (int i = tid; i < 2 * 16 * 16; i += kThreads) {
        const int t = 32 * (i >> 8) + ((i >> 4) & 15), s = 32 * (i >> 8) + 16 + (i & 15);
        s_a1[t * SP + s] = s_a2[t * SP + s] = (T)0;
    }
    bf4 a1_low[3], a2_low[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int i = w + 4 * j;
        if (i < 10) {
            const int tb = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3, sb = i - tb * (tb + 1) / 2;
            const int t = 16 * tb + col, s = 16 * sb + g4;
            const float th = s_g.c.hi[t], tl = s_g.c.lo[t];
            const f4 sh = *reinterpret_cast<const f4 *>(&s_g.c.hi[s]), sl = *reinterpret_cast<const f4 *>(&s_g.c.lo[s]);
            f4 a1, a2, wv;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = a.scale * exp2_fast((th - sh[r]) + (tl - sl[r]));
                a1[r] = aq[j][r] * d;
                a2[r] = ad[j][r] * d;
                wv[r] = a1[r] * ad[j][r];
            }
            if (sb == tb)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    a1[r] = s + r <= t ? a1[r] : 0.0f;
                    a2[r] = s + r <= t ? a2[r] : 0.0f;
                    wv[r] = s + r < t ? wv[r] : 0.0f;
                }
            // in fp64: most of a row's sum goes out against the columns' (pairs of steps that do not span t)
            const double row = sum_groups(((double)wv[0] + wv[1]) + ((double)wv[2] + wv[3]));
            if (l < 16) s_row[sb][t] = row;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const double column = sum_cols((double)wv[r]);
                if (col == 0) s_col[tb][s + r] = column;
            }
            if constexpr (PARTS == 2) {
                const bf4 u = __builtin_convertvector(a1, bf4), v = __builtin_convertvector(a2, bf4);
                *reinterpret_cast<bf4 *>(&s_a1[t * SP + s]) = u;
                *reinterpret_cast<bf4 *>(&s_a2[t * SP + s]) = v;
                a1_low[j] = __builtin_convertvector(a1 - __builtin_convertvector(u, f4), bf4);
                a2_low[j] = __builtin_convertvector(a2 - __builtin_convertvector(v, f4), bf4);
            } else {
                *reinterpret_cast<f4 *>(&s_a1[t * SP + s]) = a1;
                *reinterpret_cast<f4 *>(&s_a2[t * SP + s]) = a2;
            }
        }
    }
    // the scores' second parts, in A2's place when what is there has been read
    auto put_low = [&](const bf4 (&low)[3]) {
        lds_barrier();
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int i = w + 4 * j;
            if (i < 10) {
                const int tb = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3, sb = i - tb * (tb + 1) / 2;
                *reinterpret_cast<bf4 *>(&s_a2[(16 * tb + col) * SP + 16 * sb + g4]) = low[j];
            }
        }
        lds_barrier();
    };
    lds_barrier();

    if (w == 0) {  // dg
        const int b = l >> 4;
        double after = 0.0, ys = 0.0;
        for (int i = 0; i <= b; ++i) after += s_row[i][l];
        for (int i = b; i < 4; ++i) after -= s_col[i][l];
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            after += s_x[i][l];
            ys += s_y[i][l];
        }
        const double upto = wave_running_sum(after), yto = wave_running_sum(ys);
        const double zs = (((double)s_z[0] + s_z[1]) + ((double)s_z[2] + s_z[3])) * s_g.end;
        const double v = (lane_value(upto, 63) - upto + after) + (yto - ys) + zs;
        if (l < rows) dgp[(int64_t)l * a.H] = t0 + l < len ? (float)v : 0.0f;
    }
    // dq and dk through the scores
    auto add_scores = [&]() {
#pragma unroll
        for (int j = 0; j < JOBS; ++j) {
            const int job = w + 4 * j;
            const bool is_q = job < TILES;
            const int n0 = 16 * (is_q ? job : job - TILES);
            const T *tile = is_q ? s_k : s_q;
            const Frag<T> f0 = col_frag(tile, SN, 0, n0), f1 = col_frag(tile, SN, 32, n0);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (is_q) {
                    mma(acc[j][b], f0, row_frag(s_a2, SP, 16 * b, 0));
                    if (b >= 2) mma(acc[j][b], f1, row_frag(s_a2, SP, 16 * b, 32));
                } else {
                    if (b < 2) mma(acc[j][b], f0, col_frag(s_a2, SP, 0, 16 * b));
                    mma(acc[j][b], f1, col_frag(s_a2, SP, 32, 16 * b));
                }
            }
        }
    };
    add_scores();
    if constexpr (PARTS == 2) {
        put_low(a2_low);
        add_scores();
    }
#pragma unroll
    for (int j = 0; j < JOBS; ++j) {
        const int job = w + 4 * j;
        const bool is_q = job < TILES;
        const int n0 = 16 * (is_q ? job : job - TILES);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int t = 16 * b + col;
            f4 &v = acc[j][b];
            if (some < kC && t >= some) v = f4{0, 0, 0, 0};
            const Buffer &buf = is_q ? dq_buf : dk_buf;
            if (part) store4<float, VEC>(buf, (uint32_t)n_t, t, n0 + g4, a.N, v);
            else store4<T, VEC>(buf, (uint32_t)n_t, t, n0 + g4, a.N, v);
        }
    }
    if constexpr (PARTS == 2) put_low(a1_low);
    for (int pb = 0; pb < npb; ++pb) {  // dv: value columns 16w .. of each block
        if (npb > 1) {
            Stage<T, kPB, kThreads, VEC> d((uint32_t)a.do_t, pb * kPB, a.P);
            d.load(dp + t0 * a.do_t, some);
            if (pb) {
                fetch_adjoint(pb);
                lds_barrier();
            }
            d.store(s_d);
            lds_barrier();
        }
        f4 dv[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) dv[b] = f4{0, 0, 0, 0};
#pragma unroll
        for (int n = 0; n < NT / 32; ++n) {
            const Split<T, 2> es(e[n]);
#pragma unroll
            for (int b = 0; b < 4; ++b) mma(dv[b], es, row_frag(s_k, SN, 16 * b, 32 * n));
        }
        const Frag<T> d0 = col_frag(s_d, SV, 0, 16 * w), d1 = col_frag(s_d, SV, 32, 16 * w);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int s = 16 * b + col;
            dv[b] *= s_g.out[s];
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                const T *a1 = p ? s_a2 : s_a1;
                if (b < 2) mma(dv[b], d0, col_frag(a1, SP, 0, 16 * b));
                mma(dv[b], d1, col_frag(a1, SP, 32, 16 * b));
            }
            if (some < kC && s >= some) dv[b] = f4{0, 0, 0, 0};
            store4<T, VEC>(dv_buf, (uint32_t)dv_t, s, pb * kPB + 16 * w + g4, a.P, dv[b]);
        }
    }
}

// dq and dk of a group: the sum over its heads, in order.
template <typename T>
__global__ __launch_bounds__(kThreads) void la_group_sum_kernel(const float *dq_part, const float *dk_part, T *dq, T *dk,
                                                                int64_t n, int N, int ratio) {
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t src = i / N * ratio * N + i % N;  // [b][L][G][ratio][N]
        float q = 0.0f, k = 0.0f;
        for (int r = 0; r < ratio; ++r) {
            q += dq_part[src + (int64_t)r * N];
            k += dk_part[src + (int64_t)r * N];
        }
        dq[i] = narrow<T>(q);
        dk[i] = narrow<T>(k);
    }
}

// dg of a decay that is the same at every step: the sum over rows and steps, one workgroup per head.
__global__ __launch_bounds__(kThreads) void la_dg_sum_kernel(const float *dg_steps, float *dg, int64_t n, int H) {
    __shared__ double s[kThreads];
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) v += dg_steps[i * H + blockIdx.x];
    s[threadIdx.x] = v;
    for (int d = kThreads / 2; d > 0; d >>= 1) {
        __syncthreads();
        if ((int)threadIdx.x < d) s[threadIdx.x] += s[threadIdx.x + d];
    }
    if (threadIdx.x == 0) dg[blockIdx.x] = (float)s[0];
}

template <typename T>
hipError_t grads(const LinAttnLaunch &p, hipStream_t stream) {
    const int nt = linattn_nt(p.N);
    const dim3 grid((unsigned)(p.b * p.H * p.n_seg));
    auto launch = [&](auto vec) {
        constexpr bool VEC = decltype(vec)::value;
        if (nt == 32) la_grad_kernel<T, 32, VEC><<<grid, kThreads, 0, stream>>>(p);
        else if (nt == 64) la_grad_kernel<T, 64, VEC><<<grid, kThreads, 0, stream>>>(p);
        else la_grad_kernel<T, 128, VEC><<<grid, kThreads, 0, stream>>>(p);
    };
    if (p.vec) launch(std::true_type{});
    else launch(std::false_type{});
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.G < p.H) {
        const int64_t n = p.b * p.L * p.G * p.N, blocks = (n + kThreads - 1) / kThreads;
        la_group_sum_kernel<T><<<dim3((unsigned)(blocks < 16384 ? blocks : 16384)), kThreads, 0, stream>>>(
            p.dq_part, p.dk_part, static_cast<T *>(p.dq), static_cast<T *>(p.dk), n, p.N, p.H / p.G);
        e = hipGetLastError();
    }
    if (e == hipSuccess && !p.g_per_step) {
        la_dg_sum_kernel<<<dim3((unsigned)p.H), kThreads, 0, stream>>>(p.dg_steps, p.dg, p.b * p.L, p.H);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace
}  // namespace la

hipError_t launch_linattn_bwd(const LinAttnLaunch &p, hipStream_t stream) {
    // the last segment's own state is not needed, the first's own adjoint only for d_initial_state
    hipError_t e = launch_linattn_states(p, p.n_seg - 1, p.d_initial_state ? 0 : 1, stream);
    if (e == hipSuccess) e = launch_linattn_carry(p, true, stream);
    if (e == hipSuccess) e = p.bf16 ? la::grads<uint16_t>(p, stream) : la::grads<float>(p, stream);
    return e;
}

}  // namespace ssm
