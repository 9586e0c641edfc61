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

constexpr int kOutThreads = kLinAttnOutThreads;

struct Work {
    int64_t ib, seg, bh;
    int h, grp, p0;  // p0: first value column
};
// id: of a piece of work; n_seg: segments that are worked on.
template <int NW> __device__ __forceinline__ Work work_of(const LinAttnLaunch &a, int64_t id, int64_t n_seg) {
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

// ---- outputs: one workgroup walks the chunks of (row, head, 64 value columns, segment) in order ------------------
//
// Eight wavefronts: w % 4 names 16 value columns, w / 4 a half of the chunk's steps for the outputs and a half of N for
// the state. A wavefront keeps its columns and its half of N of the state in result tiles and updates them; the outputs
// of its columns and steps need all of N, so the state's bf16 parts pass through LDS (a sixteenth of what is read
// there). The decayed scores, 10 lower-triangular 16×16 tiles, are shared through LDS too. The next chunk's rows are
// fetched into registers, and its decays formed by a wavefront without score tiles, while this chunk is computed.
// Bound: instruction issue and LDS, not memory. b 8, L 4096, 64 heads, N 128, P 64 in bf16 takes 355 us for 0.70 GB that a
// copy moves in 134 us. By the recurrence's operations (4·N·P a step and head) that is 194 Tflop/s, 15 % of what a large
// bf16 product reaches; it makes about three times as many. A wavefront issues 390 VALU, 51 MFMA, 78 LDS and 8 memory
// instructions a chunk, and 150 clocks go to bank conflicts. Three 64-step tiles, the scores in two parts and the state's
// first parts fill half a compute unit's LDS, so 128 steps per chunk would leave one workgroup on it.
// PARTS: bf16 parts of the state, as it enters the outputs, and of the scores. Two leave 2^-16 of each product; the outputs
// are then as far off as rounding them to bf16 alone. The state in one part takes 316 us here and puts them up to 1.4
// times as far off; its second part in LDS of its own, with one workgroup on a compute unit, takes 106 us where this takes
// 68 (64 rows of 64 steps, 32 heads, 128 by 64).
template <typename T, int NT, bool VEC>
__global__ __launch_bounds__(kOutThreads) __attribute__((amdgpu_waves_per_eu(sizeof(T) == 2 && VEC ? 4 : 2)))
void la_out_kernel(LinAttnLaunch a) {
    constexpr int SN = NT + kPad<T>, SP = kC + kPad<T>, SV = kPB + kPad<T>;
    constexpr int PARTS = sizeof(T) == 2 ? 2 : 1, NF = NT / 32;  // PARTS: of the state and of the scores
    typedef typename std::conditional<sizeof(T) == 2, bf4, f4>::type Half;  // a lane's part of one result tile
    __shared__ __align__(16) T s_q[kC * SN];
    __shared__ __align__(16) T s_k[kC * SN];
    __shared__ __align__(16) T s_v[kC * SV];
    __shared__ __align__(16) T s_p[PARTS][kC * SP];  // decayed scores [t][s], s in the order spread
    // the state's operand fragments. Their second parts stand in Q's place: Q's readers are done by the barrier before they are
    // written, and the next Q is stored past a barrier after they are read. That barrier saves the 16 KB without which two
    // workgroups do not fit on a compute unit.
    typedef Half StateParts[4][NF][64][2];
    __shared__ __align__(16) StateParts s_s;
    StateParts &s_low = *reinterpret_cast<StateParts *>(&s_q[0]);
    static_assert(PARTS == 1 || sizeof(StateParts) <= sizeof(s_q), "the second parts fit in Q's place");
    __shared__ Decays s_g[2];

    const Work wk = work_of<4>(a, work_index(blockIdx.x, gridDim.x), a.n_seg);
    const int tid = threadIdx.x, w = wave_id(), l = tid & 63, col = l & 15, g4 = 4 * (l >> 4);
    const int pw = w & 3, tw = w >> 2;
    const int64_t len = row_length(a.lengths, wk.ib, a.L);
    int64_t g_stride;
    const float *gp = decays_of(a, wk, &g_stride);
    const T *qp = static_cast<const T *>(a.q) + wk.ib * a.q_b + wk.grp * a.q_h;
    const T *kp = static_cast<const T *>(a.k) + wk.ib * a.k_b + wk.grp * a.k_h;
    const T *vp = static_cast<const T *>(a.v) + wk.ib * a.v_b + wk.h * a.v_h;
    T *op = static_cast<T *>(a.o) + (wk.ib * a.L * a.H + wk.h) * a.P;
    const uint32_t o_t = (uint32_t)a.H * a.P;  // elements between steps of o
    const int p0 = wk.p0, p_wave = p0 + 16 * pw;

    // result tiles of the state: rows n0 + 16i + 4·grp + r, column p_lane
    const int n0 = tw * (NT / 2);
    const int64_t p_lane = p_wave + col;
    f4 S[NF];
    if (a.n_seg > 1) {
        const int64_t Pp = (a.P + kPB - 1) / kPB * kPB;
        const float *src = a.S + ((wk.bh * a.n_seg + wk.seg) * Pp + p_lane) * NT + n0 + g4;
#pragma unroll
        for (int i = 0; i < NF; ++i) S[i] = *reinterpret_cast<const f4 *>(src + 16 * i);
    } else {
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int n = n0 + 16 * i + g4 + r;
                S[i][r] = a.initial_state && p_lane < a.P && n < a.N
                              ? a.initial_state[(wk.bh * a.P + p_lane) * a.N + n] : 0.0f;
            }
    }
    auto put_state = [&]() {
#pragma unroll
        for (int i = 0; i < NF; ++i) {
            // four values of N of column col, 16·(tile % 2) + 4·grp into their 32, where the plain order has them
            const int tile = tw * NF + i;
            const int at = 16 * (2 * (tile & 1) + (g4 >> 3)) + col, half = g4 >> 2 & 1;
            const Half part = __builtin_convertvector(S[i], Half);
            s_s[pw][tile >> 1][at][half] = part;
            if constexpr (PARTS == 2)
                s_low[pw][tile >> 1][at][half] = __builtin_convertvector(S[i] - __builtin_convertvector(part, f4), Half);
        }
    };
    put_state();

    // the tiles right of the diagonal that a 32-step contraction touches stay zero
    for (int i = tid; i < 2 * 16 * 16; i += kOutThreads) {
        const int t = 32 * (i >> 8) + ((i >> 4) & 15), s = 32 * (i >> 8) + 16 + (i & 15);
#pragma unroll
        for (int e = 0; e < PARTS; ++e) s_p[e][t * SP + spread_of(s)] = (T)0;
    }
    lds_barrier();

    const int64_t n_chunks = (a.L + kC - 1) / kC, live = (len + kC - 1) / kC;
    const int64_t ch0 = wk.seg * a.seg_chunks, ch1 = ch0 + a.seg_chunks < n_chunks ? ch0 + a.seg_chunks : n_chunks;
    const int64_t chl = ch1 < live ? ch1 : live;  // chunks with any step of the row
    Stage<T, NT, kOutThreads, VEC> rq((uint32_t)a.q_t, 0, a.N), rk((uint32_t)a.k_t, 0, a.N);
    Stage<T, kPB, kOutThreads, VEC> rv((uint32_t)a.v_t, p0, a.P);
    // Loads and stores share one in-order counter, and a wait in a loop is for what both ways into it have outstanding.
    // So the order is kept: a chunk's outputs are stored just before the loads of the chunk after next are issued, and
    // the decays' load goes with the others, one chunk further ahead (its scan comes while this one is computed).
    float g_next = 0.0f;
    f4 res[2] = {f4{0, 0, 0, 0}, f4{0, 0, 0, 0}};
    Buffer out = buffer_of(op, 0);  // nothing to store before the first chunk
    auto store_res = [&]() {
#pragma unroll
        for (int b = 0; b < 2; ++b) store4<T, VEC>(out, o_t, 16 * (2 * tw + b) + col, p_wave + g4, a.P, res[b]);
    };
    const bool is_result = a.final_state && wk.seg == a.n_seg - 1;
    const int64_t t_first = ch0 * kC;
    Cursor cq(qp + t_first * a.q_t, a.q_t, a.N), ck(kp + t_first * a.k_t, a.k_t, a.N), cv(vp + t_first * a.v_t, a.v_t, a.P);
    Cursor cg(gp + t_first * g_stride, g_stride, 1), co(op + t_first * (int64_t)o_t, o_t, a.P);
    RowsLeft in{len - t_first}, ing{len - t_first}, outs{a.L - t_first};
    auto fetch = [&]() {
        const int rows = in.next();
        rq.load(cq.next(rows), rows);
        rk.load(ck.next(rows), rows);
        rv.load(cv.next(rows), rows);
    };
    auto fetch_g = [&]() {
        const int rows = ing.next();
        return load_g(cg.next(rows), (uint32_t)g_stride, rows);
    };
    if (ch0 < chl) {
        const float g0 = fetch_g();
        g_next = fetch_g();
        if (VEC) fetch();
        if (w == 3) s_g[0].set<true>(log_decay(g0), a.scale);
    }
    for (int64_t ch = ch0; ch < chl; ++ch) {
        const Decays &dec = s_g[(ch - ch0) & 1];
        const int all = outs.next(), some = ch + 1 == live ? (int)(len - ch * kC) : kC;
        if (!VEC) fetch();
        Frag<T> sf[PARTS][NF];
        if constexpr (PARTS == 2)
#pragma unroll
            for (int n = 0; n < NF; ++n) sf[1][n] = *reinterpret_cast<const Frag<T> *>(&s_low[pw][n][l][0]);
        rk.store(s_k);
        rv.store(s_v);
        if constexpr (PARTS == 2) lds_barrier();  // the second parts are read
        rq.store(s_q);
        float g_now = g_next;
        asm volatile("" : "+v"(g_now));  // it has arrived with the rest: no wait for it behind the next loads
        lds_barrier();
        // the state's second parts go first, before the next chunk's rows take registers
        f4 acc[2] = {f4{0, 0, 0, 0}, f4{0, 0, 0, 0}};
        if constexpr (PARTS == 2)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int n = 0; n < NF; ++n) mma(acc[b], sf[1][n], row_frag(s_q, SN, 16 * (2 * tw + b), 32 * n));
        store_res();
        out = co.next(all);
        g_next = fetch_g();
        if (VEC) fetch();  // past the last chunk: nothing

        // Through the state, and the decayed scores: a query fragment serves both. Score tile (tb, sb) holds
        // D[s][t] = k_s·q_t; a wavefront takes those of its two blocks of t and of s block pw, in two bf16 parts.
        __builtin_amdgcn_s_setprio(1);  // the workgroup that computes goes before the one that loads and stores: 3 % less time
#pragma unroll
        for (int n = 0; n < NF; ++n) sf[0][n] = *reinterpret_cast<const Frag<T> *>(&s_s[pw][n][l][0]);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int tb = 2 * tw + b;
            Frag<T> qf[NF];
#pragma unroll
            for (int n = 0; n < NF; ++n) qf[n] = row_frag(s_q, SN, 16 * tb, 32 * n);
#pragma unroll
            for (int n = 0; n < NF; ++n) mma(acc[b], sf[0][n], qf[n]);
            acc[b] *= dec.in[16 * tb + col];
            if (tb >= pw) {
                f4 sc = {0, 0, 0, 0};
#pragma unroll
                for (int n = 0; n < NF; ++n) mma(sc, row_frag(s_k, SN, 16 * pw, 32 * n), qf[n]);
                const int t = 16 * tb + col, s = 16 * pw + g4;
                const float th = dec.c.hi[t], tl = dec.c.lo[t];
                const f4 sh = *reinterpret_cast<const f4 *>(&dec.c.hi[s]), sl = *reinterpret_cast<const f4 *>(&dec.c.lo[s]);
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[r] *= a.scale * exp2_fast((th - sh[r]) + (tl - sl[r]));
                if (pw == tb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sc[r] = s + r <= t ? sc[r] : 0.0f;
                // steps s, s + 2 and s + 1, s + 3 are neighbours in the order spread
                const int at = t * SP + 32 * (pw >> 1) + 8 * (g4 >> 3) + 4 * (pw & 1) + (g4 >> 1 & 3);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    f2 v = {sc[r], sc[r + 2]};
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int e = 0; e < PARTS; ++e) {
                            const bf2 u = __builtin_convertvector(v, bf2);
                            *reinterpret_cast<bf2 *>(&s_p[e][at + 16 * r]) = u;
                            v -= __builtin_convertvector(u, f2);
                        }
                    } else {
                        *reinterpret_cast<f2 *>(&s_p[0][at + 16 * r]) = v;
                    }
                }
            }
        }
        if (w == 3) s_g[(ch + 1 - ch0) & 1].set<true>(log_decay(g_now), a.scale);
        lds_barrier();

        // From here to the next barrier the state's parts are written by the wavefronts that are done: nothing below reads them, or Q.
        const f4 through[2] = {acc[0], acc[1]};
        Frag<T> vf[2];
#pragma unroll
        for (int sp = 0; sp < 2; ++sp) vf[sp] = col_frag<true>(s_v, SV, 32 * sp, 16 * pw);
#pragma unroll
        for (int sp = 0; sp < 2; ++sp)
            if (sp <= tw)
#pragma unroll
                for (int e = 0; e < PARTS; ++e)
#pragma unroll
                    for (int b = 0; b < 2; ++b) mma(acc[b], vf[sp], row_frag(s_p[e], SP, 16 * (2 * tw + b), 32 * sp));
        // A NaN or Inf in V reaches earlier steps through the zero scores of the later ones; it also reaches each of the
        // wavefront's last 16 steps, so these tell. Then the sums are taken again over the steps up to each step's own.
        const float probe = (acc[1][0] * 0.0f + acc[1][1] * 0.0f) + (acc[1][2] * 0.0f + acc[1][3] * 0.0f);
        if (__any(probe != 0.0f)) {
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                const int tl = 16 * (2 * tw + b) + col;
                f4 v = b == 0 ? through[0] : through[1];
                for (int s = 0; s <= tl; ++s) {
                    float pr = 0.0f;
#pragma unroll
                    for (int e = 0; e < PARTS; ++e) pr += widen(s_p[e][tl * SP + spread_of(s)]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(pr, widen(s_v[s * SV + 16 * pw + g4 + r]), v[r]);
                }
                if (b == 0) acc[0] = v;
                else acc[1] = v;
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) res[b] = some < kC && 16 * (2 * tw + b) + col >= some ? f4{0, 0, 0, 0} : acc[b];

        // the state's update: V's columns scaled, in three parts where the state is an fp32 result, in two where it only
        // goes on to outputs in T (8 % less time)
        const float end = dec.end;
#pragma unroll
        for (int i = 0; i < NF; ++i) S[i] *= end;
#pragma unroll
        for (int sp = 0; sp < 2; ++sp) {
            const f4 u = *reinterpret_cast<const f4 *>(&dec.out[32 * sp + 2 * g4]);
            const f4 v = *reinterpret_cast<const f4 *>(&dec.out[32 * sp + 2 * g4 + 4]);
            auto update = [&](const auto &vs) {
#pragma unroll
                for (int i = 0; i < NF; ++i) mma(S[i], col_frag<true>(s_k, SN, 32 * sp, n0 + 16 * i), vs);
            };
            if (is_result) update(Split<T, 3>(wide(vf[sp]) * join(u, v)));
            else update(Split<T, 2>(wide(vf[sp]) * join(u, v)));
        }
        __builtin_amdgcn_s_setprio(0);
        put_state();  // its readers, and Q's, are past the last barrier
        lds_barrier();
    }
    store_res();

    // past the row's end: outputs are zero, the state stays
    for (int64_t ch = chl > ch0 ? chl : ch0; ch < ch1; ++ch) {
        const Buffer rest = rows_buffer(op + ch * kC * o_t, o_t, rows_of(ch * kC, a.L), a.P);
#pragma unroll
        for (int b = 0; b < 2; ++b)
            store4<T, VEC>(rest, o_t, 16 * (2 * tw + b) + col, p_wave + g4, a.P, f4{0, 0, 0, 0});
    }

    // what la_nonfinite_kernel asks for: whether the wavefront's part of the state the segment leaves is finite, and if it is
    // not, that part, where the lane itself had read the state entering
    if (a.bad && wk.seg + 1 < a.n_seg) {
        float probe = 0.0f;
#pragma unroll
        for (int i = 0; i < NF; ++i) probe += (S[i][0] * 0.0f + S[i][1] * 0.0f) + (S[i][2] * 0.0f + S[i][3] * 0.0f);
        const bool bad = __any(probe != 0.0f);
        const int64_t Pp = (a.P + kPB - 1) / kPB * kPB, at = wk.bh * a.n_seg + wk.seg;
        if (l == 0) a.bad[(at * (Pp / kPB) + p0 / kPB) * 8 + w] = bad;
        if (bad) {
            float *dst = a.S + (at * Pp + p_lane) * NT + n0 + g4;
#pragma unroll
            for (int i = 0; i < NF; ++i) *reinterpret_cast<f4 *>(dst + 16 * i) = S[i];
        }
    }

    if (is_result && p_lane < a.P) {
        float *dst = a.final_state + (wk.bh * a.P + p_lane) * a.N;
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n0 + 16 * i + g4 + r < a.N) dst[n0 + 16 * i + g4 + r] = S[i][r];
    }
}

// ---- a segment's own state, or its own adjoint -------------------------------------------------------------------
//
// State: S = Σ_s e^{c_end − c_s} v_s k_sᵀ over the segment. Adjoint: the gradient reaching the state that
// enters the segment from its own outputs, E = Σ_u scale·e^{c_u} do_u q_uᵀ. Workgroup (row, head, 16·NW value columns,
// segment) as above. Both walk the chunks from the far end of the decay to the near one, S from the last chunk back
// and E from the first on, so that each chunk's weights carry the decay of all chunks walked before it. The walk ends
// where that decay is below e^-200: what the rest would add is it times a state (adjoint) of the recurrence, which as
// an fp32 number is at most e^88.8, and the product is 0 in fp32 (smallest positive value e^-103.3). A NaN or Inf in the
// rest is what that leaves out: la_nonfinite_kernel sees to it. (The gradient's segments have one chunk each.)
template <typename T, int NT, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW) void la_states_kernel(LinAttnLaunch a, int64_t n_states, int64_t first_adjoint) {
    constexpr int THREADS = 64 * NW, PB = 16 * NW;
    constexpr int SN = NT + kPad<T>, SV = PB + kPad<T>;
    __shared__ __align__(16) T s_k[kC * SN];
    __shared__ __align__(16) T s_v[kC * SV];
    __shared__ Decays s_g;

    // the states of the first n_states segments, then the adjoints of those from first_adjoint on
    const int64_t blocks = a.b * a.H * ((a.P + PB - 1) / PB), n_fwd = blocks * n_states;
    const bool rev = (int64_t)blockIdx.x >= n_fwd;
    Work wk = rev ? work_of<NW>(a, work_index(blockIdx.x - n_fwd, gridDim.x - n_fwd), a.n_seg - first_adjoint)
                  : work_of<NW>(a, work_index(blockIdx.x, n_fwd), n_states);
    if (rev) wk.seg += first_adjoint;
    const int tid = threadIdx.x, w = wave_id(), l = tid & 63, col = l & 15, g4 = 4 * (l >> 4);
    const int64_t len = row_length(a.lengths, wk.ib, a.L);
    int64_t g_stride;
    const float *gp = decays_of(a, wk, &g_stride);
    const int64_t kt = rev ? a.q_t : a.k_t, vt = rev ? a.do_t : a.v_t;
    const T *kp = rev ? static_cast<const T *>(a.q) + wk.ib * a.q_b + wk.grp * a.q_h
                      : static_cast<const T *>(a.k) + wk.ib * a.k_b + wk.grp * a.k_h;
    const T *vp = rev ? static_cast<const T *>(a.dout) + wk.ib * a.do_b + wk.h * a.do_h
                      : static_cast<const T *>(a.v) + wk.ib * a.v_b + wk.h * a.v_h;
    const int p0 = wk.p0;

    f4 S[NT / 16];
#pragma unroll
    for (int i = 0; i < NT / 16; ++i) S[i] = f4{0, 0, 0, 0};
    const int64_t n_chunks = (a.L + kC - 1) / kC, live = (len + kC - 1) / kC;
    const int64_t ch0 = wk.seg * a.seg_chunks, ch1 = ch0 + a.seg_chunks < n_chunks ? ch0 + a.seg_chunks : n_chunks;
    const int64_t chl = ch1 < live ? ch1 : live;
    Stage<T, NT, THREADS, VEC> rk((uint32_t)kt, 0, a.N);
    Stage<T, PB, THREADS, VEC> rv((uint32_t)vt, p0, a.P);
    double passed = 0.0;  // in every wavefront: the sum of g over the chunks walked
    float g_next = 0.0f;
    const int64_t n = chl - ch0;
    auto start = [&](int64_t j) { return (rev ? ch0 + j : chl - 1 - j) * kC; };
    auto fetch = [&](int64_t t0) {
        const int rows = rows_of(t0, len);
        rk.load(kp + t0 * kt, rows);
        rv.load(vp + t0 * vt, rows);
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
        const double sum = wave_running_sum(log_decay(g_next)), total = lane_value(sum, 63);  // before the next loads
        // the weight of the lane's step, from all chunks walked and from this one
        const float wt = (rev ? a.scale : 1.0f) * exp_of(passed + (rev ? sum : total - sum));
        if (w == 0) s_g.out[spread_of(l)] = wt;
        passed += total;
        lds_barrier();
        if (j + 1 < n) {
            if (VEC) fetch(start(j + 1));
            g_next = fetch_g(start(j + 1));
        }
#pragma unroll
        for (int sp = 0; sp < 2; ++sp) {
            const f4 u = *reinterpret_cast<const f4 *>(&s_g.out[32 * sp + 2 * g4]);
            const f4 v = *reinterpret_cast<const f4 *>(&s_g.out[32 * sp + 2 * g4 + 4]);
            const Split<T, 3> vs(wide(col_frag<true>(s_v, SV, 32 * sp, 16 * w)) * join(u, v));
#pragma unroll
            for (int i = 0; i < NT / 16; ++i) mma(S[i], col_frag<true>(s_k, SN, 32 * sp, 16 * i), vs);
        }
        lds_barrier();
    }
    const int64_t Pp = (a.P + kPB - 1) / kPB * kPB, at = wk.bh * a.n_seg + wk.seg, p = p0 + 16 * w + col;
    if (p < Pp) {
        float *dst = (rev ? a.E : a.S) + (at * Pp + p) * NT;
#pragma unroll
        for (int i = 0; i < NT / 16; ++i) *reinterpret_cast<f4 *>(dst + 16 * i + g4) = S[i];
    }
    if (tid == 0 && p0 == 0) a.gsum[at] = passed;
}

// ---- from the segments' own states to those entering them (adjoints: leaving them), in place ---------------------
//
// One thread per four state elements steps over the segments; eight loads are kept in flight. Memory bounds it: the
// states and adjoints of all chunks of the gradient at b 4, L 2048, 24 heads, N = P = 64, 0.2 GB both ways, take 31 us
// (30 to 45 over 400 calls; 6.4 TB/s). A carry over segments of six chunks, with the chunks' states formed from zero at
// their segment's border and put together where they are used, took 8 us, but the walk and the gradient's kernel 37 us
// more.
__global__ __launch_bounds__(kThreads) void la_carry_kernel(LinAttnLaunch a, int NT) {
    const int64_t Pp = (a.P + kPB - 1) / kPB * kPB;
    const int64_t per = Pp * NT / 4;                       // four-element groups of one state: a multiple of 256
    const int64_t blocks = per / kThreads * a.b * a.H;     // the states', then (in the gradient) the adjoints'
    const bool rev = blockIdx.x >= blocks;
    const int64_t block = rev ? blockIdx.x - blocks : blockIdx.x;
    const int64_t bh = block / (per / kThreads);
    const int64_t e = block % (per / kThreads) * kThreads + threadIdx.x;
    const int64_t p = 4 * e / NT, n = 4 * e % NT;
    f4 *base = reinterpret_cast<f4 *>(rev ? a.E : a.S) + bh * a.n_seg * per + e;
    const double *gs = a.gsum + bh * a.n_seg;
    const float *first = rev ? a.d_final_state : a.initial_state;
    f4 carry = {0, 0, 0, 0};
    if (first && p < a.P)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < a.N) carry[r] = first[(bh * a.P + p) * a.N + n + r];
    constexpr int U = 8;
    for (int64_t j0 = 0; j0 < a.n_seg; j0 += U) {
        f4 own[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // the last own state (adjoint: the first, unless asked for) is not needed and may not be there
            const int64_t j = j0 + u, s = rev ? a.n_seg - 1 - j : j;
            const bool need = j < a.n_seg && (j + 1 < a.n_seg || (rev && a.d_initial_state));
            own[u] = need ? base[s * per] : f4{0, 0, 0, 0};
            d[u] = need ? exp_of(gs[s]) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t j = j0 + u, s = rev ? a.n_seg - 1 - j : j;
            if (j < a.n_seg) {
                base[s * per] = carry;
                carry = carry * d[u] + own[u];
            }
        }
    }
    if (rev && a.d_initial_state && p < a.P)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < a.N) a.d_initial_state[(bh * a.P + p) * a.N + n + r] = carry[r];
}

// ---- a NaN or Inf that a walk over a segment's own state did not reach -------------------------------------------
//
// e^-200 times a NaN or Inf is not 0: once an element of the state is one, it stays one (Inf or NaN) for all later steps, and
// so does its column of the outputs. The walk that gives the outputs meets every step and says which segments it left with
// such an element; here one workgroup per (row, head, 64 value columns) carries it into the segments after. It costs a
// launch in calls of more than one segment of more than one chunk, 4.7 us where all is finite.
template <typename T>
__global__ __launch_bounds__(kThreads) void la_nonfinite_kernel(LinAttnLaunch a, int NT) {
    const int64_t npb = (a.P + kPB - 1) / kPB, pb = blockIdx.x % npb, bh = blockIdx.x / npb;
    const int64_t ib = bh / a.H, h = bh % a.H, last = a.n_seg - 1;
    const int tid = threadIdx.x;
    auto word = [&](int64_t seg, int w) { return a.bad[((bh * a.n_seg + seg) * npb + pb) * 8 + w]; };
    uint32_t any = 0;
    for (int64_t i = tid; i < last * 8; i += kThreads) any |= word(i / 8, (int)(i % 8));
    if (!__syncthreads_or((int)any)) return;

    __shared__ int s_from[kPB];  // the first segment that a column enters with a NaN or Inf
    if (tid < kPB) s_from[tid] = (int)a.n_seg;
    __syncthreads();
    const float nan = __uint_as_float(0x7fc00000u);
    for (int64_t seg = 0; seg < last; ++seg) {
        const float *left = a.S + ((bh * a.n_seg + seg) * npb + pb) * kPB * NT;
        for (int i = tid; i < kPB * NT; i += kThreads) {
            const int p = i / NT, n = i % NT;
            if (!word(seg, p / 16 + (2 * n >= NT ? 4 : 0)) || left[i] * 0.0f == 0.0f) continue;
            atomicMin(&s_from[p], (int)seg + 1);
            if (a.final_state && pb * kPB + p < a.P && n < a.N)
                a.final_state[(bh * a.P + pb * kPB + p) * a.N + n] = nan;
        }
    }
    __syncthreads();
    const int64_t len = row_length(a.lengths, ib, a.L);
    T *o = static_cast<T *>(a.o) + (ib * a.L * a.H + h) * a.P + pb * kPB;
    const int p = tid % kPB;
    if (pb * kPB + p < a.P)
        for (int64_t t = s_from[p] * a.seg_chunks * kC + tid / kPB; t < len; t += kThreads / kPB)
            o[t * a.H * a.P + p] = narrow<T>(nan);
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
hipError_t states(const LinAttnLaunch &p, int64_t n_states, int64_t first_adjoint, hipStream_t stream) {
    const dim3 grid((unsigned)(p.b * p.H * (n_states + p.n_seg - first_adjoint)) * value_blocks(p));
    return by_width(p, [&](auto nt, auto nw, auto vec) {
        constexpr int NT = decltype(nt)::value, NW = decltype(nw)::value;
        constexpr bool VEC = decltype(vec)::value;
        la_states_kernel<T, NT, NW, VEC><<<grid, 64 * NW, 0, stream>>>(p, n_states, first_adjoint);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t nonfinite(const LinAttnLaunch &p, hipStream_t stream) {
    const dim3 grid((unsigned)(p.b * p.H) * (unsigned)((p.P + kPB - 1) / kPB));
    la_nonfinite_kernel<T><<<grid, kThreads, 0, stream>>>(p, linattn_nt(p.N));
    return hipGetLastError();
}

template <typename T>
hipError_t outputs(const LinAttnLaunch &p, hipStream_t stream) {
    const dim3 grid((unsigned)(p.b * p.H * p.n_seg) * (unsigned)((p.P + kPB - 1) / kPB));
    return by_width(p, [&](auto nt, auto, auto vec) {
        constexpr int NT = decltype(nt)::value;
        constexpr bool VEC = decltype(vec)::value;
        la_out_kernel<T, NT, VEC><<<grid, kOutThreads, 0, stream>>>(p);
        return hipGetLastError();
    });
}

}  // namespace
}  // namespace la

hipError_t launch_linattn_states(const LinAttnLaunch &p, int64_t n_states, int64_t first_adjoint, hipStream_t stream) {
    if (n_states == 0 && first_adjoint == p.n_seg) return hipSuccess;
    return p.bf16 ? la::states<uint16_t>(p, n_states, first_adjoint, stream)
                  : la::states<float>(p, n_states, first_adjoint, stream);
}

hipError_t launch_linattn_carry(const LinAttnLaunch &p, bool adjoint, hipStream_t stream) {
    const int nt = linattn_nt(p.N);
    const int64_t per = (p.P + la::kPB - 1) / la::kPB * la::kPB * nt / 4 / la::kThreads;
    la::la_carry_kernel<<<dim3((unsigned)(p.b * p.H * per * (adjoint ? 2 : 1))), la::kThreads, 0, stream>>>(p, nt);
    return hipGetLastError();
}

hipError_t launch_linattn_fwd(const LinAttnLaunch &p, hipStream_t stream) {
    if (p.n_seg > 1) {
        hipError_t e = launch_linattn_states(p, p.n_seg - 1, p.n_seg, stream);
        if (e == hipSuccess) e = launch_linattn_carry(p, false, stream);
        if (e != hipSuccess) return e;
    }
    hipError_t e = p.bf16 ? la::outputs<uint16_t>(p, stream) : la::outputs<float>(p, stream);
    if (e == hipSuccess && p.bad) e = p.bf16 ? la::nonfinite<uint16_t>(p, stream) : la::nonfinite<float>(p, stream);
    return e;
}

}  // namespace ssm
