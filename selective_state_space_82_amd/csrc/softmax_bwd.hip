// softmax_bwd.hip — gradients of softmax attention over prompts. With p_ij = 2^(scale·log2 e·q_i·k_j − lse_i·log2 e) from the
// forward call's lse, and delta_i = do_i·o_i,
//     dv_j = Σ_i p_ij do_i,   ds_ij = p_ij (do_i·v_j − delta_i),   dq_i = scale Σ_j ds_ij k_j,   dk_j = scale Σ_i ds_ij q_i,
// sums over i taken over all heads that share the key head.
//
// Three launches: delta; dk and dv by workgroups of keys that walk the queries; dq by workgroups of queries that walk the
// keys. The scores and do·v are so formed twice (7 products of queries × keys × width instead of 5), and in turn no sum is
// taken by atomics: results do not depend on the order in which workgroups run.
#include "softmax_common.h"

namespace ssm {
namespace sm {
namespace {

constexpr int kStatsLanes = 16;  // lanes to a query's row

// stats[0][h][query] = lse·log2 e, +inf for a query that saw no key (lse = −inf), that is, weights of 0; stats[1][h][query] = −do·o.
template <typename T, bool VEC>
__global__ __launch_bounds__(kSoftmaxThreads) void softmax_stats_kernel(SoftmaxLaunch a, int64_t tokens) {
    const int64_t id = (int64_t)blockIdx.x * (kSoftmaxThreads / kStatsLanes) + threadIdx.x / kStatsLanes;
    const int lane = threadIdx.x % kStatsLanes;
    if (id >= tokens * a.H) return;
    const int64_t t = id / a.H;
    const int h = (int)(id % a.H);
    const int64_t is = a.rows.cu_q ? 0 : t / a.rows.Lq, it = a.rows.cu_q ? t : t % a.rows.Lq;
    const T *dp = static_cast<const T *>(a.dout) + is * a.do_b + it * a.do_t + h * a.do_h;
    const T *op = static_cast<const T *>(a.o_in) + id * a.D;
    float sum = 0.0f;
    if constexpr (VEC) {
        for (int c = lane * kE<T>; c < a.D; c += kStatsLanes * kE<T>) {
            const u4 u = *reinterpret_cast<const u4 *>(dp + c), v = *reinterpret_cast<const u4 *>(op + c);
            T x[kE<T>], y[kE<T>];
            __builtin_memcpy(x, &u, 16);
            __builtin_memcpy(y, &v, 16);
#pragma unroll
            for (int k = 0; k < kE<T>; ++k) sum = __builtin_fmaf(widen(x[k]), widen(y[k]), sum);
        }
    } else {
        for (int c = lane; c < a.D; c += kStatsLanes) sum = __builtin_fmaf(widen(dp[c]), widen(op[c]), sum);
    }
#pragma unroll
    for (int d = 1; d < kStatsLanes; d <<= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) {
        const float lse = a.lse_in[id];
        float *out = a.stats + h * tokens + t;
        out[0] = lse == -INFINITY ? INFINITY : lse * kLog2e;
        out[tokens * a.H] = -sum;
    }
}

// dk and dv: a workgroup takes 32 keys a wavefront of one key head, their keys and values in registers, and walks the queries
// that see them, head by head of the group, in tiles of 32. While a tile's weights are formed and enter their products, so are the
// next tile's scores, and the two after are on their way into LDS.
template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(kSoftmaxThreads, DP * sizeof(T) > 128 ? 1 : 2) void softmax_dkv_kernel(SoftmaxLaunch a,
                                                                                                    SoftmaxWork work,
                                                                                                    int64_t tokens) {
    constexpr int QB = 32, NC = DP / kChunk<T>, ND = DP / 32, BK = 32 * kSoftmaxThreads / 64;
    constexpr int kTileBytes = QB * Tile<T, DP>::kRow, kStats = 2 * QB * 4;
    __shared__ __attribute__((aligned(1024))) char qt[4 * kTileBytes], dt[4 * kTileBytes];
    __shared__ __attribute__((aligned(16))) char stat_t[4 * kStats];  // lse, then −delta, of a tile's queries

    SoftmaxPlace at;
    if (!softmax_place(work, a.G, blockIdx.x, &at)) return;
    const int64_t is = at.seq;
    const int g = at.g, R = a.H / a.G, kb = at.block;  // the first keys, which most queries see, first
    const AttnSeq s = sequence(a.rows, is);
    const bool packed = a.rows.cu_q != nullptr;
    const int w = la::wave_id(), l = threadIdx.x & 63, col = l & 31, half = l >> 5;
    const int k0 = kb * BK, r0 = k0 + 32 * w, key = r0 + col;
    const int to_write = packed ? s.nk : (int)a.rows.Lk;
    if (k0 >= to_write) return;

    Frag<T> k[NC], v[NC];
    {
        const int rows = s.nk - r0 > 32 ? 32 : s.nk - r0;
        const T *kp = static_cast<const T *>(a.k) + is * a.k_b + (s.k0 + r0) * a.k_t + g * a.k_h;
        const T *vp = static_cast<const T *>(a.v) + is * a.v_b + (s.k0 + r0) * a.v_t + g * a.v_h;
        load_frags<T, DP, VEC>(k, la::rows_buffer(kp, (uint32_t)a.k_t, rows, a.D), (uint32_t)a.k_t, col, rows, a.D);
        load_frags<T, DP, VEC>(v, la::rows_buffer(vp, (uint32_t)a.v_t, rows, a.D), (uint32_t)a.v_t, col, rows, a.D);
        if (a.scale < 0.0f) {
#pragma unroll
            for (int c = 0; c < NC; ++c) negate<T>(k[c]);
        }
    }
    const int first = k0 < s.nk ? first_query(s, a.causal, k0) / QB : 0;
    const int tiles = k0 < s.nk ? (s.nq + QB - 1) / QB - first : 0;  // a head
    const float sc = scale_of(a.scale);
    // the lane's key is seen by queries lo .. nq - 1, and all of the wavefront's keys by those from all_lo on
    const int lo = key < s.nk ? first_query(s, a.causal, key) : s.nq;
    const int all_lo = r0 + 32 <= s.nk ? first_query(s, a.causal, r0 + 31) : s.nq;

    f16 dk[ND], dv[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) dk[d] = dv[d] = f16(0.0f);

    // Tiles in order, head by head of the group. Past the last nothing is read.
    const Loader<T, QB, DP, VEC> qs((uint32_t)a.q_t, a.D), ds((uint32_t)a.do_t, a.D);
    const int64_t token = (packed ? s.q0 : is * a.rows.Lq) + first * QB;
    const T *qp = static_cast<const T *>(a.q) + is * a.q_b + (s.q0 + first * QB) * a.q_t + (int64_t)g * R * a.q_h;
    const T *dop = static_cast<const T *>(a.dout) + is * a.do_b + (s.q0 + first * QB) * a.do_t + (int64_t)g * R * a.do_h;
    const float *sp = a.stats + (int64_t)g * R * tokens + token;
    const int64_t q_step = QB * a.q_t, do_step = QB * a.do_t;
    const int64_t q_turn = a.q_h - (tiles - 1) * q_step, do_turn = a.do_h - (tiles - 1) * do_step;
    int left = tiles * R, t = 0;  // tiles still to load; the next one's place among its head's
    const auto fetch = [&](int b) {
        const int rows = left > 0 ? s.nq - (first + t) * QB : 0;
        qs(qp, rows, qt + b * kTileBytes);
        ds(dop, rows, dt + b * kTileBytes);
        load_stats(sp, tokens * a.H, rows, stat_t + b * kStats);
        const bool turn = ++t == tiles;
        qp += turn ? q_turn : q_step;
        dop += turn ? do_turn : do_step;
        sp += turn ? tokens - (tiles - 1) * QB : QB;
        if (turn) t = 0;
        --left;
    };
    // scores, and do·v − delta: the sums start at −delta
    const auto start = [&](f16 &p, f16 &dp, int b) {
        p = f16(0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f4 x = *reinterpret_cast<const f4 *>(stat_t + b * kStats + QB * 4 + (8 * j + 4 * half) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) dp[4 * j + e] = x[e];
        }
    };
    const auto scores = [&](f16 &p, f16 &dp, int b) {
        start(p, dp, b);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            mma(p, row_frag<T, DP>(qt + b * kTileBytes, 0, c), k[c]);
            mma(dp, row_frag<T, DP>(dt + b * kTileBytes, 0, c), v[c]);
        }
    };
    if (tiles > 0) {
        // a fetch's instructions, which may still be on their way when the fetch before has to be there
        constexpr int FETCH = 2 * Loader<T, QB, DP, VEC>::N;
        const auto before_last = [&] {
            if (w == 0) landed_but<FETCH + 2>();
            else landed_but<FETCH>();
        };
        fetch(0);
        fetch(1);
        before_last();
        la::lds_barrier();
        int tile = 0;
        const auto step = [&](auto B, f16 &p, f16 &dp, f16 &next_p, f16 &next_dp) {
            fetch(B + 2 & 3);
            before_last();
            la::lds_barrier();
            const int i0 = (first + tile) * QB;
            tile = tile + 1 == tiles ? 0 : tile + 1;
            if (i0 < all_lo || i0 + QB > s.nq) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int row = i0 + 8 * (i >> 2) + 4 * half + (i & 3);
                    if (row < lo || row >= s.nq) p[i] = -INFINITY;
                }
            }
            // 2·NC products for the next tile's scores, then 2·UNITS with this one's weights, in steps of two: a step reads the
            // fragments of the next but one, and forms a share of the weights.
            constexpr int b = B, ahead = b + 1 & 3;
            constexpr int CH = 32 / kChunk<T>, UNITS = CH * ND, AHEAD = 2;
            const char *qn = qt + ahead * kTileBytes, *dn = dt + ahead * kTileBytes;
            const char *qc = qt + b * kTileBytes, *dc = dt + b * kTileBytes;
            Frag<T> qr[NC], dr[NC], qu[UNITS], du[UNITS], pf[CH], df[CH];
            const auto read = [&](int i) {  // for step i
                if (i < NC) {
                    qr[i] = row_frag<T, DP>(qn, 0, i);
                    dr[i] = row_frag<T, DP>(dn, 0, i);
                } else if (i < NC + UNITS) {
                    const int u = i - NC;
                    du[u] = col_frag<T, DP>(dc, kChunk<T> * (u / ND), 32 * (u % ND));
                    qu[u] = col_frag<T, DP>(qc, kChunk<T> * (u / ND), 32 * (u % ND));
                }
            };
            f4 lse[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) lse[j] = *reinterpret_cast<const f4 *>(stat_t + b * kStats + (8 * j + 4 * half) * 4);
            start(next_p, next_dp, ahead);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) read(i);
            step_end();
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                read(i + AHEAD);
                mma(next_p, qr[i], k[i]);
                mma(next_dp, dr[i], v[i]);
#pragma unroll
                for (int e = 16 * i / NC; e < 16 * (i + 1) / NC; ++e) {
                    p[e] = exp2_fast(__builtin_fmaf(p[e], sc, -lse[e / 4][e % 4]));
                    dp[e] *= p[e];
                }
                if (i == NC - 1) {
                    pf[0] = part_of<T>(p, 0);
                    df[0] = part_of<T>(dp, 0);
                }
                step_end();
            }
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
                const int c = u / ND, d = u % ND;
                read(NC + u + AHEAD);
                mma(dv[d], du[u], pf[c]);
                mma(dk[d], qu[u], df[c]);
                if (d == ND - 1 && c + 1 < CH) {
                    pf[c + 1] = part_of<T>(p, c + 1);
                    df[c + 1] = part_of<T>(dp, c + 1);
                }
                step_end();
            }
        };
        // the buffers in turn, so that their places are constants
        f16 p, dp, next_p, next_dp;
        scores(p, dp, 0);
        for (int n = tiles * R;;) {
            step(std::integral_constant<int, 0>(), p, dp, next_p, next_dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 1>(), next_p, next_dp, p, dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 2>(), p, dp, next_p, next_dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 3>(), next_p, next_dp, p, dp);
            if (--n == 0) break;
        }
        landed_but<0>();
    }

    const int64_t row = (packed ? s.k0 : is * a.rows.Lk) + r0;
    const int rows = to_write - r0 > 32 ? 32 : to_write - r0;
    const uint32_t stride = (uint32_t)(a.G * a.D);
    const Buffer kout = la::rows_buffer(static_cast<T *>(a.dk) + (row * a.G + g) * a.D, stride, rows, a.D);
    const Buffer vout = la::rows_buffer(static_cast<T *>(a.dv) + (row * a.G + g) * a.D, stride, rows, a.D);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        if (key >= s.nk) dk[d] = dv[d] = f16(0.0f);
        store_tile<T, VEC>(kout, stride, col, 32 * d, col < rows ? a.D : 0, dk[d], a.scale);
        store_tile<T, VEC>(vout, stride, col, 32 * d, col < rows ? a.D : 0, dv[d], 1.0f);
    }
}

// dq: a workgroup takes 32 queries a wavefront of one head, with their gradients in registers, and walks the keys that they
// see in tiles of 32, pipelined as above: four LDS buffers for keys, which are read one tile longer, and two for values.
template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(kSoftmaxThreads, sizeof(T) == 4 && DP > 64 ? 1 : 2) void softmax_dq_kernel(SoftmaxLaunch a,
                                                                                                        SoftmaxWork work,
                                                                                                        int64_t tokens) {
    constexpr int KB = 32, NC = DP / kChunk<T>, ND = DP / 32, BQ = 32 * kSoftmaxThreads / 64;
    constexpr int kTileBytes = KB * Tile<T, DP>::kRow;
    __shared__ __attribute__((aligned(1024))) char kt[4 * kTileBytes], vt[2 * kTileBytes];

    SoftmaxPlace at;
    if (!softmax_place(work, a.G, blockIdx.x, &at)) return;
    const int64_t is = at.seq;
    const int g = at.g, h = g * work.per + at.which, qb = work.blocks - 1 - at.block;
    const AttnSeq s = sequence(a.rows, is);
    const bool packed = a.rows.cu_q != nullptr;
    const int w = la::wave_id(), l = threadIdx.x & 63, col = l & 31, half = l >> 5;
    const int q0 = qb * BQ, r0 = q0 + 32 * w;
    const int to_write = packed ? s.nq : (int)a.rows.Lq;
    if (q0 >= to_write) return;

    const T *kp = static_cast<const T *>(a.k) + is * a.k_b + s.k0 * a.k_t + g * a.k_h;
    const T *vp = static_cast<const T *>(a.v) + is * a.v_b + s.k0 * a.v_t + g * a.v_h;
    const int last_q = (q0 + BQ < s.nq ? q0 + BQ : s.nq) - 1;
    const int keys = last_q >= q0 ? last_key(s, a.causal, last_q) + 1 : 0;
    const int tiles = (keys + KB - 1) / KB;
    const int my_last = last_key(s, a.causal, r0 + col);
    const int wave_first = last_key(s, a.causal, r0);
    const int64_t row = (packed ? s.q0 : is * a.rows.Lq) + r0;

    Frag<T> q[NC], dout[NC];
    float lse = 0.0f, less = 0.0f, rest = 0.0f;  // less: −delta; rest: the lane's half of Σ ds
    float *stat = a.stats + h * tokens + row + col;
    {
        const int rows = s.nq - r0 > 32 ? 32 : s.nq - r0;
        const T *qp = static_cast<const T *>(a.q) + is * a.q_b + (s.q0 + r0) * a.q_t + h * a.q_h;
        const T *dp = static_cast<const T *>(a.dout) + is * a.do_b + (s.q0 + r0) * a.do_t + h * a.do_h;
        load_frags<T, DP, VEC>(q, la::rows_buffer(qp, (uint32_t)a.q_t, rows, a.D), (uint32_t)a.q_t, col, rows, a.D);
        load_frags<T, DP, VEC>(dout, la::rows_buffer(dp, (uint32_t)a.do_t, rows, a.D), (uint32_t)a.do_t, col, rows, a.D);
        if (a.scale < 0.0f) {
#pragma unroll
            for (int c = 0; c < NC; ++c) negate<T>(q[c]);
        }
        if (col < rows) {
            lse = stat[0];
            less = stat[tokens * a.H];
        }
    }
    const float sc = scale_of(a.scale);
    f16 dq[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) dq[d] = f16(0.0f);

    const Loader<T, KB, DP, VEC> ks((uint32_t)a.k_t, a.D), vs((uint32_t)a.v_t, a.D);
    const int64_t k_step = KB * a.k_t, v_step = KB * a.v_t;
    int left = s.nk;  // keys from the next tile to load on
    const auto fetch = [&](int b) {
        ks(kp, left, kt + b * kTileBytes);
        vs(vp, left, vt + (b & 1) * kTileBytes);
        kp += k_step;
        vp += v_step;
        left -= KB;
    };
    // scores, and do·v − delta: the sums start at −delta
    const auto scores = [&](f16 &p, f16 &dp, int b) {
        p = f16(0.0f);
        dp = f16(less);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            mma(p, row_frag<T, DP>(kt + b * kTileBytes, 0, c), q[c]);
            mma(dp, row_frag<T, DP>(vt + (b & 1) * kTileBytes, 0, c), dout[c]);
        }
    };
    if (tiles > 0) {
        fetch(0);
        fetch(1);
        landed_but<0>();
        la::lds_barrier();
        int j0 = 0;
        const auto step = [&](auto B, f16 &p, f16 &dp, f16 &next_p, f16 &next_dp) {
            landed_but<0>();
            la::lds_barrier();
            fetch(B + 2 & 3);
            if (j0 + KB - 1 > wave_first) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (j0 + 8 * (i >> 2) + 4 * half + (i & 3) > my_last) p[i] = -INFINITY;
            }
            j0 += KB;
            scores(next_p, next_dp, B + 1 & 3);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                dp[i] *= exp2_fast(__builtin_fmaf(p[i], sc, -lse));
                rest += dp[i];
            }
#pragma unroll
            for (int c = 0; c < 32 / kChunk<T>; ++c) {
                const Split<T> df(dp, c);
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    mma<T>(dq[d], col_frag<T, DP>(kt + B * kTileBytes, kChunk<T> * c, 32 * d), df);
            }
        };
        f16 p, dp, next_p, next_dp;
        scores(p, dp, 0);
        for (int n = tiles;;) {
            step(std::integral_constant<int, 0>(), p, dp, next_p, next_dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 1>(), next_p, next_dp, p, dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 2>(), p, dp, next_p, next_dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 3>(), next_p, next_dp, p, dp);
            if (--n == 0) break;
        }
        landed_but<0>();
    }
    // Σ_j ds_ij is 0 but for the rounding of o, from which delta was formed: what is left corrects delta for dk.
    rest += other_half(rest);
    if (half == 0 && r0 + col < s.nq) stat[tokens * a.H] = less - rest;
    const int rows = to_write - r0 > 32 ? 32 : to_write - r0;
    const uint32_t stride = (uint32_t)(a.H * a.D);
    const Buffer out = la::rows_buffer(static_cast<T *>(a.dq) + (row * a.H + h) * a.D, stride, rows, a.D);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        if (r0 + col >= s.nq) dq[d] = f16(0.0f);
        store_tile<T, VEC>(out, stride, col, 32 * d, col < rows ? a.D : 0, dq[d], a.scale);
    }
}

template <typename T, int DP, bool VEC> hipError_t run(const SoftmaxLaunch &p, hipStream_t stream) {
    const int64_t tokens = p.rows.cu_q ? p.rows.Tq : p.rows.b * p.rows.Lq;
    const SoftmaxWork kw = softmax_dkv_work(p.rows, p.G), qw = softmax_dq_work(p.rows, p.H, p.G);
    constexpr int64_t per = kSoftmaxThreads / kStatsLanes;
    if (tokens > 0) {
        softmax_stats_kernel<T, VEC><<<dim3((unsigned)((tokens * p.H + per - 1) / per)), kSoftmaxThreads, 0, stream>>>(p, tokens);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (qw.blocks > 0) {
        softmax_dq_kernel<T, DP, VEC>
            <<<dim3((unsigned)softmax_groups(qw)), kSoftmaxThreads, 0, stream>>>(p, qw, tokens);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (kw.blocks > 0)
        softmax_dkv_kernel<T, DP, VEC>
            <<<dim3((unsigned)softmax_groups(kw)), kSoftmaxThreads, 0, stream>>>(p, kw, tokens);
    return hipGetLastError();
}
template <typename T> hipError_t by_width(const SoftmaxLaunch &p, hipStream_t stream) {
    if (!p.vec) return p.D <= 64 ? run<T, 64, false>(p, stream) : run<T, 128, false>(p, stream);
    if (p.D <= 32) return run<T, 32, true>(p, stream);
    if (p.D <= 64) return run<T, 64, true>(p, stream);
    if (p.D <= 96) return run<T, 96, true>(p, stream);
    return run<T, 128, true>(p, stream);
}

}  // namespace
}  // namespace sm

hipError_t launch_softmax_bwd(const SoftmaxLaunch &p, hipStream_t stream) {
    return p.bf16 ? sm::by_width<uint16_t>(p, stream) : sm::by_width<float>(p, stream);
}

}  // namespace ssm
