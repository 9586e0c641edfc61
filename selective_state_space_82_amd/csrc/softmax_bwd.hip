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

// Tiles of 32 keys that a wavefront takes.
template <typename T, int DP> constexpr int kKeyTiles = sizeof(T) == 2 ? 1 : 1;
constexpr int kStatsLanes = 16;  // lanes to a query's row

// stats[h][query] = {lse·log2 e, do·o}; a query that saw no key (lse = −inf) gets +inf, that is, weights of 0.
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
        float *out = a.stats + 2 * (h * tokens + t);
        out[0] = lse == -INFINITY ? INFINITY : lse * kLog2e;
        out[1] = sum;
    }
}

// dk and dv: a workgroup takes KT·32 keys a wavefront of one key head, their keys and values in registers, and walks the queries
// that see them, head by head of the group, in tiles of 32.
template <typename T, int DP, int KT, bool VEC>
__global__ __launch_bounds__(kSoftmaxThreads, 2) void softmax_dkv_kernel(SoftmaxLaunch a, SoftmaxWork work, int64_t tokens) {
    constexpr int QB = 32, NC = DP / kChunk<T>, ND = DP / 32, KW = 32 * KT, BK = KW * kSoftmaxThreads / 64;
    __shared__ __attribute__((aligned(1024))) char qt[2][QB * Tile<T, DP>::kRow], dt[2][QB * Tile<T, DP>::kRow];
    __shared__ __attribute__((aligned(16))) float lse_t[2][QB], delta_t[2][QB];

    SoftmaxPlace at;
    if (!softmax_place(work, a.G, blockIdx.x, &at)) return;
    const int64_t is = at.seq;
    const int g = at.g, R = a.H / a.G, kb = at.block;  // the first keys, which most queries see, first
    const AttnSeq s = sequence(a.rows, is);
    const bool packed = a.rows.cu_q != nullptr;
    const int w = la::wave_id(), l = threadIdx.x & 63, col = l & 31, half = l >> 5;
    const int k0 = kb * BK, r0 = k0 + KW * w;
    const int to_write = packed ? s.nk : (int)a.rows.Lk;
    if (k0 >= to_write) return;

    Frag<T> k[KT][NC], v[KT][NC];
#pragma unroll
    for (int u = 0; u < KT; ++u) {
        const int r = r0 + 32 * u, rows = s.nk - r > 32 ? 32 : s.nk - r;
        const T *kp = static_cast<const T *>(a.k) + is * a.k_b + (s.k0 + r) * a.k_t + g * a.k_h;
        const T *vp = static_cast<const T *>(a.v) + is * a.v_b + (s.k0 + r) * a.v_t + g * a.v_h;
        load_frags<T, DP, VEC>(k[u], la::rows_buffer(kp, (uint32_t)a.k_t, rows, a.D), (uint32_t)a.k_t, col, rows, a.D);
        load_frags<T, DP, VEC>(v[u], la::rows_buffer(vp, (uint32_t)a.v_t, rows, a.D), (uint32_t)a.v_t, col, rows, a.D);
    }
    const int first = k0 < s.nk ? first_query(s, a.causal, k0) / QB : 0;
    const int tiles = k0 < s.nk ? (s.nq + QB - 1) / QB - first : 0;  // a head
    const int off = s.nk - s.nq;
    const float sc = a.scale * kLog2e;

    f16 dk[KT][ND], dv[KT][ND];
#pragma unroll
    for (int u = 0; u < KT; ++u)
#pragma unroll
        for (int d = 0; d < ND; ++d) dk[u][d] = dv[u][d] = f16(0.0f);

    const Loader<T, QB, DP, VEC> qs((uint32_t)a.q_t, a.D), ds((uint32_t)a.do_t, a.D);
    const auto fetch = [&](int r, int tile, int b) {
        const int h = g * R + r, i0 = (first + tile) * QB;
        if (threadIdx.x < QB) {
            const int i = i0 + (int)threadIdx.x;
            const int64_t t = (packed ? s.q0 : is * a.rows.Lq) + i;
            const float *p = a.stats + 2 * (h * tokens + t);
            lse_t[b][threadIdx.x] = i < s.nq ? p[0] : 0.0f;
            delta_t[b][threadIdx.x] = i < s.nq ? p[1] : 0.0f;
        }
        qs(static_cast<const T *>(a.q) + is * a.q_b + (s.q0 + i0) * a.q_t + h * a.q_h, s.nq - i0, qt[b]);
        ds(static_cast<const T *>(a.dout) + is * a.do_b + (s.q0 + i0) * a.do_t + h * a.do_h, s.nq - i0, dt[b]);
    };
    int r = 0, tile = 0;
    if (tiles > 0) fetch(0, 0, 0);
    for (int n = 0; n < tiles * R; ++n) {
        const int i0 = (first + tile) * QB, b = n & 1;
        landed();
        la::lds_barrier();
        if (++tile == tiles) {
            tile = 0;
            ++r;
        }
        if (r < R) fetch(r, tile, b ^ 1);
        if (r0 >= s.nk || (a.causal && r0 > i0 + QB - 1 + off)) continue;
        f16 p[KT], dp[KT];
#pragma unroll
        for (int u = 0; u < KT; ++u) p[u] = dp[u] = f16(0.0f);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Frag<T> qf = row_frag<T, DP>(qt[b], 0, c), df = row_frag<T, DP>(dt[b], 0, c);
#pragma unroll
            for (int u = 0; u < KT; ++u) {
                mma(p[u], qf, k[u][c]);
                mma(dp[u], df, v[u][c]);
            }
        }
        const bool masked = i0 + QB > s.nq || r0 + KW > s.nk || (a.causal && r0 + KW - 1 > i0 + off);
#pragma unroll
        for (int u = 0; u < KT; ++u) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f4 lse = *reinterpret_cast<const f4 *>(&lse_t[b][8 * j + 4 * half]);
                const f4 delta = *reinterpret_cast<const f4 *>(&delta_t[b][8 * j + 4 * half]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[u][4 * j + e] = exp2_fast(__builtin_fmaf(p[u][4 * j + e], sc, -lse[e]));
                    dp[u][4 * j + e] = p[u][4 * j + e] * (dp[u][4 * j + e] - delta[e]);
                }
            }
            if (masked) {
                const int key = r0 + 32 * u + col;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int row = i0 + 8 * (i >> 2) + 4 * half + (i & 3);
                    if (row >= s.nq || key >= s.nk || (a.causal && key > row + off)) p[u][i] = dp[u][i] = 0.0f;
                }
            }
        }
#pragma unroll
        for (int c = 0; c < 32 / kChunk<T>; ++c) {
            Frag<T> pf[KT];
            Split<T> df[KT];
#pragma unroll
            for (int u = 0; u < KT; ++u) {
                pf[u] = part_of<T>(p[u], c);
                df[u] = Split<T>(dp[u], c);
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const Frag<T> of = col_frag<T, DP>(dt[b], kChunk<T> * c, 32 * d), qf = col_frag<T, DP>(qt[b], kChunk<T> * c, 32 * d);
#pragma unroll
                for (int u = 0; u < KT; ++u) {
                    mma(dv[u][d], of, pf[u]);
                    mma<T>(dk[u][d], qf, df[u]);
                }
            }
        }
    }

    const int64_t row = (packed ? s.k0 : is * a.rows.Lk) + r0;
    const uint32_t stride = (uint32_t)(a.G * a.D);
#pragma unroll
    for (int u = 0; u < KT; ++u) {
        const int r = r0 + 32 * u, rows = to_write - r > 32 ? 32 : to_write - r;
        const int64_t first_out = ((row + 32 * u) * a.G + g) * a.D;
        const Buffer kout = la::rows_buffer(static_cast<T *>(a.dk) + first_out, stride, rows, a.D);
        const Buffer vout = la::rows_buffer(static_cast<T *>(a.dv) + first_out, stride, rows, a.D);
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            if (r + col >= s.nk) dk[u][d] = dv[u][d] = f16(0.0f);
            store_tile<T, VEC>(kout, stride, col, 32 * d, col < rows ? a.D : 0, dk[u][d], a.scale);
            store_tile<T, VEC>(vout, stride, col, 32 * d, col < rows ? a.D : 0, dv[u][d], 1.0f);
        }
    }
}

// dq: a workgroup takes 32 queries a wavefront of one head, with their gradients in registers, and walks the keys that they
// see in tiles of 32.
template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(kSoftmaxThreads, 2) void softmax_dq_kernel(SoftmaxLaunch a, SoftmaxWork work, int64_t tokens) {
    constexpr int KB = 32, NC = DP / kChunk<T>, ND = DP / 32, BQ = 32 * kSoftmaxThreads / 64;
    __shared__ __attribute__((aligned(1024))) char kt[2][KB * Tile<T, DP>::kRow], vt[2][KB * Tile<T, DP>::kRow];

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
    const int wave_last = r0 < s.nq ? last_key(s, a.causal, (r0 + 32 < s.nq ? r0 + 32 : s.nq) - 1) : -1;
    const int64_t row = (packed ? s.q0 : is * a.rows.Lq) + r0;

    Frag<T> q[NC], dout[NC];
    float lse = 0.0f, delta = 0.0f;
    {
        const int rows = s.nq - r0 > 32 ? 32 : s.nq - r0;
        const T *qp = static_cast<const T *>(a.q) + is * a.q_b + (s.q0 + r0) * a.q_t + h * a.q_h;
        const T *dp = static_cast<const T *>(a.dout) + is * a.do_b + (s.q0 + r0) * a.do_t + h * a.do_h;
        load_frags<T, DP, VEC>(q, la::rows_buffer(qp, (uint32_t)a.q_t, rows, a.D), (uint32_t)a.q_t, col, rows, a.D);
        load_frags<T, DP, VEC>(dout, la::rows_buffer(dp, (uint32_t)a.do_t, rows, a.D), (uint32_t)a.do_t, col, rows, a.D);
        if (col < rows) {
            const float *p = a.stats + 2 * (h * tokens + row + col);
            lse = p[0];
            delta = p[1];
        }
    }
    const float sc = a.scale * kLog2e;
    f16 dq[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) dq[d] = f16(0.0f);

    const Loader<T, KB, DP, VEC> ks((uint32_t)a.k_t, a.D), vs((uint32_t)a.v_t, a.D);
    if (tiles > 0) {
        ks(kp, s.nk, kt[0]);
        vs(vp, s.nk, vt[0]);
    }
    for (int j = 0; j < tiles; ++j) {
        const int j0 = j * KB, b = j & 1;
        landed();
        la::lds_barrier();
        if (j + 1 < tiles) {
            ks(kp + (int64_t)(j0 + KB) * a.k_t, s.nk - j0 - KB, kt[b ^ 1]);
            vs(vp + (int64_t)(j0 + KB) * a.v_t, s.nk - j0 - KB, vt[b ^ 1]);
        }
        if (j0 <= wave_last) {
            f16 p = f16(0.0f), dp = f16(0.0f);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                mma(p, row_frag<T, DP>(kt[b], 0, c), q[c]);
                mma(dp, row_frag<T, DP>(vt[b], 0, c), dout[c]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                dp[i] = exp2_fast(__builtin_fmaf(p[i], sc, -lse)) * (dp[i] - delta);
            if (j0 + KB - 1 > wave_first) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (j0 + 8 * (i >> 2) + 4 * half + (i & 3) > my_last) dp[i] = 0.0f;
            }
#pragma unroll
            for (int c = 0; c < 32 / kChunk<T>; ++c) {
                const Split<T> df(dp, c);
#pragma unroll
                for (int d = 0; d < ND; ++d) mma<T>(dq[d], col_frag<T, DP>(kt[b], kChunk<T> * c, 32 * d), df);
            }
        }
    }
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
    if (kw.blocks > 0) {
        softmax_dkv_kernel<T, DP, kKeyTiles<T, DP>, VEC>
            <<<dim3((unsigned)softmax_groups(kw)), kSoftmaxThreads, 0, stream>>>(p, kw, tokens);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (qw.blocks > 0)
        softmax_dq_kernel<T, DP, VEC>
            <<<dim3((unsigned)softmax_groups(qw)), kSoftmaxThreads, 0, stream>>>(p, qw, tokens);
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
