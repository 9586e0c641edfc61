// softmax_bwd.hip — gradients of softmax attention over prompts. With p_ij = 2^(scale·log2 e·q_i·k_j − lse_i·log2 e) from the
// forward call's lse, and delta_i = do_i·o_i,
//     dv_j = Σ_i p_ij do_i,   ds_ij = p_ij (do_i·v_j − delta_i),   dq_i = scale Σ_j ds_ij k_j,   dk_j = scale Σ_i ds_ij q_i,
// sums over i taken over all heads that share the key head.
//
// Launches: with bf16 what do·o lacks as delta, and dq, each by workgroups of queries that walk the keys; dk and dv by workgroups of
// keys that walk the queries. Scores and do·v are so formed twice, with bf16 three times (7 or 9 products of queries × keys × width
// instead of 5), and in turn no sum is taken by atomics: results do not depend on the order in which workgroups run.
//
// Rounding with bf16. ds and p enter products in two parts, 2^-16. do·o is off by what o is rounded, 2^-8 of each of its values, so
// delta is summed over the keys; dq, dk and dv are then their own rounding off, 1.7e-3 of their norm, whatever keys and queries
// have in common.
//
// 130M-like layer (4 rows of 2048, 24 heads of 64, causal): 0.36 to 0.37 ms, 0.35 PFLOP/s counting five products (0.26 with one part
// each and delta from o alone, 0.30 with two parts); 9 packed documents of 463 to 4096 tokens, 32 heads on 8 key heads of 128: 2.10
// to 2.27 ms, 0.40 PFLOP/s (1.54, 1.76): 0.43 for what delta lacks at 44 % of the matrix units' time, 0.70 for dq at 56 %, 1.10 for
// dk and dv at 46 %.
#include "softmax_common.h"

namespace ssm {
namespace sm {
namespace {

// dk and dv: a workgroup takes 128 keys of one key head and walks the queries that see them, head by head of the group, in
// tiles of 32. Two wavefronts share 32 keys: the first forms their scores and weights and adds to dv, the second forms do·v and, from
// the weights that the first left in LDS in the round before, ds, and adds to dk. Each so holds one operand and one sum (one
// wavefront with both of each takes the registers of two: 36 % of the matrix instructions' rate, for want of a second
// wavefront to issue while one waits).
template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(2 * kSoftmaxThreads, DP * sizeof(T) > 128 ? 2 : 4) void softmax_dkv_kernel(SoftmaxLaunch a,
                                                                                                        SoftmaxWork work,
                                                                                                        int64_t tokens) {
    constexpr int QB = 32, NC = DP / kChunk<T>, ND = DP / 32, BK = 32 * kSoftmaxThreads / 64;
    constexpr int kTileBytes = QB * Tile<T, DP>::kRow, kStats = QB * 4, kWeights = 32 * 32 * 4;
    __shared__ __attribute__((aligned(1024))) char qt[4 * kTileBytes], dt[2 * kTileBytes], weights[2][4][kWeights];
    __shared__ __attribute__((aligned(16))) char lse_t[2 * kStats], less_t[2 * kStats];  // lse, −delta of a tile's queries

    SoftmaxPlace at;
    if (!softmax_find(work, a.rows, a.G, blockIdx.x, true, &at)) return;  // the first keys, which most queries see, first
    const int64_t is = at.seq;
    const int g = at.g, R = a.H / a.G, kb = at.block;
    const AttnSeq s = sequence(a.rows, is);
    const bool packed = a.rows.cu_q != nullptr;
    const int w = la::wave_id() & 3, l = threadIdx.x & 63, col = l & 31, half = l >> 5;
    const bool second = la::wave_id() >= 4;
    const int k0 = kb * BK, r0 = k0 + 32 * w, key = r0 + col;
    const int to_write = packed ? s.nk : (int)a.rows.Lk;
    if (k0 >= to_write) return;

    // the wavefront's operand, keys or values
    Frag<T> kv[NC];
    {
        const int rows = s.nk - r0 > 32 ? 32 : s.nk - r0;
        const T *p = second ? static_cast<const T *>(a.v) + is * a.v_b + (s.k0 + r0) * a.v_t + g * a.v_h
                            : static_cast<const T *>(a.k) + is * a.k_b + (s.k0 + r0) * a.k_t + g * a.k_h;
        const uint32_t step = (uint32_t)(second ? a.v_t : a.k_t);
        load_frags<T, DP, VEC>(kv, la::rows_buffer(p, step, rows, a.D), step, col, rows, a.D);
        if (!second) for_scale(kv, a.scale);
    }
    const int first = k0 < s.nk ? first_query(s, a.causal, k0) / QB : 0;
    const int tiles = k0 < s.nk ? (s.nq + QB - 1) / QB - first : 0;  // a head
    // The piece's rounds, a tile each, from tile t0 of head h0 of the group on; the second wavefronts take one more, the first of
    // which only starts.
    int pieces;
    const int per = softmax_piece(work, tiles * R, &pieces), begin = at.piece * per;
    if (at.piece >= pieces) return;
    const int rounds = pieces > 1 && tiles * R - begin > per ? per : tiles * R - begin;
    const int h0 = tiles > 0 ? begin / tiles : 0, t0 = tiles > 0 ? begin % tiles : 0;
    const float sc = scale_of(a.scale);
    // the lane's key is seen by queries lo .. nq - 1, and all of the wavefront's keys by those from all_lo on
    const int lo = key < s.nk ? first_query(s, a.causal, key) : s.nq;
    const int all_lo = r0 + 32 <= s.nk ? first_query(s, a.causal, r0 + 31) : s.nq;

    f16 sum[ND];  // dv, or dk
#pragma unroll
    for (int d = 0; d < ND; ++d) sum[d] = f16(0.0f);

    // Tiles in order, head by head of the group; past the last nothing is read. The first half of the workgroup loads queries, the
    // second their gradients; the first wavefront of each a tile's lse or −delta.
    const Loader<T, QB, DP, VEC> load((uint32_t)(second ? a.do_t : a.q_t), a.D);
    const int64_t token = (packed ? s.q0 : is * a.rows.Lq) + first * QB;
    const int64_t step_t = second ? a.do_t : a.q_t, step_h = second ? a.do_h : a.q_h, batch = second ? a.do_b : a.q_b;
    const T *rp = static_cast<const T *>(second ? a.dout : a.q) + is * batch + (s.q0 + first * QB) * step_t +
                  (int64_t)(g * R + h0) * step_h + t0 * QB * step_t;
    const float *sp = a.stats + (second ? tokens * a.H : 0) + (int64_t)(g * R + h0) * tokens + token + t0 * QB;
    const int64_t tile_step = QB * step_t, turn_step = step_h - (tiles - 1) * tile_step;
    int left = rounds, t = t0, stats_left = rounds, st = t0;  // still to load, and the next one's place among its head's
    const auto fetch_rows = [&](char *tile) {
        load(rp, left > 0 ? s.nq - (first + t) * QB : 0, tile);
        const bool turn = ++t == tiles;
        rp += turn ? turn_step : tile_step;
        if (turn) t = 0;
        --left;
    };
    const auto fetch_stats = [&](char *to) {
        if (w == 0) load_stats(sp, stats_left > 0 ? s.nq - (first + st) * QB : 0, to);
        const bool turn = ++st == tiles;
        sp += turn ? tokens - (tiles - 1) * QB : QB;
        if (turn) st = 0;
        --stats_left;
    };

    // In round n the first wavefronts use tile n's gradients' columns and tile n + 1's queries' rows, the second tile n's gradients'
    // rows and tile n − 1's queries' columns. Queries are loaded two rounds ahead into one of four buffers, the rest one
    // round ahead into one of two.
    if (tiles > 0 && !second) {
        fetch_rows(qt);
        fetch_rows(qt + kTileBytes);
        fetch_stats(lse_t);
        landed();
        la::lds_barrier();
        const auto scores = [&](f16 &p, int b) {
            p = f16(0.0f);
#pragma unroll
            for (int c = 0; c < NC; ++c) mma(p, row_frag<T, DP>(qt + b * kTileBytes, 0, c), kv[c]);
        };
        int tile = t0;
        const auto round = [&](auto B, f16 &p, f16 &next) {
            constexpr int b = B, odd = b & 1;
            landed();
            la::lds_barrier();
            fetch_rows(qt + (b + 2 & 3) * kTileBytes);
            fetch_stats(lse_t + (odd ^ 1) * kStats);
            const int i0 = (first + tile) * QB;
            tile = tile + 1 == tiles ? 0 : tile + 1;
            if (i0 < all_lo || i0 + QB > s.nq) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int row = i0 + 8 * (i >> 2) + 4 * half + (i & 3);
                    if (row < lo || row >= s.nq) p[i] = -INFINITY;
                }
            }
            scores(next, b + 1 & 3);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f4 lse = *reinterpret_cast<const f4 *>(lse_t + odd * kStats + (8 * j + 4 * half) * 4);
                f4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = p[4 * j + e] = exp2_fast(__builtin_fmaf(p[4 * j + e], sc, -lse[e]));
                *reinterpret_cast<f4 *>(weights[odd][w] + (64 * j + l) * 16) = x;
            }
#pragma unroll
            for (int c = 0; c < 32 / kChunk<T>; ++c) {
                const Split<T> pf(p, c);
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    mma<T>(sum[d], col_frag<T, DP>(dt + odd * kTileBytes, kChunk<T> * c, 32 * d), pf);
            }
        };
        f16 p, next;
        scores(p, 0);
        for (int n = rounds;;) {
            round(std::integral_constant<int, 0>(), p, next);
            if (--n == 0) break;
            round(std::integral_constant<int, 1>(), next, p);
            if (--n == 0) break;
            round(std::integral_constant<int, 2>(), p, next);
            if (--n == 0) break;
            round(std::integral_constant<int, 3>(), next, p);
            if (--n == 0) break;
        }
        landed();
        la::lds_barrier();
    } else if (tiles > 0) {
        fetch_rows(dt);
        fetch_stats(less_t);
        landed();
        la::lds_barrier();
        // do·v − delta: the sums start at −delta
        const auto products = [&](f16 &dp, int odd) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f4 x = *reinterpret_cast<const f4 *>(less_t + odd * kStats + (8 * j + 4 * half) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) dp[4 * j + e] = x[e];
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) mma(dp, row_frag<T, DP>(dt + odd * kTileBytes, 0, c), kv[c]);
        };
        const auto open = [&](int odd) {
            landed();
            la::lds_barrier();
            fetch_rows(dt + (odd ^ 1) * kTileBytes);
            fetch_stats(less_t + (odd ^ 1) * kStats);
        };
        const auto round = [&](auto B, f16 &dp, f16 &next) {  // B: of tile n − 1
            constexpr int b = B, odd = b & 1;
            open(odd ^ 1);
            products(next, odd ^ 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f4 x = *reinterpret_cast<const f4 *>(weights[odd][w] + (64 * j + l) * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) dp[4 * j + e] *= x[e];
            }
#pragma unroll
            for (int c = 0; c < 32 / kChunk<T>; ++c) {
                const Split<T> df(dp, c);
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    mma<T>(sum[d], col_frag<T, DP>(qt + b * kTileBytes, kChunk<T> * c, 32 * d), df);
            }
        };
        f16 dp, next;
        open(0);
        products(dp, 0);
        for (int n = rounds;;) {
            round(std::integral_constant<int, 0>(), dp, next);
            if (--n == 0) break;
            round(std::integral_constant<int, 1>(), next, dp);
            if (--n == 0) break;
            round(std::integral_constant<int, 2>(), dp, next);
            if (--n == 0) break;
            round(std::integral_constant<int, 3>(), next, dp);
            if (--n == 0) break;
        }
        landed();
    }

    const int64_t row = (packed ? s.k0 : is * a.rows.Lk) + r0;
    const uint32_t stride = (uint32_t)(a.G * a.D);
    if (pieces > 1) {
        const int64_t tokens_k = packed ? a.rows.Tk : a.rows.b * a.rows.Lk;
        const int rows = s.nk - r0 > 32 ? 32 : s.nk - r0;
        float *to = a.part + (((second ? 0 : work.splits) + at.piece) * tokens_k + row) * a.G * a.D + g * a.D;
        const Buffer out = la::rows_buffer(to, stride, rows, a.D);
#pragma unroll
        for (int d = 0; d < ND; ++d) store_tile<float, VEC>(out, stride, col, 32 * d, col < rows ? a.D : 0, sum[d], 1.0f);
        return;
    }
    const int rows = to_write - r0 > 32 ? 32 : to_write - r0;
    const Buffer out = la::rows_buffer(static_cast<T *>(second ? a.dk : a.dv) + (row * a.G + g) * a.D, stride, rows, a.D);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        if (key >= s.nk) sum[d] = f16(0.0f);
        store_tile<T, VEC>(out, stride, col, 32 * d, col < rows ? a.D : 0, sum[d], second ? a.scale : 1.0f);
    }
}

// The queries of a workgroup, 32 a wavefront, of one head, and the piece of the keys that they see, which it walks in tiles of 32.
struct QueryWalk {
    static constexpr int KB = 32, BQ = 32 * kSoftmaxThreads / 64;
    AttnSeq s;
    int64_t is, row;  // row: of the wavefront's first query among the call's tokens
    int g, h, r0, to_write, piece, pieces, begin, tiles;
    // false: nothing to do
    __device__ __forceinline__ bool set(const SoftmaxLaunch &a, const SoftmaxWork &work) {
        SoftmaxPlace at;
        if (!softmax_find(work, a.rows, a.G, blockIdx.x, false, &at)) return false;
        is = at.seq;
        g = at.g;
        h = g * work.per + at.which;
        s = sequence(a.rows, is);
        const bool packed = a.rows.cu_q != nullptr;
        const int q0 = at.block * BQ;
        r0 = q0 + 32 * la::wave_id();
        to_write = packed ? s.nq : (int)a.rows.Lq;
        if (q0 >= to_write) return false;
        const int last_q = (q0 + BQ < s.nq ? q0 + BQ : s.nq) - 1;
        const int keys = last_q >= q0 ? last_key(s, a.causal, last_q) + 1 : 0;
        const int per = softmax_piece(work, (keys + KB - 1) / KB, &pieces);
        piece = at.piece;
        if (piece >= pieces) return false;
        begin = piece * per * KB;
        tiles = ((pieces > 1 && keys - begin > per * KB ? per * KB : keys - begin) + KB - 1) / KB;
        row = (packed ? s.q0 : is * a.rows.Lq) + r0;
        return true;
    }
    __device__ __forceinline__ int rows() const { return s.nq - r0 > 32 ? 32 : s.nq - r0; }
    // the last key that query r0 + col sees, counted from the piece's first
    __device__ __forceinline__ int last(const SoftmaxLaunch &a, int col) const { return last_key(s, a.causal, r0 + col) - begin; }
    template <typename T> __device__ __forceinline__ const T *keys(const SoftmaxLaunch &a) const {
        return static_cast<const T *>(a.k) + is * a.k_b + (s.k0 + begin) * a.k_t + g * a.k_h;
    }
    template <typename T> __device__ __forceinline__ const T *values(const SoftmaxLaunch &a) const {
        return static_cast<const T *>(a.v) + is * a.v_b + (s.k0 + begin) * a.v_t + g * a.v_h;
    }
};

// The wavefront's queries and their gradients, and of the lane's query lse·log2 e, −do·o and Σ_d |do_d o_d|.
template <typename T, int DP, bool VEC>
__device__ __forceinline__ void load_queries(const SoftmaxLaunch &a, const QueryWalk &x, Frag<T> (&q)[DP / kChunk<T>],
                                             Frag<T> (&dout)[DP / kChunk<T>], float &lse, float &less, float &size) {
    constexpr int NC = DP / kChunk<T>;
    const int col = threadIdx.x & 31, rows = x.rows();
    const T *qp = static_cast<const T *>(a.q) + x.is * a.q_b + (x.s.q0 + x.r0) * a.q_t + x.h * a.q_h;
    const T *dp = static_cast<const T *>(a.dout) + x.is * a.do_b + (x.s.q0 + x.r0) * a.do_t + x.h * a.do_h;
    const uint32_t o_t = (uint32_t)(a.H * a.D);
    Frag<T> o[NC];
    load_frags<T, DP, VEC>(o, la::rows_buffer(static_cast<const T *>(a.o_in) + (x.row * a.H + x.h) * a.D, o_t, rows, a.D), o_t, col,
                           rows, a.D);
    load_frags<T, DP, VEC>(dout, la::rows_buffer(dp, (uint32_t)a.do_t, rows, a.D), (uint32_t)a.do_t, col, rows, a.D);
    load_frags<T, DP, VEC>(q, la::rows_buffer(qp, (uint32_t)a.q_t, rows, a.D), (uint32_t)a.q_t, col, rows, a.D);
    less = size = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < kE<T>; ++e) {
            const float x = (float)dout[c][e], y = (float)o[c][e];
            less = __builtin_fmaf(-x, y, less);
            size = __builtin_fmaf(__builtin_fabsf(x), __builtin_fabsf(y), size);
        }
    less += other_half(less);
    size += other_half(size);
    for_scale(q, a.scale);
    lse = INFINITY;
    if (col < rows) {
        const float given = a.lse_in[(x.row + col) * a.H + x.h];
        // a query that saw no key (lse = −inf): weights of 0
        lse = given == -INFINITY ? INFINITY : given * kLog2e;
    }
}

// What do·o lacks as delta where o is rounded to bf16: rest_i = Σ_j p_ij (do_i·v_j − do_i·o_i) over the keys of each piece. delta's
// error enters dq times Σ_j p_ij k_j: with keys that share an offset of four deviations, dq would be 8e-3 of its norm off. Two
// products are formed once more for it, by rows of tiles alone. Tiles are on their way three rounds ahead: a round of two products is
// shorter than a load takes (packed documents: 0.43 ms; 0.47 one round ahead; 0.50 with 64 queries to a wavefront, which
// halves what is read from LDS, or 256 to a workgroup, which halves what is read from the L2).
template <int DP, bool VEC>
__global__ __launch_bounds__(kSoftmaxThreads, 2) void softmax_rest_kernel(SoftmaxLaunch a, SoftmaxWork work, int64_t tokens) {
    using T = uint16_t;
    constexpr int KB = QueryWalk::KB, NC = DP / kChunk<T>, kTileBytes = KB * Tile<T, DP>::kRow;
    constexpr int kLoads = VEC ? 2 * Loader<T, KB, DP, VEC>::N : 0;  // of a tile of keys and one of values, by a wavefront
    __shared__ __attribute__((aligned(1024))) char kt[4 * kTileBytes], vt[4 * kTileBytes];

    QueryWalk x;
    if (!x.set(a, work)) return;
    const int l = threadIdx.x & 63, col = l & 31, half = l >> 5;
    const int my_last = x.last(a, col), wave_first = x.last(a, 0);
    Frag<T> q[NC], dout[NC];
    float lse, less, size, rest[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    load_queries<T, DP, VEC>(a, x, q, dout, lse, less, size);
    const float sc = scale_of(a.scale);

    const Loader<T, KB, DP, VEC> ks((uint32_t)a.k_t, a.D), vs((uint32_t)a.v_t, a.D);
    const T *kp = x.keys<T>(a), *vp = x.values<T>(a);
    const int64_t k_step = KB * a.k_t, v_step = KB * a.v_t;
    int left = x.s.nk - x.begin;  // keys from the next tile to load on
    const auto fetch = [&](int b) {
        ks(kp, left, kt + b * kTileBytes);
        vs(vp, left, vt + b * kTileBytes);
        kp += k_step;
        vp += v_step;
        left -= KB;
    };
    const auto scores = [&](f16 &p, f16 &dp, int b) {
        p = f16(0.0f);
        dp = f16(less);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            mma(p, row_frag<T, DP>(kt + b * kTileBytes, 0, c), q[c]);
            mma(dp, row_frag<T, DP>(vt + b * kTileBytes, 0, c), dout[c]);
        }
    };
    if (x.tiles > 0) {
#pragma unroll
        for (int b = 0; b < 4; ++b) fetch(b);
        landed<3 * kLoads>();
        la::lds_barrier();
        int j0 = 0;
        // tile n's sum, tile n + 1's scores, and tile n + 4 into the buffer of tile n, which all have read
        const auto step = [&](auto B, f16 &p, f16 &dp, f16 &next_p, f16 &next_dp) {
            landed<2 * kLoads>();
            la::lds_barrier();
            fetch(B);
            if (j0 + KB - 1 > wave_first) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (j0 + 8 * (i >> 2) + 4 * half + (i & 3) > my_last) {
                        p[i] = -INFINITY;
                        dp[i] = 0.0f;  // a NaN or Inf there
                    }
            }
            j0 += KB;
            scores(next_p, next_dp, B + 1 & 3);
#pragma unroll
            for (int i = 0; i < 16; ++i) rest[i & 3] = __builtin_fmaf(dp[i], exp2_fast(__builtin_fmaf(p[i], sc, -lse)), rest[i & 3]);
        };
        f16 p, dp, next_p, next_dp;
        scores(p, dp, 0);
        for (int n = x.tiles;;) {
            step(std::integral_constant<int, 0>(), p, dp, next_p, next_dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 1>(), next_p, next_dp, p, dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 2>(), p, dp, next_p, next_dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 3>(), next_p, next_dp, p, dp);
            if (--n == 0) break;
        }
        landed();
    }
    float sum = (rest[0] + rest[1]) + (rest[2] + rest[3]);
    sum += other_half(sum);
    if (half == 0 && col < x.rows()) a.rest[(x.piece * a.H + x.h) * tokens + x.row + col] = sum;
}

// dq: a workgroup takes 32 queries a wavefront of one head, with their gradients in registers, and walks the keys that they
// see in tiles of 32, pipelined as above: four LDS buffers for keys, which are read one tile longer, and two for values.
template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(kSoftmaxThreads, sizeof(T) == 4 && DP > 64 ? 1 : 2) void softmax_dq_kernel(SoftmaxLaunch a,
                                                                                                        SoftmaxWork work,
                                                                                                        int64_t tokens) {
    constexpr int KB = QueryWalk::KB, NC = DP / kChunk<T>, ND = DP / 32;
    constexpr int kTileBytes = KB * Tile<T, DP>::kRow;
    __shared__ __attribute__((aligned(1024))) char kt[4 * kTileBytes], vt[2 * kTileBytes];

    QueryWalk x;
    if (!x.set(a, work)) return;
    const int l = threadIdx.x & 63, col = l & 31, half = l >> 5;
    const int my_last = x.last(a, col), wave_first = x.last(a, 0);

    Frag<T> q[NC], dout[NC];
    float lse, less, size;  // less: −delta
    load_queries<T, DP, VEC>(a, x, q, dout, lse, less, size);
    if (col < x.rows()) {
        const int64_t at = x.h * tokens + x.row + col;
        if constexpr (sizeof(T) == 2) {
            float rest = 0.0f;
            for (int i = 0; i < x.pieces; ++i) rest += a.rest[i * a.H * tokens + at];
            // more than twice the rounding of o: o and lse are of more keys than these, whose part of delta is not here
            if (__builtin_fabsf(rest) <= 0x1p-7f * size) less -= rest;
        }
        if (half == 0 && x.piece == 0) {
            a.stats[at] = lse;
            a.stats[a.H * tokens + at] = less;
        }
    }
    const float sc = scale_of(a.scale);
    f16 dq[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) dq[d] = f16(0.0f);

    const Loader<T, KB, DP, VEC> ks((uint32_t)a.k_t, a.D), vs((uint32_t)a.v_t, a.D);
    const T *kp = x.keys<T>(a), *vp = x.values<T>(a);
    const int64_t k_step = KB * a.k_t, v_step = KB * a.v_t;
    int left = x.s.nk - x.begin;  // keys from the next tile to load on
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
    if (x.tiles > 0) {
        fetch(0);
        fetch(1);
        landed();
        la::lds_barrier();
        int j0 = 0;
        const auto step = [&](auto B, f16 &p, f16 &dp, f16 &next_p, f16 &next_dp) {
            landed();
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
            for (int i = 0; i < 16; ++i) dp[i] *= exp2_fast(__builtin_fmaf(p[i], sc, -lse));
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
        for (int n = x.tiles;;) {
            step(std::integral_constant<int, 0>(), p, dp, next_p, next_dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 1>(), next_p, next_dp, p, dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 2>(), p, dp, next_p, next_dp);
            if (--n == 0) break;
            step(std::integral_constant<int, 3>(), next_p, next_dp, p, dp);
            if (--n == 0) break;
        }
        landed();
    }
    const uint32_t stride = (uint32_t)(a.H * a.D);
    if (x.pieces > 1) {
        const int rows = x.rows();
        const Buffer out = la::rows_buffer(a.part + ((x.piece * tokens + x.row) * a.H + x.h) * a.D, stride, rows, a.D);
#pragma unroll
        for (int d = 0; d < ND; ++d) store_tile<float, VEC>(out, stride, col, 32 * d, col < rows ? a.D : 0, dq[d], 1.0f);
        return;
    }
    const int rows = x.to_write - x.r0 > 32 ? 32 : x.to_write - x.r0;
    const Buffer out = la::rows_buffer(static_cast<T *>(a.dq) + (x.row * a.H + x.h) * a.D, stride, rows, a.D);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        if (x.r0 + col >= x.s.nq) dq[d] = f16(0.0f);
        store_tile<T, VEC>(out, stride, col, 32 * d, col < rows ? a.D : 0, dq[d], a.scale);
    }
}

// Sums of pieces, in their order: of a block of queries' dq, or of a block of keys' dk and dv.
template <typename T, bool KEYS>
__global__ __launch_bounds__(kSoftmaxThreads) void softmax_bwd_join_kernel(SoftmaxLaunch a, SoftmaxWork work, SoftmaxWork join) {
    SoftmaxPlace at;
    if (!softmax_find(join, a.rows, a.G, blockIdx.x, KEYS, &at)) return;
    const AttnSeq s = sequence(a.rows, at.seq);
    const bool packed = a.rows.cu_q != nullptr;
    const int n = KEYS ? s.nk : s.nq, first = at.block * kSoftmaxBlock;
    const int rows = n - first > kSoftmaxBlock ? kSoftmaxBlock : n - first;
    if (rows <= 0) return;  // one piece
    const int tiles = KEYS ? ((s.nq + 31) / 32 - first_query(s, a.causal, first) / 32) * (a.H / a.G)
                           : (last_key(s, a.causal, first + rows - 1) + 32) / 32;
    int pieces;
    softmax_piece(work, tiles, &pieces);
    if (pieces < 2) return;
    const int64_t L = KEYS ? a.rows.Lk : a.rows.Lq, tokens = packed ? (KEYS ? a.rows.Tk : a.rows.Tq) : a.rows.b * L;
    const int l = threadIdx.x & 31, r = at.piece * 8 + (int)threadIdx.x / 32;
    // rows past the sequence's (a padded batch) are 0
    if (first + r >= (packed ? n : L)) return;
    const int m = r < rows ? pieces : 0;
    const int64_t row = (packed ? (KEYS ? s.k0 : s.q0) : at.seq * L) + first + r;
    const int heads = KEYS ? a.G : a.H, h = KEYS ? at.g : at.g * work.per + at.which;
    const int64_t apart = tokens * heads * a.D, to = (row * heads + h) * a.D;  // apart: floats of a piece
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f}, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < m; ++i) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int d = l + 32 * u;
            if (d >= a.D) continue;
            x[u] += a.part[i * apart + to + d];
            if (KEYS) y[u] += a.part[(work.splits + i) * apart + to + d];
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int d = l + 32 * u;
        if (d >= a.D) continue;
        static_cast<T *>(KEYS ? a.dk : a.dq)[to + d] = narrow<T>(x[u] * a.scale);
        if (KEYS) static_cast<T *>(a.dv)[to + d] = narrow<T>(y[u]);
    }
}

template <typename T, int DP, bool VEC> hipError_t run(const SoftmaxLaunch &p, hipStream_t stream) {
    const int64_t tokens = p.rows.cu_q ? p.rows.Tq : p.rows.b * p.rows.Lq;
    const SoftmaxWork kw = softmax_dkv_work(p.rows, p.H, p.G), qw = softmax_dq_work(p.rows, p.H, p.G);
    hipError_t e = hipSuccess;
    if (qw.blocks > 0) {
        const dim3 grid((unsigned)softmax_groups(qw));
        if constexpr (sizeof(T) == 2) {
            softmax_rest_kernel<DP, VEC><<<grid, kSoftmaxThreads, 0, stream>>>(p, qw, tokens);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        softmax_dq_kernel<T, DP, VEC><<<grid, kSoftmaxThreads, 0, stream>>>(p, qw, tokens);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (qw.splits > 1) {
            const SoftmaxWork j = softmax_join_work(qw);
            softmax_bwd_join_kernel<T, false><<<dim3((unsigned)softmax_groups(j)), kSoftmaxThreads, 0, stream>>>(p, qw, j);
        }
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (kw.blocks > 0) {
        const dim3 grid((unsigned)softmax_groups(kw));
        softmax_dkv_kernel<T, DP, VEC><<<grid, 2 * kSoftmaxThreads, 0, stream>>>(p, kw, tokens);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (kw.splits > 1) {
            const SoftmaxWork j = softmax_join_work(kw);
            softmax_bwd_join_kernel<T, true><<<dim3((unsigned)softmax_groups(j)), kSoftmaxThreads, 0, stream>>>(p, kw, j);
        }
        e = hipGetLastError();
    }
    return e;
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
