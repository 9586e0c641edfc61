// softmax_fwd.hip — softmax attention over prompts: o_i = Σ_j p_ij v_j, p = softmax_j(scale·q_i·k_j) over the keys that query i
// sees, with lse_i = log Σ_j e^(scale·q_i·k_j).
//
// One pass over the keys with the running maximum and sum of the softmax. A workgroup takes 32 queries a wavefront of one
// head and walks the keys that its queries see in tiles of 64 (fp32: 32), which go from memory straight into one of two LDS
// buffers each for keys and values while the tile before is computed. Scores and weights stay in registers (softmax_common.h).
//
// With bf16 a weight enters its product with the values in two parts, its value rounded and what that leaves, rounded: 2^-16. One part
// alone (2^-8 of every weight, each on its own) is two thirds of the result's own rounding, of 1.6e-3 of its norm: 2.06e-3 in all.
//
// What carries it: the next tile's scores are formed in the same stretch of code, without branches, as this tile's weights and
// products, so that matrix and vector instructions of one wavefront overlap; tiles that every query sees whole take no mask; the
// maximum is raised only where it has to be. 1.4B-like layer (8 rows of 4096, 32 heads on 8 key heads of 128, bf16, causal):
// 1.42 to 1.51 ms from card to card; one row of 16384, 16 heads of 128: 1.34 to 1.43 ms: three products of 0.55 TFLOP for two, 1.09 to
// 1.16 and 1.15 to 1.23 PFLOP/s of matrix instructions, where library products of 8192³ and 16384³ run at 1.14 to 1.33: the matrix
// units are busy 63 and 68 % of the time at the 1.7 GHz that the card holds then. Weights in one part take 1.11 and 1.03 ms.
// Steps measured on the way with one part (1.4B-like, ms): tiles through registers 5.59; straight into LDS without bank
// conflicts 1.46; key heads kept to an XCD 1.43; scores ahead 1.29; no masks and no path for NaN in the loop over whole
// tiles 1.10.
#include "softmax_common.h"

namespace ssm {
namespace sm {
namespace {

// Keys of a tile.
template <typename T> constexpr int kKeys = sizeof(T) == 2 ? 64 : 32;
// A running maximum is raised, and what was summed rescaled, once a score passes it by 2^8: weights are at most 2^8 then,
// and nothing else changes, for fp32 and bf16 keep their relative precision there.
constexpr float kSlack = 8.0f;

template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(kSoftmaxThreads, 2) void softmax_fwd_kernel(SoftmaxLaunch a, SoftmaxWork work) {
    constexpr int KB = kKeys<T>, NT = KB / 32, NC = DP / kChunk<T>, ND = DP / 32, BQ = 32 * kSoftmaxThreads / 64;
    constexpr int kTileBytes = KB * Tile<T, DP>::kRow;
    __shared__ __attribute__((aligned(1024))) char kt[2][kTileBytes], vt[2][kTileBytes];
    __shared__ int found;  // a NaN or Inf among the values of a tile that not every query sees whole

    SoftmaxPlace at;
    if (!softmax_find(work, a.rows, a.G, blockIdx.x, false, &at)) return;  // the last queries, which see most, first
    const int64_t is = at.seq;
    const int g = at.g, h = g * work.per + at.which, qb = at.block;
    const AttnSeq s = sequence(a.rows, is);
    const bool packed = a.rows.cu_q != nullptr;
    const int w = la::wave_id(), l = threadIdx.x & 63, col = l & 31, half = l >> 5;
    const int q0 = qb * BQ, r0 = q0 + 32 * w;
    const int to_write = packed ? s.nq : (int)a.rows.Lq;
    if (q0 >= to_write) return;

    const T *qp = static_cast<const T *>(a.q) + is * a.q_b + s.q0 * a.q_t + h * a.q_h + (int64_t)r0 * a.q_t;
    const T *kp = static_cast<const T *>(a.k) + is * a.k_b + s.k0 * a.k_t + g * a.k_h;
    const T *vp = static_cast<const T *>(a.v) + is * a.v_b + s.k0 * a.v_t + g * a.v_h;

    // tiles up to the last key that the block's last query sees; of the first `full` every query sees every key
    const int last_q = (q0 + BQ < s.nq ? q0 + BQ : s.nq) - 1;
    const int keys = last_q >= q0 ? last_key(s, a.causal, last_q) + 1 : 0;
    int pieces;
    const int per = softmax_piece(work, (keys + KB - 1) / KB, &pieces);
    if (at.piece >= pieces) return;
    // all counted from the piece's first key
    const int begin = at.piece * per * KB, n_keys = pieces > 1 && keys - begin > per * KB ? per * KB : keys - begin;
    const int tiles = (n_keys + KB - 1) / KB;
    int full = keys > 0 ? (last_key(s, a.causal, q0) + 1 - begin) / KB : 0;
    full = full < 0 ? 0 : full > tiles ? tiles : full;
    const int my_last = last_key(s, a.causal, r0 + col) - begin;  // of the lane's query
    const int wave_last = r0 < s.nq ? last_key(s, a.causal, (r0 + 32 < s.nq ? r0 + 32 : s.nq) - 1) - begin : -1;
    const int there = s.nk - begin;
    kp += begin * a.k_t;
    vp += begin * a.v_t;

    Frag<T> q[NC];
    {
        const int rows = s.nq - r0;
        load_frags<T, DP, VEC>(q, la::rows_buffer(qp, (uint32_t)a.q_t, rows > 32 ? 32 : rows, a.D), (uint32_t)a.q_t, col,
                               rows > 32 ? 32 : rows, a.D);
        for_scale(q, a.scale);
    }
    const float sc = scale_of(a.scale);

    f16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f16(0.0f);
    float m = -INFINITY, sum = 0.0f;  // sum: over the lane's half of the keys

    const Loader<T, KB, DP, VEC> ks((uint32_t)a.k_t, a.D), vs((uint32_t)a.v_t, a.D);
    // Past the last tile nothing is read: the buffer has no rows then, and zeros land in a place that nobody looks at.
    const auto load_k = [&](int j, int b) { ks(kp + (int64_t)j * KB * a.k_t, there - j * KB, kt[b]); };
    const auto load_v = [&](int j, int b) { vs(vp + (int64_t)j * KB * a.v_t, there - j * KB, vt[b]); };
    const auto scores = [&](f16(&p)[NT], int b) {
#pragma unroll
        for (int t = 0; t < NT; ++t) p[t] = f16(0.0f);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int t = 0; t < NT; ++t) mma(p[t], row_frag<T, DP>(kt[b], 32 * t, c), q[c]);
    };
    // Hides the keys of tile j that a query does not see, and, if `now`, raises the maximum where tile j's scores ask for it.
    const auto prepare = [&](f16(&p)[NT], int j, bool now, auto masked) {
        if constexpr (masked) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (j * KB + 32 * t + 8 * (i >> 2) + 4 * half + (i & 3) > my_last) p[t][i] = -INFINITY;
        }
        float top = p[0][0];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, p[t][i]);
        top = __builtin_fmaxf(top, other_half(top)) * sc;
        const bool raise = now && top > m + kSlack;  // each query by itself: its bits are its own
        if (__any(raise)) {
            const float f = raise ? exp2_fast(m - top) : 1.0f;
            m = raise ? top : m;
            sum *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] *= f;
        }
    };
    const auto weigh = [&](f16(&p)[NT]) {
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[t][i] = exp2_fast(__builtin_fmaf(p[t][i], sc, -base));
                sum += p[t][i];
            }
    };
    // Adds what tile j's scores p say, with its values in buffer b, and forms tile j + 1's scores meanwhile.
    const auto step = [&](int j, int b, f16(&p)[NT], f16(&next)[NT], auto masked) {
        landed();
        la::lds_barrier();
        load_k(j + 2, b);
        load_v(j + 1, b ^ 1);
        const char *vb = vt[b];
        if constexpr (masked) {
            if (share_not_finite<T, KB, DP>(vb)) found = 1;
            if (j * KB > wave_last) return;
        }
        scores(next, b ^ 1);
        weigh(p);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < 32 / kChunk<T>; ++c) {
                const Split<T> pf(p[t], c);
#pragma unroll
                for (int d = 0; d < ND; ++d) mma<T>(o[d], col_frag<T, DP>(vb, 32 * t + kChunk<T> * c, 32 * d), pf);
            }
    };
    if (threadIdx.x == 0) found = 0;
    if (tiles > 0) {
        load_k(0, 0);
        load_v(0, 0);
        load_k(1, 1);
        landed();
        la::lds_barrier();
        f16 p[NT], next[NT];
        scores(p, 0);
        int j = 0;
        prepare(p, 0, full > 1, std::false_type());
        for (; j + 1 < full; j += 2) {
            step(j, 0, p, next, std::false_type());
            prepare(next, j + 1, true, std::false_type());
            step(j + 1, 1, next, p, std::false_type());
            prepare(p, j + 2, j + 3 < full, std::false_type());  // the tiles from there on are prepared with their masks
        }
        for (; j < tiles; ++j) {
            prepare(p, j, true, std::true_type());
            step(j, j & 1, p, next, std::true_type());
#pragma unroll
            for (int t = 0; t < NT; ++t) p[t] = next[t];
        }
        landed();  // the loads past the last tile, before LDS is written again or given up
        la::lds_barrier();
    }
    // A masked key's weight is 0, but 0 times a NaN or Inf is not. Where there is one the block is done again, one tile after
    // the other, so that such values count as 0 in the product and make the result NaN for the queries that do see them.
    if (tiles > 0 && found) {
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] = f16(0.0f);
        m = -INFINITY;
        sum = 0.0f;
        for (int j = 0; j < tiles; ++j) {
            la::lds_barrier();
            load_k(j, 0);
            load_v(j, 0);
            landed();
            la::lds_barrier();
            f16 p[NT];
            scores(p, 0);
            prepare(p, j, true, std::true_type());
            weigh(p);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                f16 seen = f16(0.0f);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int c = 0; c < 32 / kChunk<T>; ++c) {
                        Frag<T> v = col_frag<T, DP>(vt[0], 32 * t + kChunk<T> * c, 32 * d), bad, see;
#pragma unroll
                        for (int e = 0; e < kE<T>; ++e) {
                            const int i = kE<T> * c + e;
                            const bool nf = !__builtin_isfinite((float)v[e]);
                            bad[e] = nf ? 1.0f : 0.0f;
                            if (nf) v[e] = 0.0f;
                            see[e] = j * KB + 32 * t + 8 * (i >> 2) + 4 * half + (i & 3) > my_last ? 0.0f : 1.0f;
                        }
                        mma<T>(o[d], v, Split<T>(p[t], c));
                        mma(seen, bad, see);
                    }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (seen[i] > 0.0f) o[d][i] = NAN;
            }
        }
    }
    sum += other_half(sum);

    const int64_t row = (packed ? s.q0 : is * a.rows.Lq) + r0;
    if (pieces > 1) {
        const int64_t tokens = packed ? a.rows.Tq : a.rows.b * a.rows.Lq;
        const int64_t first = (at.piece * tokens + row) * a.H + h;
        const int rows = s.nq - r0 > 32 ? 32 : s.nq - r0;
        const Buffer out = la::rows_buffer(a.part + first * a.D, (uint32_t)(a.H * a.D), rows, a.D);
#pragma unroll
        for (int d = 0; d < ND; ++d)
            store_tile<float, VEC>(out, (uint32_t)(a.H * a.D), col, 32 * d, col < rows ? a.D : 0, o[d], 1.0f);
        if (half == 0 && col < rows) {
            float *ms = a.part + work.splits * tokens * a.H * a.D + 2 * (first + (int64_t)col * a.H);
            ms[0] = m;
            ms[1] = sum;
        }
        return;
    }
    // rows past the sequence's queries (a padded batch): no keys, 0 and -inf
    const bool live = r0 + col < s.nq && !(sum == 0.0f);
    const float f = live ? 1.0f / sum : 0.0f;
    int rows = to_write - r0;
    rows = rows > 32 ? 32 : rows;
    const uint32_t stride = (uint32_t)(a.H * a.D);
    const Buffer out = la::rows_buffer(static_cast<T *>(a.o) + (row * a.H + h) * a.D, stride, rows, a.D);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        if (!live) o[d] = f16(0.0f);
        store_tile<T, VEC>(out, stride, col, 32 * d, col < rows ? a.D : 0, o[d], f);
    }
    if (a.lse && half == 0 && col < rows)
        a.lse[(row + col) * a.H + h] = live ? (m + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f : -INFINITY;
}

// The pieces of a block of queries, in their order. (Blocks with one piece are written already.)
template <typename T>
__global__ __launch_bounds__(kSoftmaxThreads) void softmax_fwd_join_kernel(SoftmaxLaunch a, SoftmaxWork work, SoftmaxWork join) {
    constexpr int KB = kKeys<T>;
    SoftmaxPlace at;
    if (!softmax_find(join, a.rows, a.G, blockIdx.x, false, &at)) return;
    const int h = at.g * work.per + at.which, q0 = at.block * kSoftmaxBlock;
    const AttnSeq s = sequence(a.rows, at.seq);
    const bool packed = a.rows.cu_q != nullptr;
    const int rows = s.nq - q0 > kSoftmaxBlock ? kSoftmaxBlock : s.nq - q0;
    if (rows <= 0) return;  // one piece
    int pieces;
    softmax_piece(work, (last_key(s, a.causal, q0 + rows - 1) + KB) / KB, &pieces);
    if (pieces < 2) return;
    const int l = threadIdx.x & 31, r = at.piece * 8 + (int)threadIdx.x / 32;
    // rows past the sequence's queries (a padded batch) are 0, -inf
    if (q0 + r >= (packed ? s.nq : a.rows.Lq)) return;
    const int n = r < rows ? pieces : 0;
    const int64_t tokens = packed ? a.rows.Tq : a.rows.b * a.rows.Lq, row = (packed ? s.q0 : at.seq * a.rows.Lq) + q0 + r;
    const int64_t to = row * a.H + h;
    const float *ms = a.part + work.splits * tokens * a.H * a.D;
    float most = -INFINITY, total = 0.0f, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < n; ++i) most = __builtin_fmaxf(most, ms[2 * (i * tokens * a.H + to)]);
    const float base = most == -INFINITY ? 0.0f : most;
    for (int i = 0; i < n; ++i) {
        const int64_t from = i * tokens * a.H + to;
        const float f = exp2_fast(ms[2 * from] - base);
        total = __builtin_fmaf(f, ms[2 * from + 1], total);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (l + 32 * u < a.D) x[u] = __builtin_fmaf(f, a.part[from * a.D + l + 32 * u], x[u]);
    }
    const bool live = !(total == 0.0f);
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (l + 32 * u < a.D) static_cast<T *>(a.o)[to * a.D + l + 32 * u] = narrow<T>(live ? x[u] / total : 0.0f);
    if (a.lse && l == 0) a.lse[to] = live ? (base + __builtin_amdgcn_logf(total)) * 0.69314718055994530942f : -INFINITY;
}

template <typename T, int DP, bool VEC> hipError_t run(const SoftmaxLaunch &p, hipStream_t stream) {
    const SoftmaxWork w = softmax_fwd_work(p.rows, p.H, p.G, p.bf16);
    const dim3 grid((unsigned)softmax_groups(w));
    softmax_fwd_kernel<T, DP, VEC><<<grid, kSoftmaxThreads, 0, stream>>>(p, w);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (w.splits > 1) {
        const SoftmaxWork j = softmax_join_work(w);
        softmax_fwd_join_kernel<T><<<dim3((unsigned)softmax_groups(j)), kSoftmaxThreads, 0, stream>>>(p, w, j);
    }
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

hipError_t launch_softmax_fwd(const SoftmaxLaunch &p, hipStream_t stream) {
    return p.bf16 ? sm::by_width<uint16_t>(p, stream) : sm::by_width<float>(p, stream);
}

}  // namespace ssm
