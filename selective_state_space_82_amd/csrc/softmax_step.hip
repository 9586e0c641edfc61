// softmax_step.hip — softmax attention of one new token a row over a paged cache of keys and values.
//
// Reading the cache is the cost: 2·D values a token and key head against 4·D·H/G operations. The heads that share a key
// head (up to 16 at once) are the columns of one 16×16 product, so that a key or value is read once for all of them: scores are
// formed transposed (keys down, heads across), a head's weights stay in the lanes that hold its scores and are the second
// operand of the product with the values (with bf16 in two parts, 2^-16, which memory hides: 0.82 ms with one as with two for the
// 512 rows below, and o 2.1e-3 of its norm off with one, 1.7e-3, its own rounding, with two). Keys come from memory straight into registers as a product's operand; values pass
// through LDS, which the transposing read takes them from. A wavefront walks tiles of its own, every fourth of its workgroup's
// piece; the four are joined in LDS, and the pieces of a row, where there are several, by a second launch. The next tile's
// keys and page numbers are on their way while a tile is computed, and so are its own values: 64 KB a workgroup of D 128.
// 512 rows of 1 to 4096 tokens, 32 heads on 8 key heads of 128, bf16, pages of 64 (4.24 GB): 0.82 ms, 5.2 TB/s, what a copy
// reaches. One row of 131072 tokens on 2 key heads: 27 us for its 256 pieces (5.1 TB/s) and 9 to join them (39 a call).
#include "softmax_common.h"

namespace ssm {
namespace sm {
namespace {

using la::f8;
template <typename T> using Wide = typename std::conditional<sizeof(T) == 2, bf8, f8>::type;  // 8 contraction values
template <typename T> constexpr int kTile = sizeof(T) == 2 ? 64 : 32;                         // keys of a wavefront's tile
// LDS row: the 8 rows (bf16; fp32: 4, every fourth) that a read down 16 columns touches at once take different banks.
template <typename T, int W> constexpr int kValStride = sizeof(T) == 2 ? W + 16 : W + 4;

// 8 values of a row at `at`, zeros from column `cols` on.
template <typename T, bool VEC> __device__ __forceinline__ Wide<T> load8(const T *row, int c, int cols) {
    Wide<T> r;
    if constexpr (VEC) {
        constexpr int N = 8 / kE<T>;
        u4 w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = c + i * kE<T> < cols ? *reinterpret_cast<const u4 *>(row + c + i * kE<T>) : u4(0u);
        __builtin_memcpy(&r, w, sizeof(r));
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = c + i < cols ? row[c + i] : T(0);
        __builtin_memcpy(&r, e, sizeof(r));
    }
    return r;
}

// Weights as an operand. bf16: in two parts, rounded to nearest and what that leaves, rounded: 2^-16.
__device__ __forceinline__ void operand(bf8 &r, const f4 &a, const f4 &b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = (__bf16)a[i];
        r[i + 4] = (__bf16)b[i];
    }
}
__device__ __forceinline__ void operand(f8 &r, const f4 &a, const f4 &b) { r = la::join(a, b); }
__device__ __forceinline__ void remainder(bf8 &r, const bf8 &p, const f4 &a, const f4 &b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = (__bf16)(a[i] - (float)p[i]);
        r[i + 4] = (__bf16)(b[i] - (float)p[i + 4]);
    }
}
__device__ __forceinline__ void remainder(f8 &, const f8 &, const f4 &, const f4 &) {}

// Columns c0 .. c0 + 15 of 32 rows of values in LDS, rows 16u + 4·grp + e (u < 2, e < 4) of lane 16·grp + col's column.
__device__ __forceinline__ bf8 value_frag(const uint16_t *tile, int stride, int c0) {
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const int l = threadIdx.x & 63, c = l & 15;
    const uint16_t *p = tile + (4 * (l >> 4) + (c >> 2)) * stride + c0 + 4 * (c & 3);
    const s4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p);
    const s4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 16 * stride));
    return __builtin_bit_cast(bf8, __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ f8 value_frag(const float *tile, int stride, int c0) {
    const int l = threadIdx.x & 63;
    const float *p = tile + 4 * (l >> 4) * stride + c0 + (l & 15);
    f8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = p[(16 * (e >> 2) + (e & 3)) * stride];
    return r;
}

// Over the four lanes that hold a column.
__device__ __forceinline__ float column_max(float v) {
    v = __builtin_fmaxf(v, __shfl_xor(v, 16));
    return __builtin_fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float column_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Tokens of a piece and how many pieces a row of n tokens has.
__device__ __forceinline__ int piece_of(const SoftmaxStepLaunch &a, int n, int *pieces) {
    int per = ((n + a.splits - 1) / a.splits + kStepTile - 1) / kStepTile * kStepTile;
    per = per < a.least ? a.least : per;
    *pieces = n > 0 ? (n + per - 1) / per : 1;
    return per;
}

template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(kSoftmaxThreads, 2) void softmax_step_kernel(SoftmaxStepLaunch a) {
    constexpr int KT = kTile<T>, NT = KT / 16, NC = DP / 32, ND = DP / 16, VS = kValStride<T, DP>, WAVES = kSoftmaxThreads / 64;
    constexpr int kValues = 32 * VS * (int)sizeof(T), kJoin = 16 * (DP + 4) * 4;  // bytes a wavefront
    constexpr int kBytes = kValues > kJoin ? kValues : kJoin;
    __shared__ __attribute__((aligned(16))) char lds[WAVES][kBytes];
    __shared__ float top_of[WAVES][16], sum_of[WAVES][16];

    const int R = a.H / a.G, groups = (R + 15) / 16;
    int64_t id = la::work_index(blockIdx.x, gridDim.x);
    const int piece = (int)(id % a.splits);
    id /= a.splits;
    const int hg = (int)(id % groups);
    id /= groups;
    const int g = (int)(id % a.G);
    const int64_t is = id / a.G;
    const int n = cached(a.pages, a.lengths, is);
    int pieces;
    const int per = piece_of(a, n, &pieces);
    if (piece >= pieces) return;
    const int end = piece == pieces - 1 ? n : (piece + 1) * per;
    const int w = la::wave_id(), l = threadIdx.x & 63, col = l & 15, grp = l >> 4;
    const int h0 = g * R + 16 * hg, heads = R - 16 * hg < 16 ? R - 16 * hg : 16;

    Wide<T> q[NC];
    {
        const T *qp = static_cast<const T *>(a.q) + is * a.q_b + (h0 + (col < heads ? col : 0)) * a.q_h;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            q[c] = load8<T, VEC>(qp, 32 * c + 8 * grp, col < heads && a.scale != 0.0f ? a.D : 0);  // as for_scale() leaves it
            if (a.scale < 0.0f) q[c] = -q[c];
        }
    }
    const float sc = scale_of(a.scale);
    const T *kc = static_cast<const T *>(a.k_cache) + g * a.D, *vc = static_cast<const T *>(a.v_cache) + g * a.D;
    const int row = a.G * a.D;
    T *vt = reinterpret_cast<T *>(lds[w]);

    f4 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f4(0.0f);
    float m = -INFINITY, sum = 0.0f;

    // Lane i's key of a tile: page and slot, and which lanes' keys there are. Keys past the end and on pages that the cache does
    // not have are read from page 0 and count for nothing.
    int page = 0, slot = 0;
    uint64_t there = 0;
    const auto find = [&](int j0) {
        const int key = j0 + (l & (KT - 1));
        const int64_t p = key < end ? page_of(a.pages, is, key) : -1;
        there = __ballot(p >= 0) & (KT == 64 ? ~UINT64_C(0) : (UINT64_C(1) << (KT & 63)) - 1);
        page = p >= 0 ? (int)p : 0;
        slot = p >= 0 ? (int)((uint32_t)key % (uint32_t)a.pages.page) : 0;
    };
    Wide<T> k[NT][NC], v[NT][NC];
    const auto load = [&](Wide<T> (&x)[NT][NC], const T *cache, int64_t stride) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const T *p = cache + (int64_t)__shfl(page, 16 * t + col) * stride + (int64_t)__shfl(slot, 16 * t + col) * row;
#pragma unroll
            for (int c = 0; c < NC; ++c) x[t][c] = load8<T, VEC>(p, 32 * c + 8 * grp, a.D);
        }
    };
    const uint64_t all = KT == 64 ? ~UINT64_C(0) : (UINT64_C(1) << (KT & 63)) - 1;

    int j0 = piece * per + w * KT;
    if (j0 < end) {
        find(j0);
        load(k, kc, a.k_page);
    }
    for (; j0 < end; j0 += WAVES * KT) {
        load(v, vc, a.v_page);
        const uint64_t mine = there;
        f4 p[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            p[t] = f4(0.0f);
#pragma unroll
            for (int c = 0; c < NC; ++c) la::mma(p[t], k[t][c], q[c]);
        }
        if (j0 + WAVES * KT < end) {
            find(j0 + WAVES * KT);
            load(k, kc, a.k_page);
        }
        if (mine != all) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(mine >> (16 * t + 4 * grp + e) & 1)) p[t][e] = -INFINITY;
                if (!(mine >> (16 * t + col) & 1)) {
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[t][c][e] = 0.0f;
                }
            }
        }
        float top = p[0][0];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = __builtin_fmaxf(top, p[t][e]);
        top = column_max(top) * sc;
        const float up = __builtin_fmaxf(m, top), base = up == -INFINITY ? 0.0f : up;
        const float f = exp2_fast(m - base);
        m = up;
        sum *= f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[t][e] = exp2_fast(__builtin_fmaf(p[t][e], sc, -base));
                sum += p[t][e];
            }
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] *= f;
#pragma unroll
        for (int u = 0; u < NT / 2; ++u) {
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    *reinterpret_cast<Wide<T> *>(vt + (16 * t + col) * VS + 32 * c + 8 * grp) = v[2 * u + t][c];
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
            Wide<T> pf, rest;
            operand(pf, p[2 * u], p[2 * u + 1]);
            remainder(rest, pf, p[2 * u], p[2 * u + 1]);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const Wide<T> x = value_frag(vt, VS, 16 * d);
                la::mma(o[d], x, pf);
                if constexpr (sizeof(T) == 2) la::mma(o[d], x, rest);
            }
        }
    }
    sum = column_sum(sum);

    // the wavefronts' parts, [head][column]
    __builtin_amdgcn_wave_barrier();
    float *own = reinterpret_cast<float *>(lds[w]);
#pragma unroll
    for (int d = 0; d < ND; ++d) *reinterpret_cast<f4 *>(own + col * (DP + 4) + 16 * d + 4 * grp) = o[d];
    if (grp == 0) {
        top_of[w][col] = m;
        sum_of[w][col] = sum;
    }
    la::lds_barrier();
    for (int i = threadIdx.x; i < heads * DP; i += kSoftmaxThreads) {
        const int h = i / DP, d = i % DP;
        if (d >= a.D) continue;
        float most = -INFINITY, total = 0.0f, x = 0.0f;
#pragma unroll
        for (int u = 0; u < WAVES; ++u) most = __builtin_fmaxf(most, top_of[u][h]);
        // a NaN score leaves the maximum as it is and makes the sum NaN; no keys: weights of 0
        const float base = most == -INFINITY ? 0.0f : most;
#pragma unroll
        for (int u = 0; u < WAVES; ++u) {
            const float f = exp2_fast(top_of[u][h] - base);
            total = __builtin_fmaf(f, sum_of[u][h], total);
            x = __builtin_fmaf(f, reinterpret_cast<const float *>(lds[u])[h * (DP + 4) + d], x);
        }
        const int64_t at = is * a.H + h0 + h;
        if (a.splits == 1) {
            static_cast<T *>(a.o)[at * a.D + d] = narrow<T>(total == 0.0f ? 0.0f : x / total);
            if (a.lse && d == 0)
                a.lse[at] = total == 0.0f ? -INFINITY : (base + __builtin_amdgcn_logf(total)) * 0.69314718055994530942f;
        } else {
            float *part = a.part + (at * a.splits + piece) * (a.D + 2);
            part[2 + d] = x;
            if (d == 0) {
                part[0] = most;
                part[1] = total;
            }
        }
    }
}

// The pieces of a row and head, in their order.
template <typename T> __global__ __launch_bounds__(kSoftmaxThreads) void softmax_join_kernel(SoftmaxStepLaunch a) {
    constexpr int WAVES = kSoftmaxThreads / 64;
    __shared__ float acc[WAVES][SSM_ATTN_MAX_D], total_of[WAVES], most_of[WAVES];
    const int64_t at = blockIdx.x, is = at / a.H;
    int pieces;
    piece_of(a, cached(a.pages, a.lengths, is), &pieces);
    const float *part = a.part + at * a.splits * (a.D + 2);
    const int w = la::wave_id(), l = threadIdx.x & 63;
    float most = -INFINITY;
    for (int i = threadIdx.x; i < pieces; i += kSoftmaxThreads) most = __builtin_fmaxf(most, part[(int64_t)i * (a.D + 2)]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) most = __builtin_fmaxf(most, __shfl_xor(most, d));
    if (l == 0) most_of[w] = most;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < WAVES; ++u) most = __builtin_fmaxf(most, most_of[u]);
    const float base = most == -INFINITY ? 0.0f : most;
    float x[2] = {0.0f, 0.0f}, total = 0.0f;
    constexpr int AT_ONCE = 8;  // pieces whose loads are on their way together
    for (int i0 = w; i0 < pieces; i0 += WAVES * AT_ONCE) {
        float f[AT_ONCE], n[AT_ONCE], y[AT_ONCE][2];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int i = i0 + WAVES * k;
            const float *p = part + (int64_t)(i < pieces ? i : 0) * (a.D + 2);
            f[k] = p[0];
            n[k] = p[1];
#pragma unroll
            for (int u = 0; u < 2; ++u) y[k][u] = l + 64 * u < a.D ? p[2 + l + 64 * u] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            if (i0 + WAVES * k >= pieces) break;
            const float e = exp2_fast(f[k] - base);
            total = __builtin_fmaf(e, n[k], total);
#pragma unroll
            for (int u = 0; u < 2; ++u) x[u] = __builtin_fmaf(e, y[k][u], x[u]);
        }
    }
    acc[w][l] = x[0];
    acc[w][l + 64] = x[1];
    if (l == 0) total_of[w] = total;
    __syncthreads();
    total = 0.0f;
#pragma unroll
    for (int u = 0; u < WAVES; ++u) total += total_of[u];
    const int d = threadIdx.x;
    if (d < a.D) {
        float y = 0.0f;
#pragma unroll
        for (int u = 0; u < WAVES; ++u) y += acc[u][d];
        static_cast<T *>(a.o)[at * a.D + d] = narrow<T>(total == 0.0f ? 0.0f : y / total);
    }
    if (a.lse && d == 0)
        a.lse[at] = total == 0.0f ? -INFINITY : (base + __builtin_amdgcn_logf(total)) * 0.69314718055994530942f;
}

template <typename T, int DP, bool VEC> hipError_t run(const SoftmaxStepLaunch &p, hipStream_t stream) {
    const int64_t groups = (p.H / p.G + 15) / 16;
    softmax_step_kernel<T, DP, VEC>
        <<<dim3((unsigned)(p.b * p.G * groups * p.splits)), kSoftmaxThreads, 0, stream>>>(p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (p.splits > 1) softmax_join_kernel<T><<<dim3((unsigned)(p.b * p.H)), kSoftmaxThreads, 0, stream>>>(p);
    return hipGetLastError();
}
template <typename T> hipError_t by_width(const SoftmaxStepLaunch &p, hipStream_t stream) {
    if (!p.vec) return p.D <= 64 ? run<T, 64, false>(p, stream) : run<T, 128, false>(p, stream);
    if (p.D <= 32) return run<T, 32, true>(p, stream);
    if (p.D <= 64) return run<T, 64, true>(p, stream);
    if (p.D <= 96) return run<T, 96, true>(p, stream);
    return run<T, 128, true>(p, stream);
}

}  // namespace
}  // namespace sm

hipError_t launch_softmax_step(const SoftmaxStepLaunch &p, hipStream_t stream) {
    return p.bf16 ? sm::by_width<uint16_t>(p, stream) : sm::by_width<float>(p, stream);
}

}  // namespace ssm
