// kv_append.hip — keys and values of new tokens into a paged cache, with the position rotation of keys and queries on the way; or the
// rotation alone, forward or back (its gradient).
//
// A token's coordinate pair m turns by the angle t·freq_m at position t. The angle is formed in turns in fp64 and reduced to
// a fraction of one before its sine and cosine are taken in fp32, so far positions lose nothing (a rounding of t·freq to
// fp32 would be 2^-8 of a turn at t = 2^17). A workgroup takes one token: its first lanes form the angles, and all go through the
// token's heads with them. Reading and writing every value once is the cost: 32 heads on 8 key heads of 128, bf16, 8 packed prompts
// of 17000 tokens in all (0.45 GB) take 87 us, 5.2 TB/s, 512 tokens 5.8 us. With a wavefront to a token both took longer (32768
// packed tokens 153 us for 139, 512 tokens 6.7 for 5.4, one 5.3 for 4.1).
#include "softmax_common.h"

namespace ssm {
namespace sm {
namespace {

constexpr int kMaxPairs = SSM_ATTN_MAX_D / 2;

// Heads of one token from `src` to up to two places, rotated. An item of work is one 16-byte piece (VEC; else one value) of the
// coordinates that stay as they are, or such a piece of each of the two coordinates of its pairs: an item reads before it
// writes, and no other touches its values, so that `src` may be a destination.
template <typename T, bool VEC> struct Mover {
    static constexpr int E = VEC ? kE<T> : 1;
    const KvAppendLaunch &a;
    const float *cs;  // cos, sin of each pair, in LDS
    __device__ __forceinline__ void move(const T *src, int64_t src_h, T *dst1, T *dst2, int heads, bool rotate) const {
        const int D = a.D, R = rotate ? a.rotary : 0, pairs = R / 2 / E, per = pairs + (D - R) / E;
        for (int i = threadIdx.x; i < heads * per; i += kAppendThreads) {
            const int h = i / per, n = i % per;
            const T *s = src + h * src_h;
            T x[E], y[E], u[E], v[E];
            if (n >= pairs) {
                const int c = R + (n - pairs) * E;
                load(x, s + c);
                store(dst1, dst2, h * D + c, x);
                continue;
            }
            // interleaved: 2E values in a row, of E pairs; otherwise E values of each half
            const int c0 = a.interleaved ? 2 * E * n : E * n, c1 = a.interleaved ? c0 + E : c0 + R / 2;
            load(x, s + c0);
            load(y, s + c1);
            if (VEC && a.interleaved) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    turn(u[2 * e], u[2 * e + 1], x[2 * e], x[2 * e + 1], E * n + e);
                    turn(v[2 * e], v[2 * e + 1], y[2 * e], y[2 * e + 1], E * n + E / 2 + e);
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) turn(u[e], v[e], x[e], y[e], E * n + e);
            }
            store(dst1, dst2, h * D + c0, u);
            store(dst1, dst2, h * D + c1, v);
        }
    }
    __device__ __forceinline__ void turn(T &u, T &v, T x, T y, int pair) const {
        const float c = cs[2 * pair], s = cs[2 * pair + 1], fx = widen(x), fy = widen(y);
        u = narrow<T>(__builtin_fmaf(fx, c, -(fy * s)));
        v = narrow<T>(__builtin_fmaf(fy, c, fx * s));
    }
    __device__ __forceinline__ void load(T (&x)[E], const T *p) const {
        if constexpr (VEC) {
            const u4 w = *reinterpret_cast<const u4 *>(p);
            __builtin_memcpy(x, &w, 16);
        } else {
            x[0] = *p;
        }
    }
    __device__ __forceinline__ void store(T *p, T *q, int at, const T (&x)[E]) const {
        if constexpr (VEC) {
            u4 w;
            __builtin_memcpy(&w, x, 16);
            if (p) *reinterpret_cast<u4 *>(p + at) = w;
            if (q) *reinterpret_cast<u4 *>(q + at) = w;
        } else {
            if (p) p[at] = x[0];
            if (q) q[at] = x[0];
        }
    }
    __device__ __forceinline__ void zero(T *p, int n) const {
        for (int i = threadIdx.x; i < n; i += kAppendThreads) p[i] = T(0);
    }
};

template <typename T, bool VEC>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(KvAppendLaunch a) {
    __shared__ float cs[2 * kMaxPairs];
    const int64_t t = blockIdx.x;
    const Mover<T, VEC> mv{a, cs};
    T *qo = a.q_out ? static_cast<T *>(a.q_out) + t * a.H * a.D : nullptr;
    T *ko = a.k_out ? static_cast<T *>(a.k_out) + t * a.G * a.D : nullptr;
    int64_t is, index, count;
    if (!locate(a.tokens, t, &is, &index, &count)) {  // a token of no row
        if (qo && a.q_out != a.q) mv.zero(qo, a.H * a.D);
        if (ko && a.k_out != a.k) mv.zero(ko, a.G * a.D);
        return;
    }
    const int64_t pos = (a.lengths ? (int64_t)a.lengths[is] - count : 0) + index;
    const int pair = threadIdx.x;
    if (a.freq && pair < a.rotary / 2) {
        double turns = (double)pos * a.freq[pair] * 0.15915494309189533577;
        turns -= __builtin_rint(turns);
        float sn, cn;
        sincospif(2.0f * (float)turns, &sn, &cn);
        cs[2 * pair] = cn;
        cs[2 * pair + 1] = a.inverse ? -sn : sn;
    }
    __syncthreads();

    const bool packed = a.tokens.cu != nullptr, turn = a.freq != nullptr;
    const int64_t ib = packed ? 0 : is, it = packed ? t : index;
    if (qo) mv.move(static_cast<const T *>(a.q) + ib * a.q_b + it * a.q_t, a.q_h, qo, nullptr, a.H, turn);
    T *kd = nullptr, *vd = nullptr;
    if (a.k_cache) {
        const int64_t page = page_of(a.pages, is, pos);
        if (page >= 0) {
            const int64_t slot = (int64_t)((uint32_t)pos % (uint32_t)a.pages.page) * a.G * a.D;
            kd = static_cast<T *>(a.k_cache) + page * a.k_page + slot;
            vd = static_cast<T *>(a.v_cache) + page * a.v_page + slot;
        }
    }
    if (kd || ko) mv.move(static_cast<const T *>(a.k) + ib * a.k_b + it * a.k_t, a.k_h, ko, kd, a.G, turn);
    if (vd) mv.move(static_cast<const T *>(a.v) + ib * a.v_b + it * a.v_t, a.v_h, vd, nullptr, a.G, false);
}

template <typename T> hipError_t run(const KvAppendLaunch &p, hipStream_t stream) {
    const dim3 grid((unsigned)p.tokens.T);
    if (p.vec) kv_append_kernel<T, true><<<grid, kAppendThreads, 0, stream>>>(p);
    else kv_append_kernel<T, false><<<grid, kAppendThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace
}  // namespace sm

hipError_t launch_kv_append(const KvAppendLaunch &p, hipStream_t stream) {
    return p.bf16 ? sm::run<uint16_t>(p, stream) : sm::run<float>(p, stream);
}

}  // namespace ssm
