// linattn_common.h — what the kernels of linear attention with a per-head decay share: the launch arguments, the
// chunk geometry, tile staging, and matrix products on fragments of 16×16×32 steps.
//
// Every product is a sum of 16×16 tiles D = A·Bᵀ over a contraction axis taken 32 at a time. Lane l = 16·grp + col
// of a wavefront supplies, for row `col` of A (and of B), the 8 contraction values 4·grp + j and 16 + 4·grp + j
// (j < 4) of the 32, and receives D[4·grp + r][col], r < 4. The order of a contraction axis is free as long as
// both operands use the same, and this one makes a result tile an operand without moving it: D's lane holds, for
// row (as an operand) `col`, four consecutive values 4·grp + r of a 16-block, so two neighbouring result tiles are
// the lane's 8 values of one contraction step. The state, kept as result tiles, is thus read as an operand in place.
#pragma once

#include <type_traits>

#include "device_common.h"
#include "launch.h"

namespace ssm {
namespace la {

constexpr int kC = 64;        // steps per chunk
constexpr int kPB = 64;       // value columns per workgroup (16 per wavefront)
constexpr int kThreads = 256; // four wavefronts
// Log-decays below this count as this: e^-1e4 is 0 in fp32, and so is every product with it, while running sums
// stay finite (−inf would turn differences of sums into NaN).
constexpr float kMinG = -1e4f;

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));

// Elements of a 16-byte access, the LDS row padding (16 bytes: rows 4 banks apart, so the 16 rows that a fragment
// read touches at once take 16 different groups of banks) and the parts that carry an fp32 operand.
template <typename T> constexpr int kVec = 16 / sizeof(T);
template <typename T> constexpr int kPad = 16 / sizeof(T);
template <typename T> using Frag = typename std::conditional<sizeof(T) == 2, bf8, f8>::type;

__device__ __forceinline__ void mma(f4 &acc, const bf8 &a, const bf8 &b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f4 &acc, const f8 &a, const f8 &b) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], acc, 0, 0, 0);
}

// Operand fragment of tile row `row0 + col`, contraction values n0 .. n0+31 along the row.
__device__ __forceinline__ bf8 row_frag(const uint16_t *tile, int stride, int row0, int n0) {
    const int l = threadIdx.x & 63;
    const uint16_t *p = tile + (row0 + (l & 15)) * stride + n0 + 4 * (l >> 4);
    const bf4 u = *reinterpret_cast<const bf4 *>(p), v = *reinterpret_cast<const bf4 *>(p + 16);
    return __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ f8 row_frag(const float *tile, int stride, int row0, int n0) {
    const int l = threadIdx.x & 63;
    const float *p = tile + (row0 + (l & 15)) * stride + n0 + 4 * (l >> 4);
    const f4 u = *reinterpret_cast<const f4 *>(p), v = *reinterpret_cast<const f4 *>(p + 16);
    return __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Operand fragment of tile column n0 + col, contraction values s0 .. s0+31 down the column. bf16: the transposing
// LDS read, which gives lane `col` of 16 lanes column `col` of the 4×16 block whose quarter rows they address.
__device__ __forceinline__ bf8 col_frag(const uint16_t *tile, int stride, int s0, int n0) {
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const int l = threadIdx.x & 63, c = l & 15;
    const uint16_t *p = tile + (s0 + 4 * (l >> 4) + (c >> 2)) * stride + n0 + 4 * (c & 3);
    const s4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p);
    const s4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 16 * stride));
    typedef short s8 __attribute__((ext_vector_type(8)));
    const s8 w = __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf8, w);
}
__device__ __forceinline__ f8 col_frag(const float *tile, int stride, int s0, int n0) {
    const int l = threadIdx.x & 63;
    const float *p = tile + (s0 + 4 * (l >> 4)) * stride + n0 + (l & 15);
    f8 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r[j] = p[j * stride];
        r[4 + j] = p[(16 + j) * stride];
    }
    return r;
}

__device__ __forceinline__ f8 wide(const bf8 &v) { return __builtin_convertvector(v, f8); }
__device__ __forceinline__ f8 wide(const f8 &v) { return v; }
__device__ __forceinline__ f8 join(const f4 &u, const f4 &v) { return __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7); }

// acc += (an fp32 operand)·b in PARTS parts: for bf16 storage the value is cut into bf16 parts, each the rounded
// remainder of those before (relative error at most 2^-8, 2^-16, 2^-24 for 1, 2, 3 parts); for f32 it is one part.
template <int PARTS> struct Parts {
    bf8 p[PARTS];
    __device__ __forceinline__ explicit Parts(f8 v) {
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
            p[i] = __builtin_convertvector(v, bf8);
            if (i + 1 < PARTS) v -= wide(p[i]);
        }
    }
};
struct Whole {
    f8 v;
    __device__ __forceinline__ explicit Whole(f8 x) : v(x) {}
};
template <typename T, int PARTS> using Split = typename std::conditional<sizeof(T) == 2, Parts<PARTS>, Whole>::type;
template <int PARTS> __device__ __forceinline__ void mma(f4 &acc, const Parts<PARTS> &a, const bf8 &b) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) mma(acc, a.p[i], b);
}
template <int PARTS> __device__ __forceinline__ void mma(f4 &acc, const bf8 &a, const Parts<PARTS> &b) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) mma(acc, a, b.p[i]);
}
__device__ __forceinline__ void mma(f4 &acc, const Whole &a, const f8 &b) { mma(acc, a.v, b); }
__device__ __forceinline__ void mma(f4 &acc, const f8 &a, const Whole &b) { mma(acc, a, b.v); }

// e^v for a difference of running sums.
__device__ __forceinline__ float exp_of(float v) { return exp2_fast(kLog2e * v); }

// Inclusive running sum over the 64 lanes of a wavefront, fp64.
__device__ __forceinline__ double wave_running_sum(double v) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double u = __shfl_up(v, d);
        if (l >= d) v += u;
    }
    return v;
}

// The lane's clamped log-decay of step t (0 past `len`).
__device__ __forceinline__ double log_decay(const float *g, int64_t stride, int64_t t, int64_t len) {
    if (t >= len) return 0.0;
    const float v = g[t * stride];
    return v < kMinG ? (double)kMinG : (double)v;
}

// Running sums of g in a chunk as fp32 hi + lo, so that their differences keep fp32's accuracy however large the
// sums are.
struct Sums {
    float hi[kC], lo[kC];
    __device__ __forceinline__ void set(int t, double c) {
        hi[t] = (float)c;
        lo[t] = (float)(c - (double)hi[t]);
    }
};

// Rows [t0, t0 + 64) × columns [c0, c0 + W) of a strided array into an LDS tile, zeros past `len` rows and `cols`
// columns; `vec` says that 16-byte accesses at multiples of kVec elements are allowed and that cols − c0 ends on one.
template <typename T, int W>
__device__ __forceinline__ void stage(T *tile, const T *src, int64_t stride, int64_t t0, int64_t len, int c0, int cols,
                                      bool vec) {
    constexpr int V = kVec<T>, PER = W / V, S = W + kPad<T>;
#pragma unroll
    for (int i = threadIdx.x; i < kC * PER; i += kThreads) {
        const int r = i / PER, c = (i % PER) * V;
        const int64_t t = t0 + r;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (t < len) {
            const T *p = src + t * stride + c0 + c;
            if (vec) {
                if (c0 + c < cols) w = *reinterpret_cast<const uint4 *>(p);
            } else {
                T e[V];
#pragma unroll
                for (int j = 0; j < V; ++j) e[j] = c0 + c + j < cols ? p[j] : (T)0;
                __builtin_memcpy(&w, e, sizeof(w));
            }
        }
        *reinterpret_cast<uint4 *>(tile + r * S + c) = w;
    }
}

// Four consecutive results row[c .. c+3] of a dense row of `cols`.
template <typename T>
__device__ __forceinline__ void store4(T *row, int c, int cols, bool vec, const f4 &v) {
    if (vec) {
        if (c < cols) {
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<bf4 *>(row + c) = __builtin_convertvector(v, bf4);
            } else {
                *reinterpret_cast<f4 *>(row + c) = v;
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (c + j < cols) row[c + j] = narrow<T>(v[j]);
}

// Steps of batch row i.
__device__ __forceinline__ int64_t row_length(const int32_t *lengths, int64_t i, int64_t L) {
    if (!lengths) return L;
    const int64_t n = lengths[i];
    return n < 0 ? 0 : (n > L ? L : n);
}

// Workgroups are dealt to the 8 XCDs in turn; this gives each XCD a contiguous run of work, so that the heads that
// share keys and queries, and the value blocks of a head, find them in one L2.
__device__ __forceinline__ int64_t work_index(int64_t block, int64_t blocks) {
    const int64_t x = block & 7, per = blocks >> 3, rest = blocks & 7;
    return x * per + (x < rest ? x : rest) + (block >> 3);
}

}  // namespace la
}  // namespace ssm
