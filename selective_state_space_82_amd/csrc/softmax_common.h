// softmax_common.h — what the kernels of softmax attention over prompts share: products on fragments of 32×32 tiles, and tiles
// of rows on their way from memory through LDS.
//
// A product D = A·Bᵀ of 32×32 tiles takes its contraction axis in chunks of 16 (bf16) or 8 (fp32) values. Lane
// l = 32·half + col of a wavefront supplies, for row `col` of A (and of B), half of the chunk's values, 16 bytes, and
// receives D[8j + 4·half + r][col], j, r < 4, as element 4j + r of its sixteen. The contraction axis' order is free as long as
// both operands use the same. Two orders are used:
//   along a row     chunk values half·E .. half·E + E − 1, one 16-byte LDS read;
//   down a column   the order in which a product's results lie in a lane: of a chunk's rows 4·half + r (and + 8 for bf16). So
//                   the results of one product, turned into weights in place, are the second operand of the next
//                   without passing through LDS, and the first operand is read down the columns of its tile: with the transposing
//                   read for bf16, value by value for fp32.
// Scores are formed transposed (keys down, queries across): a query's statistics are then sums over a lane's own elements
// and one exchange with the lane 32 away.
#pragma once

#include "linattn_common.h"
#include "launch_softmax.h"
#include "ssm_scan.h"

namespace ssm {
namespace sm {

using la::bf4;
using la::bf8;
using la::Buffer;
using la::f4;
using la::kOutside;
typedef float f16 __attribute__((ext_vector_type(16)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

template <typename T> constexpr int kE = 16 / sizeof(T);   // a lane's values of a chunk
template <typename T> constexpr int kChunk = 2 * kE<T>;    // contraction values of a chunk
template <typename T> using Frag = typename std::conditional<sizeof(T) == 2, bf8, f4>::type;

__device__ __forceinline__ void mma(f16 &acc, const bf8 &a, const bf8 &b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f16 &acc, const f4 &a, const f4 &b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], acc, 0, 0, 0);
}

// Elements between the rows of an LDS tile of W columns. read_rows: 16-byte reads of 16 rows at once take all banks (rows 4
// banks apart beyond whole turns). read_cols: the 4 rows of a transposing read lie 16 banks apart (bf16), the two of a
// read by value 32 (fp32). A tile read both ways takes the first.
template <typename T, int W> constexpr int kRowStride = W + 16 / sizeof(T);
template <typename T, int W> constexpr int kColStride =
    sizeof(T) == 2 ? (W % 64 == 32 ? W : W % 128 == 96 ? W : W + 32) : W + 8;

// Row `row0 + col`, values n0 + E·half on, of a tile.
template <typename T> __device__ __forceinline__ Frag<T> row_frag(const T *tile, int stride, int row0, int n0) {
    const int l = threadIdx.x & 63;
    return *reinterpret_cast<const Frag<T> *>(tile + (row0 + (l & 31)) * stride + n0 + kE<T> * (l >> 5));
}
// Column `col0 + col`, rows s0 .. s0 + chunk − 1 in the order above, of a tile.
__device__ __forceinline__ bf8 col_frag(const uint16_t *tile, int stride, int s0, int col0) {
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const int l = threadIdx.x & 63, c = l & 15;
    const uint16_t *p = tile + (s0 + 4 * (l >> 5) + (c >> 2)) * stride + col0 + (l & 16) + 4 * (c & 3);
    const s4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p);
    const s4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 8 * stride));
    return __builtin_bit_cast(bf8, __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ f4 col_frag(const float *tile, int stride, int s0, int col0) {
    const int l = threadIdx.x & 63;
    const float *p = tile + (s0 + 4 * (l >> 5)) * stride + col0 + (l & 31);
    return f4{p[0], p[stride], p[2 * stride], p[3 * stride]};
}

// Elements of chunk c of a lane's sixteen results as an operand in the order down a column. bf16: rounded to nearest, 2^-8.
template <typename T> __device__ __forceinline__ Frag<T> part_of(const f16 &x, int c) {
    if constexpr (sizeof(T) == 2) {
        bf8 r;
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = (__bf16)x[8 * c + j];
        return r;
    } else {
        return f4{x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]};
    }
}

// A row of a strided matrix in memory as fragments in registers: row `row0 + col` (zeros from row `rows` on, columns from
// `cols` on), all DP columns.
template <typename T, int DP, bool VEC>
__device__ __forceinline__ void load_frags(Frag<T> (&f)[DP / kChunk<T>], const Buffer &buf, uint32_t stride, int row, int rows,
                                           int cols) {
    const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int c = 0; c < DP / kChunk<T>; ++c) {
        const int n0 = kChunk<T> * c + kE<T> * half;
        u4 w;
        if constexpr (VEC) {
            const uint32_t at = row < rows && n0 < cols ? (uint32_t)(row * stride + n0) * (uint32_t)sizeof(T) : kOutside;
            w = __builtin_amdgcn_raw_buffer_load_b128(buf, at, 0, 0);
        } else {
            T e[kE<T>];
#pragma unroll
            for (int k = 0; k < kE<T>; ++k) {
                const uint32_t at =
                    row < rows && n0 + k < cols ? (uint32_t)(row * stride + n0 + k) * (uint32_t)sizeof(T) : kOutside;
                if constexpr (sizeof(T) == 2) e[k] = (T)__builtin_amdgcn_raw_buffer_load_b16(buf, at, 0, 0);
                else e[k] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(buf, at, 0, 0));
            }
            __builtin_memcpy(&w, e, sizeof(w));
        }
        f[c] = __builtin_bit_cast(Frag<T>, w);
    }
}

// Whether a 16-byte piece holds a NaN or Inf.
template <typename T> __device__ __forceinline__ bool not_finite(const u4 &w) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) bad = bad || (~w[i] & 0x7f80u) == 0 || (~w[i] & 0x7f800000u) == 0;
        else bad = bad || (~w[i] & 0x7f800000u) == 0;
    }
    return bad;
}

// ROWS rows × W columns on their way into an LDS tile, zeros past the rows and columns there are. A thread holds its pieces
// between load and store, so that a tile is fetched while the one before is computed.
template <typename T, int ROWS, int W, bool VEC> struct Stage {
    static constexpr int E = kE<T>, PER = W / E, PIECES = ROWS * PER, N = (PIECES + kSoftmaxThreads - 1) / kSoftmaxThreads;
    u4 w[N];
    // first: row 0, column 0 of the tile, the same in every lane; rows: how many there are (0 and below: none)
    __device__ __forceinline__ void load(const T *first, uint32_t stride, int rows, int cols) {
        rows = rows > ROWS ? ROWS : rows;
        const Buffer buf = la::rows_buffer(first, stride, rows, cols);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int id = (int)threadIdx.x + j * kSoftmaxThreads, r = id / PER, c = id % PER * E;
            if constexpr (VEC) {
                const uint32_t at = r < rows && c < cols ? (r * stride + c) * (uint32_t)sizeof(T) : kOutside;
                w[j] = __builtin_amdgcn_raw_buffer_load_b128(buf, at, 0, 0);
            } else {
                T e[E];
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const uint32_t at = r < rows && c + k < cols ? (r * stride + c + k) * (uint32_t)sizeof(T) : kOutside;
                    if constexpr (sizeof(T) == 2) e[k] = (T)__builtin_amdgcn_raw_buffer_load_b16(buf, at, 0, 0);
                    else e[k] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(buf, at, 0, 0));
                }
                __builtin_memcpy(&w[j], e, sizeof(w[j]));
            }
        }
    }
    __device__ __forceinline__ void store(T *tile, int stride) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int id = (int)threadIdx.x + j * kSoftmaxThreads;
            if (PIECES % kSoftmaxThreads == 0 || id < PIECES)
                *reinterpret_cast<u4 *>(tile + id / PER * stride + id % PER * E) = w[j];
        }
    }
    __device__ __forceinline__ bool bad() const {
        bool b = false;
#pragma unroll
        for (int j = 0; j < N; ++j) b = b || not_finite<T>(w[j]);
        return b;
    }
};

// Of the lane's value and that of the lane 32 away.
__device__ __forceinline__ float other_half(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float((threadIdx.x & 32) ? a[0] : a[1]);
}

// The scale times log2 e, and whether the queries change sign for it: weights are then 2^(|scale|·log2 e·s − maximum). A scale of 0
// counts as 2^-126 (scores below 2^-100 of any input that fp32 products can hold: the same weights), so that masked
// scores of −inf stay what they are.
__device__ __forceinline__ float scale_of(float scale) {
    return __builtin_fmaxf(__builtin_fabsf(scale) * kLog2e, 1.17549435e-38f);
}
template <typename T> __device__ __forceinline__ void negate(Frag<T> &f) { f = -f; }

// Results [8j + 4·half + r][col] as rows of a matrix: row `row` (the lane's), columns n0 + 8j + 4·half + r.
template <typename T, bool VEC>
__device__ __forceinline__ void store_tile(const Buffer &buf, uint32_t stride, int row, int n0, int cols, const f16 &x, float f) {
    const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        la::store4<T, VEC>(buf, stride, row, n0 + 8 * j + 4 * half, cols,
                           f4{x[4 * j] * f, x[4 * j + 1] * f, x[4 * j + 2] * f, x[4 * j + 3] * f});
}

}  // namespace sm
}  // namespace ssm
