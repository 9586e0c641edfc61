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

// An LDS tile of rows of W columns, without padding between them, so that loads can go from memory straight into LDS, 64
// pieces of 16 bytes at a time in the order of the lanes. Banks are spread by where a row's pieces stand: piece p of row r at place
// p ^ turn(r). So 16 rows read 16 bytes each at one piece, the 4 rows × 64 bytes of a transposing read (bf16) and the two rows, 4
// apart, of 128 bytes each of a read by value (fp32) lie in different banks.
template <typename T, int W> struct Tile {
    static constexpr int kPitch = W == 96 ? 128 : W;                    // columns between rows
    static constexpr int kRow = kPitch * (int)sizeof(T), kPer = kRow / 16;  // bytes and pieces of a row
    __device__ static __forceinline__ int turn(int r) {
        if constexpr (kRow == 512) return (r & 3) | (r >> 3 & 1) << 2 | (r >> 2 & 1) << 3;
        else if constexpr (kRow == 256) return (r & 3) << 2 | (r >> 2 & 3);
        else if constexpr (kRow == 128) return (r >> 1 & 1) << 2 | (r >> 2 & 3);
        else return r >> 2 & 3;
    }
    // byte offset of piece p of row r
    __device__ static __forceinline__ int at(int r, int p) { return r * kRow + 16 * (p ^ turn(r)); }
};

// Row `row0 + col` (row0 a multiple of 32), chunk c of a tile.
template <typename T, int W> __device__ __forceinline__ Frag<T> row_frag(const char *tile, int row0, int c) {
    const int l = threadIdx.x & 63;
    return *reinterpret_cast<const Frag<T> *>(tile + row0 * Tile<T, W>::kRow + Tile<T, W>::at(l & 31, 2 * c + (l >> 5)));
}
// Column `col0 + col`, rows s0 .. s0 + chunk − 1 (s0 a multiple of the chunk) in the order above, of a tile.
template <typename T, int W> __device__ __forceinline__ Frag<T> col_frag(const char *tile, int s0, int col0) {
    const int l = threadIdx.x & 63;
    using X = Tile<T, W>;
    if constexpr (sizeof(T) == 2) {
        typedef __attribute__((address_space(3))) s4 lds_s4;
        const int c = l & 15, r = 4 * (l >> 5) + (c >> 2), p = col0 / 8 + (l >> 4 & 1) * 2 + (c >> 1 & 1), e = 8 * (c & 1);
        const char *q = tile + s0 * X::kRow + e;
        const s4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(q + X::at(r, p)));
        const s4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(q + X::at(r + 8, p)));
        return __builtin_bit_cast(bf8, __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        f4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = (s0 & 15) + 4 * (l >> 5) + e, p = col0 / 4 + (l >> 2 & 7);
            x[e] = *reinterpret_cast<const float *>(tile + (s0 & ~15) * X::kRow + X::at(r, p) + 4 * (l & 3));
        }
        return x;
    }
}

// Elements of chunk c of a lane's sixteen results as an operand in the order down a column. bf16: rounded to nearest, 2^-8.
template <typename T> __device__ __forceinline__ Frag<T> part_of(const f16 &x, int c) {
    if constexpr (sizeof(T) == 2) {
        la::f8 y;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[8 * c + j];
        return __builtin_convertvector(y, bf8);
    } else {
        return f4{x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]};
    }
}
// The same in two parts for bf16, the second the rounded remainder of the first: 2^-16.
template <typename T> struct Split {
    Frag<T> p, rest;
    Split() = default;
    __device__ __forceinline__ Split(const f16 &x, int c) : p(part_of<T>(x, c)) {
        if constexpr (sizeof(T) == 2) {
            const u4 w = __builtin_bit_cast(u4, p);
            la::f8 y;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[j] = x[8 * c + j] - __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
            rest = __builtin_convertvector(y, bf8);
        }
    }
};
template <typename T> __device__ __forceinline__ void mma(f16 &acc, const Frag<T> &a, const Split<T> &b) {
    mma(acc, a, b.p);
    if constexpr (sizeof(T) == 2) mma(acc, a, b.rest);
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

// Whether the thread's share of a tile of ROWS rows holds a NaN or Inf.
template <typename T, int ROWS, int W> __device__ __forceinline__ bool share_not_finite(const char *tile) {
    constexpr int PIECES = ROWS * Tile<T, W>::kPer;
    typedef unsigned short us2 __attribute__((ext_vector_type(2)));
    us2 most = us2(0);  // the upper 16 bits say it for fp32 as well
#pragma unroll
    for (int j = 0; j < (PIECES + kSoftmaxThreads - 1) / kSoftmaxThreads; ++j) {
        const int id = (int)threadIdx.x + j * kSoftmaxThreads;
        if (PIECES < kSoftmaxThreads && id >= PIECES) break;
        const u4 w = *reinterpret_cast<const u4 *>(tile + 16 * id);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            most = __builtin_elementwise_max(most, __builtin_bit_cast(us2, w[i] & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fff0000u)));
    }
    return most[0] >= 0x7f80 || most[1] >= 0x7f80;
}

// ROWS rows × W columns of a strided matrix into an LDS tile, by four wavefronts; zeros past the rows and columns there are.
// VEC: straight into LDS, 16 bytes a lane, through a buffer that ends with the last row; the instructions are written out, for the
// compiler would have every later read of LDS wait for a load that it knows to go there, also one from the other
// buffer. A wavefront waits for its own with landed() before the barrier that hands the tile over. The compiler puts no wait states
// into written-out code: one has to lie between a scalar write of m0 and the load that goes to LDS by it, five between a vector
// instruction's write of a scalar register (readfirstlane, a spilled one's readlane) and a load that reads it. m0 is a reserved
// register that the compiler writes right before each use of its own, so none of its values can be lost here. Otherwise element by
// element through registers.
template <typename T, int ROWS, int W, bool VEC> struct Loader {
    using X = Tile<T, W>;
    static constexpr int E = kE<T>, PIECES = ROWS * X::kPer, N = (PIECES + kSoftmaxThreads - 1) / kSoftmaxThreads;
    static_assert(PIECES % kSoftmaxThreads == 0 || (PIECES < kSoftmaxThreads && PIECES % 64 == 0), "whole instructions");
    // A workgroup's threads cover kStep rows at a time. Where a row's turn repeats after as many, one offset serves all pieces.
    static constexpr int kStep = kSoftmaxThreads / X::kPer, kOffsets = kStep % 16 == 0 ? 1 : N;
    uint32_t at[VEC ? kOffsets : 1];  // of the lane's pieces, in bytes from row 0
    uint32_t stride;
    int cols;
    // a tile is loaded by 256 threads; of a workgroup of 512, each half loads its own
    __device__ static __forceinline__ int thread() { return (int)threadIdx.x % kSoftmaxThreads; }
    __device__ __forceinline__ Loader(uint32_t stride_, int cols_) : stride(stride_), cols(cols_) {
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < kOffsets; ++j) {
                const int id = thread() + j * kSoftmaxThreads, r = id / X::kPer, c = (id % X::kPer ^ X::turn(r)) * E;
                at[j] = c < cols ? (r * stride + c) * (uint32_t)sizeof(T) : kOutside;
            }
        }
    }
    // first: row 0 of the tile, column 0, the same in every lane; rows: how many there are from it on
    __device__ __forceinline__ void operator()(const T *first, int rows, char *tile) const {
        rows = rows > ROWS ? ROWS : rows;
        const uint32_t bytes = rows > 0 ? (uint32_t)((rows - 1) * stride + cols) * (uint32_t)sizeof(T) : 0u;
        if constexpr (VEC) {
            const uint64_t a = reinterpret_cast<uint64_t>(first);
            const u4 buf = {(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                            (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
                            (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00027000u};
            const int w = la::wave_id() % (kSoftmaxThreads / 64);
            if (PIECES < kSoftmaxThreads && w * 64 >= PIECES) return;
            const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)tile + w * 1024;
#pragma unroll
            for (int j = 0; j < N; ++j)
                asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                             :
                             : "s"(lds + j * kSoftmaxThreads * 16), "v"(at[kOffsets == 1 ? 0 : j]), "s"(buf),
                               "s"(kOffsets == 1 ? j * kStep * stride * (uint32_t)sizeof(T) : 0u)
                             : "memory");
        } else {
            const Buffer buf = la::buffer_of(first, bytes);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int id = thread() + j * kSoftmaxThreads, r = id / X::kPer, c = (id % X::kPer ^ X::turn(r)) * E;
                if (PIECES < kSoftmaxThreads && id >= PIECES) break;
                T e[E];
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const uint32_t off = r < rows && c + k < cols ? (r * stride + c + k) * (uint32_t)sizeof(T) : kOutside;
                    if constexpr (sizeof(T) == 2) e[k] = (T)__builtin_amdgcn_raw_buffer_load_b16(buf, off, 0, 0);
                    else e[k] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(buf, off, 0, 0));
                }
                u4 w;
                __builtin_memcpy(&w, e, sizeof(w));
                *reinterpret_cast<u4 *>(tile + 16 * id) = w;
            }
        }
    }
};
// 32 values from `first` on into LDS, one a lane, by one wavefront; zeros past the first `rows`.
__device__ __forceinline__ void load_stats(const float *first, int rows, char *lds) {
    const int l = threadIdx.x & 63;
    const uint64_t a = reinterpret_cast<uint64_t>(first);
    const u4 buf = {(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                    (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
                    (uint32_t)__builtin_amdgcn_readfirstlane(rows > 32 ? 128 : rows > 0 ? rows * 4 : 0), 0x00027000u};
    if (l < 32)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
                     :
                     : "s"((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds), "v"(l * 4u), "s"(buf)
                     : "memory");
}
// The wavefront's loads into LDS are there, but for the last `left`.
template <int left = 0> __device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(%0)" ::"i"(left) : "memory"); }

// The value of the lane 32 away.
__device__ __forceinline__ float other_half(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float((threadIdx.x & 32) ? a[0] : a[1]);
}

// Weights are 2^(scale_of(scale)·s − maximum) of scores s of a product's one operand as for_scale() leaves it: negated for a negative
// scale, zeros for a scale of 0. So the factor is above 0 and finite (a scale of more than 2^128 / log2 e counts as that), and masked
// scores of −inf stay what they are.
__device__ __forceinline__ float scale_of(float scale) {
    return scale == 0.0f ? 1.0f : __builtin_fminf(__builtin_fabsf(scale) * kLog2e, 3.40282347e38f);
}
template <typename F, int N> __device__ __forceinline__ void for_scale(F (&f)[N], float scale) {
    if (scale > 0.0f) return;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = scale < 0.0f ? -f[i] : F(0.0f);
}

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
