// linattn_common.h — what the kernels of linear attention with a per-head decay share: the launch arguments, the
// chunk geometry, tile staging, and matrix products on fragments of 16×16×32 steps.
//
// Every product is a sum of 16×16 tiles D = A·Bᵀ over a contraction axis taken 32 at a time. Lane l = 16·grp + col
// of a wavefront supplies, for row `col` of A (and of B), 8 of the 32 contraction values, and receives
// D[4·grp + r][col], r < 4. The order of a contraction axis is free as long as both operands use the same:
//   plain    values 8·grp .. 8·grp + 7: one 16-byte LDS read along a row (bf16), which moves 128 bytes a clock (two of
//            8 bytes each: 64);
//   spread   8·(grp % 2) + grp / 2 + 2j, and the same + 16, j < 4: rows two apart, which lie 8 LDS banks apart at the row
//            distances used here, so that the 32 lanes of a transposing read down 16 columns touch 64 different
//            banks (8.5 clocks for 1 KB; in the plain order, where they meet in half of them, 12).
#pragma once

#include <type_traits>

#include "device_common.h"
#include "launch_attn.h"

namespace ssm {
namespace la {

constexpr int kC = 64;        // steps per chunk
constexpr int kPB = 64;       // value columns per workgroup; P is padded to it in scratch
constexpr int kThreads = kLinAttnThreads;  // four wavefronts
// Log-decays below this count as this: e^-1e4 is 0 in fp32, and so is every product with it, while running sums
// stay finite (−inf would turn differences of sums into NaN).
constexpr float kMinG = -1e4f;

typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
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

// The wavefront's number in its workgroup, as a scalar.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }

// Workgroup barrier that orders LDS only: the next chunk's loads and the outputs' stores stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Operand fragment of tile row `row0 + col`, contraction values n0 .. n0+31 along the row.
__device__ __forceinline__ bf8 row_frag(const uint16_t *tile, int stride, int row0, int n0) {
    const int l = threadIdx.x & 63;
    return *reinterpret_cast<const bf8 *>(tile + (row0 + (l & 15)) * stride + n0 + 8 * (l >> 4));
}
__device__ __forceinline__ f8 row_frag(const float *tile, int stride, int row0, int n0) {
    const int l = threadIdx.x & 63;
    const float *p = tile + (row0 + (l & 15)) * stride + n0 + 8 * (l >> 4);
    const f4 u = *reinterpret_cast<const f4 *>(p), v = *reinterpret_cast<const f4 *>(p + 4);
    return __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Operand fragment of tile column n0 + col, contraction values s0 .. s0+31 down the column, in the order plain or
// spread. bf16: the transposing LDS read, which gives lane `col` of 16 lanes column `col` of the 4×16 block whose
// quarter rows they address.
template <bool SPREAD = false> __device__ __forceinline__ bf8 col_frag(const uint16_t *tile, int stride, int s0, int n0) {
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const int l = threadIdx.x & 63, c = l & 15, g = l >> 4;
    const int row = SPREAD ? 8 * (g & 1) + (g >> 1) + 2 * (c >> 2) : 8 * g + (c >> 2);
    const uint16_t *p = tile + (s0 + row) * stride + n0 + 4 * (c & 3);
    const s4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p);
    const s4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + (SPREAD ? 16 : 4) * stride));
    typedef short s8 __attribute__((ext_vector_type(8)));
    const s8 w = __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf8, w);
}
template <bool SPREAD = false> __device__ __forceinline__ f8 col_frag(const float *tile, int stride, int s0, int n0) {
    const int l = threadIdx.x & 63, g = l >> 4;
    const float *p = tile + (s0 + (SPREAD ? 8 * (g & 1) + (g >> 1) : 8 * g)) * stride + n0 + (l & 15);
    f8 r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = p[(SPREAD ? 2 * (j & 3) + 16 * (j >> 2) : j) * stride];
    return r;
}
// Where step s of a chunk stands in the order spread (8·grp + j of its 32).
__device__ __forceinline__ int spread_of(int s) {
    return (s & 32) + 8 * ((s >> 3 & 1) + 2 * (s & 1)) + 4 * (s >> 4 & 1) + (s >> 1 & 3);
}

__device__ __forceinline__ f8 wide(const bf8 &v) { return __builtin_convertvector(v, f8); }
__device__ __forceinline__ f8 wide(const f8 &v) { return v; }
__device__ __forceinline__ f8 join(const f4 &u, const f4 &v) { return __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7); }

// acc += (an fp32 operand)·b in PARTS parts: for bf16 storage the value is cut into bf16 parts, each the rounded
// remainder of those before (relative error at most 2^-8, 2^-16, 2^-24 for 1, 2, 3 parts); for f32 it is one part.
template <int PARTS> struct Parts {
    bf8 p[PARTS];
    Parts() = default;
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
    Whole() = default;
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

// e^v of a running sum or a difference of two: 2^(hi + lo) = 2^hi·(1 + lo·ln 2), so that neither v's nor its product's
// rounding to fp32 is left, which at v = -60 would be 4e-6 of the result. (A factor near 1 keeps 0 and Inf what they are.)
__device__ __forceinline__ float exp_of(double v) {
    const double e = v * 1.4426950408889634074;
    const float hi = (float)e, lo = (float)(e - (double)hi);
    return exp2_fast(hi) * (1.0f + 0.69314718055994530942f * lo);
}

// Inclusive running sum over the 64 lanes of a wavefront, fp64: data-parallel moves inside each row of 16 lanes (lanes
// shifted in from outside add 0), then the totals of the rows before.
template <int CTRL> __device__ __forceinline__ double row_shift(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_running_sum(double v) {
    v += row_shift<0x111>(v);
    v += row_shift<0x112>(v);
    v += row_shift<0x114>(v);
    v += row_shift<0x118>(v);
    const double r0 = lane_value(v, 15), r1 = lane_value(v, 31), r2 = lane_value(v, 47);
    const int row = (threadIdx.x & 63) >> 4;
    return v + (row == 0 ? 0.0 : row == 1 ? r0 : row == 2 ? r0 + r1 : (r0 + r1) + r2);
}

// The clamped log-decay.
__device__ __forceinline__ double log_decay(float v) { return v < kMinG ? (double)kMinG : (double)v; }

// Running sums of g in a chunk, in units of log 2, as fp32 hi + lo, so that their differences keep fp32's accuracy
// however large the sums are; decay(t, s) = e^{c_t − c_s}.
struct Sums {
    float hi[kC], lo[kC];
    __device__ __forceinline__ void set(int t, double c) {
        const double e = c * 1.4426950408889634074;
        const float h = (float)e;
        hi[t] = h;
        lo[t] = (float)(e - (double)h);
    }
};

// What a chunk's decays are needed for: pairs of steps, from the chunk's start (times a factor), to its end, across.
struct Decays {
    Sums c;
    __attribute__((aligned(16))) float in[kC], out[kC];
    float end;
    // By one wavefront, lane t for step t; `out` in the order spread or as the steps are.
    template <bool SPREAD> __device__ __forceinline__ void set(double g, float factor) {
        const int l = threadIdx.x & 63;
        const double sum = wave_running_sum(g), total = lane_value(sum, 63);
        c.set(l, sum);
        in[l] = factor * exp_of(sum);
        out[SPREAD ? spread_of(l) : l] = exp_of(total - sum);
        if (l == 63) end = exp_of(total);
    }
};

// A buffer descriptor of `bytes` from `first` on (the same in every lane): loads outside give 0, stores outside are
// dropped, so a chunk's edge needs no branch (which would make every load wait for the one before).
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void *first, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(first), 0, (int)bytes, 0x00027000);
}
constexpr uint32_t kOutside = 0xfffffff0u;  // past every buffer: 64 rows of 2^24 fp32 elements end below it

// `rows` rows (0 .. 64) of `cols` elements, `stride` elements apart.
template <typename T> __device__ __forceinline__ Buffer rows_buffer(const T *first, uint32_t stride, int rows, int cols) {
    return buffer_of(first, rows > 0 ? (uint32_t)((rows - 1) * stride + cols) * (uint32_t)sizeof(T) : 0u);
}

// The log-decay of the lane's step in a chunk of `rows` rows (0 past them), not yet clamped; first: that of row 0.
__device__ __forceinline__ float load_g(const Buffer &buf, uint32_t stride, int rows) {
    const int l = threadIdx.x & 63;
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buf, l < rows ? l * stride * 4u : kOutside, 0, 0));
}
__device__ __forceinline__ float load_g(const float *first, uint32_t stride, int rows) {
    return load_g(rows_buffer(first, stride, rows, 1), stride, rows);
}

// Rows of a chunk × columns [c0, c0 + W) of a strided array on their way into an LDS tile, zeros past the rows and
// columns there are. VEC: 16-byte accesses at multiples of kVec elements are allowed, `cols` is one of them, and
// rows are at least `cols` apart, so that the buffer's end alone cuts off the rows; otherwise element by element. A
// thread holds its pieces between load and store, so that a chunk is fetched while the one before is computed.
template <typename T, int W, int THREADS, bool VEC> struct Stage {
    static constexpr int V = kVec<T>, PER = W / V, S = W + kPad<T>, PIECES = kC * PER,
                         N = (PIECES + THREADS - 1) / THREADS, STEP = THREADS / PER;  // rows between a thread's pieces
    static_assert(THREADS % PER == 0, "a thread's pieces are in one column");
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    u4 w[N];
    uint32_t at;  // of the first piece, in bytes from row 0
    int c0, cols;
    uint32_t stride;
    __device__ __forceinline__ Stage(uint32_t stride_, int c0_, int cols_) : c0(c0_), cols(cols_), stride(stride_) {
        const int c = c0 + (int)(threadIdx.x % PER) * V;
        at = c < cols && (int)threadIdx.x < PIECES ? (threadIdx.x / PER * stride + c) * (uint32_t)sizeof(T) : kOutside;
    }
    // first: row 0 of the chunk, column 0, the same in every lane
    __device__ __forceinline__ void load(const T *first, int rows) { load(rows_buffer(first, stride, rows, cols), rows); }
    __device__ __forceinline__ void load(const Buffer &buf, int rows) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if constexpr (VEC) {
                w[j] = __builtin_amdgcn_raw_buffer_load_b128(buf, at, j * STEP * stride * (uint32_t)sizeof(T), 0);
            } else {
                const int r = threadIdx.x / PER + j * STEP, c = c0 + (int)(threadIdx.x % PER) * V;
                T e[V];
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const bool mine = r < rows && (int)threadIdx.x < PIECES && c + k < cols;
                    const uint32_t off = mine ? (r * stride + c + k) * (uint32_t)sizeof(T) : kOutside;
                    if constexpr (sizeof(T) == 2) e[k] = (T)__builtin_amdgcn_raw_buffer_load_b16(buf, off, 0, 0);
                    else e[k] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(buf, off, 0, 0));
                }
                __builtin_memcpy(&w[j], e, sizeof(w[j]));
            }
        }
    }
    __device__ __forceinline__ void store(T *tile) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (PIECES % THREADS == 0 || (int)threadIdx.x < PIECES)
                *reinterpret_cast<u4 *>(tile + (threadIdx.x / PER + j * STEP) * S + threadIdx.x % PER * V) = w[j];
        }
    }
};

// Four consecutive results (row r, columns c .. c+3) of dense rows in `buf` (rows_buffer), `stride` elements apart.
template <typename T, bool VEC>
__device__ __forceinline__ void store4(const Buffer &buf, uint32_t stride, int r, int c, int cols, const f4 &v) {
    const uint32_t at = (r * stride + c) * (uint32_t)sizeof(T);  // r is a lane's own
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    if constexpr (VEC) {
        const uint32_t off = c < cols ? at : kOutside;
        if constexpr (sizeof(T) == 2)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, __builtin_convertvector(v, bf4)), buf, off, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), buf, off, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t off = c + j < cols ? at + j * (uint32_t)sizeof(T) : kOutside;
            if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(narrow<T>(v[j]), buf, off, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[j]), buf, off, 0, 0);
        }
    }
}

// Rows of a chunk that starts at step t0, of a row of `len` steps.
__device__ __forceinline__ int rows_of(int64_t t0, int64_t len) {
    const int64_t n = len - t0;
    return n > kC ? kC : n < 0 ? 0 : (int)n;
}

// The chunks of a strided array in order, without products on the way: the place and byte count of the next one's rows,
// of `left` rows in all.
struct Cursor {
    const char *at;
    int64_t step;      // bytes from one chunk to the next
    uint32_t full, row;// bytes of a whole chunk, and between rows
    template <typename T> __device__ __forceinline__ Cursor(const T *first, int64_t stride, int cols)
        : at(reinterpret_cast<const char *>(first)), step(stride * kC * (int64_t)sizeof(T)),
          full((uint32_t)((kC - 1) * stride + cols) * (uint32_t)sizeof(T)), row((uint32_t)stride * (uint32_t)sizeof(T)) {}
    // the chunk's buffer, rows: 0 .. 64 of them; then on to the next
    __device__ __forceinline__ Buffer next(int rows) {
        const Buffer b = buffer_of(at, rows > 0 ? full - (kC - rows) * row : 0u);
        at += step;
        return b;
    }
};
// Rows still to come, counted down by chunks: the next chunk's.
struct RowsLeft {
    int64_t left;
    __device__ __forceinline__ int next() {
        const int n = left > kC ? kC : left < 0 ? 0 : (int)left;
        left -= kC;
        return n;
    }
};

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
