// layernorm.hip — layer norm and its gradient.
//
// The norm of the Mamba block (page "Mambaとは？Transformer以外の系列モデル", section Mamba blockのarchitecture), or of
// each head's output with a weight row per head. y = w ⊙ x̂ + bias, x̂ = (x − μ)·r, r = 1/sqrt(σ² + eps);
//     dx = r·(w ⊙ dy − avg(w ⊙ dy) − x̂·avg(w ⊙ dy ⊙ x̂)),  dw = Σ_rows dy ⊙ x̂,  dbias = Σ_rows dy.
// Memory bounds both: a row is read once, into the registers of the LR lanes that share it (K 16-byte pieces each),
// so that the mean, the centred variance and the output come from one read. A workgroup keeps to rows of one weight
// row and walks them with that row's weight, bias and partial dw, dbias in registers. Forward, 32768 rows of 2048 in bf16:
// 64 us (4.2 TB/s; a copy of as much takes 52). Gradient, 8192 rows of 768 in fp32: 18 us and 4.5 us for the sum of the
// partial rows (a copy of as much 15); 524288 rows of 128 in bf16 with 32 weight rows: 88 us (4.6 TB/s; a copy 78).
#include <type_traits>

#include "device_common.h"
#include "launch_attn.h"

namespace ssm {
namespace ln {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f8 __attribute__((ext_vector_type(8)));

template <typename T> constexpr int kV = 16 / sizeof(T);

// A 16-byte piece of a row as fp32, zeros past d.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load_piece(const T *row, int c, int d) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if constexpr (VEC) {
        if (c < d) w = *reinterpret_cast<const uint4 *>(row + c);
    } else {
        T e[kV<T>];
#pragma unroll
        for (int j = 0; j < kV<T>; ++j) e[j] = c + j < d ? row[c + j] : (T)0;
        __builtin_memcpy(&w, e, sizeof(w));
    }
    return w;
}
template <typename T> __device__ __forceinline__ void spread(const uint4 &w, float *f);
template <> __device__ __forceinline__ void spread<float>(const uint4 &w, float *f) {
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y); f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
}
template <> __device__ __forceinline__ void spread<uint16_t>(const uint4 &w, float *f) {
    f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_piece(T *row, int c, int d, const float *f) {
    if constexpr (VEC) {
        if (c < d) {
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<f4 *>(row + c) = f4{f[0], f[1], f[2], f[3]};
            } else {
                *reinterpret_cast<bf8 *>(row + c) =
                    __builtin_convertvector((f8{f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]}), bf8);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < kV<T>; ++j)
            if (c + j < d) row[c + j] = narrow<T>(f[j]);
    }
}

// Sums of two values over the LR lanes of a row, for all of them. `buf`: a row for each parity of calls, so that one
// barrier per call is enough.
template <int LR>
__device__ __forceinline__ void row_sums(float &u, float &v, float2 (*buf)[16], int &turn) {
#pragma unroll
    for (int d = 1; d < (LR < 64 ? LR : 64); d <<= 1) {
        u += __shfl_xor(u, d);
        v += __shfl_xor(v, d);
    }
    if constexpr (LR > 64) {
        float2 *b = buf[turn];
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) b[threadIdx.x >> 6] = make_float2(u, v);
        __syncthreads();
        u = v = 0.0f;
#pragma unroll
        for (int i = 0; i < LR / 64; ++i) {
            u += b[i].x;
            v += b[i].y;
        }
    }
}

// Columns of a lane: pieces lr, lr + LR, ... of the row.
template <typename T, int LR, int K> struct Lay {
    static constexpr int V = kV<T>, E = K * V, THREADS = LR > 256 ? LR : 256, SLOTS = THREADS / LR;
    __device__ static int col(int i) { return ((int)(threadIdx.x % LR) + LR * i) * V; }
};

// Rows of a workgroup: weight row blockIdx.x mod w_rows, every SLOTS·(workgroups per weight row)-th of its rows.
struct Rows {
    int64_t wr, first, step, count;
    __device__ Rows(const NormLaunch &a, int slots, int slot) {
        wr = blockIdx.x % a.w_rows;
        const int64_t per = gridDim.x / a.w_rows;
        first = (blockIdx.x / a.w_rows) * slots + slot;
        step = per * slots;
        count = a.rows / a.w_rows;
    }
};

template <typename T, int LR, int K, bool VEC>
__global__ __launch_bounds__((Lay<T, LR, K>::THREADS)) void norm_fwd_kernel(NormLaunch a) {
    typedef Lay<T, LR, K> Y;
    __shared__ float2 s_buf[2][16];
    int turn = 0;
    const int d = (int)a.d, lr = threadIdx.x % LR;
    const Rows rows(a, Y::SLOTS, threadIdx.x / LR);
    const float inv_d = 1.0f / (float)d;
    float w[Y::E], bias[Y::E];
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
        for (int j = 0; j < Y::V; ++j) {
            const int c = Y::col(i) + j;
            w[i * Y::V + j] = a.w && c < d ? a.w[rows.wr * d + c] : 1.0f;
            bias[i * Y::V + j] = a.bias && c < d ? a.bias[rows.wr * d + c] : 0.0f;
        }
    uint4 ahead[K];  // the next row's pieces, fetched while this one is computed
    auto fetch = [&](int64_t m) {
        const T *x = static_cast<const T *>(a.x) + (m * a.w_rows + rows.wr) * a.x_stride;
#pragma unroll
        for (int i = 0; i < K; ++i)
            ahead[i] = m < rows.count ? load_piece<T, VEC>(x, Y::col(i), d) : make_uint4(0, 0, 0, 0);
    };
    fetch(rows.first);
    // all lanes of a workgroup take as many turns as its first row, so that its barriers meet
    for (int64_t m0 = rows.first - threadIdx.x / LR; m0 < rows.count; m0 += rows.step) {
        const int64_t m = m0 + threadIdx.x / LR;
        const bool live = m < rows.count;
        const int64_t row = m * a.w_rows + rows.wr;
        float f[Y::E];
        float sum = 0.0f, none = 0.0f;
#pragma unroll
        for (int i = 0; i < K; ++i) spread<T>(ahead[i], f + i * Y::V);
        fetch(m + rows.step);
#pragma unroll
        for (int e = 0; e < Y::E; ++e) sum += f[e];
        row_sums<LR>(sum, none, s_buf, turn);
        const float mean = sum * inv_d;
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int j = 0; j < Y::V; ++j) {
                const int e = i * Y::V + j;
                f[e] -= mean;
                sq = Y::col(i) + j < d ? __builtin_fmaf(f[e], f[e], sq) : sq;
            }
        row_sums<LR>(sq, none, s_buf, turn);
        const float rstd = 1.0f / sqrtf(sq * inv_d + a.eps);
        if (!live) continue;
        if (lr == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        T *y = static_cast<T *>(a.y) + row * d;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            float o[Y::V];
#pragma unroll
            for (int j = 0; j < Y::V; ++j) {
                const int e = i * Y::V + j;
                o[j] = __builtin_fmaf(f[e] * rstd, w[e], bias[e]);
            }
            store_piece<T, VEC>(y, Y::col(i), d, o);
        }
    }
}

template <typename T, int LR, int K, bool VEC>
__global__ __launch_bounds__((Lay<T, LR, K>::THREADS)) void norm_bwd_kernel(NormLaunch a) {
    typedef Lay<T, LR, K> Y;
    __shared__ float2 s_buf[2][16];
    __shared__ float s_part[Y::SLOTS > 1 ? (Y::SLOTS * LR * Y::E) : 1];
    int turn = 0;
    const int d = (int)a.d, slot = threadIdx.x / LR;
    const Rows rows(a, Y::SLOTS, slot);
    const float inv_d = 1.0f / (float)d;
    float w[Y::E], dw[Y::E], db[Y::E];
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
        for (int j = 0; j < Y::V; ++j) {
            const int c = Y::col(i) + j, e = i * Y::V + j;
            w[e] = a.w && c < d ? a.w[rows.wr * d + c] : 1.0f;
            dw[e] = db[e] = 0.0f;
        }
    uint4 px[K], pd[K];  // the next row's pieces, fetched while this one is computed
    float next_mean, next_rstd;
    auto fetch = [&](int64_t m) {
        const int64_t row = m * a.w_rows + rows.wr;
        const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
        const T *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
        const bool live = m < rows.count;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            px[i] = live ? load_piece<T, VEC>(x, Y::col(i), d) : make_uint4(0, 0, 0, 0);
            pd[i] = live ? load_piece<T, VEC>(dy, Y::col(i), d) : make_uint4(0, 0, 0, 0);
        }
        next_mean = live ? a.mean_in[row] : 0.0f;
        next_rstd = live ? a.rstd_in[row] : 0.0f;
    };
    fetch(rows.first);
    for (int64_t m0 = rows.first - slot; m0 < rows.count; m0 += rows.step) {
        const int64_t m = m0 + slot;
        const bool live = m < rows.count;
        const int64_t row = m * a.w_rows + rows.wr;
        const float mean = next_mean, rstd = next_rstd;
        float xh[Y::E], g[Y::E];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            spread<T>(px[i], xh + i * Y::V);
            spread<T>(pd[i], g + i * Y::V);
        }
        fetch(m + rows.step);
#pragma unroll
        for (int i = 0; i < K; ++i) {
#pragma unroll
            for (int j = 0; j < Y::V; ++j) {
                const int e = i * Y::V + j;
                xh[e] = Y::col(i) + j < d ? (xh[e] - mean) * rstd : 0.0f;
                dw[e] = __builtin_fmaf(g[e], xh[e], dw[e]);
                db[e] += g[e];
                g[e] *= w[e];
                s1 += g[e];
                s2 = __builtin_fmaf(g[e], xh[e], s2);
            }
        }
        row_sums<LR>(s1, s2, s_buf, turn);
        if (!live) continue;
        s1 *= inv_d;
        s2 *= inv_d;
        T *dx = static_cast<T *>(a.y) + row * d;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            float o[Y::V];
#pragma unroll
            for (int j = 0; j < Y::V; ++j) {
                const int e = i * Y::V + j;
                o[j] = rstd * (g[e] - s1 - xh[e] * s2);
            }
            store_piece<T, VEC>(dx, Y::col(i), d, o);
        }
    }
    if (!a.part) return;
    // the workgroup's dw and dbias: over its slots in order
    float *out = a.part + 2 * (int64_t)blockIdx.x * d;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float *v = which ? db : dw;
        if constexpr (Y::SLOTS > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < Y::E; ++e) s_part[e * Y::THREADS + threadIdx.x] = v[e];
            __syncthreads();
            if (slot == 0)
#pragma unroll
                for (int e = 0; e < Y::E; ++e) {
                    float t = 0.0f;
#pragma unroll 4
                    for (int s = 0; s < Y::SLOTS; ++s) t += s_part[e * Y::THREADS + s * LR + threadIdx.x];
                    v[e] = t;
                }
        }
        if (slot == 0)
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int j = 0; j < Y::V; ++j)
                    if (Y::col(i) + j < d) out[which * d + Y::col(i) + j] = v[i * Y::V + j];
    }
}

// dw and dbias from the workgroups' partial sums: 16 columns of one weight row per workgroup (64-byte pieces of the
// partial rows), 64 interleaved runs of partial sums each, joined in order. With 64 columns and 4 runs, 12 workgroups of
// 256 dependent loads each took 78 us for 768 columns and 1024 partial rows.
__global__ __launch_bounds__(1024) void norm_part_sum_kernel(const float *part, float *dw, float *dbias, int64_t d,
                                                             int64_t w_rows, int64_t per) {
    __shared__ float s[2][64][17];
    const int64_t blocks = (d + 15) / 16;
    const int col = threadIdx.x & 15, run = threadIdx.x >> 4;
    for (int64_t block = blockIdx.x; block < w_rows * blocks; block += gridDim.x) {
        const int64_t wr = block / blocks, c = block % blocks * 16 + col;
        float u = 0.0f, v = 0.0f;
        if (c < d) {
#pragma unroll 4
            for (int64_t i = run; i < per; i += 64) {
                const float *p = part + 2 * (i * w_rows + wr) * d + c;
                u += p[0];
                v += p[d];
            }
        }
        s[0][run][col] = u;
        s[1][run][col] = v;
        for (int h = 32; h > 0; h >>= 1) {
            __syncthreads();
            if (run < h) {
                s[0][run][col] += s[0][run + h][col];
                s[1][run][col] += s[1][run + h][col];
            }
        }
        if (run == 0 && c < d) {
            if (dw) dw[wr * d + c] = s[0][0][col];
            if (dbias) dbias[wr * d + c] = s[1][0][col];
        }
        __syncthreads();  // every sum of this block is read
    }
}

__global__ __launch_bounds__(256) void norm_zero_kernel(float *dw, float *dbias, int64_t n) {
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += gridDim.x * (int64_t)256) {
        if (dw) dw[i] = 0.0f;
        if (dbias) dbias[i] = 0.0f;
    }
}

// Workgroups per weight row: enough to give the device `most` workgroups in all, no more than have rows.
int64_t groups(int64_t rows, int64_t w_rows, int slots, int64_t most) {
    const int64_t need = (rows / w_rows + slots - 1) / slots;
    const int64_t cap = most / w_rows > 1 ? most / w_rows : 1;
    return need < cap ? need : cap;
}
constexpr int64_t kFwdGroups = 2048;
// Workgroups of the launches that walk over columns in steps of the grid, far below HIP's limit of threads.
unsigned walking(int64_t n) { return (unsigned)(n < 65536 ? n : 65536); }
// The gradient's workgroups also write a row of partial sums each: 512 of them, but 1024 where a lane has one piece of a row
// of one wavefront or less, whose registers (under 90) let that many be resident at once. Over 2^25 elements, 1024 against 512:
//   one piece a lane: fp32 d 64 81 us against 87, 192 78 against 108, 256 82 against 88; bf16 d 64 50 against 65, 128 43
//   against 44, 320 45 against 57, 512 42 against 43;
//   the rest: fp32 d 128 86 us against 81, 320 82 against 86, 512 86 against 79, 768 91 against 83, 2048 90 against 80, 8192 125
//   against 102; bf16 d 192 56 against 48, 256 54 against 47, 768 51 against 44, 2048 50 against 50, 8192 104 against 70.
template <int LR, int K> constexpr int64_t kBwdGroups = K == 1 && LR <= 64 ? 1024 : 512;
// the most of them for either type: one piece a lane holds rows of up to 64·8
int64_t most_bwd_groups(int64_t d) { return d <= 512 ? 1024 : 512; }

// f(LR, K): the lanes of a row and their pieces; at most 16 elements of a row to a lane, so that the gradient's row,
// its weight and its two partial sums stay in registers with the next row on its way. Past d = 8192 they do not quite: the
// 1024 lanes have 128 registers each, and the gradient spills 59 (bf16) to 113 (fp32, rows of odd width) of them.
template <typename T, typename F> hipError_t by_width(int64_t d, F f) {
    const int64_t n = (d + kV<T> - 1) / kV<T>;
#define SSM_LN(LR, K) if (n <= (LR) * (K)) return f(std::integral_constant<int, LR>{}, std::integral_constant<int, K>{})
    SSM_LN(16, 1);
    SSM_LN(16, 2);
    SSM_LN(64, 1);
    SSM_LN(64, 2);
    if constexpr (sizeof(T) == 4) SSM_LN(64, 4);
    if constexpr (sizeof(T) == 2) SSM_LN(256, 1);  // fp32: no wider than the one before
    SSM_LN(256, 2);
    if constexpr (sizeof(T) == 4) SSM_LN(256, 4);
    if constexpr (sizeof(T) == 2) SSM_LN(1024, 1);
    SSM_LN(1024, 2);
    if constexpr (sizeof(T) == 4) SSM_LN(1024, 4);
#undef SSM_LN
    return hipErrorInvalidValue;
}

template <typename T> hipError_t fwd(const NormLaunch &p, hipStream_t stream) {
    return by_width<T>(p.d, [&](auto lr, auto k) {
        constexpr int LR = decltype(lr)::value, K = decltype(k)::value;
        typedef Lay<T, LR, K> Y;
        const int64_t n = groups(p.rows, p.w_rows, Y::SLOTS, kFwdGroups) * p.w_rows;
        if (p.vec) norm_fwd_kernel<T, LR, K, true><<<dim3((unsigned)n), Y::THREADS, 0, stream>>>(p);
        else norm_fwd_kernel<T, LR, K, false><<<dim3((unsigned)n), Y::THREADS, 0, stream>>>(p);
        return hipGetLastError();
    });
}

template <typename T> hipError_t bwd(const NormLaunch &p, hipStream_t stream) {
    return by_width<T>(p.d, [&](auto lr, auto k) {
        constexpr int LR = decltype(lr)::value, K = decltype(k)::value;
        typedef Lay<T, LR, K> Y;
        const int64_t per = groups(p.rows, p.w_rows, Y::SLOTS, kBwdGroups<LR, K>);
        const dim3 grid((unsigned)(per * p.w_rows));
        if (p.vec) norm_bwd_kernel<T, LR, K, true><<<grid, Y::THREADS, 0, stream>>>(p);
        else norm_bwd_kernel<T, LR, K, false><<<grid, Y::THREADS, 0, stream>>>(p);
        hipError_t e = hipGetLastError();
        if (e == hipSuccess && p.part) {
            norm_part_sum_kernel<<<dim3(walking(p.w_rows * ((p.d + 15) / 16))), 1024, 0, stream>>>(
                p.part, p.dw, p.dbias, p.d, p.w_rows, per);
            e = hipGetLastError();
        }
        return e;
    });
}

}  // namespace
}  // namespace ln

int64_t layernorm_part_floats(int64_t rows, int64_t d, int64_t w_rows) {
    // the most workgroups any layout launches: one row each, or the cap, or one per weight row
    const int64_t per = ln::groups(rows, w_rows, 1, ln::most_bwd_groups(d));
    return 2 * per * w_rows * d;
}

hipError_t launch_layernorm_fwd(const NormLaunch &p, hipStream_t stream) {
    return p.bf16 ? ln::fwd<uint16_t>(p, stream) : ln::fwd<float>(p, stream);
}

hipError_t launch_layernorm_bwd(const NormLaunch &p, hipStream_t stream) {
    if (p.rows == 0) {
        const int64_t n = p.w_rows * p.d;
        ln::norm_zero_kernel<<<dim3(ln::walking((n + 255) / 256)), 256, 0, stream>>>(p.dw, p.dbias, n);
        return hipGetLastError();
    }
    return p.bf16 ? ln::bwd<uint16_t>(p, stream) : ln::bwd<float>(p, stream);
}

}  // namespace ssm
