// linattn_step.hip — linear attention with a per-head decay, one token on a stored state.
//
// S ← e^g S + v kᵀ, o = scale·S q per (row, head) (page "Mambaとは？Transformer以外の系列モデル", section training、
// prefill、decodeでは計算の姿が違う). The state's read and write are the cost: 8·P·N bytes per head against 5·P·N
// operations. A workgroup takes 64 rows of P of one head; LR lanes share a row of N in 16-byte pieces, so every load
// and store of a wavefront covers whole rows, and all of a lane's loads are issued before the first is used. 512 rows of
// 64 heads, N 128, P 64 (2.16 GB) take 416 us: 5.2 TB/s, what a copy reaches. One row of 24 heads takes 5.3 us on the
// device, and the call 11.5 us on the host.
#include "linattn_common.h"

namespace ssm {
namespace la {
namespace {

constexpr int kRows = 64;  // rows of P per workgroup, 16 per wavefront

template <typename T, int LR, int NV>
__global__ __launch_bounds__(kThreads) void la_step_kernel(float *state, LinAttnLaunch a, bool vec) {
    constexpr int RW = 64 / LR, U = 16 / RW;  // rows per wavefront at once, and passes over them
    const int npb = (a.P + kRows - 1) / kRows;
    int64_t id = work_index(blockIdx.x, gridDim.x);
    const int pb = (int)(id % npb);
    id /= npb;
    const int h = (int)(id % a.H), grp = h / (a.H / a.G);
    const int64_t ib = id / a.H;
    const int w = wave_id(), l = threadIdx.x & 63, lr = l % LR;
    const int p0 = pb * kRows + 16 * w + l / LR;

    float *sp = state + (ib * a.H + h) * (int64_t)a.P * a.N;
    const T *qp = static_cast<const T *>(a.q) + ib * a.q_b + grp * a.q_h;
    const T *kp = static_cast<const T *>(a.k) + ib * a.k_b + grp * a.k_h;
    const T *vp = static_cast<const T *>(a.v) + ib * a.v_b + h * a.v_h;
    T *op = static_cast<T *>(a.o) + (ib * a.H + h) * (int64_t)a.P;

    f4 s[U][NV];
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = p0 + u * RW;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int n = 4 * (lr + LR * i);
            s[u][i] = f4{0, 0, 0, 0};
            if (p < a.P) {
                if (vec) {
                    if (n < a.N) s[u][i] = *reinterpret_cast<const f4 *>(sp + (int64_t)p * a.N + n);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (n + r < a.N) s[u][i][r] = sp[(int64_t)p * a.N + n + r];
                }
            }
        }
        v[u] = p < a.P ? widen(vp[p]) : 0.0f;
    }
    f4 q[NV], k[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int n = 4 * (lr + LR * i) + r;
            q[i][r] = n < a.N ? widen(qp[n]) : 0.0f;
            k[i][r] = n < a.N ? widen(kp[n]) : 0.0f;
        }
    const float gv = a.g_per_step ? a.g[ib * a.H + h] : a.g[h];
    const float decay = exp_of(log_decay(gv));
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = p0 + u * RW;
        float o = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int n = 4 * (lr + LR * i);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                s[u][i][r] = __builtin_fmaf(decay, s[u][i][r], v[u] * k[i][r]);
                o = n + r < a.N ? __builtin_fmaf(s[u][i][r], q[i][r], o) : o;
            }
            if (p < a.P) {
                if (vec) {
                    if (n < a.N) *reinterpret_cast<f4 *>(sp + (int64_t)p * a.N + n) = s[u][i];
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (n + r < a.N) sp[(int64_t)p * a.N + n + r] = s[u][i][r];
                }
            }
        }
#pragma unroll
        for (int d = 1; d < LR; d <<= 1) o += __shfl_xor(o, d);
        if (lr == 0 && p < a.P) op[p] = narrow<T>(a.scale * o);
    }
}

template <typename T>
hipError_t step(float *state, const LinAttnLaunch &p, hipStream_t stream) {
    const dim3 grid((unsigned)(p.b * p.H * ((p.P + kRows - 1) / kRows)));
    const bool vec = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(state) % 16 == 0;
    if (p.N <= 16) la_step_kernel<T, 4, 1><<<grid, kThreads, 0, stream>>>(state, p, vec);
    else if (p.N <= 32) la_step_kernel<T, 8, 1><<<grid, kThreads, 0, stream>>>(state, p, vec);
    else if (p.N <= 64) la_step_kernel<T, 16, 1><<<grid, kThreads, 0, stream>>>(state, p, vec);
    else la_step_kernel<T, 16, 2><<<grid, kThreads, 0, stream>>>(state, p, vec);
    return hipGetLastError();
}

}  // namespace
}  // namespace la

hipError_t launch_linattn_step(float *state, const LinAttnLaunch &p, hipStream_t stream) {
    return p.bf16 ? la::step<uint16_t>(state, p, stream) : la::step<float>(state, p, stream);
}

}  // namespace ssm
