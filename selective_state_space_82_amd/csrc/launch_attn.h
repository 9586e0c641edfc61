// launch_attn.h — launch arguments and launchers of linear attention and layer norm, apart from launch.h's so that the scan's
// measurements, which go by the sources they are of, do not turn on them.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ssm {

// Linear attention with a per-head decay (validated by the ABI layer). The steps are cut into n_seg segments of
// seg_chunks chunks of 64; S and E are the segments' states and adjoints, [b·H][n_seg][⌈P/64⌉·64][NT] floats with
// NT = linattn_nt(N), first the segments' own, then those entering (S) and leaving (E) them.
struct LinAttnLaunch {
    const void *q, *k, *v, *dout;
    const float *g;
    bool g_per_step;
    float scale;
    const float *initial_state, *d_final_state;
    const int32_t *lengths;
    void *o, *dq, *dk, *dv;
    float *dg, *final_state, *d_initial_state;
    int64_t b, L;
    int H, G, N, P;
    bool bf16;
    int64_t q_b, q_t, q_h, k_b, k_t, k_h, v_b, v_t, v_h, do_b, do_t, do_h;  // elements
    int64_t seg_chunks, n_seg;
    float *S, *E;
    double *gsum;          // [b·H][n_seg] sums of g
    uint32_t *bad;         // [b·H][n_seg][⌈P/64⌉][8 wavefronts]: whether the state a segment leaves holds a NaN or Inf
    float *dg_steps;       // [b][L][H] when g_per_step is false
    float *dq_part, *dk_part;  // [b][L][H][N] when G < H
    bool vec;              // every input and output row takes 16-byte accesses at multiples of 16 bytes
};
// HIP takes fewer than 2^32 threads to a launch; the ABI layer refuses what would need more.
inline bool launchable(int64_t workgroups, int64_t threads) { return workgroups <= ((INT64_C(1) << 32) - 1) / threads; }
constexpr int kLinAttnThreads = 256, kLinAttnOutThreads = 512;
// Value columns per workgroup of the segment states' walk, 16 to a wavefront.
inline int64_t linattn_cols(int64_t P) { return P > 64 ? 128 : 64; }
inline int linattn_nt(int64_t N) { return N <= 32 ? 32 : N <= 64 ? 64 : 128; }
hipError_t launch_linattn_fwd(const LinAttnLaunch &p, hipStream_t stream);
hipError_t launch_linattn_bwd(const LinAttnLaunch &p, hipStream_t stream);
hipError_t launch_linattn_step(float *state, const LinAttnLaunch &p, hipStream_t stream);
// The own states of the first n_states segments and the own adjoints of those from first_adjoint on, in one launch.
hipError_t launch_linattn_states(const LinAttnLaunch &p, int64_t n_states, int64_t first_adjoint, hipStream_t stream);
// From own states (and, if `adjoint`, own adjoints) to those entering (leaving) the segments, in place, in one launch.
hipError_t launch_linattn_carry(const LinAttnLaunch &p, bool adjoint, hipStream_t stream);

// Layer norm (validated by the ABI layer).
struct NormLaunch {
    const void *x, *dy;
    const float *w, *bias, *mean_in, *rstd_in;
    void *y;                 // dx in the gradient
    float *mean, *rstd, *dw, *dbias;
    int64_t rows, d, w_rows, x_stride, dy_stride;
    float eps;
    bool bf16;
    float *part;             // gradient: partial sums of dw, dbias
    bool vec;                // 16-byte accesses allowed on every row
};
// Threads of a workgroup; there is one at least for each weight row.
inline int64_t layernorm_threads(int64_t d) { return d > 4096 ? 1024 : 256; }
hipError_t launch_layernorm_fwd(const NormLaunch &p, hipStream_t stream);
hipError_t launch_layernorm_bwd(const NormLaunch &p, hipStream_t stream);
int64_t layernorm_part_floats(int64_t rows, int64_t d, int64_t w_rows);

}  // namespace ssm
