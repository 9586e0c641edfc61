// launch_softmax.h — launch arguments and launchers of softmax attention (prompts, their gradient, one token over a paged
// cache) and of the cache's append and the position rotation.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "softmax_index.h"

namespace ssm {

// Attention over prompts and its gradient (validated by the ABI layer).
struct SoftmaxLaunch {
    const void *q, *k, *v, *o_in, *dout;
    const float *lse_in;
    float scale;
    bool causal, bf16;
    AttnRows rows;
    int H, G, D;
    int64_t q_b, q_t, q_h, k_b, k_t, k_h, v_b, v_t, v_h, do_b, do_t, do_h;  // elements
    void *o, *dq, *dk, *dv;
    float *lse;
    float *stats;  // gradient: per head and query, [H][tokens][2]: lse·log2 e and scale·delta
    bool vec;      // every row takes 16-byte accesses
};
// Queries of a workgroup of the forward kernel and of the gradients' for the queries, and keys of the gradients' for the keys.
int softmax_fwd_block(const SoftmaxLaunch &p);
int softmax_dq_block(const SoftmaxLaunch &p);
int softmax_dkv_block(const SoftmaxLaunch &p);
constexpr int kSoftmaxThreads = 256;
hipError_t launch_softmax_fwd(const SoftmaxLaunch &p, hipStream_t stream);
hipError_t launch_softmax_bwd(const SoftmaxLaunch &p, hipStream_t stream);

// One new token a row over a paged cache (validated by the ABI layer). The keys of a row are cut into at most `splits` pieces
// of at least `least` tokens, joined by a second launch where splits > 1.
struct SoftmaxStepLaunch {
    const void *q, *k_cache, *v_cache;
    Pages pages;
    const int32_t *lengths;
    float scale;
    bool bf16;
    int64_t b;
    int H, G, D;
    int64_t q_b, q_h, k_page, v_page;  // elements
    void *o;
    float *lse;
    int splits, least;
    float *part;  // [b][H][splits][D + 2]: maximum, sum, unnormalised output
    bool vec;
};
constexpr int kStepTile = 64;  // keys a wavefront takes at once
hipError_t launch_softmax_step(const SoftmaxStepLaunch &p, hipStream_t stream);

// Rotation by position, and the append to a paged cache (validated by the ABI layer).
struct KvAppendLaunch {
    const void *q, *k, *v;  // q, v may be null
    void *q_out, *k_out;    // may be null
    void *k_cache, *v_cache;  // null: rotation alone
    Pages pages;
    const int32_t *lengths;  // tokens of each row with the new ones; null: as many as are new
    NewTokens tokens;
    const double *freq;      // [rotary / 2], null: no rotation
    int rotary;
    bool interleaved, inverse, bf16, vec;
    int H, G, D;
    int64_t q_b, q_t, q_h, k_b, k_t, k_h, v_b, v_t, v_h;
    int64_t k_page, v_page;
};
constexpr int kAppendThreads = 256;
hipError_t launch_kv_append(const KvAppendLaunch &p, hipStream_t stream);

}  // namespace ssm
