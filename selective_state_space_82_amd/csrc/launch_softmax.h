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
    float *stats;  // gradient: [2][H][tokens]: lse·log2 e and −delta of each head and query
    float *rest;   // gradient with bf16: [splits][H][tokens]: what do·o lacks as delta, of each piece
    float *part;   // results of pieces, where a walk is cut (SoftmaxWork): the forward call's [splits][tokens][H][D], then
                   // maximum and sum [splits][tokens][H][2]; dq's [splits][tokens][H][D]; dk's [splits][tokens][G][D], then dv's
    bool vec;      // every row takes 16-byte accesses
};
constexpr int kSoftmaxThreads = 256;
// Work of a launch: for every sequence and key head `per` times `blocks` blocks (of queries of the heads that share it, or of
// its keys). Workgroups are dealt to the 8 XCDs in turn, and each XCD has an L2 of its own, so that the work on one key head
// should be in one; but sequences may differ in length, so that each should be spread over all. Units are therefore key heads, or,
// where a sequence has fewer than 8, every `parts`-th block of one, and dealt to the XCDs in turn; an XCD takes its units one
// after the other. (Units as runs of neighbours: 9 sequences of 100 to 4096 tokens, 8 key heads, gradient 6.5 ms.)
// Where there are too few of these to fill the device, the tiles that a block walks are cut into up to `splits` pieces of at
// least `least` tiles, a workgroup each, and a second launch joins them.
struct SoftmaxWork {
    int64_t units, each;  // each: workgroups of a unit
    int parts, per, blocks, splits, least;
    bool across;  // an XCD takes the first block of each of its units, then the second of each, ...; otherwise unit by unit
};  // workgroups number less than 2^24
inline SoftmaxWork softmax_work(int64_t b, int64_t G, int64_t per, int64_t blocks, int64_t splits, int64_t least) {
    const int64_t parts = G >= 8 || blocks < 2 ? 1 : ((8 + G - 1) / G < blocks ? (8 + G - 1) / G : blocks);
    const int64_t units = b * G * parts, each = per * splits * ((blocks + parts - 1) / parts);
    // The last unit's longest blocks should not start when all else is done: where a unit does not fill an XCD (32 compute units,
    // two workgroups each) and there are rounds enough for that to matter. (4 sequences of 2048, 24 heads, gradient: 314 us unit
    // by unit, 264 across; 8 of 4096, 32 heads on 8 key heads, forward: 1091 and 1139.)
    return {units, each, (int)parts, (int)per, (int)blocks, (int)splits, (int)least,
            each < 64 && (units + 7) / 8 * each >= 128};
}
inline int64_t softmax_groups(const SoftmaxWork &w) { return (w.units + 7) / 8 * 8 * w.each; }
// Of a workgroup: sequence, key head, which of the `per`, which block counted from the first to be taken, which piece of it;
// false: none.
struct SoftmaxPlace {
    int64_t seq;
    int g, which, block, piece;
};
SSM_BOTH bool softmax_place(const SoftmaxWork &w, int64_t G, uint32_t id, SoftmaxPlace *p) {
    const uint32_t turn = id >> 3, each = (uint32_t)w.each, mine = ((uint32_t)w.units + 7) / 8;  // an XCD's units
    const uint32_t unit = (w.across ? turn % mine : turn / each) * 8 + (id & 7), at = w.across ? turn / mine : turn % each;
    const uint32_t head = unit / (uint32_t)w.parts, part = unit % (uint32_t)w.parts, row = at / (uint32_t)w.splits;
    p->seq = head / (uint32_t)G;
    p->g = (int)(head % (uint32_t)G);
    p->piece = (int)(at % (uint32_t)w.splits);
    p->which = (int)(row % (uint32_t)w.per);
    p->block = (int)(row / (uint32_t)w.per * (uint32_t)w.parts + part);
    return unit < (uint32_t)w.units && p->block < w.blocks;
}
// Tiles of each piece of a walk of `tiles`, and how many pieces it has.
SSM_BOTH int softmax_piece(const SoftmaxWork &w, int tiles, int *pieces) {
    int per = (tiles + w.splits - 1) / w.splits;
    per = per < w.least ? w.least : per;
    *pieces = tiles > per ? (tiles + per - 1) / per : 1;
    return per;
}

// The work of joining a block's pieces: 16 workgroups to a block, 32 lanes to each of its 128 rows.
inline SoftmaxWork softmax_join_work(SoftmaxWork w) {
    w.each = w.each / w.splits * 16;
    w.splits = 16;
    w.across = false;
    return w;
}

// The forward kernel and the gradient's for the queries take 128 queries to a workgroup, the gradient's for the keys 128 keys.
constexpr int kSoftmaxBlock = 128;
constexpr int64_t kSoftmaxLeast = 256;  // keys or queries of a piece
// Blocks that there are, of b sequences of at most L tokens: packed sequences have as many as their tokens say, or b more.
inline int64_t softmax_blocks(const AttnRows &r, int64_t L, int64_t tokens) {
    const int64_t all = r.b * ((L + kSoftmaxBlock - 1) / kSoftmaxBlock), some = tokens / kSoftmaxBlock + (r.b < tokens ? r.b : tokens);
    return r.cu_q && some < all ? some : all;
}
// Pieces for `groups` blocks of walks of up to `tiles` tiles where `fill` workgroups fill the device; `launched`: blocks that
// a launch has workgroups for, which many packed sequences of different lengths leave mostly empty (2^16 of them start in 30 us).
inline int64_t softmax_splits(int64_t groups, int64_t launched, int64_t tiles, int64_t least, int64_t fill) {
    int64_t n = groups > 0 ? (fill + groups - 1) / groups : 1;
    if (n > 1 && n * launched > (INT64_C(1) << 16)) n = (INT64_C(1) << 16) / launched;
    const int64_t most = (tiles + least - 1) / least;
    n = n < 16 ? n : 16;
    n = n < most ? n : most;
    return n > 1 ? n : 1;
}
inline SoftmaxWork softmax_query_work(const AttnRows &r, int64_t H, int64_t G, int64_t keys) {
    const int64_t least = kSoftmaxLeast / keys;
    const int64_t blocks = (r.Lq + kSoftmaxBlock - 1) / kSoftmaxBlock;
    const int64_t splits =
        softmax_splits(softmax_blocks(r, r.Lq, r.Tq) * H, r.b * blocks * H, (r.Lk + keys - 1) / keys, least, 1024);
    return softmax_work(r.b, G, H / G, blocks, splits, least);
}
inline SoftmaxWork softmax_fwd_work(const AttnRows &r, int64_t H, int64_t G, bool bf16) {
    return softmax_query_work(r, H, G, bf16 ? 64 : 32);  // keys of a tile
}
inline SoftmaxWork softmax_dq_work(const AttnRows &r, int64_t H, int64_t G) { return softmax_query_work(r, H, G, 32); }
inline SoftmaxWork softmax_dkv_work(const AttnRows &r, int64_t H, int64_t G) {
    const int64_t blocks = (r.Lk + kSoftmaxBlock - 1) / kSoftmaxBlock, least = kSoftmaxLeast / 32;
    const int64_t splits = softmax_splits(softmax_blocks(r, r.Lk, r.Tk) * G, r.b * blocks * G, (r.Lq + 31) / 32 * (H / G), least, 512);
    return softmax_work(r.b, G, 1, blocks, splits, least);
}
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
