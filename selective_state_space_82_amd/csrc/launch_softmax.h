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
//
// Packed sequences may be many and most of them far shorter than the longest. Where workgroups for the longest's blocks of each
// would be more than 2^16 (which start in 30 us), a launch has them for slots of a block instead: sequence i has those from
// ⌊cu_i/128⌋ + i on, of which there are enough whatever its length, ⌊tokens/128⌋ + b in all, and a workgroup finds its sequence in
// the offsets (softmax_find). (Lengths of exponential spread, bf16, forward and gradient, by sequences and by slots: 2^21 workgroups for
// 1024 sequences of up to 8192, 138726 tokens, 32 heads on 8 key heads of 128: 5.4 and 2.3 ms, 18.5 and 8.3 ms; 1.1·2^16 for 96 of
// up to 4096, 24 heads of 64: 3.7 and 2.9, 13.9 and 11.0; 2^17 for 128 of up to 4096, 32 heads on 8 of 128: 8.2 and 8.2, 36.7 and
// 36.8. Below 2^16 calls are as they were.)
struct SoftmaxWork {
    int64_t units, each;  // each: workgroups of a unit
    int parts, per, blocks, splits, least;
    bool across;  // an XCD takes the first block of each of its units, then the second of each, ...; otherwise unit by unit
    int block = 0, most = 0;  // by slots: tokens of a block (0: by sequences), and blocks of the longest sequence
};  // workgroups number less than 2^24
inline SoftmaxWork softmax_work(int64_t b, int64_t G, int64_t per, int64_t blocks, int64_t splits, int64_t least) {
    const int64_t parts = G >= 8 || blocks < 2 ? 1 : ((8 + G - 1) / G < blocks ? (8 + G - 1) / G : blocks);
    const int64_t units = b * G * parts, each = per * splits * ((blocks + parts - 1) / parts);
    // The last unit's longest blocks should not start when all else is done: where a unit does not fill an XCD (32 compute units,
    // two workgroups each) and there are rounds enough for that to matter. Measured on both sides, unit by unit and across, us
    // (bf16, causal; workgroups of a unit; of an XCD): 16; 192: forward 116 and 100, gradient 427 and 366. 32; 128: 147 and 131,
    // 531 and 477. 48; 192: 438 and 407, 1725 and 1636. 64; 256: 731 and 694, 2915 and 2874. 96; 192: 812 and 786, 3190 and 3136.
    // With four heads to a key head, whose tiles a unit shares: 32; 256: 134 and 126. 32; 512: 247 and 268. 32; 1024: 510 and
    // 563. 64; 512: 413 and 424. Below the second border: 32; 64: 103 and 96. So the rule is right where it matters most and within
    // 10 % elsewhere.
    return {units, each, (int)parts, (int)per, (int)blocks, (int)splits, (int)least,
            each < 64 && (units + 7) / 8 * each >= 128};
}
// By slots: all sequences' blocks of a key head as if they were one sequence's, spread so that each XCD has as many units.
inline SoftmaxWork softmax_slot_work(int64_t G, int64_t per, int64_t slots, int64_t splits, int64_t least, int64_t block, int64_t most) {
    int64_t parts = G % 8 == 0 ? 1 : G % 4 == 0 ? 2 : G % 2 == 0 ? 4 : 8;
    parts = parts < slots ? parts : slots;
    return {G * parts, per * splits * ((slots + parts - 1) / parts), (int)parts, (int)per, (int)slots, (int)splits, (int)least, false,
            (int)block, (int)most};
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
// The same with the block's place in its sequence, of queries (the last first) or of keys (the first first).
SSM_BOTH bool softmax_find(const SoftmaxWork &w, const AttnRows &r, int64_t G, uint32_t id, bool keys, SoftmaxPlace *p) {
    if (!softmax_place(w, G, id, p)) return false;
    const int at = keys ? p->block : w.blocks - 1 - p->block;
    p->block = at;
    if (w.block == 0) return true;
    const int32_t *cu = keys ? r.cu_k : r.cu_q;
    const int64_t tokens = keys ? r.Tk : r.Tq;
    int64_t lo = 0, hi = r.b, first = clamp_to(cu[0], 0, tokens) / w.block;  // lo's first slot <= at, where offsets rise
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2, from = clamp_to(cu[mid], 0, tokens) / w.block + mid;
        if (from <= at) {
            lo = mid;
            first = from;
        } else {
            hi = mid;
        }
    }
    p->seq = lo;
    p->block = (int)(at - first);
    return at >= first && at - first < w.most;
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
// a launch has workgroups for, of which packed sequences of different lengths leave some empty (2^16 of them start in 30 us).
inline int64_t softmax_splits(int64_t groups, int64_t launched, int64_t tiles, int64_t least, int64_t fill) {
    int64_t n = groups > 0 ? (fill + groups - 1) / groups : 1;
    if (n > 1 && n * launched > (INT64_C(1) << 16)) n = (INT64_C(1) << 16) / launched;
    const int64_t most = (tiles + least - 1) / least;
    n = n < 16 ? n : 16;
    n = n < most ? n : most;
    return n > 1 ? n : 1;
}
// Slots of packed sequences of at most L tokens for `heads` workgroups a block, or 0: by sequences.
inline int64_t softmax_slots(const AttnRows &r, int64_t L, int64_t tokens, int64_t heads) {
    const int64_t all = r.b * ((L + kSoftmaxBlock - 1) / kSoftmaxBlock), slots = tokens / kSoftmaxBlock + r.b;
    return r.cu_q && slots < all && all * heads > (INT64_C(1) << 16) ? slots : 0;
}
inline SoftmaxWork softmax_query_work(const AttnRows &r, int64_t H, int64_t G, int64_t keys) {
    const int64_t least = kSoftmaxLeast / keys;
    const int64_t blocks = (r.Lq + kSoftmaxBlock - 1) / kSoftmaxBlock, slots = softmax_slots(r, r.Lq, r.Tq, H);
    const int64_t splits = softmax_splits(softmax_blocks(r, r.Lq, r.Tq) * H, (slots > 0 ? slots : r.b * blocks) * H,
                                          (r.Lk + keys - 1) / keys, least, 1024);
    return slots > 0 ? softmax_slot_work(G, H / G, slots, splits, least, kSoftmaxBlock, blocks)
                     : softmax_work(r.b, G, H / G, blocks, splits, least);
}
inline SoftmaxWork softmax_fwd_work(const AttnRows &r, int64_t H, int64_t G, bool bf16) {
    return softmax_query_work(r, H, G, bf16 ? 64 : 32);  // keys of a tile
}
inline SoftmaxWork softmax_dq_work(const AttnRows &r, int64_t H, int64_t G) { return softmax_query_work(r, H, G, 32); }
inline SoftmaxWork softmax_dkv_work(const AttnRows &r, int64_t H, int64_t G) {
    const int64_t blocks = (r.Lk + kSoftmaxBlock - 1) / kSoftmaxBlock, least = kSoftmaxLeast / 32;
    const int64_t slots = softmax_slots(r, r.Lk, r.Tk, G);
    const int64_t splits = softmax_splits(softmax_blocks(r, r.Lk, r.Tk) * G, (slots > 0 ? slots : r.b * blocks) * G,
                                          (r.Lq + 31) / 32 * (H / G), least, 512);
    return slots > 0 ? softmax_slot_work(G, 1, slots, splits, least, kSoftmaxBlock, blocks)
                     : softmax_work(r.b, G, 1, blocks, splits, least);
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
