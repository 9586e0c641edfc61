// softmax_index.h — where the sequences of softmax attention and the tokens of a paged cache lie: the arithmetic on lengths,
// offsets and pages that come from device memory, clamped so that no value of theirs leads outside of a tensor. Plain C++
// for the host and the device.
#pragma once

#include <cstdint>

#if defined(__HIPCC__)
#define SSM_BOTH __host__ __device__ __forceinline__
#else
#define SSM_BOTH inline
#endif

namespace ssm {

// Sequences of queries and keys. Packed: cu_q and cu_k hold b + 1 offsets into Tq and Tk tokens. Otherwise b rows of Lq and Lk
// tokens, of which len_q[i] and len_k[i] count (all where null). No sequence is longer than Lq or Lk.
struct AttnRows {
    const int32_t *cu_q, *cu_k, *len_q, *len_k;
    int64_t b, Lq, Lk, Tq, Tk;
};

struct AttnSeq {
    int64_t q0, k0;  // packed: first token; otherwise 0
    int nq, nk;
};

SSM_BOTH int64_t clamp_to(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : (v > hi ? hi : v); }

SSM_BOTH void packed_range(const int32_t *cu, int64_t i, int64_t total, int64_t most, int64_t *first, int *n) {
    const int64_t a = clamp_to(cu[i], 0, total), e = clamp_to(cu[i + 1], a, total);
    *first = a;
    *n = (int)(e - a < most ? e - a : most);
}

SSM_BOTH AttnSeq sequence(const AttnRows &r, int64_t i) {
    AttnSeq s{0, 0, (int)r.Lq, (int)r.Lk};
    if (r.cu_q) {
        packed_range(r.cu_q, i, r.Tq, r.Lq, &s.q0, &s.nq);
        packed_range(r.cu_k, i, r.Tk, r.Lk, &s.k0, &s.nk);
    } else {
        if (r.len_q) s.nq = (int)clamp_to(r.len_q[i], 0, r.Lq);
        if (r.len_k) s.nk = (int)clamp_to(r.len_k[i], 0, r.Lk);
    }
    return s;
}

// The last key that query i of a sequence sees (-1: none).
SSM_BOTH int last_key(const AttnSeq &s, bool causal, int i) {
    const int last = s.nk - 1, own = i + s.nk - s.nq;
    return causal && own < last ? (own < -1 ? -1 : own) : last;
}
// The first query that sees key j (nq: none).
SSM_BOTH int first_query(const AttnSeq &s, bool causal, int j) {
    const int i = causal ? j - (s.nk - s.nq) : 0;
    return i < 0 ? 0 : (i > s.nq ? s.nq : i);
}

// A paged cache: row i's token t is in slot t mod page of page table[i·max_pages + t / page].
struct Pages {
    const int32_t *table;
    int64_t max_pages, n_pages;
    int32_t page;
};

// The page of a row's token t, or -1 where the table has none in range.
SSM_BOTH int64_t page_of(const Pages &p, int64_t i, int64_t t) {
    if (t < 0 || t >= p.max_pages * p.page) return -1;
    const int64_t at = p.table[i * p.max_pages + (int64_t)((uint32_t)t / (uint32_t)p.page)];
    return at >= 0 && at < p.n_pages ? at : -1;
}

// Tokens of row i in the cache, as far as its pages go.
SSM_BOTH int cached(const Pages &p, const int32_t *lengths, int64_t i) {
    return (int)clamp_to(lengths[i], 0, p.max_pages * p.page);
}

// New tokens in packed order, of b rows: row r has those from first_of(r) to first_of(r + 1). Packed: by cu; otherwise L a
// row, of which len[r] count.
struct NewTokens {
    const int32_t *cu, *len;
    int64_t b, L, T;  // T tokens in all
};
// Which row token t belongs to, its index there and how many the row has; false: to none.
SSM_BOTH bool locate(const NewTokens &n, int64_t t, int64_t *row, int64_t *index, int64_t *count) {
    if (!n.cu) {
        *row = n.L == 1 ? t : t / n.L;
        *index = t - *row * n.L;
        *count = n.len ? clamp_to(n.len[*row], 0, n.L) : n.L;
        return *index < *count;
    }
    int64_t lo = 0, hi = n.b;  // cu[lo] <= t < cu[hi], if offsets rise
    if (t < n.cu[0] || t >= n.cu[n.b]) return false;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (n.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    *row = lo;
    *index = t - n.cu[lo];
    *count = (int64_t)n.cu[lo + 1] - n.cu[lo];
    return *index < *count;
}

}  // namespace ssm
