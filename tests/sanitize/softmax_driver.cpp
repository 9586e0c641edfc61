// softmax_driver.cpp — the index arithmetic of softmax attention and the paged cache (softmax_index.h) and the host code behind
// its C ABI, run on the CPU under the sanitizers with stub launchers. Exits 0 only if every check holds.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "launch_softmax.h"
#include "ssm_scan.h"

namespace ssm {
int g_launches = 0;
SoftmaxLaunch g_last;
SoftmaxStepLaunch g_step;
KvAppendLaunch g_append;
hipError_t launch_softmax_fwd(const SoftmaxLaunch &p, hipStream_t) { ++g_launches; g_last = p; return hipSuccess; }
hipError_t launch_softmax_bwd(const SoftmaxLaunch &p, hipStream_t) { ++g_launches; g_last = p; return hipSuccess; }
hipError_t launch_softmax_step(const SoftmaxStepLaunch &p, hipStream_t) { ++g_launches; g_step = p; return hipSuccess; }
hipError_t launch_kv_append(const KvAppendLaunch &p, hipStream_t) { ++g_launches; g_append = p; return hipSuccess; }
}  // namespace ssm

static int failures = 0;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); ++failures; } } while (0)

static void sequences() {
    using namespace ssm;
    // any offsets, however wrong, give tokens inside
    const int32_t values[] = {INT32_MIN, -7, 0, 1, 5, 9, 10, 11, 40, INT32_MAX};
    for (const int32_t a : values)
        for (const int32_t e : values)
            for (const int64_t total : {0, 1, 10})
                for (const int64_t most : {0, 1, 4, 100}) {
                    const int32_t cu[2] = {a, e};
                    const AttnSeq s = sequence({cu, cu, nullptr, nullptr, 1, most, most, total, total}, 0);
                    CHECK(s.q0 >= 0 && s.nq >= 0 && s.q0 + s.nq <= total && s.nq <= most);
                    CHECK(s.k0 == s.q0 && s.nk == s.nq);
                    if (a >= 0 && e >= a && e <= total && e - a <= most) CHECK(s.q0 == a && s.nq == e - a);
                }
    for (const int32_t n : values) {
        const int32_t len[1] = {n};
        const AttnSeq s = sequence({nullptr, nullptr, len, nullptr, 1, 10, 20, 0, 0}, 0);
        CHECK(s.nq == (n < 0 ? 0 : n > 10 ? 10 : n) && s.nk == 20 && s.q0 == 0 && s.k0 == 0);
    }
    for (int nq = 0; nq < 6; ++nq)
        for (int nk = 0; nk < 6; ++nk)
            for (const bool causal : {false, true}) {
                const AttnSeq s{0, 0, nq, nk};
                for (int i = 0; i < nq; ++i) {
                    int last = -1;
                    for (int j = 0; j < nk; ++j)
                        if (!causal || j <= i + nk - nq) last = j;
                    CHECK(last_key(s, causal, i) == last);
                }
                for (int j = 0; j < nk; ++j) {
                    int first = nq;
                    for (int i = nq - 1; i >= 0; --i)
                        if (last_key(s, causal, i) >= j) first = i;
                    CHECK(first_query(s, causal, j) == first);
                }
            }
}

static void pages() {
    using namespace ssm;
    const std::vector<int32_t> table = {3, -1, 7, 8, INT32_MAX, INT32_MIN};  // two rows of three pages, 8 pages
    const Pages p{table.data(), 3, 8, 5};
    for (int64_t row = 0; row < 2; ++row)
        for (int64_t t = -20; t < 40; ++t) {
            const int64_t got = page_of(p, row, t);
            if (t < 0 || t >= 15) CHECK(got == -1);
            else {
                const int32_t e = table[(size_t)(row * 3 + t / 5)];
                CHECK(got == (e >= 0 && e < 8 ? e : -1));
            }
        }
    CHECK(page_of(p, 0, INT64_C(1) << 40) == -1 && page_of(p, 0, -(INT64_C(1) << 40)) == -1);
    const int32_t lens[4] = {INT32_MIN, 0, 15, INT32_MAX};
    CHECK(cached(p, lens, 0) == 0 && cached(p, lens, 1) == 0 && cached(p, lens, 2) == 15 && cached(p, lens, 3) == 15);
}

static void tokens() {
    using namespace ssm;
    int64_t row = 0, index = 0, count = 0;
    const std::vector<int32_t> cu = {2, 2, 5, 5, 9};
    const NewTokens n{cu.data(), nullptr, 4, 0, 12};
    for (int64_t t = 0; t < 12; ++t) {
        const bool in = locate(n, t, &row, &index, &count);
        CHECK(in == (t >= 2 && t < 9));
        if (in) CHECK(cu[(size_t)row] + index == t && t < cu[(size_t)row + 1] && count == cu[(size_t)row + 1] - cu[(size_t)row]);
    }
    // falling offsets: a row inside all the same
    const std::vector<int32_t> bad = {0, 9, -4, INT32_MAX, 6, 20};
    for (int64_t t = 0; t < 30; ++t)
        if (locate({bad.data(), nullptr, 5, 0, 30}, t, &row, &index, &count)) CHECK(row >= 0 && row < 5 && index >= 0 && index < count);
    const int32_t len[3] = {4, -2, 9};
    for (int64_t t = 0; t < 12; ++t) {
        const bool in = locate({nullptr, len, 3, 4, 12}, t, &row, &index, &count);
        CHECK(row == t / 4 && index == t % 4 && in == (row != 1));
    }
    CHECK(locate({nullptr, nullptr, 9, 1, 9}, 7, &row, &index, &count) && row == 7 && index == 0 && count == 1);
}

// Every block of every sequence and head is some workgroup's, once, and a sequence's work is spread over the XCDs.
static void places() {
    using namespace ssm;
    for (const int64_t b : {1, 2, 5})
        for (const int64_t G : {1, 3, 7, 8, 12})
            for (const int64_t per : {1, 4})
                for (const int64_t splits : {1, 3})
                    for (const int64_t blocks : {0, 1, 2, 5, 16, 33}) {
                        const SoftmaxWork w = softmax_work(b, G, per, blocks, splits, 8);
                        std::vector<int> seen((size_t)(b * G * per * blocks * splits), 0), of(8, 0);
                        for (int64_t id = 0; id < softmax_groups(w); ++id) {
                            SoftmaxPlace p;
                            if (!softmax_place(w, G, (uint32_t)id, &p)) continue;
                            CHECK(p.seq >= 0 && p.seq < b && p.g >= 0 && p.g < G && p.which < per && p.block >= 0 &&
                                  p.block < blocks && p.piece >= 0 && p.piece < splits);
                            ++seen[(size_t)((((p.seq * G + p.g) * per + p.which) * blocks + p.block) * splits + p.piece)];
                            if (p.seq == 0) ++of[(size_t)(id & 7)];
                        }
                        for (const int n : seen) CHECK(n == 1);
                        if (blocks >= 8)
                            for (const int n : of) CHECK(n > 0);
                    }
    // pieces cover a walk, none of them empty
    for (int splits = 1; splits < 17; ++splits)
        for (const int least : {4, 8})
            for (int tiles = 0; tiles < 200; ++tiles) {
                SoftmaxWork w{};
                w.splits = splits;
                w.least = least;
                int pieces = 0;
                const int per = softmax_piece(w, tiles, &pieces);
                CHECK(pieces >= 1 && pieces <= splits && (int64_t)per * pieces >= tiles);
                CHECK(pieces == 1 || (pieces - 1) * per < tiles);
                CHECK(pieces == 1 || per >= least);
            }
    const AttnRows one{nullptr, nullptr, nullptr, nullptr, 1, 4096, 4096, 0, 0};
    CHECK(softmax_fwd_work(one, 2, 1, true).splits == 16 && softmax_fwd_work(one, 32, 1, true).splits == 1);
    CHECK(softmax_dkv_work(one, 2, 1).splits == 16);
    const int32_t cu[2] = {0, 0};
    const AttnRows packed{cu, cu, nullptr, nullptr, 64, 4096, 4096, 1280, 1280};  // few tokens of many short sequences
    CHECK(softmax_blocks(packed, 4096, 1280) == 74);
}

static void host_code() {
    using namespace ssm;
    alignas(16) static char mem[64][4096];
    const auto at = [](int i) { return (void *)mem[i]; };
    const auto fl = [&](int i) { return (float *)at(i); };
    const auto in = [&](int i) { return (const int32_t *)at(i); };
    ssm_attn_rows_t rows{nullptr, nullptr, nullptr, nullptr, 2, 3, 3, 0, 0};
    int launches = g_launches;
    CHECK(ssm_attn_fwd(at(0), at(1), at(2), 1.0f, 1, &rows, at(3), fl(4), 2, 1, 8, SSM_F32, nullptr, nullptr, 0, nullptr) == SSM_OK);
    CHECK(g_launches == ++launches && g_last.vec && g_last.q_t == 16 && g_last.q_b == 48 && g_last.k_t == 8);
    CHECK(ssm_attn_fwd((char *)at(0) + 4, at(1), at(2), 1.0f, 1, &rows, at(3), nullptr, 2, 1, 8, SSM_F32, nullptr, nullptr, 0,
                       nullptr) == SSM_OK);
    CHECK(g_launches == ++launches && !g_last.vec);
    rows.Lq = 0;
    CHECK(ssm_attn_fwd(nullptr, at(1), at(2), 1.0f, 1, &rows, nullptr, nullptr, 2, 1, 8, SSM_F32, nullptr, nullptr, 0,
                       nullptr) == SSM_OK);
    CHECK(g_launches == launches);
    rows = {in(10), in(11), nullptr, nullptr, 2, 5, 5, 7, 7};
    int64_t need = 0;
    CHECK(ssm_attn_fwd_workspace(&rows, 2, 1, 8, SSM_BF16, &need) == SSM_OK && need == 0);
    CHECK(ssm_attn_bwd_workspace(&rows, 2, 1, 8, &need) == SSM_OK && need == 256);
    CHECK(ssm_attn_bwd(at(0), at(1), at(2), at(3), fl(4), at(5), 1.0f, 0, &rows, at(6), at(7), at(8), 2, 1, 8, SSM_BF16, nullptr,
                       at(9), need, nullptr) == SSM_OK);
    CHECK(g_launches == ++launches && g_last.bf16 && !g_last.causal && g_last.q_b == 0 && g_last.stats == at(9));
    CHECK(ssm_attn_bwd(at(0), at(1), at(2), at(3), fl(4), at(5), 1.0f, 0, &rows, at(6), at(7), at(8), 2, 1, 8, SSM_BF16, nullptr,
                       at(9), need - 1, nullptr) == SSM_ERR_SCRATCH);
    // pieces: none for short rows, more where few rows have to fill the device, one at least for 4096 tokens
    const ssm_pages_t g{in(20), 4, 16, 1 << 16, 0, 0};
    struct { int64_t b, H, G, max_len, pieces; } plans[] = {{1, 2, 2, 256, 1}, {1, 2, 2, 257, 2}, {1, 24, 24, 1000, 4},
                                                            {512, 32, 8, 4096, 1}, {512, 32, 8, 4097, 2},
                                                            {1, 16, 2, 131072, 256}, {64, 1, 1, 131072, 32}};
    for (const auto &p : plans) {
        CHECK(ssm_attn_step_workspace(p.b, p.H, p.G, 64, &g, p.max_len, &need) == SSM_OK);
        CHECK(need == (p.pieces > 1 ? p.b * p.H * p.pieces * 66 * 4 : 0));
    }
    const ssm_pages_t two{in(20), 2, 4, 3, 2 * 4 * 8, 2 * 4 * 8};  // both caches in one pool
    CHECK(ssm_attn_step(at(0), at(1), (char *)at(1) + 4 * 8 * 4, &two, in(21), 1.0f, at(3), nullptr, 2, 2, 1, 8, 0, 0, 0, SSM_F32,
                        nullptr, 0, nullptr) == SSM_OK);
    CHECK(g_launches == ++launches && g_step.vec && g_step.splits == 1 && g_step.k_page == 64);
    const ssm_tokens_t t{nullptr, nullptr, 2, 1, 2};
    CHECK(ssm_kv_append(at(0), at(2), at(3), at(4), nullptr, at(1), (char *)at(1) + 4 * 8 * 4, &two, in(21), &t, (double *)at(22), 8,
                        0, 2, 1, 8, SSM_F32, nullptr, nullptr) == SSM_OK);
    CHECK(g_launches == ++launches && g_append.vec && g_append.rotary == 8);
    CHECK(ssm_kv_append(at(0), at(2), at(3), at(4), nullptr, at(1), (char *)at(1) + 4 * 8 * 4 - 4, &two, in(21), &t, nullptr, 0, 0,
                        2, 1, 8, SSM_F32, nullptr, nullptr) == SSM_ERR_ALIAS);
    CHECK(ssm_rope(at(0), at(0), nullptr, &t, (double *)at(22), 6, 0, 1, 2, 8, 0, 0, 0, SSM_F32, nullptr) == SSM_OK);
    CHECK(g_launches == ++launches && !g_append.vec && g_append.inverse && !g_append.k_cache);
}

int main() {
    sequences();
    pages();
    tokens();
    places();
    host_code();
    if (failures == 0) std::printf("all host paths behaved\n");
    return failures != 0;
}
