// softmax_limits_driver.cpp — the host code of softmax attention at the sizes where its plans end: every call is answered without
// overflow on the way; and the slots of packed sequences, which workgroups find by the offsets. Built with the sanitizers and run on
// the CPU with stub launchers. Exits 0 only if every check holds.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "launch_softmax.h"
#include "ssm_scan.h"

namespace ssm {
hipError_t launch_softmax_fwd(const SoftmaxLaunch &, hipStream_t) { return hipSuccess; }
hipError_t launch_softmax_bwd(const SoftmaxLaunch &, hipStream_t) { return hipSuccess; }
hipError_t launch_softmax_step(const SoftmaxStepLaunch &, hipStream_t) { return hipSuccess; }
hipError_t launch_kv_append(const KvAppendLaunch &, hipStream_t) { return hipSuccess; }
}  // namespace ssm

static int failures = 0;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); ++failures; } } while (0)

static void sizes() {
    const int32_t cu[2] = {0, 0};
    const int64_t L30 = INT64_C(1) << 30, lens[] = {0, 1, 128, 129, 1 << 20, L30, L30 + 1, INT64_MAX};
    const int64_t rows[] = {1, 3, 1 << 20, L30, INT32_MAX - 1, INT64_C(1) << 40, INT64_MAX};
    const int64_t heads[][2] = {{1, 1}, {64, 8}, {1024, 1}, {1 << 17, 1 << 17}, {1 << 24, 1}};
    int64_t good = 0;
    for (const int64_t b : rows)
        for (const int64_t Lq : lens)
            for (const int64_t Lk : lens)
                for (const auto &h : heads)
                    for (const int64_t D : {1, 128})
                        for (const int64_t tokens : {INT64_C(-1), INT64_C(0), Lq, (int64_t)INT32_MAX})
                            for (const bool packed : {false, true}) {
                                ssm_attn_rows_t r{packed ? cu : nullptr, packed ? cu : nullptr, nullptr, nullptr, b, Lq, Lk,
                                                  tokens, tokens};
                                int64_t n = -1;
                                ssm_status_t st = ssm_attn_fwd_workspace(&r, h[0], h[1], D, SSM_BF16, &n);
                                CHECK(st == SSM_ERR_SHAPE || (st == SSM_OK && n >= 0));
                                good += st == SSM_OK;
                                st = ssm_attn_bwd_workspace(&r, h[0], h[1], D, &n);
                                CHECK(st == SSM_ERR_SHAPE || (st == SSM_OK && n >= 0));
                            }
    CHECK(good > 0);
}

// Every block of every sequence and head is some workgroup's, once, wherever the sequences lie among the tokens; with offsets
// that are wrong, what a workgroup is given lies inside all the same.
static void slots() {
    using namespace ssm;
    uint32_t seed = 1;
    const auto next = [&](uint32_t n) { seed = seed * 1664525u + 1013904223u; return (seed >> 8) % n; };
    const int64_t groups[] = {1, 2, 3, 8, 12};
    const int32_t odd[] = {INT32_MIN, -3, 100, 5000, INT32_MAX};
    for (int round = 0; round < 60; ++round) {
        const int64_t b = 1 + next(40), G = groups[next(5)], per = 1 + next(3), splits = 1 + next(3);
        std::vector<int32_t> cu{(int32_t)next(300)};
        int64_t longest = 0;
        for (int64_t i = 0; i < b; ++i) {
            const int32_t n = next(3) == 0 ? 0 : (int32_t)next(next(4) == 0 ? 2000 : 200);
            cu.push_back(cu.back() + n);
            longest = longest < n ? n : longest;
        }
        const int64_t tokens = cu.back() + next(300), most = (longest + 127) / 128;
        const SoftmaxWork w = softmax_slot_work(G, per, tokens / kSoftmaxBlock + b, splits, 8, kSoftmaxBlock, most);
        for (const bool wrong : {false, true}) {
            if (wrong)
                for (int k = 0; k < 5; ++k) cu[next((uint32_t)cu.size())] = odd[next(5)];
            const AttnRows r{cu.data(), cu.data(), nullptr, nullptr, b, longest, longest, tokens, tokens};
            for (const bool keys : {false, true}) {
                std::vector<int> seen((size_t)(b * G * per * splits * (most + 1)), 0);
                for (int64_t id = 0; id < softmax_groups(w); ++id) {
                    SoftmaxPlace p;
                    if (!softmax_find(w, r, G, (uint32_t)id, keys, &p)) continue;
                    CHECK(p.seq >= 0 && p.seq < b && p.g >= 0 && p.g < G && p.which >= 0 && p.which < per && p.block >= 0 &&
                          p.block < most && p.piece >= 0 && p.piece < splits);
                    if (p.seq < 0 || p.seq >= b || p.block < 0 || p.block > most) continue;
                    ++seen[(size_t)((((p.seq * G + p.g) * per + p.which) * splits + p.piece) * (most + 1) + p.block)];
                }
                if (wrong) continue;
                for (int64_t i = 0; i < b; ++i)
                    for (int64_t k = 0; k < G * per * splits; ++k)
                        for (int64_t blk = 0; blk <= most; ++blk) {
                            const int n = seen[(size_t)((i * G * per * splits + k) * (most + 1) + blk)];
                            if (blk * 128 < cu[(size_t)i + 1] - cu[(size_t)i]) CHECK(n == 1);
                            else CHECK(n <= 1);
                        }
            }
        }
    }
    // a launch by slots only where one by sequences would be mostly empty
    const int32_t cu[2] = {0, 0};
    const AttnRows many{cu, cu, nullptr, nullptr, 1024, 8192, 8192, 131072, 131072}, few{cu, cu, nullptr, nullptr, 9, 4096, 4096, 20000, 20000};
    CHECK(softmax_fwd_work(many, 32, 8, true).block == 128 && softmax_groups(softmax_fwd_work(many, 32, 8, true)) == 2048 * 32);
    CHECK(softmax_dkv_work(many, 32, 8).block == 128 && softmax_dq_work(few, 32, 8).block == 0);
    const AttnRows full{cu, cu, nullptr, nullptr, 512, 1024, 1024, 512 * 1024, 512 * 1024}, rows{nullptr, nullptr, nullptr, nullptr, 512, 1024, 1024, 0, 0};
    CHECK(softmax_fwd_work(full, 32, 8, true).block == 0 && softmax_fwd_work(rows, 32, 8, true).block == 0);
}

int main() {
    sizes();
    slots();
    if (failures == 0) std::printf("all limits held\n");
    return failures != 0;
}
