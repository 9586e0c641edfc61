// softmax_limits_driver.cpp — the host code of softmax attention at the sizes where its plans end: every call is answered without
// overflow on the way, built with the sanitizers and run on the CPU with stub launchers. Exits 0 only if every check holds.
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

int main() {
    sizes();
    if (failures == 0) std::printf("all limits held\n");
    return failures != 0;
}
