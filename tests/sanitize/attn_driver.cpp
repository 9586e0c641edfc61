// attn_driver.cpp — drives abi_attn.cpp's host code with stub launchers under the sanitizers: sizes at and past every
// limit (products that would overflow included), strides, workspaces, and calls that reach a launcher, whose arguments
// (segments, workspace pieces, access widths) are checked against the shapes.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "launch.h"
#include "ssm_scan.h"

namespace ssm {
extern int g_launches;
extern LinAttnLaunch g_last;
extern NormLaunch g_last_norm;
}  // namespace ssm

#define CHECK(x)                                                          \
    do {                                                                  \
        if (!(x)) {                                                       \
            std::printf("line %d: %s\n", __LINE__, #x);                   \
            std::exit(1);                                                 \
        }                                                                 \
    } while (0)

static char *at(int64_t i) { return reinterpret_cast<char *>((INT64_C(1) << 44) + (i << 42)); }  // never dereferenced

static ssm_status_t fwd(int64_t b, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, ssm_dtype_t t = SSM_F32,
                        const ssm_linattn_strides_t *st = nullptr, void *ws = at(20), int64_t wb = INT64_C(1) << 41) {
    return ssm_linattn_fwd(at(0), at(1), at(2), (const float *)at(3), 1, 1.0f, nullptr, nullptr, at(4), (float *)at(5), b, L,
                           H, G, N, P, t, st, ws, wb, nullptr);
}
static ssm_status_t bwd(int64_t b, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int ps = 1) {
    return ssm_linattn_bwd(at(0), at(1), at(2), (const float *)at(3), ps, 1.0f, nullptr, nullptr, at(4), nullptr, at(5),
                           at(6), at(7), (float *)at(8), (float *)at(9), b, L, H, G, N, P, SSM_BF16, nullptr, at(20),
                           INT64_C(1) << 41, nullptr);
}

int main() {
    const int64_t big[] = {INT64_MIN, -1, 0, 1, 2, 63, 64, 65, 1000, INT64_C(1) << 24, INT64_C(1) << 31, INT64_C(1) << 40,
                           INT64_C(1) << 62, INT64_MAX};
    for (int64_t x : big)
        for (int64_t y : big) {
            int64_t n = 0;
            (void)fwd(x, y, 2, 1, 16, 16);
            (void)fwd(1, x, y, 1, 16, 16);
            (void)fwd(1, 64, y, x, 16, 16);
            (void)fwd(1, 64, 2, 1, x, y);
            (void)bwd(x, y, 2, 1, 16, 16);
            (void)ssm_linattn_workspace(1, x, y, 4, 2, 128, 64, SSM_BF16, 0, &n);
            (void)ssm_layernorm_bwd_workspace(x, y, 1, &n);
            (void)ssm_layernorm_bwd_workspace(x, 64, y, &n);
            (void)ssm_layernorm_fwd(at(0), nullptr, nullptr, at(4), nullptr, nullptr, x, 64, 1, y, 1e-5f, SSM_F32, nullptr);
            ssm_linattn_strides_t s{x, y, x, y, x, y, x, y, x, y, x, y};
            (void)fwd(2, 100, 4, 2, 16, 16, SSM_F32, &s);
        }
    for (int t : {2, 7, INT32_MAX}) CHECK(fwd(1, 64, 2, 1, 16, 16, (ssm_dtype_t)t) == SSM_ERR_UNSUPPORTED);

    // a call's launch: segments cover the chunks, pieces of the workspace lie in it in order
    for (int64_t L : {1, 64, 65, 1000, 4096, 100000})
        for (int64_t H : {1, 8, 300}) {
            int64_t need = 0;
            CHECK(ssm_linattn_workspace(0, 1, L, H, 1, 64, 100, SSM_F32, 1, &need) == SSM_OK);
            ssm::g_launches = 0;
            CHECK(fwd(1, L, H, 1, 64, 100, SSM_F32, nullptr, need ? at(20) : nullptr, need) == SSM_OK);
            CHECK(ssm::g_launches == 1);
            const ssm::LinAttnLaunch &p = ssm::g_last;
            const int64_t chunks = (L + 63) / 64;
            CHECK(p.n_seg >= 1 && p.seg_chunks >= 1 && (p.n_seg - 1) * p.seg_chunks < chunks &&
                  p.n_seg * p.seg_chunks >= chunks);
            CHECK((p.n_seg > 1) == (need > 0));
            if (need) {
                CHECK((char *)p.S == at(20) && (char *)p.gsum >= (char *)(p.S + H * p.n_seg * 128 * 64));
                CHECK((char *)(p.gsum + H * p.n_seg) <= at(20) + need);
                CHECK(fwd(1, L, H, 1, 64, 100, SSM_F32, nullptr, at(20), need - 1) == SSM_ERR_SCRATCH);
            }
        }
    for (int ps : {0, 1}) {
        int64_t need = 0;
        CHECK(ssm_linattn_workspace(1, 2, 200, 6, 3, 40, 72, SSM_BF16, ps, &need) == SSM_OK && need > 0);
        CHECK(bwd(2, 200, 6, 3, 40, 72, ps) == SSM_OK);
        const ssm::LinAttnLaunch &p = ssm::g_last;
        const int64_t state = 128 * 64, n = 2 * 6 * p.n_seg;
        CHECK((char *)(p.S + n * state) <= (char *)p.gsum && (char *)(p.gsum + n) <= (char *)p.E);
        CHECK((char *)(p.E + n * state) <= (char *)p.dq_part);
        CHECK(p.dq_part + 2 * 200 * 6 * 40 <= p.dk_part && (char *)(p.dk_part + 2 * 200 * 6 * 40) <= at(20) + need);
        CHECK((p.dg_steps != nullptr) == (ps == 0));
    }
    // 16-byte accesses only where every row allows them
    ssm_linattn_strides_t s{0, 64, 32, 0, 64, 32, 0, 64, 32, 0, 0, 0};
    CHECK(fwd(1, 100, 2, 2, 32, 32, SSM_F32, &s) == SSM_OK && ssm::g_last.vec);
    s.v_t = 66;
    CHECK(fwd(1, 100, 2, 2, 32, 32, SSM_F32, &s) == SSM_OK && !ssm::g_last.vec);
    s.v_t = 0;  // one value row for all steps
    CHECK(fwd(1, 100, 2, 2, 32, 32, SSM_F32, &s) == SSM_OK && !ssm::g_last.vec);
    CHECK(fwd(1, 1, 2, 2, 32, 32, SSM_F32, &s) == SSM_OK && ssm::g_last.vec);
    CHECK(fwd(1, 100, 2, 2, 31, 32) == SSM_OK && !ssm::g_last.vec);

    // norm: dense strides are filled in, a caller's kept
    CHECK(ssm_layernorm_fwd(at(0), nullptr, nullptr, at(4), nullptr, nullptr, 10, 64, 5, 0, 1e-5f, SSM_F32, nullptr) == SSM_OK);
    CHECK(ssm::g_last_norm.x_stride == 64 && ssm::g_last_norm.vec);
    CHECK(ssm_layernorm_fwd(at(0), nullptr, nullptr, at(4), nullptr, nullptr, 10, 64, 5, 65, 1e-5f, SSM_F32, nullptr) == SSM_OK);
    CHECK(ssm::g_last_norm.x_stride == 65 && !ssm::g_last_norm.vec);
    std::printf("all host paths behaved\n");
    return 0;
}
