// attn_stubs.cpp — stand-ins for the launchers behind abi_attn.cpp, so that its host code (validation, planning,
// workspace layout, dispatch) can run under the sanitizers on a machine without a GPU. Each notes its call and touches no
// device memory.
#include "launch.h"

namespace ssm {

int g_launches = 0;
LinAttnLaunch g_last;
NormLaunch g_last_norm;

hipError_t launch_fill_zero(float *, int64_t, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_linattn_fwd(const LinAttnLaunch &p, hipStream_t) { ++g_launches; g_last = p; return hipSuccess; }
hipError_t launch_linattn_bwd(const LinAttnLaunch &p, hipStream_t) { ++g_launches; g_last = p; return hipSuccess; }
hipError_t launch_linattn_step(float *, const LinAttnLaunch &p, hipStream_t) { ++g_launches; g_last = p; return hipSuccess; }
hipError_t launch_layernorm_fwd(const NormLaunch &p, hipStream_t) { ++g_launches; g_last_norm = p; return hipSuccess; }
hipError_t launch_layernorm_bwd(const NormLaunch &p, hipStream_t) { ++g_launches; g_last_norm = p; return hipSuccess; }
int64_t layernorm_part_floats(int64_t rows, int64_t d, int64_t w_rows) {
    const int64_t per = rows / w_rows < 512 ? rows / w_rows : 512;
    return 2 * (per > 0 ? per : 1) * w_rows * d;
}

}  // namespace ssm
