// host_util.h — what the library's host code shares: argument checks, the device's compute units and the
// stream-ordered scratch pool.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <mutex>

#include "ssm_scan.h"

namespace ssm {

inline bool valid_dtype(ssm_dtype_t t) { return t == SSM_F32 || t == SSM_BF16; }

// a * b without overflow past 2^62 (sizes are far below that in practice)
inline bool mul_ok(int64_t a, int64_t b, int64_t *out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > (INT64_C(1) << 62) / a) return false;
    *out = a * b;
    return true;
}

struct Span {
    const void *p;
    int64_t bytes;
};

inline bool overlaps(const Span &u, const Span &v) {
    if (!u.p || !v.p || u.bytes <= 0 || v.bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(u.p), a1 = a0 + (uintptr_t)u.bytes;
    const uintptr_t b0 = reinterpret_cast<uintptr_t>(v.p), b1 = b0 + (uintptr_t)v.bytes;
    return a0 < b1 && b0 < a1;
}

// Compute units of the current device, cached per device id.
inline int cu_count() {
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
        cache[dev] = n;
    }
    return cache[dev];
}

// Stream-ordered scratch comes from a memory pool the library creates on each device at first use. Its
// release threshold is at the maximum, so freed scratch stays in that pool across synchronisations and
// repeated calls do not pay for re-mapping it. The device's default pool is left as the caller set it.
// Should the pool not be created, scratch comes from the default pool as it stands.
inline hipMemPool_t scratch_pool() {
    static std::mutex mu;
    static hipMemPool_t pools[64] = {};
    static bool tried[64] = {false};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!tried[dev]) {
        tried[dev] = true;
        hipMemPoolProps props{};
        props.allocType = hipMemAllocationTypePinned;
        props.handleTypes = hipMemHandleTypeNone;
        props.location.type = hipMemLocationTypeDevice;
        props.location.id = dev;
        hipMemPool_t pool = nullptr;
        if (hipMemPoolCreate(&pool, &props) == hipSuccess && pool) {
            uint64_t threshold = UINT64_MAX;
            (void)hipMemPoolSetAttribute(pool, hipMemPoolAttrReleaseThreshold, &threshold);
            pools[dev] = pool;
        }
    }
    return pools[dev];
}

inline hipError_t scratch_alloc(void **p, size_t bytes, hipStream_t stream) {
    hipMemPool_t pool = scratch_pool();
    if (pool) return hipMallocFromPoolAsync(p, bytes, pool, stream);
    return hipMallocAsync(p, bytes, stream);
}

}  // namespace ssm
