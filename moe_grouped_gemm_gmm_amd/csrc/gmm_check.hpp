// Argument checks and error reporting shared by the C-ABI sources.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gmm.h"

namespace gmm {
namespace abi {

// Records the calling thread's last error message and returns status.
int fail(int status, const char* fmt, ...);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;

inline int check_ptr(const void* p, const char* name) {
    if (p == nullptr) return fail(GMM_ERR_NULL, "%s is NULL", name);
    if (!aligned16(p)) return fail(GMM_ERR_ALIGN, "%s is not 16-byte aligned", name);
    return GMM_OK;
}

inline int check_opt_ptr(const void* p, const char* name) {
    if (p != nullptr && !aligned16(p)) return fail(GMM_ERR_ALIGN, "%s is not 16-byte aligned", name);
    return GMM_OK;
}

inline int check_groups(int64_t M, int64_t G) {
    if (M < 0 || M > kMaxDim) return fail(GMM_ERR_SHAPE, "M=%lld out of range", (long long)M);
    if (G < 1 || G > GMM_MAX_GROUPS)
        return fail(GMM_ERR_SHAPE, "G=%lld outside [1, %d]", (long long)G, GMM_MAX_GROUPS);
    return GMM_OK;
}

inline int check_mult(int64_t v, int64_t mult, const char* name) {
    if (v < mult || v > kMaxDim || v % mult != 0)
        return fail(GMM_ERR_SHAPE, "%s=%lld must be a positive multiple of %lld", name,
                    (long long)v, (long long)mult);
    return GMM_OK;
}

inline int check_out_dtype(int dt, const char* name) {
    if (dt != GMM_BF16 && dt != GMM_F32)
        return fail(GMM_ERR_DTYPE, "%s dtype %d is not GMM_BF16 or GMM_F32", name, dt);
    return GMM_OK;
}

// Bytes of the status block at the start of every workspace (word 0: the
// device status of the last call that used it).
constexpr size_t kWsStatusBytes = 256;

inline int check_ws(const void* ws, size_t ws_bytes, size_t need) {
    if (ws == nullptr || ws_bytes < need)
        return fail(GMM_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed%s", ws == nullptr ? 0 : ws_bytes,
                    need, ws == nullptr ? " (ws is NULL)" : "");
    if (!aligned16(ws)) return fail(GMM_ERR_ALIGN, "ws is not 16-byte aligned");
    return GMM_OK;
}

inline int32_t* ws_status(void* ws) { return reinterpret_cast<int32_t*>(ws); }

inline int hip_status(hipError_t e) {
    if (e != hipSuccess) return fail(GMM_ERR_HIP, "HIP launch failed: %s", hipGetErrorString(e));
    return GMM_OK;
}

#define GMM_TRY(expr)                 \
    do {                              \
        int _rc = (expr);             \
        if (_rc != GMM_OK) return _rc; \
    } while (0)

}  // namespace abi
}  // namespace gmm
