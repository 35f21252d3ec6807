// C ABI of the gated expert block and of 8-bit activation checkpoints
// (declared in include/gmm_ffn.h): host-side argument checks, then launches
// on the caller's stream.  Nothing here allocates or synchronises.
#include <hip/hip_runtime.h>

#include "../../include/gmm_ffn.h"
#include "gmm_check.hpp"
#include "gmm_launch.hpp"

using namespace gmm::abi;

namespace {

// A launch holds fewer than 2^32 threads: workgroups of 256 in one grid.
constexpr int64_t kMaxGrid = (int64_t(1) << 24) - 1;

// A tensor with one row per row of the problem: may be NULL when there are none.
int check_rows_ptr(const void* p, const char* name, int64_t M) {
    return M == 0 ? check_opt_ptr(p, name) : check_ptr(p, name);
}

// A tensor given in bf16 or as a checkpoint (codes and scales), exactly one.
int check_kept(const void* plain, const uint8_t* q, const uint8_t* scale, const char* name, int64_t M) {
    if (plain != nullptr && (q != nullptr || scale != nullptr))
        return fail(GMM_ERR_DTYPE, "%s is given in bf16 and as a checkpoint", name);
    if ((q != nullptr) != (scale != nullptr))
        return fail(GMM_ERR_NULL, "%s: codes and scales are needed together", name);
    if (plain == nullptr && q == nullptr && M > 0) return fail(GMM_ERR_NULL, "%s is NULL", name);
    GMM_TRY(check_opt_ptr(plain, name));
    GMM_TRY(check_opt_ptr(q, name));
    return check_opt_ptr(scale, name);
}

int check_blocks(int64_t M, int64_t K) {
    if (M < 0 || M > kMaxDim) return fail(GMM_ERR_SHAPE, "M=%lld out of range", (long long)M);
    GMM_TRY(check_mult(K, gmm::kMx8BlockSize, "K"));
    if (M * (K / 8) > kMaxDim * 256) return fail(GMM_ERR_SHAPE, "tensor too large");
    return GMM_OK;
}

// Widths of the fused weights: 2N columns have to fit an int too.
int check_widths(int64_t M, int64_t K, int64_t N, int64_t G) {
    GMM_TRY(check_groups(M, G));
    GMM_TRY(check_mult(K, 64, "K"));
    GMM_TRY(check_mult(N, 64, "N"));
    if (N > kMaxDim / 2) return fail(GMM_ERR_SHAPE, "N=%lld out of range", (long long)N);
    return GMM_OK;
}

// The smallest tiles any of the grouped kernels cuts an operation into.
int check_grid(int64_t blocks) {
    if (blocks > kMaxGrid) return fail(GMM_ERR_SHAPE, "grid too large");
    return GMM_OK;
}

gmm::FfnArgs args_of(const int32_t* group_sizes, int64_t M, int64_t K, int64_t NN, int64_t G, void* ws) {
    gmm::FfnArgs a = {};
    a.group_sizes = group_sizes;
    a.M = (int)M;
    a.K = (int)K;
    a.NN = (int)NN;
    a.G = (int)G;
    a.status = ws_status(ws);
    return a;
}

const uint16_t* u16(const void* p) { return reinterpret_cast<const uint16_t*>(p); }

}  // namespace

extern "C" {

int gmm_quantize_mx8(const void* x, int x_dtype, int64_t M, int64_t K, uint8_t* q, uint8_t* scale, void* stream) {
    if (x_dtype != GMM_BF16 && x_dtype != GMM_F32)
        return fail(GMM_ERR_DTYPE, "x dtype %d is not GMM_BF16 or GMM_F32", x_dtype);
    GMM_TRY(check_blocks(M, K));
    GMM_TRY(check_rows_ptr(x, "x", M));
    GMM_TRY(check_rows_ptr(q, "q", M));
    GMM_TRY(check_rows_ptr(scale, "scale", M));
    if (M == 0) return GMM_OK;
    return hip_status(gmm::launch_quantize_mx8(x, x_dtype == GMM_BF16, M, K, q, scale, (hipStream_t)stream));
}

int gmm_dequantize_mx8(const uint8_t* q, const uint8_t* scale, int64_t M, int64_t K, void* out, int out_dtype,
                       void* stream) {
    GMM_TRY(check_out_dtype(out_dtype, "out"));
    GMM_TRY(check_blocks(M, K));
    GMM_TRY(check_rows_ptr(q, "q", M));
    GMM_TRY(check_rows_ptr(scale, "scale", M));
    GMM_TRY(check_rows_ptr(out, "out", M));
    if (M == 0) return GMM_OK;
    return hip_status(gmm::launch_dequantize_mx8(q, scale, M, K, out, out_dtype == GMM_BF16, (hipStream_t)stream));
}

int gmm_bf16_swiglu(const void* lhs, const void* rhs, const int32_t* group_sizes, int64_t M, int64_t K, int64_t N,
                    int64_t G, void* out, int out_dtype, void* gu, uint8_t* gu_q, uint8_t* gu_scale, void* ws,
                    size_t ws_bytes, void* stream) {
    GMM_TRY(check_out_dtype(out_dtype, "out"));
    GMM_TRY(check_widths(M, K, N, G));
    GMM_TRY(check_rows_ptr(lhs, "lhs", M));
    GMM_TRY(check_ptr(rhs, "rhs"));
    GMM_TRY(check_ptr(group_sizes, "group_sizes"));
    GMM_TRY(check_rows_ptr(out, "out", M));
    if (gu != nullptr || gu_q != nullptr || gu_scale != nullptr) GMM_TRY(check_kept(gu, gu_q, gu_scale, "gu", M));
    GMM_TRY(check_grid(gmm::gated_fwd_blocks(M, N, G)));
    GMM_TRY(check_ws(ws, ws_bytes, gmm_workspace_bytes(GMM_OP_BF16_SWIGLU, M, K, N, G)));
    if (M == 0) return GMM_OK;
    gmm::FfnArgs a = args_of(group_sizes, M, K, 2 * N, G, ws);
    a.a = u16(lhs);
    a.b = u16(rhs);
    a.out = out;
    a.gu = reinterpret_cast<uint16_t*>(gu);
    a.gu_q = gu_q;
    a.gu_s = gu_scale;
    return hip_status(gmm::launch_gated_fwd(a, out_dtype == GMM_BF16, (hipStream_t)stream));
}

int gmm_bf16_swiglu_bwd(const void* dh, const void* rhs, const int32_t* group_sizes, const void* lhs,
                        const uint8_t* lhs_q, const uint8_t* lhs_scale, const void* gu, const uint8_t* gu_q,
                        const uint8_t* gu_scale, int64_t M, int64_t K, int64_t N, int64_t G, void* dx, int dx_dtype,
                        void* dw, int dw_dtype, void* h, void* ws, size_t ws_bytes, void* stream) {
    if (dx != nullptr) GMM_TRY(check_out_dtype(dx_dtype, "dx"));
    if (dw != nullptr) GMM_TRY(check_out_dtype(dw_dtype, "dw"));
    GMM_TRY(check_widths(M, K, N, G));
    GMM_TRY(check_rows_ptr(dh, "dh", M));
    GMM_TRY(check_ptr(group_sizes, "group_sizes"));
    GMM_TRY(check_kept(gu, gu_q, gu_scale, "gu", M));
    if (dx != nullptr) GMM_TRY(check_ptr(rhs, "rhs"));
    if (dw != nullptr) GMM_TRY(check_kept(lhs, lhs_q, lhs_scale, "lhs", M));
    if (dx == nullptr && dw == nullptr && h == nullptr && M > 0)
        return fail(GMM_ERR_NULL, "dx, dw and h are all NULL");
    GMM_TRY(check_opt_ptr(dx, "dx"));
    GMM_TRY(check_opt_ptr(dw, "dw"));
    GMM_TRY(check_opt_ptr(h, "h"));
    GMM_TRY(check_grid(M * (N / 8) / 256 + 1));
    GMM_TRY(check_grid(gmm::ffn_dx_blocks(M, K, G)));
    GMM_TRY(check_grid(gmm::ffn_dw_blocks(K, 2 * N, G)));
    GMM_TRY(check_ws(ws, ws_bytes, gmm_workspace_bytes(GMM_OP_BF16_SWIGLU_BWD, M, K, N, G)));
    hipStream_t s = (hipStream_t)stream;
    uint16_t* dp = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + kWsStatusBytes);
    if (M > 0)
        GMM_TRY(hip_status(gmm::launch_gated_grad(dh, gu, gu_q, gu_scale, group_sizes, (int)M, (int)N, (int)G, dp, h,
                                                  ws_status(ws), s)));
    gmm::FfnArgs x = args_of(group_sizes, M, K, 2 * N, G, ws), w = x;
    x.a = dp;
    x.b = u16(rhs);
    x.out = dx;
    w.a = u16(lhs);
    w.aq = lhs_q;
    w.as = lhs_scale;
    w.b = dp;
    w.out = dw;
    const bool want_dx = dx != nullptr && M > 0;
    if (want_dx && dw != nullptr)
        return hip_status(gmm::launch_ffn_bwd(x, dx_dtype == GMM_BF16, w, dw_dtype == GMM_BF16, s));
    if (want_dx) return hip_status(gmm::launch_ffn_dx(x, dx_dtype == GMM_BF16, s));
    if (dw != nullptr) return hip_status(gmm::launch_ffn_dw(w, dw_dtype == GMM_BF16, s));
    return GMM_OK;
}

int tgmm_mx8(const uint8_t* x_q, const uint8_t* x_scale, const void* dy, const int32_t* group_sizes, int64_t M,
             int64_t K, int64_t N, int64_t G, void* dw, int out_dtype, void* ws, size_t ws_bytes, void* stream) {
    GMM_TRY(check_out_dtype(out_dtype, "dw"));
    GMM_TRY(check_widths(M, K, N, G));
    GMM_TRY(check_rows_ptr(x_q, "x_q", M));
    GMM_TRY(check_rows_ptr(x_scale, "x_scale", M));
    GMM_TRY(check_rows_ptr(dy, "dy", M));
    GMM_TRY(check_ptr(group_sizes, "group_sizes"));
    GMM_TRY(check_ptr(dw, "dw"));
    GMM_TRY(check_grid(gmm::ffn_dw_blocks(K, N, G)));
    GMM_TRY(check_ws(ws, ws_bytes, gmm_workspace_bytes(GMM_OP_TGMM_MX8, M, K, N, G)));
    gmm::FfnArgs a = args_of(group_sizes, M, K, N, G, ws);
    a.aq = x_q;
    a.as = x_scale;
    a.b = u16(dy);
    a.out = dw;
    return hip_status(gmm::launch_ffn_dw(a, out_dtype == GMM_BF16, (hipStream_t)stream));
}

}  // extern "C"
