// C ABI of the calls around the experts' products (declared in
// include/gmm_moe.h): host-side argument checks, then launches on the caller's
// stream.  Nothing here allocates or synchronises.
#include <hip/hip_runtime.h>

#include "../../include/gmm_moe.h"
#include "gmm_check.hpp"
#include "gmm_launch.hpp"
#include "gmm_moe.hpp"

using namespace gmm::abi;

namespace {

// A tensor with one row per row of the problem: may be NULL when there are none.
int check_rows_ptr(const void* p, const char* name, int64_t rows) {
    return rows == 0 ? check_opt_ptr(p, name) : check_ptr(p, name);
}

int check_slots(int64_t T, int64_t k) {
    if (T < 0 || T > kMaxDim) return fail(GMM_ERR_SHAPE, "T=%lld out of range", (long long)T);
    if (k < 1 || k > GMM_MAX_TOPK) return fail(GMM_ERR_SHAPE, "k=%lld outside [1, %d]", (long long)k, GMM_MAX_TOPK);
    if (T * k > kMaxDim) return fail(GMM_ERR_SHAPE, "T k=%lld out of range", (long long)(T * k));
    return GMM_OK;
}

int check_route(int64_t T, int64_t E, int64_t k, int score, int logits_dtype) {
    GMM_TRY(check_out_dtype(logits_dtype, "logits"));
    if (score != GMM_SCORE_SOFTMAX && score != GMM_SCORE_SIGMOID)
        return fail(GMM_ERR_DTYPE, "score %d is not GMM_SCORE_SOFTMAX or GMM_SCORE_SIGMOID", score);
    if (E < 1 || E > GMM_MAX_GROUPS) return fail(GMM_ERR_SHAPE, "E=%lld outside [1, %d]", (long long)E, GMM_MAX_GROUPS);
    GMM_TRY(check_slots(T, k));
    if (k > E) return fail(GMM_ERR_SHAPE, "k=%lld of E=%lld experts", (long long)k, (long long)E);
    return GMM_OK;
}

int check_move(int64_t T, int64_t k, int64_t M, int64_t K) {
    GMM_TRY(check_slots(T, k));
    if (M < 0 || M > kMaxDim) return fail(GMM_ERR_SHAPE, "M=%lld out of range", (long long)M);
    return check_mult(K, 8, "K");
}

gmm::RouteArgs route_args(const void* logits, const float* bias, int64_t T, int64_t E, int64_t k, int score,
                          int normalize, float scale) {
    return gmm::RouteArgs{logits, bias, T, (int)E, (int)k, score == GMM_SCORE_SIGMOID, normalize != 0, scale};
}

gmm::MoveArgs move_args(const int32_t* row_of, const int32_t* slot_of, const float* weights, int64_t T, int64_t k,
                        int64_t M, int64_t K) {
    return gmm::MoveArgs{row_of, slot_of, weights, T, M, (int)k, K};
}

// A launch holds fewer than 2^32 threads: workgroups of 256 in one grid.
constexpr int64_t kMaxGrid = (int64_t(1) << 24) - 1;

int check_grid(int64_t blocks) {
    if (blocks > kMaxGrid) return fail(GMM_ERR_SHAPE, "grid too large");
    return GMM_OK;
}

int check_linear(int64_t M, int64_t K, int64_t N, int64_t G, int act) {
    GMM_TRY(check_groups(M, G));
    GMM_TRY(check_mult(K, 64, "K"));
    GMM_TRY(check_mult(N, 64, "N"));
    if (act < GMM_ACT_NONE || act > GMM_ACT_GELU_TANH) return fail(GMM_ERR_DTYPE, "act %d is not a gmm_activation", act);
    return GMM_OK;
}

gmm::FfnArgs linear_args(const int32_t* group_sizes, int64_t M, int64_t K, int64_t N, int64_t G, void* ws) {
    gmm::FfnArgs a = {};
    a.group_sizes = group_sizes;
    a.M = (int)M;
    a.K = (int)K;
    a.NN = (int)N;
    a.G = (int)G;
    a.status = ws_status(ws);
    return a;
}

const uint16_t* u16(const void* p) { return reinterpret_cast<const uint16_t*>(p); }

}  // namespace

extern "C" {

int gmm_route(const void* logits, int logits_dtype, const float* bias, int64_t T, int64_t E, int64_t k, int score,
              int normalize, float scale, int32_t* ids, float* weights, void* stream) {
    GMM_TRY(check_route(T, E, k, score, logits_dtype));
    GMM_TRY(check_rows_ptr(logits, "logits", T));
    GMM_TRY(check_opt_ptr(bias, "bias"));
    GMM_TRY(check_rows_ptr(ids, "ids", T));
    GMM_TRY(check_rows_ptr(weights, "weights", T));
    if (T == 0) return GMM_OK;
    return hip_status(gmm::launch_route(route_args(logits, bias, T, E, k, score, normalize, scale),
                                        logits_dtype == GMM_BF16, ids, weights, (hipStream_t)stream));
}

int gmm_route_bwd(const float* dweights, const void* logits, int logits_dtype, const int32_t* ids, int64_t T, int64_t E,
                  int64_t k, int score, int normalize, float scale, void* dlogits, int dlogits_dtype, void* stream) {
    GMM_TRY(check_out_dtype(dlogits_dtype, "dlogits"));
    GMM_TRY(check_route(T, E, k, score, logits_dtype));
    GMM_TRY(check_rows_ptr(dweights, "dweights", T));
    GMM_TRY(check_rows_ptr(logits, "logits", T));
    GMM_TRY(check_rows_ptr(ids, "ids", T));
    GMM_TRY(check_rows_ptr(dlogits, "dlogits", T));
    if (T == 0) return GMM_OK;
    return hip_status(gmm::launch_route_bwd(route_args(logits, nullptr, T, E, k, score, normalize, scale),
                                            logits_dtype == GMM_BF16, dweights, ids, dlogits,
                                            dlogits_dtype == GMM_BF16, (hipStream_t)stream));
}

int gmm_sort_tokens(const int32_t* ids, int64_t T, int64_t k, int64_t first, int64_t G, int64_t M,
                    int32_t* group_sizes, int32_t* row_of, int32_t* slot_of, void* ws, size_t ws_bytes, void* stream) {
    GMM_TRY(check_slots(T, k));
    GMM_TRY(check_groups(M, G));
    if (first < 0 || first > kMaxDim) return fail(GMM_ERR_SHAPE, "first=%lld out of range", (long long)first);
    GMM_TRY(check_rows_ptr(ids, "ids", T));
    GMM_TRY(check_ptr(group_sizes, "group_sizes"));
    GMM_TRY(check_rows_ptr(row_of, "row_of", T));
    GMM_TRY(check_rows_ptr(slot_of, "slot_of", M));
    GMM_TRY(check_ws(ws, ws_bytes, gmm_workspace_bytes(GMM_OP_SORT_TOKENS, T * k, 0, 0, G)));
    int32_t* counts = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kWsStatusBytes);
    return hip_status(gmm::launch_sort_tokens(ids, (int)(T * k), (int)first, (int)G, (int)M, group_sizes, row_of,
                                              slot_of, counts, ws_status(ws), (hipStream_t)stream));
}

int gmm_dispatch(const void* x, int dtype, const int32_t* row_of, const int32_t* slot_of, int64_t T, int64_t k,
                 int64_t M, int64_t K, void* out, void* stream) {
    GMM_TRY(check_out_dtype(dtype, "x"));
    GMM_TRY(check_move(T, k, M, K));
    GMM_TRY(check_rows_ptr(x, "x", T));
    GMM_TRY(check_rows_ptr(row_of, "row_of", T));
    GMM_TRY(check_rows_ptr(slot_of, "slot_of", M));
    GMM_TRY(check_rows_ptr(out, "out", M));
    if (M == 0) return GMM_OK;
    return hip_status(gmm::launch_dispatch(move_args(row_of, slot_of, nullptr, T, k, M, K), x, dtype == GMM_BF16, out,
                                           (hipStream_t)stream));
}

int gmm_combine(const void* y, int y_dtype, const int32_t* row_of, const float* weights, const void* residual,
                int64_t T, int64_t k, int64_t M, int64_t K, void* out, int out_dtype, void* stream) {
    GMM_TRY(check_out_dtype(y_dtype, "y"));
    GMM_TRY(check_out_dtype(out_dtype, "out"));
    GMM_TRY(check_move(T, k, M, K));
    GMM_TRY(check_rows_ptr(y, "y", M));
    GMM_TRY(check_rows_ptr(row_of, "row_of", T));
    GMM_TRY(check_opt_ptr(weights, "weights"));
    GMM_TRY(check_opt_ptr(residual, "residual"));
    GMM_TRY(check_rows_ptr(out, "out", T));
    if (T == 0) return GMM_OK;
    return hip_status(gmm::launch_combine(move_args(row_of, nullptr, weights, T, k, M, K), y, y_dtype == GMM_BF16,
                                          residual, out, out_dtype == GMM_BF16, (hipStream_t)stream));
}

int gmm_combine_bwd(const void* dout, int dout_dtype, const void* y, int y_dtype, const int32_t* row_of,
                    const int32_t* slot_of, const float* weights, int64_t T, int64_t k, int64_t M, int64_t K, void* dy,
                    float* dweights, void* stream) {
    GMM_TRY(check_out_dtype(dout_dtype, "dout"));
    GMM_TRY(check_out_dtype(y_dtype, "y"));
    GMM_TRY(check_move(T, k, M, K));
    GMM_TRY(check_rows_ptr(dout, "dout", T));
    GMM_TRY(check_rows_ptr(row_of, "row_of", T));
    if (dy == nullptr && dweights == nullptr && T > 0 && M > 0)
        return fail(GMM_ERR_NULL, "dy and dweights are both NULL");
    GMM_TRY(check_opt_ptr(dy, "dy"));
    GMM_TRY(check_opt_ptr(dweights, "dweights"));
    if (dy != nullptr) {
        GMM_TRY(check_rows_ptr(slot_of, "slot_of", M));
        GMM_TRY(check_rows_ptr(weights, "weights", T));
    }
    if (dweights != nullptr) GMM_TRY(check_rows_ptr(y, "y", M));
    if (dy == nullptr && dweights == nullptr) return GMM_OK;
    return hip_status(gmm::launch_combine_bwd(move_args(row_of, slot_of, weights, T, k, M, K), dout,
                                              dout_dtype == GMM_BF16, y, y_dtype == GMM_BF16, dy, dweights,
                                              (hipStream_t)stream));
}

int gmm_bf16_linear(const void* lhs, const void* rhs, const int32_t* group_sizes, int64_t M, int64_t K, int64_t N,
                    int64_t G, const void* bias, int bias_dtype, int act, const void* residual, void* out,
                    int out_dtype, void* pre, void* ws, size_t ws_bytes, void* stream) {
    GMM_TRY(check_out_dtype(out_dtype, "out"));
    if (bias != nullptr) GMM_TRY(check_out_dtype(bias_dtype, "bias"));
    GMM_TRY(check_linear(M, K, N, G, act));
    GMM_TRY(check_rows_ptr(lhs, "lhs", M));
    GMM_TRY(check_ptr(rhs, "rhs"));
    GMM_TRY(check_ptr(group_sizes, "group_sizes"));
    GMM_TRY(check_opt_ptr(bias, "bias"));
    GMM_TRY(check_opt_ptr(residual, "residual"));
    GMM_TRY(check_rows_ptr(out, "out", M));
    GMM_TRY(check_opt_ptr(pre, "pre"));
    GMM_TRY(check_grid(gmm::linear_fwd_blocks(M, N, G)));
    GMM_TRY(check_ws(ws, ws_bytes, gmm_workspace_bytes(GMM_OP_BF16_LINEAR, M, K, N, G)));
    if (M == 0) return GMM_OK;
    gmm::FfnArgs a = linear_args(group_sizes, M, K, N, G, ws);
    a.a = u16(lhs);
    a.b = u16(rhs);
    a.out = out;
    a.gu = reinterpret_cast<uint16_t*>(pre);
    a.bias = bias;
    a.bias_bf16 = bias_dtype == GMM_BF16;
    a.residual = residual;
    a.act = act;
    return hip_status(gmm::launch_linear_fwd(a, out_dtype == GMM_BF16, (hipStream_t)stream));
}

int gmm_bf16_linear_bwd(const void* dout, const void* rhs, const int32_t* group_sizes, const void* lhs,
                        const void* pre, int act, int64_t M, int64_t K, int64_t N, int64_t G, void* dx, int dx_dtype,
                        void* dw, int dw_dtype, void* db, int db_dtype, void* ws, size_t ws_bytes, void* stream) {
    if (dx != nullptr) GMM_TRY(check_out_dtype(dx_dtype, "dx"));
    if (dw != nullptr) GMM_TRY(check_out_dtype(dw_dtype, "dw"));
    if (db != nullptr) GMM_TRY(check_out_dtype(db_dtype, "db"));
    GMM_TRY(check_linear(M, K, N, G, act));
    GMM_TRY(check_rows_ptr(dout, "dout", M));
    GMM_TRY(check_ptr(group_sizes, "group_sizes"));
    if (act != GMM_ACT_NONE) GMM_TRY(check_rows_ptr(pre, "pre", M));
    else GMM_TRY(check_opt_ptr(pre, "pre"));
    if (dx != nullptr) GMM_TRY(check_ptr(rhs, "rhs"));
    if (dw != nullptr) GMM_TRY(check_rows_ptr(lhs, "lhs", M));
    if (dx == nullptr && dw == nullptr && db == nullptr && M > 0)
        return fail(GMM_ERR_NULL, "dx, dw and db are all NULL");
    GMM_TRY(check_opt_ptr(dx, "dx"));
    GMM_TRY(check_opt_ptr(dw, "dw"));
    GMM_TRY(check_opt_ptr(db, "db"));
    GMM_TRY(check_grid(gmm::linear_part_words(M, N, G) / 64));
    if (db != nullptr) GMM_TRY(check_grid(gmm::linear_db_blocks(N, G)));
    GMM_TRY(check_grid(gmm::ffn_dx_blocks(M, K, G)));
    GMM_TRY(check_grid(gmm::ffn_dw_blocks(K, N, G)));
    GMM_TRY(check_ws(ws, ws_bytes, gmm_workspace_bytes(GMM_OP_BF16_LINEAR_BWD, M, K, N, G)));
    hipStream_t s = (hipStream_t)stream;
    uint16_t* dpre = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + kWsStatusBytes);
    float* part = reinterpret_cast<float*>(dpre + M * N);
    const bool products = dx != nullptr || dw != nullptr;
    GMM_TRY(hip_status(gmm::launch_linear_grad(dout, pre, act, group_sizes, (int)M, (int)N, (int)G,
                                               products ? dpre : nullptr, db, db_dtype == GMM_BF16, part, ws_status(ws), s)));
    gmm::FfnArgs x = linear_args(group_sizes, M, K, N, G, ws), w = x;
    x.a = act == GMM_ACT_NONE ? u16(dout) : dpre;
    x.b = u16(rhs);
    x.out = dx;
    w.a = u16(lhs);
    w.b = x.a;
    w.out = dw;
    const bool want_dx = dx != nullptr && M > 0;
    if (want_dx && dw != nullptr)
        return hip_status(gmm::launch_ffn_bwd(x, dx_dtype == GMM_BF16, w, dw_dtype == GMM_BF16, s));
    if (want_dx) return hip_status(gmm::launch_ffn_dx(x, dx_dtype == GMM_BF16, s));
    if (dw != nullptr) return hip_status(gmm::launch_ffn_dw(w, dw_dtype == GMM_BF16, s));
    return GMM_OK;
}

}  // extern "C"
