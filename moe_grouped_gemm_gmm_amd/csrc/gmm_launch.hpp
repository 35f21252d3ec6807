// Internal launchers behind the C ABI of gmm.h.  Arguments are already
// validated by gmm_api.cpp; each launcher only enqueues kernels on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_config.hpp"

namespace gmm {

// Compute units of the current device (queried once).
inline int device_cus() {
    static const int cus = [] {
        int dev = 0, n = 0;
        if (hipGetDevice(&dev) != hipSuccess ||
            hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
            n = 256;
        return n;
    }();
    return cus;
}

// Every grouped launcher takes `status`: a device int32 that block 0 of the
// launch sets to the call's device status (bits kDevSumGtM, kDevNegativeSize
// of gmm_device.hpp; 0 when group_sizes keeps the contract).

// Bytes of the library-owned device scratch behind gmm_fp8_fwd_noalloc, and
// its device address on the current device (found once per device).
constexpr size_t kNoallocScratchBytes = 4096;
hipError_t noalloc_scratch(void** ptr, size_t* bytes);

// Streaming read of `bytes` (a multiple of 64 KB) with one 64 KB slice per
// workgroup; sink has one word per slice.
hipError_t launch_probe_stream_read(const void* buf, int64_t bytes, uint32_t* sink,
                                    hipStream_t stream);

hipError_t launch_group_metadata(const int32_t* group_sizes, int G, int M, int tm,
                                 int32_t* offsets, int32_t* work, int capacity,
                                 int32_t* num_work, int32_t* status, hipStream_t stream);

// x_bf16: true for bf16 input, false for fp32.
hipError_t launch_quantize_lhs(const void* x, bool x_bf16, int64_t M, int64_t K, uint8_t* q,
                               float* scale, hipStream_t stream);

hipError_t launch_quantize_rhs(const void* w, bool w_bf16, int64_t G, int64_t K, int64_t N,
                               uint8_t* q, float* scale, hipStream_t stream);

// Logical [G,K,N] E4M3 codes into the packed order of launch_quantize_rhs.
hipError_t launch_pack_rhs(const uint8_t* q, int64_t G, int64_t K, int64_t N, uint8_t* packed,
                           hipStream_t stream);

// s = a/448 and its guarded inverse for n block abs-maxima (the quantisers'
// own device routines).
hipError_t launch_quant_scales(const float* amax, int64_t n, float* scale, float* inv,
                               hipStream_t stream);

// MXFP4 weights in the forward's packed operand order (codes G*K*N/2 bytes,
// E8M0 scales G*K*N/32 bytes).
hipError_t launch_quantize_rhs_mxfp4(const void* w, bool w_bf16, int64_t G, int64_t K, int64_t N,
                                     uint8_t* q, uint8_t* scale, hipStream_t stream);

// int4 weights (codes in [-8, 7], 128x128 fp32 block scales s = a/7) in the
// forward's packed operand order (G*K*N/2 bytes); and int4 codes made
// elsewhere (int8 values, logical [G,K,N]) into that order.
hipError_t launch_quantize_rhs_int4(const void* w, bool w_bf16, int64_t G, int64_t K, int64_t N,
                                    uint8_t* q, float* scale, hipStream_t stream);
hipError_t launch_pack_rhs_int4(const int8_t* q, int64_t G, int64_t K, int64_t N, uint8_t* packed,
                                hipStream_t stream);

// lhs_kind: 0 = E4M3 codes + lhs_scale, 1 = bf16, 2 = fp32.
hipError_t launch_fp8_fwd(const TileConfig& cfg, const void* lhs, int lhs_kind, const float* lhs_scale,
                          const uint8_t* rhs, const float* rhs_scale,
                          const int32_t* group_sizes, int M, int K, int N, int G, void* out,
                          bool out_bf16, uint8_t* q_out, float* scale_out, int32_t* status, hipStream_t stream);

// Fused gate+up: rhs has 2N columns (gate, then up); out = silu(gate) * up,
// [M,N]; act_q/act_scale (both or neither) the 1x128 quantised activation.
hipError_t launch_fp8_fwd_swiglu(const TileConfig& cfg, const void* lhs, int lhs_kind, const float* lhs_scale,
                                 const uint8_t* rhs, const float* rhs_scale,
                                 const int32_t* group_sizes, int M, int K, int N, int G,
                                 void* out, bool out_bf16, uint8_t* act_q, float* act_scale,
                                 int32_t* status, hipStream_t stream);

// FP8 (1x128) LHS against packed MXFP4 weights.
hipError_t launch_fp8_mxfp4_fwd(const TileConfig& cfg, const void* lhs, int lhs_kind, const float* lhs_scale,
                                const uint8_t* rhs_q, const uint8_t* rhs_scale,
                                const int32_t* group_sizes, int M, int K, int N, int G, void* out,
                                bool out_bf16, int32_t* status, hipStream_t stream);

// FP8 (1x128) LHS against packed int4 weights with 128x128 fp32 block scales.
hipError_t launch_fp8_int4_fwd(const TileConfig& cfg, const void* lhs, int lhs_kind, const float* lhs_scale,
                               const uint8_t* rhs_q, const float* rhs_scale,
                               const int32_t* group_sizes, int M, int K, int N, int G, void* out,
                               bool out_bf16, int32_t* status, hipStream_t stream);

hipError_t launch_bf16_fwd(const TileConfig& cfg, const void* lhs, const void* rhs, const int32_t* group_sizes, int M,
                           int K, int N, int G, void* out, bool out_bf16, int32_t* status, hipStream_t stream);

hipError_t launch_bf16_dx(const TileConfig& cfg, const void* dy, const void* w, const int32_t* group_sizes, int M,
                          int K, int N, int G, void* dx, bool out_bf16, int32_t* status, hipStream_t stream);

hipError_t launch_tgmm(const TileConfig& cfg, const void* x, const void* dy, const int32_t* group_sizes, int M, int K,
                       int N, int G, void* dw, bool out_bf16, int32_t* status, hipStream_t stream);

constexpr int64_t kMx8BlockSize = 32;   // values that share a checkpoint scale

// 8-bit checkpoints (gmm_mx8.hpp): codes [M,K] and E8M0 scales [M,K/32] of x,
// and the values back.
hipError_t launch_quantize_mx8(const void* x, bool x_bf16, int64_t M, int64_t K, uint8_t* q, uint8_t* scale,
                               hipStream_t stream);
hipError_t launch_dequantize_mx8(const uint8_t* q, const uint8_t* scale, int64_t M, int64_t K, void* out,
                                 bool out_bf16, hipStream_t stream);

// dP [M,2N] (bf16) of h = silu(gate) * up from dh [M,N] and P in bf16 (gu) or
// as a checkpoint (gu_q, gu_s); h, when given, receives the recomputed h.
hipError_t launch_gated_grad(const void* dh, const void* gu, const uint8_t* gu_q, const uint8_t* gu_s,
                             const int32_t* group_sizes, int M, int N, int G, void* dgu, void* h,
                             int32_t* status, hipStream_t stream);

// Operands of the gated block's grouped products.  NN is the column count of
// the second operand (2N for the fused gate and up weights).
struct FfnArgs {
    const uint16_t* a;                    // x [M,K], or dP [M,NN] for dx
    const uint8_t *aq, *as;               // x as a checkpoint (the weight gradient; else NULL)
    const uint16_t* b;                    // w [G,K,NN], or dP / dy [M,NN] for the weight gradient
    const int32_t* group_sizes;
    int M, K, NN, G;
    void* out;                            // h [M,NN/2], dx [M,K] or dw [G,K,NN]
    uint16_t* gu;                         // the forward's P, or NULL
    uint8_t *gu_q, *gu_s;                 // the forward's P as a checkpoint, or NULL
    int ntiles_c, ntiles_r, nblocks, cap;   // set by the launcher (cap: rows of a load-wave item)
    int32_t* status;
};
hipError_t launch_gated_fwd(const FfnArgs& a, bool out_bf16, hipStream_t stream);
hipError_t launch_ffn_dx(const FfnArgs& a, bool out_bf16, hipStream_t stream);
hipError_t launch_ffn_dw(const FfnArgs& a, bool out_bf16, hipStream_t stream);
// Both, in one launch where that pays.
hipError_t launch_ffn_bwd(const FfnArgs& x, bool x_bf16, const FfnArgs& w, bool w_bf16, hipStream_t stream);

// The kernel and tiles that a call takes (decided by its sizes alone; M >= 1).
enum FfnKernel { kFfnFewRows = 1, kFfnTiles = 2, kFfnLoadWaves = 3, kFfnBoth = 4 };
struct FfnChoice {
    int kernel, waves, rows, cols;   // FfnKernel; waves of a workgroup; rows and columns of a tile
};
FfnChoice gated_fwd_choice(int M, int K, int NN, int G, bool keep_mx8);
FfnChoice ffn_dx_choice(int M, int K, int NN, int G);
FfnChoice ffn_dw_choice(int K, int NN, int G);
// dX's choice in a backward call for dX and dW: kFfnBoth when one launch computes both.
FfnChoice ffn_bwd_choice(int M, int K, int NN, int G);

// Upper bounds of these launches' grids.
int64_t gated_fwd_blocks(int64_t M, int64_t N, int64_t G);
int64_t ffn_dx_blocks(int64_t M, int64_t K, int64_t G);
int64_t ffn_dw_blocks(int64_t K, int64_t NN, int64_t G);

}  // namespace gmm
