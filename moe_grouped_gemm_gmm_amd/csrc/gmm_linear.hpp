// Epilogue of the plain grouped product, pre = x . w[g] + b[g], out = act(pre)
// + residual, and the activations' slopes (device side).  Everything is in
// fp32; out is rounded once, and pre, where it is kept, once to bf16.
//
// The activations are written so that small results keep their digits: z times
// a sigmoid for SiLU and the tanh form of GELU (1 + tanh(u) = 2 / (1 +
// exp(-2u))), z erfc(-z / sqrt 2) / 2 for GELU, whose 1 + erf would cancel for
// z below -3.  An exponential that overflows gives 0.
#pragma once

#include "gmm_launch.hpp"
#include "gmm_mx8.hpp"

#include <type_traits>

namespace gmm {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

__device__ __forceinline__ float logistic(float u) { return 1.0f / (1.0f + expf(-u)); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == kActRelu) return z > 0.0f ? z : 0.0f;
    else if constexpr (ACT == kActSilu) return z * logistic(z);
    else if constexpr (ACT == kActGelu) return 0.5f * z * erfcf(-z * kSqrtHalf);
    else if constexpr (ACT == kActGeluTanh) return z * logistic(kTanhScale * (z + kTanhCubic * z * z * z));
    else return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
    else if constexpr (ACT == kActSilu) {
        const float s = logistic(z);
        return s + z * s * (1.0f - s);
    } else if constexpr (ACT == kActGelu) {
        return 0.5f * erfcf(-z * kSqrtHalf) + z * kInvSqrt2Pi * expf(-0.5f * z * z);
    } else if constexpr (ACT == kActGeluTanh) {
        const float s = logistic(kTanhScale * (z + kTanhCubic * z * z * z));
        return s + z * s * (1.0f - s) * (kTanhScale * (1.0f + 3.0f * kTanhCubic * z * z));
    } else return 1.0f;
}

// f(ACT) for the call's activation, the same in the whole grid.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
        case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
        case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
        case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
        default: break;
    }
}

// N (4 or 8) consecutive values of a tensor in bf16 or fp32.
template <int N>
__device__ __forceinline__ void load_n(const void* p, bool bf16, int64_t e, float (&v)[N]) {
    if (bf16) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint2 d = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + e + i);
            v[i] = bf16_lo(d.x);
            v[i + 1] = bf16_hi(d.x);
            v[i + 2] = bf16_lo(d.y);
            v[i + 3] = bf16_hi(d.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 d = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + e + i);
            v[i] = d.x;
            v[i + 1] = d.y;
            v[i + 2] = d.z;
            v[i + 3] = d.w;
        }
    }
}

// b[g, col ..], zeros without a bias.
template <int N>
__device__ __forceinline__ void linear_bias(const FfnArgs& a, int g, int col, float (&v)[N]) {
    if (a.bias != nullptr) {
        load_n<N>(a.bias, a.bias_bf16 != 0, (int64_t)g * a.NN + col, v);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
    }
}

// N (4 or 8) consecutive bf16 or fp32 results of one row.
template <bool BF16, int N>
__device__ __forceinline__ void store_n(void* p, int64_t e, const float (&v)[N]) {
    if constexpr (!BF16) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            store_out(static_cast<float*>(p) + e + i, make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
    } else if constexpr (N == 4) {
        store_out(static_cast<uint16_t*>(p) + e, make_uint2(pack_rne(v[0], v[1]), pack_rne(v[2], v[3])));
    } else {
        store_out(static_cast<uint16_t*>(p) + e, make_uint4(pack_rne(v[0], v[1]), pack_rne(v[2], v[3]),
                                                            pack_rne(v[4], v[5]), pack_rne(v[6], v[7])));
    }
}

// From the sums z of N columns of a row to everything the call writes there.
template <bool OUT_BF16, int N>
__device__ __forceinline__ void linear_finish(const FfnArgs& a, int row, int col, const float (&bias)[N], float (&z)[N]) {
    const int64_t e = (int64_t)row * a.NN + col;
    float r[N];
    if (a.residual != nullptr) load_n<N>(a.residual, OUT_BF16, e, r);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] += bias[i];
    if (a.gu != nullptr) store_n<true, N>(a.gu, e, z);
    with_act(a.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = act_value<decltype(act)::value>(z[i]);
    });
    if (a.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] += r[i];
    }
    store_n<OUT_BF16, N>(a.out, e, z);
}

}  // namespace gmm
