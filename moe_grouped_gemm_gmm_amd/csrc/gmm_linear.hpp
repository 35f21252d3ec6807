// Epilogue of the plain grouped product, pre = x . w[g] + b[g], out = act(pre)
// + residual, and the activations' slopes (device side).  Everything is in
// fp32; out is rounded once, and pre, where it is kept, once to bf16.
//
// The activations are written so that small results keep their digits, from
// the hardware's 2^x and 1/x: an epilogue runs them on every output, and with
// library exponentials and divisions SiLU alone cost the 128 x 128 tiles a third
// of their time (3000 rows, 8 experts, K = 512, N = 2048: 19.5 us, 16.2 so; no activation 15.3).
//   SiLU, tanh form of GELU: z / (1 + exp(-u)), since 1 + tanh(v) = 2 / (1 +
//     exp(-2v)).  An exponential that overflows gives 0.
//   GELU: with h = erfc(|z| / sqrt 2) / 2 it is z h for z < 0 and z (1 - h)
//     above; 1 + erf would cancel below -3.  h = exp(-z^2 / 2) q(t), t = 1 / (1 +
//     |z| / (2 sqrt 2)): q is a polynomial of degree 9, fitted to erfc(x)
//     exp(x^2) / 2 on 0 <= x <= 14 by least squares on relative errors,
//     reweighted until they are level; off by 3.3e-7 of the value at most,
//     evaluated in fp32.
#pragma once

#include "gmm_launch.hpp"
#include "gmm_mx8.hpp"

#include <type_traits>

namespace gmm {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

constexpr float kLog2E = 1.44269504088896341f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

__device__ __forceinline__ float logistic(float u) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * u));
}

// exp(-z^2 / 2), and erfc(|z| / sqrt 2) / 2 over it.
__device__ __forceinline__ float gauss(float z) { return __builtin_amdgcn_exp2f(-0.5f * kLog2E * (z * z)); }
__device__ __forceinline__ float half_erfcx(float z) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(z), 0.35355339059327376f, 1.0f));
    float q = -2.940962091e-02f;
    q = __builtin_fmaf(q, t, 1.416352689e-01f);
    q = __builtin_fmaf(q, t, -2.421303689e-01f);
    q = __builtin_fmaf(q, t, 1.371632516e-01f);
    q = __builtin_fmaf(q, t, -1.183455344e-02f);
    q = __builtin_fmaf(q, t, 1.005925909e-01f);
    q = __builtin_fmaf(q, t, 1.217964739e-01f);
    q = __builtin_fmaf(q, t, 1.411384493e-01f);
    q = __builtin_fmaf(q, t, 1.410487443e-01f);
    return __builtin_fmaf(q, t, -2.655870617e-07f);
}
// P(x <= z) of a standard normal, given gauss(z).
__device__ __forceinline__ float normal_cdf(float z, float e) {
    const float h = e * half_erfcx(z);
    return z < 0.0f ? h : 1.0f - h;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == kActRelu) return z <= 0.0f ? 0.0f : z;   // a NaN stays one
    else if constexpr (ACT == kActSilu) return z * logistic(z);
    else if constexpr (ACT == kActGelu) return z * normal_cdf(z, gauss(z));
    else if constexpr (ACT == kActGeluTanh) return z * logistic(kTanhScale * (z + kTanhCubic * z * z * z));
    else return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    else if constexpr (ACT == kActSilu) {
        const float s = logistic(z);
        return s + z * s * (1.0f - s);
    } else if constexpr (ACT == kActGelu) {
        const float e = gauss(z);
        return normal_cdf(z, e) + z * kInvSqrt2Pi * e;
    } else if constexpr (ACT == kActGeluTanh) {
        // s (1 - s) is 0 long before z^2 overflows: the bound keeps 0 times infinity out
        const float s = logistic(kTanhScale * (z + kTanhCubic * z * z * z)), z2 = fminf(z * z, 0x1p100f);
        return s + z * s * (1.0f - s) * (kTanhScale * (1.0f + 3.0f * kTanhCubic * z2));
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

// From the sums z of N columns of a row to everything the call writes there; r:
// the residual's values, if there is one.
template <bool OUT_BF16, int N>
__device__ __forceinline__ void linear_finish(const FfnArgs& a, int row, int col, const float (&bias)[N],
                                              const float (&r)[N], float (&z)[N]) {
    const int64_t e = (int64_t)row * a.NN + col;
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

// The same with the residual read here.
template <bool OUT_BF16, int N>
__device__ __forceinline__ void linear_finish(const FfnArgs& a, int row, int col, const float (&bias)[N], float (&z)[N]) {
    float r[N];
    if (a.residual != nullptr) load_n<N>(a.residual, OUT_BF16, (int64_t)row * a.NN + col, r);
    linear_finish<OUT_BF16, N>(a, row, col, bias, r, z);
}

// Eight values of the residual as they are stored, and as fp32.
template <bool BF16>
struct ResidualVec {
    uint4 d[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* p, int64_t e) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + e * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) d[i] = q[i];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (BF16) {
            v[0] = bf16_lo(d[0].x); v[1] = bf16_hi(d[0].x); v[2] = bf16_lo(d[0].y); v[3] = bf16_hi(d[0].y);
            v[4] = bf16_lo(d[0].z); v[5] = bf16_hi(d[0].z); v[6] = bf16_lo(d[0].w); v[7] = bf16_hi(d[0].w);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(d[i].x);
                v[4 * i + 1] = __uint_as_float(d[i].y);
                v[4 * i + 2] = __uint_as_float(d[i].z);
                v[4 * i + 3] = __uint_as_float(d[i].w);
            }
        }
    }
};

}  // namespace gmm
