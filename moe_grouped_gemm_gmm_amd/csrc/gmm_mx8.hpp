// The 8-bit checkpoint format (device side): blocks of 32 consecutive values
// of a row share a power-of-two scale, kept as an E8M0 byte c standing for
// 2^(c - 127); each value is an E4M3 code of value / 2^(c - 127).
//
// c is the smallest with max|v| <= 448 * 2^(c - 127) (0 for an all-zero
// block), so the largest value of a block never saturates: with max|v| =
// m * 2^k, 1 <= m < 2, and 448 = 1.75 * 2^8, c - 127 is k - 8 for m <= 1.75
// and k - 7 above, which is one comparison on the bits of max|v|.  Scaling by
// a power of two is exact, so the only rounding is the E4M3 one (half a step,
// 2^-4 of the value), and a value read back has 4 significant bits: it is
// exact in bf16, and the bf16 MFMAs of the backward pass see exactly what the
// checkpoint stands for.
#pragma once

#include "gmm_device.hpp"

namespace gmm {

constexpr int kMx8Block = 32;

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// E8M0 byte of a block from the bits of its max|v|.
__device__ __forceinline__ uint32_t mx8_scale_code(uint32_t amax_bits) {
    const int c = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(c, 0);
}

// 2^(127 - c), the factor that codes are made with (c <= 247).
__device__ __forceinline__ float mx8_inverse(uint32_t c) { return __uint_as_float((254u - c) << 23); }

// 2^(c - 127), the factor that codes are read with.
__device__ __forceinline__ float mx8_scale(uint32_t c) {
    return __uint_as_float(c == 0 ? 0x00400000u : c << 23);
}

// Bits of |v|, 0 for a NaN: it keeps its NaN code under any scale, and the
// block's other values theirs.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(fmaxf(fabsf(v), 0.0f)); }

// Four E4M3 codes -> their values times s.
__device__ __forceinline__ void mx8_values4(uint32_t codes, float s, float (&v)[4]) {
    const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
    const v2f hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
    v[0] = lo[0] * s;
    v[1] = lo[1] * s;
    v[2] = hi[0] * s;
    v[3] = hi[1] * s;
}

// Two fp32 -> packed bf16, round to nearest even (one instruction on gfx950).
__device__ __forceinline__ uint32_t pack_rne(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi});
}

// Maximum over the four lanes l % 16, +16, +32, +48 (non-negative floats as
// bits): the 16- and 32-lane swaps of gfx950 put each lane's partner beside
// its own value.
__device__ __forceinline__ uint32_t max_over_rows16(uint32_t u) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t m = max(a[0], a[1]);
    const u32x2 b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return max(b[0], b[1]);
}

}  // namespace gmm
