// Element-wise kernels of the gated expert block's training path: the 8-bit
// checkpoint written and read back, and the gradient of silu(gate) * up.
#include "gmm_launch.hpp"
#include "gmm_mx8.hpp"

namespace gmm {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Eight consecutive values of a row as fp32.
struct Bf16Source {
    const uint16_t* p;
    __device__ void load8(int64_t e, float (&v)[8]) const {
        const u32x4 d = *reinterpret_cast<const u32x4*>(p + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(d[i]);
            v[2 * i + 1] = bf16_hi(d[i]);
        }
    }
};
struct F32Source {
    const float* p;
    __device__ void load8(int64_t e, float (&v)[8]) const {
        const float4 a = *reinterpret_cast<const float4*>(p + e), b = *reinterpret_cast<const float4*>(p + e + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

// One thread per 8 values, four neighbouring lanes per block of 32; rows are
// whole blocks, so the tensor is one run of n / 32 blocks.
template <typename Src>
__global__ __launch_bounds__(256) void quantize_mx8_kernel(Src src, int64_t n8, uint8_t* __restrict__ q,
                                                           uint8_t* __restrict__ scale) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= n8) return;   // n8 is a multiple of 4: a block's four lanes leave together
    float v[8];
    src.load8(8 * t, v);
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
    const uint32_t c = mx8_scale_code(__float_as_uint(max_over_4(a)));
    const float inv = mx8_inverse(c);
    *reinterpret_cast<uint2*>(q + 8 * t) =
        make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                   e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    if ((t & 3) == 0) scale[t >> 2] = (uint8_t)c;
}

template <bool OUT_BF16>
__global__ __launch_bounds__(256) void dequantize_mx8_kernel(const uint8_t* __restrict__ q,
                                                             const uint8_t* __restrict__ scale, int64_t n8,
                                                             void* __restrict__ out) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= n8) return;
    const uint2 d = *reinterpret_cast<const uint2*>(q + 8 * t);
    const float s = mx8_scale(scale[t >> 2]);
    float a[4], b[4];
    mx8_values4(d.x, s, a);
    mx8_values4(d.y, s, b);
    if constexpr (OUT_BF16) {
        store_out(reinterpret_cast<uint16_t*>(out) + 8 * t,
                  make_uint4(pack_rne(a[0], a[1]), pack_rne(a[2], a[3]), pack_rne(b[0], b[1]), pack_rne(b[2], b[3])));
    } else {
        float* o = reinterpret_cast<float*>(out) + 8 * t;
        store_out(o, make_float4(a[0], a[1], a[2], a[3]));
        store_out(o + 4, make_float4(b[0], b[1], b[2], b[3]));
    }
}

// Gradient of h = silu(g) * u, s = 1 / (1 + exp(-g)):
//   dg = dh * u * s * (1 + g * (1 - s)),   du = dh * g * s.
// Everything in fp32; dg and du are rounded once, to bf16, because they are
// the operands of the two bf16 products that follow.  exp(-g) overflowing to
// infinity gives s = 0 and both gradients 0.
struct GatedGrad {
    float dg, du, h;
};
__device__ __forceinline__ GatedGrad gated_grad(float dh, float g, float u) {
    const float s = 1.0f / (1.0f + expf(-g));
    const float gs = g * s;
    GatedGrad r;
    r.du = dh * gs;
    r.dg = dh * u * (s + gs * (1.0f - s));
    r.h = gs * u;
    return r;
}

// One thread per 8 columns of one row: dh [M,N], P = (gate, up) [M,2N] in
// bf16 or as an 8-bit checkpoint; writes dP [M,2N] and, when h is given, the
// recomputed h [M,N].  Rows past the groups' total hold anything: their dP is
// never read, their h is written as zeros.
template <bool MX8>
__global__ __launch_bounds__(256) void gated_grad_kernel(const uint16_t* __restrict__ dh,
                                                         const uint16_t* __restrict__ gu,
                                                         const uint8_t* __restrict__ gu_q,
                                                         const uint8_t* __restrict__ gu_s,
                                                         const int32_t* __restrict__ group_sizes, int M, int N, int G,
                                                         uint16_t* __restrict__ dgu, uint16_t* __restrict__ h,
                                                         int32_t* __restrict__ status) {
    __shared__ int s_total;
    if (blockIdx.x == 0 && threadIdx.x >= 64 && threadIdx.x < 128) {
        const int st = group_status(group_sizes, G, M);
        if (threadIdx.x == 64) status[0] = st;
    }
    if (h != nullptr) {   // the same for the whole grid
        if (threadIdx.x < 64) {
            int carry = 0;
            for (int base = 0; base < G; base += 64) carry = group_chunk(group_sizes, G, M, base, carry).next_carry;
            if (threadIdx.x == 0) s_total = min(carry, M);
        }
        __syncthreads();
    }
    const int per_row = N >> 3;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= (int64_t)M * per_row) return;
    const int64_t row = t / per_row;
    const int col = (int)(t - row * per_row) * 8;
    float d[8], g[8], u[8];
    Bf16Source{dh}.load8(row * N + col, d);
    const int64_t pg = row * 2 * N + col, pu = pg + N;
    if constexpr (MX8) {
        const float sg = mx8_scale(gu_s[pg >> 5]), su = mx8_scale(gu_s[pu >> 5]);
        const uint2 cg = *reinterpret_cast<const uint2*>(gu_q + pg), cu = *reinterpret_cast<const uint2*>(gu_q + pu);
        mx8_values4(cg.x, sg, *reinterpret_cast<float(*)[4]>(g));
        mx8_values4(cg.y, sg, *reinterpret_cast<float(*)[4]>(g + 4));
        mx8_values4(cu.x, su, *reinterpret_cast<float(*)[4]>(u));
        mx8_values4(cu.y, su, *reinterpret_cast<float(*)[4]>(u + 4));
    } else {
        Bf16Source{gu}.load8(pg, g);
        Bf16Source{gu}.load8(pu, u);
    }
    GatedGrad r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = gated_grad(d[i], g[i], u[i]);
    *reinterpret_cast<uint4*>(dgu + pg) = make_uint4(pack_rne(r[0].dg, r[1].dg), pack_rne(r[2].dg, r[3].dg),
                                                     pack_rne(r[4].dg, r[5].dg), pack_rne(r[6].dg, r[7].dg));
    *reinterpret_cast<uint4*>(dgu + pu) = make_uint4(pack_rne(r[0].du, r[1].du), pack_rne(r[2].du, r[3].du),
                                                     pack_rne(r[4].du, r[5].du), pack_rne(r[6].du, r[7].du));
    if (h != nullptr) {
        const bool used = row < s_total;
        const uint4 v = make_uint4(pack_rne(r[0].h, r[1].h), pack_rne(r[2].h, r[3].h), pack_rne(r[4].h, r[5].h),
                                   pack_rne(r[6].h, r[7].h));
        store_out(h + row * N + col, used ? v : make_uint4(0, 0, 0, 0));
    }
}

}  // namespace

// Threads of one launch of the two kernels above; a launch holds fewer than
// 2^32, so tensors of 2^34 values and more take several.  A multiple of a
// block's four lanes.
constexpr int64_t kChunk = int64_t(1) << 31;

hipError_t launch_quantize_mx8(const void* x, bool x_bf16, int64_t M, int64_t K, uint8_t* q, uint8_t* scale,
                               hipStream_t stream) {
    const int64_t total = M * K / 8;
    for (int64_t first = 0; first < total; first += kChunk) {
        const int64_t n8 = total - first < kChunk ? total - first : kChunk;
        const dim3 grid((unsigned)((n8 + 255) / 256)), block(256);
        if (x_bf16)
            hipLaunchKernelGGL((quantize_mx8_kernel<Bf16Source>), grid, block, 0, stream,
                               Bf16Source{reinterpret_cast<const uint16_t*>(x) + 8 * first}, n8, q + 8 * first,
                               scale + first / 4);
        else
            hipLaunchKernelGGL((quantize_mx8_kernel<F32Source>), grid, block, 0, stream,
                               F32Source{reinterpret_cast<const float*>(x) + 8 * first}, n8, q + 8 * first,
                               scale + first / 4);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_dequantize_mx8(const uint8_t* q, const uint8_t* scale, int64_t M, int64_t K, void* out,
                                 bool out_bf16, hipStream_t stream) {
    const int64_t total = M * K / 8;
    for (int64_t first = 0; first < total; first += kChunk) {
        const int64_t n8 = total - first < kChunk ? total - first : kChunk;
        const dim3 grid((unsigned)((n8 + 255) / 256)), block(256);
        char* o = static_cast<char*>(out) + first * (out_bf16 ? 16 : 32);
        if (out_bf16)
            hipLaunchKernelGGL((dequantize_mx8_kernel<true>), grid, block, 0, stream, q + 8 * first, scale + first / 4,
                               n8, o);
        else
            hipLaunchKernelGGL((dequantize_mx8_kernel<false>), grid, block, 0, stream, q + 8 * first,
                               scale + first / 4, n8, o);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_gated_grad(const void* dh, const void* gu, const uint8_t* gu_q, const uint8_t* gu_s,
                             const int32_t* group_sizes, int M, int N, int G, void* dgu, void* h,
                             int32_t* status, hipStream_t stream) {
    const int64_t n = (int64_t)M * (N / 8);
    const dim3 grid((unsigned)((n + 255) / 256)), block(256);
    const uint16_t* d = reinterpret_cast<const uint16_t*>(dh);
    uint16_t* o = reinterpret_cast<uint16_t*>(dgu);
    uint16_t* ho = reinterpret_cast<uint16_t*>(h);
    if (gu_q != nullptr)
        hipLaunchKernelGGL((gated_grad_kernel<true>), grid, block, 0, stream, d, nullptr, gu_q, gu_s, group_sizes, M, N,
                           G, o, ho, status);
    else
        hipLaunchKernelGGL((gated_grad_kernel<false>), grid, block, 0, stream, d,
                           reinterpret_cast<const uint16_t*>(gu), nullptr, nullptr, group_sizes, M, N, G, o, ho, status);
    return hipGetLastError();
}

}  // namespace gmm
