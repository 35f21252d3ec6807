// The top-k router of a mixture-of-experts layer and its gradient.
//
// W lanes of a wave take one token's logits, V consecutive experts a lane, so
// the order of (lane, place in the lane) is the order of the experts: of
// several equal keys the lowest lane's first one is the lowest index.  k
// rounds each find the largest key left: V - 1 maxima in the lane, log2 W lane
// moves, a ballot for the lowest lane that holds it.  Choice j stays in lane j
// (k <= W always), where the weights are made.
//
// Keys are compared as integers in the order of the numbers they stand for,
// 0 for an expert that is off or already taken.  Without a bias a key is the
// logit itself (the scores are monotonic in it), exact.  With a bias it is
// score + bias in 64 bits: scores that differ in the last bits of 32 would
// change places with every change of the arithmetic.  The weights and their
// gradient are in 32 bits.
#include "gmm_launch.hpp"
#include "gmm_moe.hpp"
#include "gmm_mx8.hpp"

#include <cfloat>
#include <type_traits>

namespace gmm {

namespace {

constexpr float kOff = -__builtin_huge_valf();

// ---- reductions over the aligned groups of W lanes that share a token; every
// lane gets the result.  The order of the additions is the same in every call.
template <int W, typename Op>
__device__ __forceinline__ uint32_t over_lanes(uint32_t x, Op op) {
    if constexpr (W >= 2) x = op(x, dpp<kDppXor1>(x));
    if constexpr (W >= 4) x = op(x, dpp<kDppXor2>(x));
    if constexpr (W >= 8) x = op(x, dpp<kDppHalfMirror>(x));
    if constexpr (W >= 16) x = op(x, dpp<kDppMirror>(x));
    if constexpr (W >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = op(p[0], p[1]);
    }
    if constexpr (W >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        x = op(p[0], p[1]);
    }
    return x;
}
template <int W>
__device__ __forceinline__ float sum_lanes(float x) {
    return __uint_as_float(over_lanes<W>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
template <int W>
__device__ __forceinline__ float max_lanes(float x) {
    return __uint_as_float(over_lanes<W>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
template <int W>
__device__ __forceinline__ uint32_t max_key(uint32_t x) {
    return over_lanes<W>(x, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// One exchange of 64-bit values between the lanes of a group: step s of log2 W.
template <int S>
__device__ __forceinline__ uint64_t exchange(uint64_t x) {
    uint32_t l = (uint32_t)x, h = (uint32_t)(x >> 32);
    if constexpr (S < 4) {
        constexpr int c = S == 0 ? kDppXor1 : (S == 1 ? kDppXor2 : (S == 2 ? kDppHalfMirror : kDppMirror));
        l = dpp<c>(l);
        h = dpp<c>(h);
    } else {
        l = (uint32_t)__shfl_xor((int)l, 1 << S, 64);
        h = (uint32_t)__shfl_xor((int)h, 1 << S, 64);
    }
    return (uint64_t)h << 32 | l;
}
template <int W, int S = 0, typename Op>
__device__ __forceinline__ uint64_t over_lanes64(uint64_t x, Op op) {
    if constexpr ((1 << S) < W) return over_lanes64<W, S + 1>(op(x, exchange<S>(x)), op);
    return x;
}
template <int W>
__device__ __forceinline__ uint64_t max_key(uint64_t x) {
    return over_lanes64<W>(x, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
}
template <int W>
__device__ __forceinline__ double sum_lanes(double x) {
    return __longlong_as_double((long long)over_lanes64<W>((uint64_t)__double_as_longlong(x), [](uint64_t a, uint64_t b) {
        return (uint64_t)__double_as_longlong(__longlong_as_double((long long)a) + __longlong_as_double((long long)b));
    }));
}

// Integers in the order of the floating-point numbers; NaN is not given here.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t ordered(double f) {
    const uint64_t u = (uint64_t)__double_as_longlong(f);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}

// A logit as the router takes it: kOff where the expert is off, +infinity as
// the largest number, one zero.
__device__ __forceinline__ float clean(float l) { return l > kOff ? fminf(l, FLT_MAX) + 0.0f : kOff; }

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
    if constexpr (BF16) return bf16_lo(reinterpret_cast<const uint16_t*>(p)[i]);
    else return reinterpret_cast<const float*>(p)[i];
}

// Experts e0 .. e0 + V - 1 of the row that starts at element `row`, kOff from E
// on.  `vec`: E is a multiple of 4, so groups of four are aligned.
template <int V, bool BF16>
__device__ __forceinline__ void load_logits(const void* p, int64_t row, int e0, int E, bool vec, float (&l)[V]) {
    if (V >= 4 && vec) {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            if (e0 + v >= E) {
#pragma unroll
                for (int i = 0; i < 4 && v + i < V; ++i) l[v + i] = kOff;
            } else if constexpr (V >= 4) {
                if constexpr (BF16) {
                    const uint2 d = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + row + e0 + v);
                    l[v] = bf16_lo(d.x);
                    l[v + 1] = bf16_hi(d.x);
                    l[v + 2] = bf16_lo(d.y);
                    l[v + 3] = bf16_hi(d.y);
                } else {
                    const float4 d = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + row + e0 + v);
                    l[v] = d.x;
                    l[v + 1] = d.y;
                    l[v + 2] = d.z;
                    l[v + 3] = d.w;
                }
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? logit_at<BF16>(p, row + e0 + v) : kOff;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = clean(l[v]);
}

// Maximum (0 where every expert is off) and 1 / sum of exp(l - maximum) (0 there)
// of a token.
template <int W, int V>
__device__ __forceinline__ void softmax_of(const float (&l)[V], float& top, float& inv) {
    float m = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
    m = max_lanes<W>(m);
    top = m > kOff ? m : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) s += expf(l[v] - top);
    s = sum_lanes<W>(s);
    inv = s > 0.0f ? 1.0f / s : 0.0f;
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// score / sum of scores over a token's choices, choice j in lane j; l is kOff
// where there is none.  Both sums are of scores times exp(-m), m the largest
// chosen logit (sigmoid: if it is below 0), so that they cannot vanish.
template <int W>
__device__ __forceinline__ float chosen_share(float l, bool sigmoid_score) {
    const float top = max_lanes<W>(l), m = top > kOff ? top : 0.0f;
    float s;
    if (sigmoid_score) s = l >= 0.0f ? sigmoid(l) : expf(l - fminf(m, 0.0f)) / (1.0f + expf(l));
    else s = expf(l - m);
    const float sum = sum_lanes<W>(s);
    return sum > 0.0f ? s / sum : 0.0f;
}

template <int W, int V, bool BF16, bool BIAS>
__global__ __launch_bounds__(256) void route_kernel(const RouteArgs a, int32_t* __restrict__ ids,
                                                    float* __restrict__ weights) {
    using Key = typename std::conditional<BIAS, uint64_t, uint32_t>::type;
    const int lane = lane_id(), sub = lane % W, E = a.E, k = a.k;
    const bool vec = E % 4 == 0;
    const int64_t stride = (int64_t)gridDim.x * (256 / W);
    // whole waves stay together: the last tokens' lanes without one repeat the last
    for (int64_t t0 = (int64_t)blockIdx.x * (256 / W) + (threadIdx.x / 64) * (64 / W); t0 < a.T; t0 += stride) {
        const int64_t t = min(t0 + lane / W, a.T - 1);
        float l[V];
        load_logits<V, BF16>(a.logits, t * E, sub * V, E, vec, l);
        float top = 0.0f, inv = 0.0f;
        if (!a.sigmoid && !a.normalize) softmax_of<W, V>(l, top, inv);
        Key key[V];
        if constexpr (BIAS) {
            double s[V];
            if (a.sigmoid) {
#pragma unroll
                for (int v = 0; v < V; ++v) s[v] = 1.0 / (1.0 + exp(-(double)l[v]));
            } else {
                float m = l[0];
#pragma unroll
                for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
                m = max_lanes<W>(m);
                double sum = 0.0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    s[v] = l[v] > kOff ? exp((double)l[v] - (double)m) : 0.0;
                    sum += s[v];
                }
                sum = sum_lanes<W>(sum);
#pragma unroll
                for (int v = 0; v < V; ++v) s[v] /= sum;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = sub * V + v;
                const double b = e < E ? s[v] + (double)a.bias[e] : 0.0;
                key[v] = l[v] > kOff && b > (double)kOff ? ordered(b + 0.0) : 0;
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = l[v] > kOff ? ordered(l[v]) : 0;
        }
        int my_id = -1;
        float my_l = kOff;
        for (int j = 0; j < k; ++j) {
            Key best = key[0];
#pragma unroll
            for (int v = 1; v < V; ++v) best = key[v] > best ? key[v] : best;
            const Key m = max_key<W>(best);
            const unsigned long long held = __ballot(best == m);
            int id, owner;
            if constexpr (W == 64) {
                owner = __ffsll((long long)held) - 1;
            } else {
                owner = __ffsll((long long)(held >> (lane - sub) & ((1ull << W) - 1ull))) - 1;
            }
            int at = 0;
            float lv = l[0];
#pragma unroll
            for (int v = V - 1; v >= 0; --v)
                if (key[v] == m) {
                    at = v;
                    lv = l[v];
                }
            if constexpr (V > 1) {   // W == 64: the owner is the wave's
                id = owner * V + lane_value(at, owner);
            } else {
                id = owner;
            }
            float lj;
            if constexpr (!BIAS) lj = from_ordered((uint32_t)m);
            else if constexpr (W == 64) lj = __int_as_float(lane_value(__float_as_int(lv), owner));
            else lj = __shfl(lv, lane - sub + owner, 64);
            if (sub == j && m != 0) {
                my_id = id;
                my_l = lj;
            }
            if (sub == owner) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (V == 1 || v == at) key[v] = 0;
            }
        }
        float w;
        if (a.normalize) w = chosen_share<W>(my_l, a.sigmoid);
        else if (a.sigmoid) w = sigmoid(my_l);
        else w = expf(my_l - top) * inv;
        if (sub < k && t0 + lane / W < a.T) {
            ids[t * k + sub] = my_id;
            weights[t * k + sub] = my_id >= 0 ? a.scale * w : 0.0f;
        }
    }
}

template <int W, int V, bool BF16, bool OUT_BF16>
__global__ __launch_bounds__(256) void route_bwd_kernel(const RouteArgs a, const float* __restrict__ dweights,
                                                        const int32_t* __restrict__ ids, void* __restrict__ dlogits) {
    const int lane = lane_id(), sub = lane % W, E = a.E, k = a.k;
    const bool vec = E % 4 == 0;
    const int64_t stride = (int64_t)gridDim.x * (256 / W);
    for (int64_t t0 = (int64_t)blockIdx.x * (256 / W) + (threadIdx.x / 64) * (64 / W); t0 < a.T; t0 += stride) {
        const int64_t t = min(t0 + lane / W, a.T - 1);
        const bool mine = t0 + lane / W < a.T;
        int id = sub < k ? ids[t * k + sub] : -1;
        float dw = sub < k ? dweights[t * k + sub] : 0.0f;
        id = id >= 0 && id < E ? id : -1;
        const float lj = id >= 0 ? clean(logit_at<BF16>(a.logits, t * E + id)) : kOff;
        const bool on = lj > kOff;
        if (!on) {
            id = -1;
            dw = 0.0f;
        }
        // what choice j adds at its expert: its part of the gradient itself, or
        // (dense) its weight's gradient
        const bool dense = !a.sigmoid && !a.normalize;
        float g = dw, dot = 0.0f, l[V], top = 0.0f, inv = 0.0f;
        if (dense) {
            load_logits<V, BF16>(a.logits, t * E, sub * V, E, vec, l);
            softmax_of<W, V>(l, top, inv);
            dot = sum_lanes<W>(on ? expf(lj - top) * inv * dw : 0.0f);
        } else if (a.normalize) {
            const float q = chosen_share<W>(lj, a.sigmoid);
            g = a.scale * q * (dw - sum_lanes<W>(q * dw));
            if (a.sigmoid) g *= 1.0f / (1.0f + expf(lj));
        } else {
            g = on ? a.scale * dw * sigmoid(lj) * (1.0f / (1.0f + expf(lj))) : 0.0f;
        }
        float d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = 0.0f;
        for (int j = 0; j < k; ++j) {
            int e;
            float gj;
            if constexpr (W == 64) {
                e = lane_value(id, j);
                gj = __int_as_float(lane_value(__float_as_int(g), j));
            } else {
                e = __shfl(id, lane - sub + j, 64);
                gj = __shfl(g, lane - sub + j, 64);
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (e == sub * V + v) d[v] += gj;
        }
        if (dense) {
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = a.scale * (expf(l[v] - top) * inv) * (d[v] - dot);
        }
        if (!mine) continue;
        const int64_t o = t * E + sub * V;
        if (V >= 4 && vec) {
#pragma unroll
            for (int v = 0; v + 3 < V; v += 4) {
                if (sub * V + v >= E) break;
                if constexpr (OUT_BF16)
                    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(dlogits) + o + v) =
                        make_uint2(pack_rne(d[v], d[v + 1]), pack_rne(d[v + 2], d[v + 3]));
                else
                    *reinterpret_cast<float4*>(reinterpret_cast<float*>(dlogits) + o + v) =
                        make_float4(d[v], d[v + 1], d[v + 2], d[v + 3]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (sub * V + v >= E) break;
                if constexpr (OUT_BF16) reinterpret_cast<uint16_t*>(dlogits)[o + v] = (uint16_t)pack_rne(d[v], d[v]);
                else reinterpret_cast<float*>(dlogits)[o + v] = d[v];
            }
        }
    }
}

// Lanes and experts a lane for E experts.
template <typename F>
hipError_t with_lanes(int E, F f) {
    using std::integral_constant;
    if (E <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    if (E <= 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (E <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    if (E <= 64) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (E <= 256) return f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if (E <= 1024) return f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
    return f(integral_constant<int, 64>{}, integral_constant<int, 64>{});
}

dim3 token_grid(int64_t T, int W) {
    const int64_t blocks = (T + 256 / W - 1) / (256 / W);
    return dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20));
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, bool logits_bf16, int32_t* ids, float* weights, hipStream_t stream) {
    return with_lanes(a.E, [&](auto w, auto v) {
        constexpr int W = decltype(w)::value, V = decltype(v)::value;
        const dim3 grid = token_grid(a.T, W), block(256);
        if (a.bias != nullptr) {
            if (logits_bf16) hipLaunchKernelGGL((route_kernel<W, V, true, true>), grid, block, 0, stream, a, ids, weights);
            else hipLaunchKernelGGL((route_kernel<W, V, false, true>), grid, block, 0, stream, a, ids, weights);
        } else {
            if (logits_bf16) hipLaunchKernelGGL((route_kernel<W, V, true, false>), grid, block, 0, stream, a, ids, weights);
            else hipLaunchKernelGGL((route_kernel<W, V, false, false>), grid, block, 0, stream, a, ids, weights);
        }
        return hipGetLastError();
    });
}

hipError_t launch_route_bwd(const RouteArgs& a, bool logits_bf16, const float* dweights, const int32_t* ids,
                            void* dlogits, bool out_bf16, hipStream_t stream) {
    return with_lanes(a.E, [&](auto w, auto v) {
        constexpr int W = decltype(w)::value, V = decltype(v)::value;
        const dim3 grid = token_grid(a.T, W), block(256);
        if (logits_bf16) {
            if (out_bf16)
                hipLaunchKernelGGL((route_bwd_kernel<W, V, true, true>), grid, block, 0, stream, a, dweights, ids, dlogits);
            else
                hipLaunchKernelGGL((route_bwd_kernel<W, V, true, false>), grid, block, 0, stream, a, dweights, ids, dlogits);
        } else {
            if (out_bf16)
                hipLaunchKernelGGL((route_bwd_kernel<W, V, false, true>), grid, block, 0, stream, a, dweights, ids, dlogits);
            else
                hipLaunchKernelGGL((route_bwd_kernel<W, V, false, false>), grid, block, 0, stream, a, dweights, ids, dlogits);
        }
        return hipGetLastError();
    });
}

}  // namespace gmm
