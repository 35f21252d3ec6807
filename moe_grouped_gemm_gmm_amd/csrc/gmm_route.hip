// The top-k router of a mixture-of-experts layer and its gradient.
//
// W lanes of a wave take one token's logits, V consecutive experts a lane, so
// the order of (lane, place in the lane) is the order of the experts: of
// several equal keys the lowest lane's first one is the lowest index.  k
// rounds each find the largest key left: V / 2 three-way maxima in the lane,
// log2 W lane moves, a ballot for the lowest lane that holds it.  Choice j
// stays in lane j (k <= W always), where the weights are made.
//
// Without a bias a key is the logit itself (the scores are monotonic in it),
// exact.  With a bias it is score + bias in 64 bits: scores that differ in the
// last bits of 32 would change places with every change of the arithmetic.
// Such keys are first compared in 32 bits; only where two that follow each
// other among the k + 1 largest are closer than twice their error is the
// wave's choice made again in 64.  How many tokens that takes depends on the data
// (65536 tokens of 256 experts, fp32, k = 8, us: normal logits of deviation 1.2 and
// biases of 0.05 35, logits of deviation 15 with biases of 0 138, where most of the
// softmax's scores are closer to each other than the largest one's error; with a
// sigmoid, whose scores crowd at 1 then, 150).  The weights and their gradient are in 32 bits.
//
// What bounds it: the forward's instructions (65536 tokens of 256 experts, k =
// 8: 20 us for 71 MB, which a copy's 5 TB/s moves in 14; one wave a token took
// 54), the gradient's memory (25 us for 138 MB, the copy 28; 44 with a wave a
// token, which spent as many instructions on its lane moves).
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
// Maxima of numbers (no NaN gets here).  In asm: fmaxf also has to quieten
// signalling NaNs, an instruction more for each operand of unknown origin.  The
// compiler takes the result for a vector instruction's and keeps the two wait
// states before a lane move reads it.
__device__ __forceinline__ float max2(float a, float b) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
template <int W>
__device__ __forceinline__ float max_lanes(float x) {
    return __uint_as_float(over_lanes<W>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(max2(__uint_as_float(a), __uint_as_float(b)));
    }));
}
__device__ __forceinline__ float min2(float a, float b) {
    float r;
    asm("v_min_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
template <int V>
__device__ __forceinline__ float max_of(const float (&x)[V]) {
    float m = x[0];
#pragma unroll
    for (int v = 1; v + 1 < V; v += 2) m = max3(m, x[v], x[v + 1]);
    return V % 2 == 0 ? max2(m, x[V - 1]) : m;
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
__device__ __forceinline__ uint64_t max_lanes(uint64_t x) {
    return over_lanes64<W>(x, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
}
template <int V>
__device__ __forceinline__ uint64_t max_of(const uint64_t (&x)[V]) {
    uint64_t m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = x[v] > m ? x[v] : m;
    return m;
}
template <int W>
__device__ __forceinline__ double sum_lanes(double x) {
    return __longlong_as_double((long long)over_lanes64<W>((uint64_t)__double_as_longlong(x), [](uint64_t a, uint64_t b) {
        return (uint64_t)__double_as_longlong(__longlong_as_double((long long)a) + __longlong_as_double((long long)b));
    }));
}

// An integer in the order of the floating-point numbers; NaN is not given here.
__device__ __forceinline__ uint64_t ordered(double f) {
    const uint64_t u = (uint64_t)__double_as_longlong(f);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}

// What a key that is off, or taken already, reads as.
template <typename Key>
__device__ __forceinline__ Key no_key();
template <>
__device__ __forceinline__ float no_key<float>() { return kOff; }
template <>
__device__ __forceinline__ uint64_t no_key<uint64_t>() { return 0; }

// A lane's key as a scalar, and equality of scalars' bits (keys have one zero).
__device__ __forceinline__ uint32_t lane_bits(uint32_t k, int lane) { return (uint32_t)lane_value((int)k, lane); }
__device__ __forceinline__ uint32_t lane_bits(float k, int lane) { return lane_bits(__float_as_uint(k), lane); }
__device__ __forceinline__ uint64_t lane_bits(uint64_t k, int lane) {
    return (uint64_t)lane_bits((uint32_t)(k >> 32), lane) << 32 | lane_bits((uint32_t)k, lane);
}

// A logit as the router takes it: kOff where the expert is off (-infinity or
// any NaN), +infinity as the largest number, one zero.
__device__ __forceinline__ float clean(float l) {
    return l > kOff ? __builtin_amdgcn_fmed3f(l, -FLT_MAX, FLT_MAX) + 0.0f : kOff;
}

// exp by the hardware's 2^x: the product's rounding moves it by |x| 2^-24 of
// itself, as much as the rounding of the difference x that it is given; results
// below the smallest normal number are 0.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
    if constexpr (BF16) return bf16_lo(reinterpret_cast<const uint16_t*>(p)[i]);
    else return reinterpret_cast<const float*>(p)[i];
}

// Values e0 .. e0 + V - 1 of the row of E that starts at element `row`, kOff from
// E on.  `vec`: E is a multiple of 4, so groups of four are aligned.
template <int V, bool BF16>
__device__ __forceinline__ void load_row(const void* p, int64_t row, int e0, int E, bool vec, float (&l)[V]) {
    if constexpr (V >= 4) {
        if (vec) {
#pragma unroll
            for (int v = 0; v < V; v += 4) {
                if (e0 + v >= E) {
                    l[v] = l[v + 1] = l[v + 2] = l[v + 3] = kOff;
                } else if constexpr (BF16) {
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
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? logit_at<BF16>(p, row + e0 + v) : kOff;
}
template <int V, bool BF16>
__device__ __forceinline__ void load_logits(const void* p, int64_t row, int e0, int E, bool vec, float (&l)[V]) {
    load_row<V, BF16>(p, row, e0, E, vec, l);
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = clean(l[v]);
}

// exp(l - maximum) of a token's logits and 1 / their sum (0 where every expert is off).
template <int W, int V>
__device__ __forceinline__ void softmax_of(const float (&l)[V], float (&e)[V], float& top, float& inv) {
    const float m = max_lanes<W>(max_of<V>(l));
    top = m > kOff ? m : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        e[v] = exp_of(l[v] - top);
        s += e[v];
    }
    s = sum_lanes<W>(s);
    inv = s > 0.0f ? __builtin_amdgcn_rcpf(s) : 0.0f;
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
    else s = exp_of(l - m);
    const float sum = sum_lanes<W>(s);
    return sum > 0.0f ? s / sum : 0.0f;
}

// k rounds: the j-th largest key's expert and the key in lane j of the token's
// W (-1 and no_key where none is left); returns the key of round k (`more`) or
// no_key.  key is used up.
template <int W, int V, typename Key>
__device__ __forceinline__ Key choose(Key (&key)[V], int k, bool more, int& my_id, Key& my_key) {
    const int lane = lane_id(), sub = lane % W;
    const Key none = no_key<Key>();
    my_id = -1;
    my_key = none;
    for (int j = 0; j < k; ++j) {
        const Key best = max_of<V>(key), m = max_lanes<W>(best);
        const unsigned long long held = __ballot(best == m);
        int id = -1;
        if constexpr (W == 64) {   // one token a wave: where the key is, and its removal, are scalar
            if (lane_bits(m, 0) == lane_bits(none, 0)) return none;
            const int owner = __ffsll((long long)held) - 1;
            bool found = false;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (found || lane_bits(key[v], owner) != lane_bits(m, 0)) continue;
                found = true;
                id = owner * V + v;
                key[v] = lane == owner ? none : key[v];
            }
        } else {
            static_assert(W <= 16, "a token's lanes are in one half of the ballot");
            const uint32_t half = lane < 32 ? (uint32_t)held : (uint32_t)(held >> 32);
            const int owner = __ffs((int)(half >> (lane & 31 & ~(W - 1)) & ((1u << W) - 1u))) - 1;
            int at = 0;
            bool open = sub == owner;   // the first of the owner's equal keys
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool hit = open && key[v] == m;
                at = hit ? v : at;
                key[v] = hit ? none : key[v];
                open = open && !hit;
            }
            if constexpr (V == 1) {
                id = owner;
            } else {
                id = owner * V + __shfl(at, (lane & ~(W - 1)) + owner, 64);
            }
            if (m == none) id = -1;
        }
        my_id = sub == j ? id : my_id;
        my_key = sub == j ? m : my_key;
    }
    return more ? max_lanes<W>(max_of<V>(key)) : none;
}

// Batcher's odd-even merge sort of V numbers: the pairs that are compared.
template <int V>
struct SortPairs {
    int a[V * V], b[V * V], n;
    constexpr SortPairs() : a(), b(), n(0) {
        for (int p = 1; p < V; p *= 2)
            for (int q = p; q >= 1; q /= 2)
                for (int j = q % p; j + q < V; j += 2 * q)
                    for (int i = 0; i < q && i + j + q < V; ++i)
                        if ((i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                            a[n] = i + j;
                            b[n] = i + j + q;
                            ++n;
                        }
    }
};

// choose<W, V, float> for many rounds: each lane sorts its keys first (63
// comparisons of two instructions for 16), so that a round looks at one key a
// lane and the owner's others move up.  The places that sorting forgets are
// found again at the end: lane j reads its choice's owner's keys from `row`
// (W V words of LDS of the token's own) and takes the first that is equal, or
// the next one where the choice before it is the same key of the same lane.
template <int W, int V>
__device__ __forceinline__ float choose_sorted(const float (&key)[V], int k, bool more, float* row, int& my_id,
                                               float& my_key) {
    static_assert(W == 16 && V % 4 == 0, "a token's lanes are a row of 16");
    constexpr SortPairs<V> pairs;
    const int lane = lane_id(), sub = lane % W;
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = key[v];
#pragma unroll
    for (int c = 0; c < pairs.n; ++c) {
        const float hi = max2(s[pairs.a[c]], s[pairs.b[c]]), lo = min2(s[pairs.a[c]], s[pairs.b[c]]);
        s[pairs.a[c]] = hi;
        s[pairs.b[c]] = lo;
    }
    my_key = kOff;
    int my_owner = 0;
    for (int j = 0; j < k; ++j) {
        const float m = max_lanes<W>(s[0]);
        const unsigned long long held = __ballot(s[0] == m);
        const uint32_t half = lane < 32 ? (uint32_t)held : (uint32_t)(held >> 32);
        const int owner = __ffs((int)(half >> (lane & 16) & 0xffffu)) - 1;
        const bool pop = sub == owner;
#pragma unroll
        for (int v = 0; v < V / 2 - 1; ++v) s[v] = pop ? s[v + 1] : s[v];
        if (k > V / 2) {   // further keys only matter with more rounds than V / 2
#pragma unroll
            for (int v = V / 2 - 1; v < V - 1; ++v) s[v] = pop ? s[v + 1] : s[v];
            s[V - 1] = pop ? kOff : s[V - 1];
        }
        my_key = sub == j ? m : my_key;
        my_owner = sub == j ? owner : my_owner;
    }
    auto sync = [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); };
    sync();   // the last token's reads
#pragma unroll
    for (int v = 0; v < V; v += 4)
        *reinterpret_cast<float4*>(row + V * sub + v) = make_float4(key[v], key[v + 1], key[v + 2], key[v + 3]);
    sync();
    // how many choices just before this one are the same key of the same lane
    int skip = 0;
    const float key_before = __shfl_up(my_key, 1, W);   // by every lane: an idle one would give nothing
    const int owner_before = __shfl_up(my_owner, 1, W);
    const bool same = sub > 0 && sub < k && key_before == my_key && owner_before == my_owner;
    unsigned long long run = __ballot(same);
    if (run != 0) {
        const uint32_t half = lane < 32 ? (uint32_t)run : (uint32_t)(run >> 32);
        const uint32_t mine = half >> (lane & 16) & 0xffffu;        // bit j: choice j repeats choice j - 1
        skip = __clz((int)~(mine << (31 - sub)));                   // ones from bit sub down
    }
    int at = -1;
#pragma unroll
    for (int v = 0; v < V; v += 4) {
        const float4 d = *reinterpret_cast<const float4*>(row + V * my_owner + v);
        const float x[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool hit = x[i] == my_key;
            at = hit && skip == 0 ? v + i : at;
            skip -= hit ? 1 : 0;
        }
    }
    my_id = my_key > kOff ? V * my_owner + at : -1;
    return more ? max_lanes<W>(s[0]) : kOff;
}

// The choice of token t by keys in 64 bits, 64 lanes of VX experts; choice j in
// lane j.  top: the token's largest logit.
template <int VX, bool BF16>
__device__ __forceinline__ int exact_choice(const RouteArgs& a, int64_t t, float top) {
    const int lane = lane_id(), E = a.E;
    uint64_t key[VX];
    double s[VX], sum = 0.0;
#pragma unroll
    for (int v = 0; v < VX; ++v) {
        const int e = lane * VX + v;
        const float l = e < E ? clean(logit_at<BF16>(a.logits, t * E + e)) : kOff;
        s[v] = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : (l > kOff ? exp((double)l - (double)top) : 0.0);
        key[v] = l > kOff;
        sum += s[v];
    }
    sum = a.sigmoid ? 1.0 : sum_lanes<64>(sum);
#pragma unroll
    for (int v = 0; v < VX; ++v) {
        const double z = s[v] / sum + (double)a.bias[min(lane * VX + v, E - 1)];
        key[v] = key[v] != 0 && z > (double)kOff ? ordered(z + 0.0) : 0;
    }
    int id;
    uint64_t unused;
    choose<64, VX, uint64_t>(key, a.k, false, id, unused);
    return id;
}

// Keys score + bias in 32 bits, kOff where the expert is off.  key: the
// exponentials of a softmax (not read for a sigmoid).
template <int V>
__device__ __forceinline__ void biased_keys(const RouteArgs& a, const float (&l)[V], const float (&b)[V], float inv,
                                            float (&key)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float x = a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + exp_of(-l[v])) : key[v] * inv;
        const float z = x + b[v] + 0.0f;
        key[v] = l[v] > kOff && z > kOff ? z : kOff;
    }
}

template <int W, int V, bool BF16, bool BIAS>
__global__ __launch_bounds__(256, BIAS && W * V <= 256 ? 4 : 1) void route_kernel(const RouteArgs a, int32_t* __restrict__ ids,
                                                    float* __restrict__ weights) {
    // Sorting a lane's keys pays from five rounds on (65536 tokens, 256 experts,
    // scores of a softmax, us by rounds alone / sorted: k 4 17.9 / 18.1, 5 19.9 /
    // 18.6, 8 24.8 / 19.9, 16 39.0 / 27.8).
    constexpr bool kSorts = W == 16 && V >= 8;
    __shared__ __attribute__((aligned(16))) float rows[kSorts ? 256 / W : 1][kSorts ? W * V : 4];
    const int lane = lane_id(), sub = lane % W, E = a.E, k = a.k;
    const bool vec = E % 4 == 0;
    const int64_t stride = (int64_t)gridDim.x * (256 / W);
    auto pick = [&](float (&key)[V], bool more, int& my_id, float& my_key) {
        if constexpr (kSorts)
            if (k >= 5) return choose_sorted<W, V>(key, k, more, rows[threadIdx.x / W], my_id, my_key);
        return choose<W, V, float>(key, k, more, my_id, my_key);
    };
    // whole waves stay together: the last tokens' lanes without one repeat the last
    for (int64_t t0 = (int64_t)blockIdx.x * (256 / W) + (threadIdx.x / 64) * (64 / W); t0 < a.T; t0 += stride) {
        const int64_t t = min(t0 + lane / W, a.T - 1);
        float l[V], s[V], top = 0.0f, inv = 0.0f;
        load_logits<V, BF16>(a.logits, t * E, sub * V, E, vec, l);
        if (!a.sigmoid && (BIAS || !a.normalize)) softmax_of<W, V>(l, s, top, inv);
        int my_id;
        float my_l;
        if constexpr (!BIAS) {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = l[v];
            pick(s, false, my_id, my_l);
        } else {
            float b[V];
            load_row<V, false>(a.bias, 0, sub * V, E, vec, b);
            biased_keys<V>(a, l, b, inv, s);
            float my_key;
            const float next = pick(s, true, my_id, my_key);
            // Twice the error of a key.  A sigmoid is off by less than 4 u of it (u = 2^-24: its exponential by (2 |l|
            // + 2) u, of which s (1 - s) counts, the sum and the reciprocal); a softmax, d below the top, by (2 d + 80)
            // u of it (the differences and products of d, a sum of at most 70 roundings), so by less than 2^-17 of
            // the top's score, which is inv; score + bias by half a step.
            const int group = lane & ~(W - 1), beside = group | ((sub + 1) & (W - 1));
            const float after_lane = __shfl(my_key, beside, 64), after = sub + 1 < k ? after_lane : next;
            const float tol = (a.sigmoid ? 0x1p-20f : 0x1p-16f * inv) + 0x1p-23f * (fabsf(my_key) + fabsf(after));
            // Equal logits with equal biases are the same key in 64 bits too, and in the order of their indices.
            my_l = my_id >= 0 ? clean(logit_at<BF16>(a.logits, t * E + my_id)) : kOff;
            const float my_b = my_id >= 0 ? a.bias[my_id] : 0.0f;
            const float l_after = __shfl(my_l, beside, 64), b_after = __shfl(my_b, beside, 64);
            bool close = sub < k && my_id >= 0 && after > kOff && !(my_key - after > tol);
            const bool edge = close && sub == k - 1;   // against keys that were not chosen: all that are as near
            close = close && !edge && !(my_l == l_after && my_b == b_after);
            if (__ballot(edge) != 0) {
                const int last = group + k - 1;
                const float m = __shfl(my_key, last, 64), lm = __shfl(my_l, last, 64), bm = __shfl(my_b, last, 64),
                            tm = __shfl(tol, last, 64);
                const bool asked = __shfl((int)edge, last, 64) != 0;   // by every lane: an idle one would give nothing
                bool other = false;
                constexpr int C = V < 4 ? V : 4;
#pragma unroll 1
                for (int v = 0; v < V; v += C) {   // read again: the registers are the common path's
                    const int e = sub * V + v;
                    float x[C], key[C], bias[C];
                    load_logits<C, BF16>(a.logits, t * E, e, E, vec, x);
                    load_row<C, false>(a.bias, 0, e, E, vec, bias);
#pragma unroll
                    for (int c = 0; c < C; ++c) key[c] = exp_of(x[c] - top);
                    biased_keys<C>(a, x, bias, inv, key);
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        other = other || (key[c] > kOff && !(fabsf(key[c] - m) > tm) && !(x[c] == lm && bias[c] == bm));
                }
                close = close || (asked && other);
            }
            constexpr unsigned long long kGroup = W == 64 ? ~0ull : (1ull << (W % 64)) - 1ull;
            unsigned long long open = __ballot(close);
            while (open != 0) {   // one token after the other, by the whole wave
                const int base = (__ffsll((long long)open) - 1) & ~(W - 1);
                open &= ~(kGroup << base);
                const int id = exact_choice<(W * V + 63) / 64, BF16>(
                    a, min(t0 + base / W, a.T - 1), __int_as_float(lane_value(__float_as_int(top), base)));
                const int mine = __shfl(id, sub, 64);
                my_id = group == base ? mine : my_id;
                my_l = my_id >= 0 ? clean(logit_at<BF16>(a.logits, t * E + my_id)) : kOff;
            }
        }
        float w;
        if (a.normalize) w = chosen_share<W>(my_l, a.sigmoid);
        else if (a.sigmoid) w = sigmoid(my_l);
        else w = exp_of(my_l - top) * inv;
        if (sub < k && t0 + lane / W < a.T) {
            ids[t * k + sub] = my_id;
            weights[t * k + sub] = my_id >= 0 ? a.scale * w : 0.0f;
        }
    }
}

// Where the gradient's lanes have their experts: place v of lane `sub` (the
// order does not matter here, so a group's lanes read and write whole lines).
template <int W, int V>
__device__ __forceinline__ int expert_at(int sub, int v) { return V < 4 ? sub * V + v : 4 * W * (v / 4) + 4 * sub + v % 4; }

// The choices' values added up at their experts: x[v] of expert_at(v) from g of
// the expert id (or -1) in lane j < k, by way of `row` in LDS, W V words of the
// token's own.  Ids that a router made differ, and one write each does; where
// some are equal (found by writing the lane and reading it back) the lanes add
// one after the other.
template <int W, int V>
__device__ __forceinline__ void scatter_choices(int id, float g, int k, float* row, float (&x)[V]) {
    const int sub = lane_id() % W;
    int* owner = reinterpret_cast<int*>(row);
    auto sync = [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); };
    sync();   // the last token's reads
#pragma unroll
    for (int v = 0; v < V; v += V < 4 ? 1 : 4) {
        if constexpr (V < 4) row[expert_at<W, V>(sub, v)] = 0.0f;
        else *reinterpret_cast<float4*>(row + expert_at<W, V>(sub, v)) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    sync();
    if (id >= 0) owner[id] = sub;
    sync();
    const bool shared = id >= 0 && owner[id] != sub;
    sync();
    if (__ballot(shared) == 0) {
        if (id >= 0) row[id] = g;
    } else {
        if (id >= 0) row[id] = 0.0f;
        for (int j = 0; j < k; ++j) {
            sync();
            if (sub == j && id >= 0) row[id] += g;
        }
    }
    sync();
#pragma unroll
    for (int v = 0; v < V; v += V < 4 ? 1 : 4) {
        if constexpr (V < 4) {
            x[v] = row[expert_at<W, V>(sub, v)];
        } else {
            const float4 d = *reinterpret_cast<const float4*>(row + expert_at<W, V>(sub, v));
            x[v] = d.x;
            x[v + 1] = d.y;
            x[v + 2] = d.z;
            x[v + 3] = d.w;
        }
    }
}

template <int W, int V, bool BF16, bool OUT_BF16>
__global__ __launch_bounds__(256) void route_bwd_kernel(const RouteArgs a, const float* __restrict__ dweights,
                                                        const int32_t* __restrict__ ids, void* dlogits) {
    __shared__ __attribute__((aligned(16))) float rows[256 / W][W * V];
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
        float g = dw, dot = 0.0f, s[V], d[V];
        if (dense) {
            float l[V], top, inv;
#pragma unroll
            for (int v = 0; v < V; v += V < 4 ? 1 : 4) {
                const int e = expert_at<W, V>(sub, v);
                if constexpr (V < 4) load_logits<1, BF16>(a.logits, t * E, e, E, vec, reinterpret_cast<float(&)[1]>(l[v]));
                else load_logits<4, BF16>(a.logits, t * E, e, E, vec, reinterpret_cast<float(&)[4]>(l[v]));
            }
            softmax_of<W, V>(l, s, top, inv);
            dot = sum_lanes<W>(on ? exp_of(lj - top) * inv * dw : 0.0f);
            const float c = a.scale * inv;
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] *= c;
        } else if (a.normalize) {
            const float q = chosen_share<W>(lj, a.sigmoid);
            g = a.scale * q * (dw - sum_lanes<W>(q * dw));
            if (a.sigmoid) g *= 1.0f / (1.0f + expf(lj));
        } else {
            g = on ? a.scale * dw * sigmoid(lj) * (1.0f / (1.0f + expf(lj))) : 0.0f;
        }
        scatter_choices<W, V>(id, g, k, rows[threadIdx.x / W], d);
        if (dense) {
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = s[v] * (d[v] - dot);
        }
        if (!mine) continue;
        const int64_t o = t * E;
#pragma unroll
        for (int v = 0; v < V; v += V < 4 ? 1 : 4) {
            const int e = expert_at<W, V>(sub, v);
            if (e >= E) break;
            if (V >= 4 && vec) {
                if constexpr (V >= 4) {
                    if constexpr (OUT_BF16)
                        store_out(reinterpret_cast<uint16_t*>(dlogits) + o + e,
                                  make_uint2(pack_rne(d[v], d[v + 1]), pack_rne(d[v + 2], d[v + 3])));
                    else
                        store_out(reinterpret_cast<float*>(dlogits) + o + e,
                                  make_float4(d[v], d[v + 1], d[v + 2], d[v + 3]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < (V < 4 ? 1 : 4); ++i) {
                    if (e + i >= E) break;
                    if constexpr (OUT_BF16) reinterpret_cast<uint16_t*>(dlogits)[o + e + i] = (uint16_t)pack_rne(d[v + i], d[v + i]);
                    else reinterpret_cast<float*>(dlogits)[o + e + i] = d[v + i];
                }
            }
        }
    }
}

// Lanes and experts a lane for E experts.  16 lanes a token (four tokens a
// wave) share the lane moves and ballots of a round between four tokens; 64
// give the shortest rounds and the most waves, which few tokens need (below 8192
// tokens of 256 experts both take the time of a launch, 65536 47.2 / 25.3 us
// before a lane's keys were sorted).
template <typename F>
hipError_t with_lanes(int E, int k, bool many, F f) {
    using std::integral_constant;
    constexpr integral_constant<int, 16> w16;
    constexpr integral_constant<int, 64> w64;
    if (E <= 16) return f(w16, integral_constant<int, 1>{});
    if (E <= 64) return k <= 16 ? f(w16, integral_constant<int, 4>{}) : f(w64, integral_constant<int, 1>{});
    if (E <= 128 && k <= 16 && many) return f(w16, integral_constant<int, 8>{});
    if (E <= 256) return k <= 16 && many ? f(w16, integral_constant<int, 16>{}) : f(w64, integral_constant<int, 4>{});
    if (E <= 512) return f(w64, integral_constant<int, 8>{});
    if (E <= 1024) return f(w64, integral_constant<int, 16>{});
    return f(w64, integral_constant<int, 64>{});
}

constexpr int64_t kManyTokens = 8192;

dim3 token_grid(int64_t T, int W) {
    const int64_t blocks = (T + 256 / W - 1) / (256 / W);
    return dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20));
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, bool logits_bf16, int32_t* ids, float* weights, hipStream_t stream) {
    return with_lanes(a.E, a.k, a.T >= kManyTokens, [&](auto w, auto v) {
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
    return with_lanes(a.E, a.k, a.T >= kManyTokens, [&](auto w, auto v) {
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
