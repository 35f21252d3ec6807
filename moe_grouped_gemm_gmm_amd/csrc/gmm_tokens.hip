// Tokens sorted by expert and back: the order of the slots, and the rows moved
// into it and out of it with their weights and gradients.
//
// The order is a counting sort that keeps equal experts in slot order.  A
// workgroup counts the experts of its run of slots in LDS; a slot's row is
//     slots of lower experts + slots of its expert in earlier runs
//     + in earlier waves of the run + in earlier slots of the wave,
// the last from ballots on the expert's bits, so nothing depends on the order
// in which workgroups or atomics run (the LDS atomics only count).
//
// Moving rows is bound by memory: a workgroup takes one token and touches the
// token's k rows, whole rows at a time, so that every byte of the sorted buffer
// crosses the chip once.  The token's own row is read once instead of k times; the
// gradient of combine takes the choices that have a row in pieces of 8, 4, 2 and 1
// and reads it again, from the cache, for each (twice with 6 choices, four times
// with 15).  Stores, and the loads of the sorted buffer, are
// nontemporal: with 8192 tokens of 8 rows of 4 KB a buffer fills the last-level
// cache and pushes out what the next kernel reads (there and back 155 -> 118 us,
// its gradient 178 -> 159; dispatch and the product that reads the rows 162 -> 144
// with 2048 tokens, 279 -> 265 with 8192; smaller ones take the same time).
#include "gmm_launch.hpp"
#include "gmm_moe.hpp"
#include "gmm_mx8.hpp"

#include <type_traits>

namespace gmm {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------- the order --

constexpr int kRun = 1024;        // slots of a run, the least
constexpr int kMaxRuns = 1024;
constexpr int kSumRuns = 64;      // up to here (and 256 experts) every workgroup adds up the runs before its own
constexpr int kOneRun = 4096;     // up to here (and 1024 experts) one workgroup does everything

struct Runs {
    int count, slots;   // slots: of one run, a multiple of 256
};
Runs runs_of(int64_t n) {
    const int64_t c = (n + kRun - 1) / kRun, r = c < 1 ? 1 : (c < kMaxRuns ? c : kMaxRuns);
    const int64_t s = ((n + r - 1) / r + 255) / 256 * 256;
    return Runs{(int)(n > 0 ? (n + s - 1) / s : 1), (int)(s > 0 ? s : 256)};
}

// The local expert of a slot, G where it has none here.
__device__ __forceinline__ int expert_of(const int32_t* __restrict__ ids, int slot, int end, int first, int G) {
    if (slot >= end) return G;
    const unsigned e = (unsigned)ids[slot] - (unsigned)first;
    return ids[slot] >= 0 && e < (unsigned)G ? (int)e : G;
}

// counts[run, g]: slots of expert g in the run.
template <int GMAX>
__global__ __launch_bounds__(256) void count_kernel(const int32_t* __restrict__ ids, int n, int first, int G, int run,
                                                    int32_t* __restrict__ counts) {
    __shared__ int hist[GMAX];
    for (int g = threadIdx.x; g < G; g += 256) hist[g] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * run;
    const int hi = (int)(lo + run < n ? lo + run : n);
    for (int64_t s = lo + threadIdx.x; s < hi; s += 256) {
        const int e = expert_of(ids, (int)s, hi, first, G);
        if (e < G) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += 256) counts[(int64_t)blockIdx.x * G + g] = hist[g];
}

// counts[run, g] -> slots of expert g in earlier runs, and totals[g] behind
// them: 16 experts a workgroup, each of 64 threads a sixty-fourth of the runs,
// so that 512 runs (524288 slots) are one batch of loads a thread and stay in
// registers (4.4 us; with a quarter of the workgroups and two passes 7).
__global__ __launch_bounds__(1024) void scan_kernel(int32_t* __restrict__ counts, int runs, int G) {
    __shared__ int part[64][16];
    const int across = threadIdx.x & 15, seg = threadIdx.x >> 4, g = blockIdx.x * 16 + across;
    const int per = (runs + 63) / 64, lo = min(runs, seg * per), hi = min(runs, lo + per);
    const bool mine = g < G && lo < hi;
    constexpr int kHeld = kMaxRuns / 64;
    int c[kHeld], sum = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        c[i] = mine && lo + i < hi ? counts[(int64_t)(lo + i) * G + g] : 0;
        sum += c[i];
    }
    part[seg][across] = sum;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < seg; ++w) before += part[w][across];
    if (g < G && seg == 63) counts[(int64_t)runs * G + g] = before + sum;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        if (mine && lo + i < hi) counts[(int64_t)(lo + i) * G + g] = before;
        before += c[i];
    }
}

enum Before { kAlone = 0, kSum = 1, kScanned = 2 };   // one run; runs added up here; runs added up by scan_kernel

// Rows of a run's slots.  NW waves, each a contiguous NW-th of the run.
template <int NW, int GMAX, int BEFORE>
__global__ __launch_bounds__(64 * NW) void place_kernel(const int32_t* __restrict__ ids, int n, int first, int G,
                                                        int M, int run, int runs, const int32_t* __restrict__ counts,
                                                        int32_t* __restrict__ group_sizes, int32_t* __restrict__ row_of,
                                                        int32_t* __restrict__ slot_of, int32_t* __restrict__ status) {
    constexpr int NT = 64 * NW, EPT = (GMAX + NT - 1) / NT;
    __shared__ int next[NW][GMAX];   // counts of each wave, then the row of its next slot of each expert
    __shared__ int wave_sum[NW];
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
    for (int e = tid; e < NW * GMAX; e += NT) next[e / GMAX][e % GMAX] = 0;
    __syncthreads();
    const int64_t run_lo = (int64_t)blockIdx.x * run;
    const int run_hi = (int)(run_lo + run < n ? run_lo + run : n);
    const int part = (run + NT - 1) / NT * 64;
    const int64_t lo = run_lo + (int64_t)wave * part;
    const int hi = (int)(lo + part < run_hi ? lo + part : run_hi);
    for (int64_t s = lo + lane; s < hi; s += 64) {
        const int e = expert_of(ids, (int)s, hi, first, G);
        if (e < G) atomicAdd(&next[wave][e], 1);
    }
    __syncthreads();
    // the runs before and all runs of every expert, PARTS threads an expert
    constexpr int PARTS = BEFORE == kSum ? NT / GMAX : 1;
    static_assert(BEFORE != kSum || PARTS > 1, "several threads an expert");
    __shared__ int part_before[PARTS][PARTS > 1 ? GMAX : 1], part_total[PARTS][PARTS > 1 ? GMAX : 1];
    if constexpr (PARTS > 1) {
        const int g = tid % GMAX, q = tid / GMAX;
        const int per = (runs + PARTS - 1) / PARTS, r0 = min(runs, q * per), r1 = min(runs, r0 + per);
        int b = 0, t = 0;
        if (g < G) {
#pragma unroll 16
            for (int r = r0; r < r1; ++r) {
                const int c = counts[(int64_t)r * G + g];
                t += c;
                b += r < (int)blockIdx.x ? c : 0;
            }
        }
        part_before[q][g] = b;
        part_total[q][g] = t;
        __syncthreads();
    }
    // thread t: experts t EPT .. + EPT - 1, so that a scan over threads is one over experts
    int before[EPT], total[EPT], sum = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int g = tid * EPT + i;
        before[i] = total[i] = 0;
        if (g < G) {
            if constexpr (BEFORE == kAlone) {
                for (int w = 0; w < NW; ++w) total[i] += next[w][g];
            } else if constexpr (PARTS > 1) {
                for (int q = 0; q < PARTS; ++q) {
                    before[i] += part_before[q][g];
                    total[i] += part_total[q][g];
                }
            } else {
                before[i] = counts[(int64_t)blockIdx.x * G + g];
                total[i] = counts[(int64_t)runs * G + g];
            }
        }
        sum += total[i];
    }
    const int incl = wave_incl_scan(sum);
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int base = incl - sum, all = 0;
    for (int w = 0; w < NW; ++w) {
        base += w < wave ? wave_sum[w] : 0;
        all += wave_sum[w];
    }
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int g = tid * EPT + i;
        if (g >= G) break;
        if (blockIdx.x == 0) group_sizes[g] = min(base + total[i], M) - min(base, M);
        int row = base + before[i];
        for (int w = 0; w < NW; ++w) {
            const int c = next[w][g];
            next[w][g] = row;
            row += c;
        }
        base += total[i];
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) status[0] = all > M ? kDevSumGtM : 0;
    for (int64_t r = (int64_t)all + (int64_t)blockIdx.x * NT + tid; r < M; r += (int64_t)gridDim.x * NT) slot_of[r] = -1;
    const int bits = 32 - __clz(G);   // of G itself: the slots without an expert match each other too
    for (int64_t s0 = lo; s0 < hi; s0 += 64) {
        const int s = (int)s0 + lane;
        const int e = expert_of(ids, s, hi, first, G);
        unsigned long long same = ~0ull;   // lanes of the same expert
        for (int b = 0; b < bits; ++b) {
            const unsigned long long m = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? m : ~m;
        }
        const unsigned long long below = same & ((1ull << lane) - 1ull);
        int row = -1;
        if (e < G) row = next[wave][e] + __popcll(below);
        __builtin_amdgcn_wave_barrier();
        if (e < G && below == 0) next[wave][e] = row + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (s < hi) {
            const bool fits = row >= 0 && row < M;
            row_of[s] = fits ? row : -1;
            if (fits) slot_of[row] = s;
        }
    }
}

// ------------------------------------------------------------ moved rows --

// 16 bytes of a row as fp32 values, and back.
template <bool BF16>
struct Vec {
    static constexpr int N = BF16 ? 8 : 4;
    __device__ static void get(const u32x4& d, float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                v[2 * i] = bf16_lo(d[i]);
                v[2 * i + 1] = bf16_hi(d[i]);
            } else {
                v[i] = __uint_as_float(d[i]);
            }
        }
    }
};
// N consecutive values read or written as bf16 or fp32.
template <bool BF16, int N>
__device__ __forceinline__ void get_n(const void* p, int64_t e, float (&v)[N]) {
    constexpr int V = Vec<BF16>::N;
    if constexpr (N >= V) {
#pragma unroll
        for (int i = 0; i < N; i += V) {
            float u[V];
            Vec<BF16>::get(*reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + (e + i) * (BF16 ? 2 : 4)), u);
#pragma unroll
            for (int q = 0; q < V; ++q) v[i + q] = u[q];
        }
    } else {   // four bf16 values
        const uint2 d = *reinterpret_cast<const uint2*>(static_cast<const char*>(p) + e * 2);
        v[0] = bf16_lo(d.x);
        v[1] = bf16_hi(d.x);
        v[2] = bf16_lo(d.y);
        v[3] = bf16_hi(d.y);
    }
}
template <bool BF16, int N>
__device__ __forceinline__ void put_n(void* p, int64_t e, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        if constexpr (!BF16)
            store_out(reinterpret_cast<float*>(p) + e + i, make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
        else if constexpr (N == 4)
            store_out(reinterpret_cast<uint16_t*>(p) + e, make_uint2(pack_rne(v[0], v[1]), pack_rne(v[2], v[3])));
        else if (i % 8 == 0)
            store_out(reinterpret_cast<uint16_t*>(p) + e + i,
                      make_uint4(pack_rne(v[i], v[i + 1]), pack_rne(v[i + 2], v[i + 3]), pack_rne(v[i + 4], v[i + 5]),
                                 pack_rne(v[i + 6], v[i + 7])));
    }
}

// The rows of a token's choices: lane j < k holds choice j's row and weight;
// `mask` has the choices that have a row.
struct Choices {
    int row;
    float w;
    unsigned long long mask;
};
__device__ __forceinline__ Choices choices_of(const MoveArgs& a, int64_t t) {
    Choices c;
    const int lane = lane_id();
    c.row = lane < a.k ? a.row_of[t * a.k + lane] : -1;
    c.w = lane < a.k && a.weights != nullptr ? a.weights[t * a.k + lane] : 1.0f;
    c.mask = __ballot(c.row >= 0 && c.row < a.M);
    return c;
}

constexpr int kTailRows = 16;   // rows a unit behind the tokens' looks at

// Zeros in the rows r0 .. r0 + 15 of out that no slot owns (row_bytes a
// multiple of 16), by TPT threads.
template <int TPT>
__device__ __forceinline__ void zero_unowned(const MoveArgs& a, int64_t r0, void* out, int64_t row_bytes) {
    const int lane = lane_id();
    const int64_t r = r0 + lane, slots = a.T * a.k;
    bool none = false;
    if (lane < kTailRows && r < a.M) {
        const int s = a.slot_of[r];
        none = s < 0 || s >= slots;
    }
    for (unsigned long long m = __ballot(none); m != 0; m &= m - 1) {
        char* p = static_cast<char*>(out) + (r0 + __ffsll((long long)m) - 1) * row_bytes;
        for (int64_t b = 16 * (int64_t)(threadIdx.x % TPT); b < row_bytes; b += 16 * TPT)
            store_out(p + b, make_uint4(0u, 0u, 0u, 0u));
    }
}

// A unit is a token, or 16 rows of the sorted buffer to look for unowned ones.
// TPT threads take one: the workgroup, or (rows of up to 2 KB) each of its waves
// another.
__device__ __forceinline__ int64_t move_units(const MoveArgs& a) { return a.T + (a.M + kTailRows - 1) / kTailRows; }
template <int TPT>
__device__ __forceinline__ int64_t first_unit() {
    return (int64_t)blockIdx.x * (256 / TPT) + __builtin_amdgcn_readfirstlane(threadIdx.x / TPT);
}
template <int TPT>
__device__ __forceinline__ int64_t unit_step() { return (int64_t)gridDim.x * (256 / TPT); }

template <int TPT>
__global__ __launch_bounds__(256) void dispatch_kernel(const MoveArgs a, const char* __restrict__ x, int64_t row_bytes,
                                                       char* __restrict__ out) {
    for (int64_t u = first_unit<TPT>(); u < move_units(a); u += unit_step<TPT>()) {
        if (u >= a.T) {
            zero_unowned<TPT>(a, (u - a.T) * kTailRows, out, row_bytes);
            continue;
        }
        const Choices c = choices_of(a, u);
        if (c.mask == 0) continue;
        for (int64_t b = 16 * (int64_t)(threadIdx.x % TPT); b < row_bytes; b += 16 * TPT) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(x + u * row_bytes + b);
            for (unsigned long long m = c.mask; m != 0; m &= m - 1)
                store_out(out + (int64_t)lane_value(c.row, __ffsll((long long)m) - 1) * row_bytes + b,
                          make_uint4(v[0], v[1], v[2], v[3]));
        }
    }
}

// 16 bytes of row `row` of a matrix of `pitch`-byte rows, as stored; no other
// workgroup reads them.
__device__ __forceinline__ u32x4 row_vec(const void* p, int64_t row, int64_t pitch, int64_t b) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + row * pitch + b));
}

__device__ __forceinline__ float wave_sum_f(float x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
    return x;
}

// The first B choices of the mask, taken off it.  Their rows are loaded before
// any is used.
template <int B>
__device__ __forceinline__ void take_choices(unsigned long long& mask, int (&j)[B]) {
#pragma unroll
    for (int i = 0; i < B; ++i) {
        j[i] = __ffsll((long long)mask) - 1;
        mask &= mask - 1;
    }
}

// s += weights * rows of B choices.
template <bool Y_BF16, int B>
__device__ __forceinline__ void add_rows(const Choices& c, unsigned long long& mask, const void* y, int64_t pitch,
                                         int64_t b, float (&s)[Vec<Y_BF16>::N]) {
    constexpr int N = Vec<Y_BF16>::N;
    int j[B];
    take_choices<B>(mask, j);
    u32x4 d[B];
#pragma unroll
    for (int i = 0; i < B; ++i) d[i] = row_vec(y, lane_value(c.row, j[i]), pitch, b);
#pragma unroll
    for (int i = 0; i < B; ++i) {
        const float w = __int_as_float(lane_value(__float_as_int(c.w), j[i]));
        float v[N];
        Vec<Y_BF16>::get(d[i], v);
#pragma unroll
        for (int q = 0; q < N; ++q) s[q] = __builtin_fmaf(w, v[q], s[q]);
    }
}

template <int TPT, bool Y_BF16, bool OUT_BF16, bool RES>
__global__ __launch_bounds__(256) void combine_kernel(const MoveArgs a, const void* __restrict__ y, const void* residual,
                                                      void* out) {
    constexpr int N = Vec<Y_BF16>::N, kBytes = Y_BF16 ? 2 : 4;
    const int64_t pitch = a.K * kBytes;
    for (int64_t t = first_unit<TPT>(); t < a.T; t += unit_step<TPT>()) {
        const Choices c = choices_of(a, t);
        const int n = __popcll(c.mask);
        for (int64_t e = N * (int64_t)(threadIdx.x % TPT); e < a.K; e += N * TPT) {
            float s[N];
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = 0.0f;
            if constexpr (RES) get_n<OUT_BF16, N>(residual, t * a.K + e, s);
            unsigned long long mask = c.mask;
            for (int i = n >> 3; i > 0; --i) add_rows<Y_BF16, 8>(c, mask, y, pitch, e * kBytes, s);
            if (n & 4) add_rows<Y_BF16, 4>(c, mask, y, pitch, e * kBytes, s);
            if (n & 2) add_rows<Y_BF16, 2>(c, mask, y, pitch, e * kBytes, s);
            if (n & 1) add_rows<Y_BF16, 1>(c, mask, y, pitch, e * kBytes, s);
            put_n<OUT_BF16, N>(out, t * a.K + e, s);
        }
    }
}

// dy rows and, where wanted, partial dot products of B choices: acc[i] of the
// thread's columns.
template <int TPT, bool D_BF16, bool Y_BF16, int B>
__device__ __forceinline__ void grad_rows(const MoveArgs& a, const Choices& c, unsigned long long& mask, int64_t t,
                                          const void* dout, const void* y, void* dy, bool dots, float* part,
                                          float* dweights) {
    constexpr int N = Vec<Y_BF16>::N, kBytes = Y_BF16 ? 2 : 4;
    int j[B];
    take_choices<B>(mask, j);
    float acc[B];
#pragma unroll
    for (int i = 0; i < B; ++i) acc[i] = 0.0f;
    for (int64_t e = N * (int64_t)(threadIdx.x % TPT); e < a.K; e += N * TPT) {
        float d[N];
        get_n<D_BF16, N>(dout, t * a.K + e, d);
        u32x4 r[B];
        if (dots) {
#pragma unroll
            for (int i = 0; i < B; ++i) r[i] = row_vec(y, lane_value(c.row, j[i]), a.K * kBytes, e * kBytes);
        }
        if (dy != nullptr) {
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const float w = __int_as_float(lane_value(__float_as_int(c.w), j[i]));
                float v[N];
#pragma unroll
                for (int q = 0; q < N; ++q) v[q] = w * d[q];
                put_n<Y_BF16, N>(dy, (int64_t)lane_value(c.row, j[i]) * a.K + e, v);
            }
        }
        if (dots) {
#pragma unroll
            for (int i = 0; i < B; ++i) {
                float v[N];
                Vec<Y_BF16>::get(r[i], v);
#pragma unroll
                for (int q = 0; q < N; ++q) acc[i] = __builtin_fmaf(d[q], v[q], acc[i]);
            }
        }
    }
    if (!dots) return;
#pragma unroll
    for (int i = 0; i < B; ++i) acc[i] = wave_sum_f(acc[i]);
    if constexpr (TPT == 64) {
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (lane_id() == 0) dweights[t * a.k + j[i]] = acc[i];
    } else {   // the four waves' parts, in their order
        __syncthreads();
        if (lane_id() == 0) {
#pragma unroll
            for (int i = 0; i < B; ++i) part[(threadIdx.x >> 6) * 8 + i] = acc[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (threadIdx.x == i) dweights[t * a.k + j[i]] = ((part[i] + part[8 + i]) + part[16 + i]) + part[24 + i];
    }
}

template <int TPT, bool D_BF16, bool Y_BF16>
__global__ __launch_bounds__(256) void combine_bwd_kernel(const MoveArgs a, const void* __restrict__ dout, const void* y,
                                                          void* dy, float* __restrict__ dweights) {
    __shared__ float part[32];
    const int64_t units = dy != nullptr ? move_units(a) : a.T;
    const bool dots = dweights != nullptr;
    for (int64_t u = first_unit<TPT>(); u < units; u += unit_step<TPT>()) {
        if (u >= a.T) {
            zero_unowned<TPT>(a, (u - a.T) * kTailRows, dy, a.K * (Y_BF16 ? 2 : 4));
            continue;
        }
        const Choices c = choices_of(a, u);
        const int lane = threadIdx.x % TPT, n = __popcll(c.mask);
        if (dots && lane < a.k && !(c.mask >> lane & 1)) dweights[u * a.k + lane] = 0.0f;
        unsigned long long mask = c.mask;
        for (int i = n >> 3; i > 0; --i) grad_rows<TPT, D_BF16, Y_BF16, 8>(a, c, mask, u, dout, y, dy, dots, part, dweights);
        if (n & 4) grad_rows<TPT, D_BF16, Y_BF16, 4>(a, c, mask, u, dout, y, dy, dots, part, dweights);
        if (n & 2) grad_rows<TPT, D_BF16, Y_BF16, 2>(a, c, mask, u, dout, y, dy, dots, part, dweights);
        if (n & 1) grad_rows<TPT, D_BF16, Y_BF16, 1>(a, c, mask, u, dout, y, dy, dots, part, dweights);
    }
}

dim3 unit_grid(int64_t units, int tpt) {
    const int64_t blocks = (units + 256 / tpt - 1) / (256 / tpt);
    return dim3((unsigned)(blocks < 1 ? 1 : (blocks < (1 << 20) ? blocks : 1 << 20)));
}

// Threads a token takes for rows of `bytes` bytes.
bool wave_a_token(int64_t bytes) { return bytes <= 2048; }

template <int NW, int GMAX, int BEFORE>
hipError_t place(const int32_t* ids, int n, int first, int G, int M, Runs r, const int32_t* counts, int32_t* group_sizes,
                 int32_t* row_of, int32_t* slot_of, int32_t* status, hipStream_t stream) {
    hipLaunchKernelGGL((place_kernel<NW, GMAX, BEFORE>), dim3((unsigned)r.count), dim3(64 * NW), 0, stream, ids, n, first,
                       G, M, r.slots, r.count, counts, group_sizes, row_of, slot_of, status);
    return hipGetLastError();
}

// One workgroup orders the slots; nothing is kept between launches.
bool one_run(int64_t n, int64_t G) { return n <= kOneRun && G <= 1024; }

}  // namespace

int64_t sort_count_words(int64_t n, int64_t G) { return G <= 0 || one_run(n, G) ? 0 : ((int64_t)runs_of(n > 0 ? n : 0).count + 1) * G; }

hipError_t launch_sort_tokens(const int32_t* ids, int n, int first, int G, int M, int32_t* group_sizes, int32_t* row_of,
                              int32_t* slot_of, int32_t* counts, int32_t* status, hipStream_t stream) {
    if (one_run(n, G)) {
        const Runs one{1, n > 0 ? n : 1};
        if (G <= 256)
            return place<16, 256, kAlone>(ids, n, first, G, M, one, counts, group_sizes, row_of, slot_of, status, stream);
        return place<16, 1024, kAlone>(ids, n, first, G, M, one, counts, group_sizes, row_of, slot_of, status, stream);
    }
    const Runs r = runs_of(n);
    if (G <= 256)
        hipLaunchKernelGGL((count_kernel<256>), dim3((unsigned)r.count), dim3(256), 0, stream, ids, n, first, G, r.slots, counts);
    else
        hipLaunchKernelGGL((count_kernel<4096>), dim3((unsigned)r.count), dim3(256), 0, stream, ids, n, first, G, r.slots, counts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (r.count <= kSumRuns && G <= 256)
        return place<16, 256, kSum>(ids, n, first, G, M, r, counts, group_sizes, row_of, slot_of, status, stream);
    hipLaunchKernelGGL(scan_kernel, dim3((unsigned)((G + 15) / 16)), dim3(1024), 0, stream, counts, r.count, G);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (G <= 256)
        return place<16, 256, kScanned>(ids, n, first, G, M, r, counts, group_sizes, row_of, slot_of, status, stream);
    if (G <= 1024)
        return place<16, 1024, kScanned>(ids, n, first, G, M, r, counts, group_sizes, row_of, slot_of, status, stream);
    return place<4, 4096, kScanned>(ids, n, first, G, M, r, counts, group_sizes, row_of, slot_of, status, stream);
}

hipError_t launch_dispatch(const MoveArgs& a, const void* x, bool bf16, void* out, hipStream_t stream) {
    const int64_t units = a.T + (a.M + kTailRows - 1) / kTailRows, bytes = a.K * (bf16 ? 2 : 4);
    if (wave_a_token(bytes))
        hipLaunchKernelGGL((dispatch_kernel<64>), unit_grid(units, 64), dim3(256), 0, stream, a,
                           static_cast<const char*>(x), bytes, static_cast<char*>(out));
    else
        hipLaunchKernelGGL((dispatch_kernel<256>), unit_grid(units, 256), dim3(256), 0, stream, a,
                           static_cast<const char*>(x), bytes, static_cast<char*>(out));
    return hipGetLastError();
}

namespace {

// f(TPT, first type is bf16, second type is bf16)
template <typename F>
hipError_t with_types(bool wave, bool p, bool q, F f) {
    using std::integral_constant;
    auto types = [&](auto tpt) {
        constexpr integral_constant<bool, true> yes;
        constexpr integral_constant<bool, false> no;
        if (p) return q ? f(tpt, yes, yes) : f(tpt, yes, no);
        return q ? f(tpt, no, yes) : f(tpt, no, no);
    };
    return wave ? types(integral_constant<int, 64>{}) : types(integral_constant<int, 256>{});
}

}  // namespace

hipError_t launch_combine(const MoveArgs& a, const void* y, bool y_bf16, const void* residual, void* out, bool out_bf16,
                          hipStream_t stream) {
    return with_types(wave_a_token(a.K * (y_bf16 ? 2 : 4)), y_bf16, out_bf16, [&](auto tpt, auto yb, auto ob) {
        constexpr int TPT = decltype(tpt)::value;
        constexpr bool YB = decltype(yb)::value, OB = decltype(ob)::value;
        const dim3 grid = unit_grid(a.T, TPT), block(256);
        if (residual != nullptr)
            hipLaunchKernelGGL((combine_kernel<TPT, YB, OB, true>), grid, block, 0, stream, a, y, residual, out);
        else
            hipLaunchKernelGGL((combine_kernel<TPT, YB, OB, false>), grid, block, 0, stream, a, y, residual, out);
        return hipGetLastError();
    });
}

hipError_t launch_combine_bwd(const MoveArgs& a, const void* dout, bool dout_bf16, const void* y, bool y_bf16, void* dy,
                              float* dweights, hipStream_t stream) {
    const int64_t units = a.T + (dy != nullptr ? (a.M + kTailRows - 1) / kTailRows : 0);
    return with_types(wave_a_token(a.K * (y_bf16 ? 2 : 4)), dout_bf16, y_bf16, [&](auto tpt, auto db, auto yb) {
        constexpr int TPT = decltype(tpt)::value;
        constexpr bool DB = decltype(db)::value, YB = decltype(yb)::value;
        hipLaunchKernelGGL((combine_bwd_kernel<TPT, DB, YB>), unit_grid(units, TPT), dim3(256), 0, stream, a, dout, y, dy,
                           dweights);
        return hipGetLastError();
    });
}

}  // namespace gmm
