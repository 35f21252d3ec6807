// Grouped products of the gated expert block for gfx950: its forward, and the
// products of its backward pass.
//
//   kGated   P = x . w[g],  h = silu(P[:, :N]) * P[:, N:]   (reduce over K)
//   kBwdX    dx = dP . w[g]^T                               (reduce over 2N)
//   kBwdW    dw[g] = x_g^T dP_g                             (reduce over rows)
//   kBwdWQ   the same with x from an 8-bit checkpoint
//
// Operands move from global memory to LDS with the load-to-LDS instructions
// into a ring of S stages (gmm_tile.hpp); each wave owns 64 x 64 of the tile.
// The gated forward's tile holds gate columns in its left half and the up
// columns of the same outputs in its right half, and a wave owns 32 of each,
// so gate and up of one output meet in one lane's accumulators and the
// activation, the product and the checkpoint of P are an epilogue on
// registers.
#include "gmm_launch.hpp"
#include "gmm_mx8.hpp"
#include "gmm_tile.hpp"

namespace gmm {

namespace {

enum FfnMode { kGated = 0, kBwdX = 1, kBwdW = 2, kBwdWQ = 3 };
enum Save { kSaveNone = 0, kSaveBf16 = 1, kSaveMx8 = 2 };

struct FfnItem {
    int g, row0, lo, hi, c0, red_lo, red_hi;
};

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// Rows [lo, hi) x `bytes` bytes from byte column `col` of a matrix of
// `pitch`-byte rows, written as zeros by all threads (bytes, col and pitch
// multiples of 4).
__device__ __forceinline__ void zero_block(void* base, int64_t pitch, int lo, int hi, int64_t col, int bytes,
                                           int nthr) {
    const int w = bytes >> 2;
    for (int e = threadIdx.x; e < (hi - lo) * w; e += nthr)
        *reinterpret_cast<uint32_t*>(static_cast<char*>(base) + (int64_t)(lo + e / w) * pitch + col + 4 * (e % w)) = 0u;
}

// Work item of a workgroup; every mode's block 0 also writes the call's
// device status word.  TR x TC: tile rows and columns of the product.
template <int MODE, int TR, int TC, int NTHR>
__device__ __forceinline__ bool ffn_item(const FfnArgs& a, int* s_info, FfnItem& it) {
    const int lane = lane_id(), wave = threadIdx.x >> 6;
    if (wave == 1 && blockIdx.x == 0) {
        const int st = group_status(a.group_sizes, a.G, a.M);
        if (lane == 0) a.status[0] = st;
    }
    if constexpr (MODE == kBwdW || MODE == kBwdWQ) {
        if (wave == 0) {
            const TgmmTile tt = tgmm_tile(a.group_sizes, a.G, a.M, a.ntiles_r * a.ntiles_c,
                                          xcd_remap(blockIdx.x, a.nblocks), a.placement);
            if (lane == 0) { s_info[0] = tt.row_lo; s_info[1] = tt.row_hi; s_info[2] = tt.g; s_info[3] = tt.t; }
        }
        __syncthreads();
        it.red_lo = s_info[0];
        it.red_hi = s_info[1];
        it.g = s_info[2];
        if (it.g < 0) return false;
        it.row0 = (s_info[3] / a.ntiles_c) * TR;
        it.c0 = (s_info[3] % a.ntiles_c) * TC;
        it.lo = it.row0;
        it.hi = min(it.row0 + TR, a.K);
        return true;
    } else {
        if (wave == 0) {
            int col;
            const WorkItem wi = balanced_work_item<true>(a.group_sizes, a.G, a.M, TR, a.ntiles_c, blockIdx.x, col);
            if (lane == 0) { s_info[0] = wi.g; s_info[1] = wi.lo; s_info[2] = wi.hi; s_info[3] = col; }
        }
        __syncthreads();
        it.g = s_info[0];
        if (it.g < 0) return false;
        it.row0 = it.lo = s_info[1];
        it.hi = s_info[2];
        it.c0 = s_info[3] * (MODE == kGated ? TC / 2 : TC);
        it.red_lo = 0;
        it.red_hi = MODE == kGated ? a.K : a.NN;
        return true;
    }
}

// Rows past the last group: zeros in every output the call produces.
template <int MODE, bool OUT_BF16, int SAVE, int TC, int NTHR>
__device__ __forceinline__ void zero_tail(const FfnArgs& a, const FfnItem& it) {
    const int N = a.NN / 2;
    const int ocols = MODE == kGated ? N : a.K;
    const int n = min(MODE == kGated ? TC / 2 : TC, ocols - it.c0);
    constexpr int kOut = OUT_BF16 ? 2 : 4;
    zero_block(a.out, (int64_t)ocols * kOut, it.lo, it.hi, (int64_t)it.c0 * kOut, n * kOut, NTHR);
    if constexpr (SAVE == kSaveBf16) {
        zero_block(a.gu, (int64_t)a.NN * 2, it.lo, it.hi, (int64_t)it.c0 * 2, n * 2, NTHR);
        zero_block(a.gu, (int64_t)a.NN * 2, it.lo, it.hi, (int64_t)(N + it.c0) * 2, n * 2, NTHR);
    }
    if constexpr (SAVE == kSaveMx8) {
        zero_block(a.gu_q, a.NN, it.lo, it.hi, it.c0, n, NTHR);
        zero_block(a.gu_q, a.NN, it.lo, it.hi, N + it.c0, n, NTHR);
        for (int e = threadIdx.x; e < (it.hi - it.lo) * (n / 32); e += NTHR) {
            uint8_t* p = a.gu_s + (int64_t)(it.lo + e / (n / 32)) * (a.NN / 32) + it.c0 / 32 + e % (n / 32);
            p[0] = 0;
            p[N / 32] = 0;
        }
    }
}

// Epilogue of the gated forward for a TR x TC tile (gate columns, then up
// columns) held as 64 x 64 wave blocks: acc[i][0..1] gate, acc[i][2..3] up;
// lane (lr, lg) holds row 16i + lr and columns 16j + 4lg .. +3 of its wave's
// 32.  Everything leaves through LDS (`sm`, idle by now) so that global
// stores cover whole row segments.
template <bool OUT_BF16, int SAVE, int TR, int TC, int WN, int NTHR>
__device__ __forceinline__ void gated_epilogue(const FfnArgs& a, const FfnItem& it, v4f (&acc)[4][4],
                                               uint16_t* sm) {
    constexpr int H = TC / 2;
    const int tid = threadIdx.x, lane = lane_id();
    const int wm = (tid >> 6) / WN, wn = (tid >> 6) % WN, lr = lane & 15, lg = lane >> 4;
    const int N = a.NN / 2, rows = it.hi - it.lo;
    if constexpr (SAVE == kSaveBf16) {
        constexpr int P = TC + 8;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint2*>(sm + (wm * 64 + 16 * i + lr) * P + (j < 2 ? 0 : H) + wn * 32 + 16 * (j & 1) + 4 * lg) =
                    make_uint2(pack_rne(acc[i][j][0], acc[i][j][1]), pack_rne(acc[i][j][2], acc[i][j][3]));
        __syncthreads();
        for (int e = tid; e < rows * (TC / 8); e += NTHR) {
            const int r = e / (TC / 8), c = (e % (TC / 8)) * 8;
            const int col = it.c0 + (c < H ? c : c - H);
            if (col < N)
                store_out(a.gu + (int64_t)(it.lo + r) * a.NN + (c < H ? 0 : N) + col,
                          *reinterpret_cast<const uint4*>(sm + r * P + c));
        }
        __syncthreads();
    }
    if constexpr (SAVE == kSaveMx8) {
        // a wave's 32 gate (and up) columns of a row are one block, spread
        // over the lanes lr, lr + 16, lr + 32, lr + 48
        constexpr int P = TC + 16, NS = TC / 32;
        uint8_t* cm = reinterpret_cast<uint8_t*>(sm);
        uint8_t* ss = cm + TR * P;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const v4f v0 = acc[i][2 * p], v1 = acc[i][2 * p + 1];
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) m = max(m, max(abs_bits(v0[k]), abs_bits(v1[k])));
                const uint32_t c = mx8_scale_code(max_over_rows16(m));
                const float inv = mx8_inverse(c);
                const int r = wm * 64 + 16 * i + lr;
                uint8_t* d = cm + r * P + p * H + wn * 32 + 4 * lg;
                *reinterpret_cast<uint32_t*>(d) = e4m3x4(v0[0] * inv, v0[1] * inv, v0[2] * inv, v0[3] * inv);
                *reinterpret_cast<uint32_t*>(d + 16) = e4m3x4(v1[0] * inv, v1[1] * inv, v1[2] * inv, v1[3] * inv);
                if (lg == 0) ss[r * NS + p * WN + wn] = (uint8_t)c;
            }
        __syncthreads();
        for (int e = tid; e < rows * (TC / 16); e += NTHR) {
            const int r = e / (TC / 16), c = (e % (TC / 16)) * 16;
            const int col = it.c0 + (c < H ? c : c - H);
            if (col < N)
                store_out(a.gu_q + (int64_t)(it.lo + r) * a.NN + (c < H ? 0 : N) + col,
                          *reinterpret_cast<const uint4*>(cm + r * P + c));
        }
        for (int e = tid; e < rows * (NS / 2); e += NTHR) {   // pairs of scale bytes: 64 columns
            const int r = e / (NS / 2), k = (e % (NS / 2)) * 2;
            const int p = k / WN, b = k % WN;
            if (it.c0 + b * 32 < N)
                *reinterpret_cast<uint16_t*>(a.gu_s + (int64_t)(it.lo + r) * (a.NN / 32) + (p * N + it.c0) / 32 + b) =
                    *reinterpret_cast<const uint16_t*>(ss + r * NS + k);
        }
        __syncthreads();
    }
    if constexpr (OUT_BF16) {
        constexpr int P = H + 8;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const v4f g = acc[i][j], u = acc[i][j + 2];
                *reinterpret_cast<uint2*>(sm + (wm * 64 + 16 * i + lr) * P + wn * 32 + 16 * j + 4 * lg) =
                    make_uint2(pack_rne(silu_mul(g[0], u[0]), silu_mul(g[1], u[1])),
                               pack_rne(silu_mul(g[2], u[2]), silu_mul(g[3], u[3])));
            }
        __syncthreads();
        for (int e = tid; e < rows * (H / 8); e += NTHR) {
            const int r = e / (H / 8), c = (e % (H / 8)) * 8;
            if (it.c0 + c < N)
                store_out(reinterpret_cast<uint16_t*>(a.out) + (int64_t)(it.lo + r) * N + it.c0 + c,
                          *reinterpret_cast<const uint4*>(sm + r * P + c));
        }
    } else {
        constexpr int P = H + 4;
        float* fm = reinterpret_cast<float*>(sm);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const v4f g = acc[i][j], u = acc[i][j + 2];
                *reinterpret_cast<float4*>(fm + (wm * 64 + 16 * i + lr) * P + wn * 32 + 16 * j + 4 * lg) =
                    make_float4(silu_mul(g[0], u[0]), silu_mul(g[1], u[1]), silu_mul(g[2], u[2]), silu_mul(g[3], u[3]));
            }
        __syncthreads();
        for (int e = tid; e < rows * (H / 4); e += NTHR) {
            const int r = e / (H / 4), c = (e % (H / 4)) * 4;
            if (it.c0 + c < N)
                store_out(reinterpret_cast<float*>(a.out) + (int64_t)(it.lo + r) * N + it.c0 + c,
                          *reinterpret_cast<const float4*>(fm + r * P + c));
        }
    }
}

// 16 E4M3 codes of one checkpoint block -> 16 bf16 values (exact).
__device__ __forceinline__ void mx8_expand16(const u32x4& codes, uint32_t scale_code, u32x4& lo, u32x4& hi) {
    const float s = mx8_scale(scale_code);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        float v[4];
        mx8_values4(codes[d], s, v);
        const uint32_t p0 = pack_rne(v[0], v[1]), p1 = pack_rne(v[2], v[3]);
        if (d < 2) {
            lo[2 * d] = p0;
            lo[2 * d + 1] = p1;
        } else {
            hi[2 * d - 4] = p0;
            hi[2 * d - 3] = p1;
        }
    }
}

// WM x WN waves of 64 x 64, S stages, RES workgroups per CU.
template <int MODE, bool OUT_BF16, int SAVE, int S, int RES, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, RES * WM * WN / 4) void ffn_kernel(const FfnArgs a) {
    using D = DmaShape<S, RES, WM, WN>;
    constexpr int RD = D::kRD, TR = D::kTR, TC = D::kTC, NW = D::kWaves, NB = RD / 32, NTHR = 64 * NW;
    constexpr int NIA = MODE == kBwdWQ ? 0 : D::kInstrA, NIB = D::kInstrB, kSt = D::kStage;
    static_assert((WM == 2 && WN == 2) || (WM == 4 && WN == 2) || (WM == 2 && WN == 4), "2 x 2, 4 x 2 or 2 x 4 waves");
    static_assert(RES * S * kSt * 2 <= 163840 - 1024, "the rings of RES workgroups fit the LDS");
    static_assert(MODE != kBwdWQ || (NB == 1 && S >= 3 && TR * RD == NTHR * 16), "one 16-code chunk per thread");
    constexpr bool kW = MODE == kBwdW || MODE == kBwdWQ;   // both operands transposed
    constexpr bool A_TR = kW, B_TR = MODE != kBwdX, kSpread = kW;
    __shared__ __attribute__((aligned(1024))) uint16_t ring[S * kSt];
    __shared__ int s_info[5];
    static_assert(MODE != kGated || TR * (TC + 16) * 2 <= S * kSt * 2, "epilogue staging fits the ring");

    const int tid = threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    FfnItem it;
    if (!ffn_item<MODE, TR, TC, NTHR>(a, s_info, it)) return;
    if (!kW && it.g == a.G) {
        zero_tail<MODE, OUT_BF16, SAVE, TC, NTHR>(a, it);
        return;
    }
    const int K = a.K, NN = a.NN, N = NN / 2;
    const int g = it.g, row0 = it.row0, hi = it.hi, c0 = it.c0, red_lo = it.red_lo, red_hi = it.red_hi;

    // ---- global element offsets of this lane's load-to-LDS instructions at
    //      reduction index 0; rows and columns past the operand are clamped
    //      to its last ones (they only reach outputs that are not stored)
    const int lda = MODE == kGated ? K : NN;
    const uint16_t* wg = a.b + (kW ? 0 : (int64_t)g * K * NN);
    int64_t a_off[NIA > 0 ? NIA : 1], b_off[NIB];
    int a_row[NIA > 0 ? NIA : 1], b_row[NIB];
#pragma unroll
    for (int i = 0; i < NIA; ++i) {
        const int j = NIA * wave + i;
        if constexpr (kW) {
            const DmaLane d = dma_trans<kSpread, TR>(j, lane);
            a_row[i] = d.row;
            a_off[i] = min(row0 + d.col, K - 8);
        } else {
            const DmaLane d = dma_direct<RD, D::kChunks, D::kRows>(j, lane);
            a_row[i] = 0;
            a_off[i] = (int64_t)min(row0 + d.row, hi - 1) * lda + d.col;
        }
    }
#pragma unroll
    for (int i = 0; i < NIB; ++i) {
        const int j = NIB * wave + i;
        if constexpr (MODE == kBwdX) {
            const DmaLane d = dma_direct<RD, D::kChunks, D::kRows>(j, lane);
            b_row[i] = 0;
            b_off[i] = (int64_t)min(c0 + d.row, K - 1) * NN + d.col;
        } else {
            const DmaLane d = dma_trans<kSpread, TC>(j, lane);
            b_row[i] = d.row;
            if constexpr (MODE == kGated)
                b_off[i] = d.col < TC / 2 ? min(c0 + d.col, N - 8) : N + min(c0 + d.col - TC / 2, N - 8);
            else
                b_off[i] = min(c0 + d.col, NN - 8);
        }
    }
    auto issue = [&](int t, int stage) {
        const int r0 = red_lo + t * RD;
        uint16_t* sa = ring + stage * kSt;
        uint16_t* sb = sa + D::kSliceA;
#pragma unroll
        for (int i = 0; i < NIA; ++i) {
            const uint16_t* pa;
            if constexpr (kW)
                pa = a.a + (int64_t)min(r0 + a_row[i], red_hi - 1) * K + a_off[i];
            else
                pa = a.a + a_off[i] + r0;
            __builtin_amdgcn_global_load_lds(pa, (GMM_LDS void*)(sa + (NIA * wave + i) * 512), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < NIB; ++i) {
            const uint16_t* pb;
            if constexpr (kW)
                pb = a.b + (int64_t)min(r0 + b_row[i], red_hi - 1) * NN + b_off[i];
            else if constexpr (MODE == kGated)
                pb = wg + (int64_t)(r0 + b_row[i]) * NN + b_off[i];
            else
                pb = wg + b_off[i] + r0;
            __builtin_amdgcn_global_load_lds(pb, (GMM_LDS void*)(sb + (NIB * wave + i) * 512), 16, 0, 0);
        }
    };

    // ---- checkpointed x: thread t takes the 16 codes of columns
    //      16 (t % TR/16) .. +15 of slice row t / (TR/16), expands them and
    //      writes the 32-byte chunk the transposed layout has there
    constexpr int CPR = TR / 16;
    const int qrow = tid / CPR, qchunk = tid % CPR;
    const int qcol = min(row0 + 16 * qchunk, K - 16);
    u32x4 qd;
    uint32_t qs = 0;
    auto fetch_codes = [&](int t) {
        const int64_t m = min(red_lo + t * RD + qrow, red_hi - 1);
        qd = *reinterpret_cast<const u32x4*>(a.aq + m * K + qcol);
        qs = a.as[m * (K >> 5) + (qcol >> 5)];
    };
    auto put_codes = [&](int t, int stage) {
        u32x4 l, h;
        mx8_expand16(qd, qs, l, h);
        if (red_lo + t * RD + qrow >= red_hi) l = h = u32x4{0u, 0u, 0u, 0u};
        uint16_t* p = ring + stage * kSt + qrow * TR + 16 * (qchunk ^ trans_key<kSpread>(qrow));
        *reinterpret_cast<u32x4*>(p) = l;
        *reinterpret_cast<u32x4*>(p + 8) = h;
    };

    const int wm = (tid >> 6) / WN, wn = (tid >> 6) % WN;
    const int lr = lane & 15, lg = lane >> 4;
    v4f acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    constexpr int kHalfA = (kSpread ? 16 : 4) * TR * 2, kBlkA = 32 * TR * 2;
    constexpr int kHalfB = (kSpread ? 16 : 4) * TC * 2, kBlkB = 32 * TC * 2;
    const unsigned ring_lds = (unsigned)(uintptr_t)(GMM_LDS uint16_t*)ring;
    unsigned a_tr[4], b_tr[4], a_dir[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a_tr[i] = tr_addr<kSpread, TR>(lg, wm * 64 + i * 16, lr);
        // the gated tile: blocks 0, 1 gate columns, 2, 3 the same up columns
        const int bc = MODE == kGated ? (i < 2 ? 0 : TC / 2) + wn * 32 + (i & 1) * 16 : wn * 64 + i * 16;
        b_tr[i] = tr_addr<kSpread, TC>(lg, bc, lr);
        const int row = wm * 64 + i * 16 + lr;
        a_dir[i] = (unsigned)(2 * (row * RD + 8 * (lg ^ direct_key<RD>(row))));
    }

    const int nsl = (red_hi - red_lo + RD - 1) / RD;
#pragma unroll
    for (int t = 0; t < S - 1; ++t)
        if (t < nsl) issue(t, t);
    if constexpr (MODE == kBwdWQ) {
        // slices 0 .. S-3 now; slice u >= S-2 is fetched S-1 steps ahead and
        // written one step later
#pragma unroll
        for (int t = 0; t < S - 2; ++t)
            if (t < nsl) {
                fetch_codes(t);
                put_codes(t, t);
            }
        if (S - 2 < nsl) fetch_codes(S - 2);
    }
    int stage = 0;
    for (int t = 0; t < nsl; ++t) {
        if constexpr (MODE == kBwdWQ) {
            // codes of slice t + S - 2 were fetched last step; the wait for
            // them covers every older load, slice t's included
            const int st = stage + S - 2 >= S ? stage - 2 : stage + S - 2;
            if (t + S - 2 < nsl) put_codes(t + S - 2, st);
        }
        if (t + S - 2 < nsl) wait_vmem<(NIA + NIB) * (S - 2)>(); else wait_vmem<0>();
        stage_barrier();
        if (t + S - 1 < nsl) {
            issue(t + S - 1, stage == 0 ? S - 1 : stage - 1);
            if constexpr (MODE == kBwdWQ) fetch_codes(t + S - 1);
        }
        const uint16_t* ta = ring + stage * kSt;
        const uint16_t* tb = ta + D::kSliceA;
        const unsigned sbase = ring_lds + (unsigned)(stage * kSt * 2);
        v8bf atr[2][4], btr[2][4];
        const unsigned bs = sbase + (unsigned)(D::kSliceA * 2);
        if constexpr (!A_TR && B_TR && NB == 1) {
            const unsigned ad[4] = {sbase + a_dir[0], sbase + a_dir[1], sbase + a_dir[2], sbase + a_dir[3]};
            const unsigned bd[4] = {bs + b_tr[0], bs + b_tr[1], bs + b_tr[2], bs + b_tr[3]};
            direct_tr_slice<kHalfB>(atr[0], btr[0], ad, bd);
        } else if constexpr (A_TR && B_TR && NB == 1) {
            const unsigned ad[4] = {sbase + a_tr[0], sbase + a_tr[1], sbase + a_tr[2], sbase + a_tr[3]};
            const unsigned bd[4] = {bs + b_tr[0], bs + b_tr[1], bs + b_tr[2], bs + b_tr[3]};
            tr_slice_pair<kHalfA, kHalfB>(atr[0], btr[0], ad, bd);
        } else {
            if constexpr (A_TR) {
                const unsigned ad[4] = {sbase + a_tr[0], sbase + a_tr[1], sbase + a_tr[2], sbase + a_tr[3]};
                tr_slice<NB, kHalfA, kBlkA>(atr, ad);
            }
            if constexpr (B_TR) {
                const unsigned bd[4] = {bs + b_tr[0], bs + b_tr[1], bs + b_tr[2], bs + b_tr[3]};
                tr_slice<NB, kHalfB, kBlkB>(btr, bd);
            }
        }
        const int valid = red_hi - (red_lo + t * RD);
#pragma unroll
        for (int s = 0; s < NB; ++s) {
            v8bf af[4], bf[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (A_TR || (B_TR && NB == 1))
                    af[i] = atr[s][i];
                else
                    af[i] = swz_read_direct<RD>(ta, wm * 64 + i * 16 + lr, s * 4 + lg);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (B_TR)
                    bf[j] = btr[s][j];
                else
                    bf[j] = swz_read_direct<RD>(tb, wn * 64 + j * 16 + lr, s * 4 + lg);
            }
            if constexpr (kW) {   // rows past the group's end repeat its last row: dropped
                if (valid < RD) {
#pragma unroll
                    for (int i = 0; MODE == kBwdW && i < 4; ++i) af[i] = zero_rows_past<kSpread>(af[i], s, lg, valid);
#pragma unroll
                    for (int j = 0; j < 4; ++j) bf[j] = zero_rows_past<kSpread>(bf[j], s, lg, valid);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    __syncthreads();

    if constexpr (MODE == kGated) {
        gated_epilogue<OUT_BF16, SAVE, TR, TC, WN, NTHR>(a, it, acc, ring);
    } else {
        // each wave stages its 64 x 64 block and stores whole row segments
        const int ocols = MODE == kBwdX ? K : NN;
        const int64_t obase = kW ? (int64_t)g * K * NN : 0;
        const int col0 = c0 + wn * 64;
        if (col0 >= ocols) return;   // widths are multiples of 64
        if constexpr (OUT_BF16) {
            constexpr int kEpiRow = 64 + 8;
            static_assert(NW * 64 * kEpiRow <= S * kSt, "epilogue staging fits the ring");
            uint16_t* ep = ring + (tid >> 6) * 64 * kEpiRow;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint2*>(ep + (16 * i + lr) * kEpiRow + 16 * j + 4 * lg) =
                        make_uint2(pack_rne(acc[i][j][0], acc[i][j][1]), pack_rne(acc[i][j][2], acc[i][j][3]));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const int orow = lane >> 3, ocol = (lane & 7) * 8;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int r = 8 * q + orow;
                const uint4 v = *reinterpret_cast<const uint4*>(ep + r * kEpiRow + ocol);
                const int row = row0 + wm * 64 + r;
                if (row < hi)
                    store_out(reinterpret_cast<uint16_t*>(a.out) + obase + (int64_t)row * ocols + col0 + ocol, v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = row0 + wm * 64 + i * 16 + lr;
                if (row >= hi) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + obase + (int64_t)row * ocols + col0 + 16 * j + 4 * lg) =
                        make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
            }
        }
    }
}

template <int MODE, bool OUT_BF16, int SAVE, int S, int RES, int WM, int WN>
hipError_t launch(FfnArgs a, hipStream_t stream) {
    constexpr int TR = 64 * WM, TC = 64 * WN;
    int64_t nblocks;
    if constexpr (MODE == kBwdW || MODE == kBwdWQ) {
        a.ntiles_r = (a.K + TR - 1) / TR;
        a.ntiles_c = (a.NN + TC - 1) / TC;
        nblocks = (int64_t)a.G * a.ntiles_r * a.ntiles_c;
    } else {
        const int cols = MODE == kGated ? a.NN / 2 : a.K, tc = MODE == kGated ? TC / 2 : TC;
        a.ntiles_r = 0;
        a.ntiles_c = (cols + tc - 1) / tc;
        nblocks = max_work_items(a.M, a.G < a.M ? a.G : a.M, TR) * a.ntiles_c;
    }
    if (nblocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    a.nblocks = (int)nblocks;
    hipLaunchKernelGGL((ffn_kernel<MODE, OUT_BF16, SAVE, S, RES, WM, WN>), dim3((unsigned)nblocks), dim3(64 * WM * WN),
                       0, stream, a);
    return hipGetLastError();
}

// ------------------------------------------------------------- few rows --
// The gated forward for few rows per expert (a serving step): the work is
// reading each busy expert's weights once, so the tile is TR = 16 MB rows by
// CT gate + CT up columns, small enough that a handful of experts covers the
// chip, and the workgroup's NW waves split K between them: wave v takes the
// 32-deep slices v, v + NW, ...  Each wave feeds its own ring of S stages by
// load-to-LDS and never meets the others before the end, so no barrier stands
// in the stream of loads.  The partial sums meet in LDS, added in wave order.
//
// Stage layout: x as direct rows of 32; the weights as rows of CT gate and CT
// up columns in 32-byte chunks, chunk k at k ^ key: the 8 rows that one pass
// of a transposed read covers (0-3 and 8-11 of 16) fall on each bank once.
//
// What bounds it: a pass over one token's 8 experts (33 MB) takes 17.7 us, of
// which 3.4 us are launch and prologue; a bare read of as many cold bytes
// takes 10.4 us.  Deeper rings and more waves change nothing; weights that lie
// contiguously for each workgroup would (14 us), but the layout is the
// caller's.
template <int CT>
__device__ __forceinline__ int few_key(int r) {
    return CT == 32 ? ((r >> 1) & 1) | ((r >> 2) & 2) : (r >> 3) & 1;
}

// The reads of a slice in one asm block (one wait): MB direct fragments of x
// and the NF transposed ones of the weights, second half 4 rows on.
template <int MB, int NF, int HALF>
__device__ __forceinline__ void few_slice(v8bf (&fa)[MB], v8bf (&fb)[NF], const unsigned (&da)[MB],
                                          const unsigned (&ba)[NF]) {
    static_assert((MB == 1 || MB == 2 || MB == 4) && (NF == 2 || NF == 4), "1, 2 or 4 row blocks, 2 or 4 column blocks");
    if constexpr (MB == 4 && NF == 4) {
        direct_tr_slice<HALF>(fa, fb, da, ba);
        return;
    }
    // rows past MB read the last block again
    v4i d[4];
    u64 o[8];
    if constexpr (NF == 4)
        asm volatile(
            "ds_read_b128 %0, %10\n\t"
            "ds_read_b128 %1, %11\n\t"
            "ds_read_b64_tr_b16 %2, %12\n\t"
            "ds_read_b64_tr_b16 %3, %12 offset:%16\n\t"
            "ds_read_b64_tr_b16 %4, %13\n\t"
            "ds_read_b64_tr_b16 %5, %13 offset:%16\n\t"
            "ds_read_b64_tr_b16 %6, %14\n\t"
            "ds_read_b64_tr_b16 %7, %14 offset:%16\n\t"
            "ds_read_b64_tr_b16 %8, %15\n\t"
            "ds_read_b64_tr_b16 %9, %15 offset:%16\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(d[0]), "=&v"(d[1]), "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]), "=&v"(o[4]), "=&v"(o[5]),
              "=&v"(o[6]), "=&v"(o[7])
            : "v"(da[0]), "v"(da[MB - 1]), "v"(ba[0]), "v"(ba[1]), "v"(ba[NF - 2]), "v"(ba[NF - 1]), "i"(HALF)
            : "memory");
    else if constexpr (MB <= 2)
        asm volatile(
            "ds_read_b128 %0, %6\n\t"
            "ds_read_b128 %1, %7\n\t"
            "ds_read_b64_tr_b16 %2, %8\n\t"
            "ds_read_b64_tr_b16 %3, %8 offset:%10\n\t"
            "ds_read_b64_tr_b16 %4, %9\n\t"
            "ds_read_b64_tr_b16 %5, %9 offset:%10\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(d[0]), "=&v"(d[1]), "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3])
            : "v"(da[0]), "v"(da[MB - 1]), "v"(ba[0]), "v"(ba[1]), "i"(HALF)
            : "memory");
    else
        asm volatile(
            "ds_read_b128 %0, %8\n\t"
            "ds_read_b128 %1, %9\n\t"
            "ds_read_b128 %2, %10\n\t"
            "ds_read_b128 %3, %11\n\t"
            "ds_read_b64_tr_b16 %4, %12\n\t"
            "ds_read_b64_tr_b16 %5, %12 offset:%14\n\t"
            "ds_read_b64_tr_b16 %6, %13\n\t"
            "ds_read_b64_tr_b16 %7, %13 offset:%14\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3])
            : "v"(da[0]), "v"(da[1 % MB]), "v"(da[2 % MB]), "v"(da[3 % MB]), "v"(ba[0]), "v"(ba[1]), "i"(HALF)
            : "memory");
#pragma unroll
    for (int i = 0; i < MB; ++i) fa[i] = __builtin_bit_cast(v8bf, d[i]);
#pragma unroll
    for (int i = 0; i < NF; ++i) fb[i] = __builtin_bit_cast(v8bf, u64x2{o[2 * i], o[2 * i + 1]});
}

template <bool OUT_BF16, int SAVE, int MB, int CT, int NW, int S>
__global__ __launch_bounds__(64 * NW, 1) void gated_few_kernel(const FfnArgs a) {
    constexpr int TR = 16 * MB, NTHR = 64 * NW, NF = CT / 8, NI = CT / 8;
    constexpr int kA = TR * 32, kB = 64 * CT, kSt = kA + kB;   // elements
    constexpr int kRow = 2 * CT + 4;                           // fp32 staging row
    constexpr int kRing = NW * S * kSt;
    __shared__ __attribute__((aligned(1024))) uint16_t ring[kRing];
    __shared__ int s_info[5];
    static_assert(NW * TR * kRow * 2 <= kRing, "the partial sums fit the rings");
    static_assert(kRing * 2 <= 163840 - 1024, "the rings fit the LDS");

    const int tid = threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    FfnItem it;
    if (!ffn_item<kGated, TR, 2 * CT, NTHR>(a, s_info, it)) return;
    if (it.g == a.G) {
        zero_tail<kGated, OUT_BF16, SAVE, 2 * CT, NTHR>(a, it);
        return;
    }
    const int K = a.K, NN = a.NN, N = NN / 2;
    uint16_t* mine = ring + wave * S * kSt;
    int64_t a_off[MB], b_off[NI];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const DmaLane d = dma_direct<32, 4, 16>(i, lane);
        a_off[i] = (int64_t)min(it.row0 + d.row, it.hi - 1) * K + d.col;
    }
    constexpr int LPR = CT / 4;   // lanes per row of 2 CT columns
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int r = (64 / LPR) * i + lane / LPR, p = lane % LPR;
        const int col = 16 * ((p >> 1) ^ few_key<CT>(r)) + 8 * (p & 1);
        b_off[i] = (int64_t)r * NN + it.c0 + (col < CT ? col : N + col - CT);
    }
    const uint16_t* wg = a.b + (int64_t)it.g * K * NN;
    auto issue = [&](int i, int stage) {
        const int r0 = 32 * (wave + NW * i);
        uint16_t* sa = mine + stage * kSt;
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            const uint16_t* pa = a.a + a_off[j] + r0;
            __builtin_amdgcn_global_load_lds(pa, (GMM_LDS void*)(sa + j * 512), 16, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const uint16_t* pb = wg + (int64_t)r0 * NN + b_off[j];
            __builtin_amdgcn_global_load_lds(pb, (GMM_LDS void*)(sa + kA + j * 512), 16, 0, 0);
        }
    };
    const int lr = lane & 15, lg = lane >> 4;
    const unsigned base = (unsigned)(uintptr_t)(GMM_LDS uint16_t*)mine;
    unsigned a_dir[MB], b_tr[NF];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int row = 16 * i + lr;
        a_dir[i] = base + (unsigned)(2 * (row * 32 + 8 * (lg ^ direct_key<32>(row))));
    }
#pragma unroll
    for (int i = 0; i < NF; ++i) {
        const int r = 8 * lg + (lr >> 2);
        b_tr[i] = base + (unsigned)(2 * (kA + r * 2 * CT + 16 * (i ^ few_key<CT>(r)) + (lr & 3) * 4));
    }
    v4f acc[MB][NF];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    const int ns = (K / 32 - wave + NW - 1) / NW;   // this wave's slices
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        if (i < ns) issue(i, i);
    int stage = 0;
    for (int i = 0; i < ns; ++i) {
        if (i + S - 2 < ns) wait_vmem<(NI + MB) * (S - 2)>(); else wait_vmem<0>();
        if (i + S - 1 < ns) issue(i + S - 1, stage == 0 ? S - 1 : stage - 1);
        const unsigned so = (unsigned)(stage * kSt * 2);
        unsigned da[MB], ba[NF];
#pragma unroll
        for (int j = 0; j < MB; ++j) da[j] = a_dir[j] + so;
#pragma unroll
        for (int j = 0; j < NF; ++j) ba[j] = b_tr[j] + so;
        v8bf af[MB], bf[NF];
        few_slice<MB, NF, 4 * 4 * CT>(af, bf, da, ba);
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int j = 0; j < NF; ++j)
                acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], af[m], acc[m][j], 0, 0, 0);
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    __syncthreads();   // every wave is done with its ring
    float* part = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < NF; ++j)
            *reinterpret_cast<v4f*>(part + (wave * TR + 16 * m + lr) * kRow + 16 * j + 4 * lg) = acc[m][j];
    __syncthreads();
    // CT / 4 threads a row, 4 gate and 4 up columns each
    constexpr int TPR = CT / 4;
    for (int e = tid; e < TR * TPR; e += NTHR) {
        const int r = e / TPR, c = (e % TPR) * 4, row = it.row0 + r;
        if (row >= it.hi) continue;   // the lanes of a row together
        v4f g = v4f{0.f, 0.f, 0.f, 0.f}, u = g;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            g += *reinterpret_cast<const v4f*>(part + (w * TR + r) * kRow + c);
            u += *reinterpret_cast<const v4f*>(part + (w * TR + r) * kRow + CT + c);
        }
        const float h0 = silu_mul(g[0], u[0]), h1 = silu_mul(g[1], u[1]), h2 = silu_mul(g[2], u[2]),
                    h3 = silu_mul(g[3], u[3]);
        const int64_t o = (int64_t)row * N + it.c0 + c, pg = (int64_t)row * NN + it.c0 + c;
        if constexpr (OUT_BF16)
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + o) =
                make_uint2(pack_rne(h0, h1), pack_rne(h2, h3));
        else
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + o) = make_float4(h0, h1, h2, h3);
        if constexpr (SAVE == kSaveBf16) {
            *reinterpret_cast<uint2*>(a.gu + pg) = make_uint2(pack_rne(g[0], g[1]), pack_rne(g[2], g[3]));
            *reinterpret_cast<uint2*>(a.gu + pg + N) = make_uint2(pack_rne(u[0], u[1]), pack_rne(u[2], u[3]));
        }
        if constexpr (SAVE == kSaveMx8) {
            static_assert(SAVE != kSaveMx8 || CT == 32, "a row's columns are one block");
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const v4f v = p == 0 ? g : u;
                const uint32_t m = max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3])));
                const uint32_t sc = mx8_scale_code(__float_as_uint(max_over_8(__uint_as_float(m))));
                const float inv = mx8_inverse(sc);
                *reinterpret_cast<uint32_t*>(a.gu_q + pg + p * N) =
                    e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                if ((e & 7) == 0) a.gu_s[(pg + p * N) >> 5] = (uint8_t)sc;
            }
        }
    }
}

template <bool OUT_BF16, int SAVE, int MB, int CT, int NW, int S>
hipError_t launch_few(FfnArgs a, hipStream_t stream) {
    a.ntiles_c = a.NN / 2 / CT;
    a.nblocks = (int)(max_work_items(a.M, a.G < a.M ? a.G : a.M, 16 * MB) * a.ntiles_c);
    hipLaunchKernelGGL((gated_few_kernel<OUT_BF16, SAVE, MB, CT, NW, S>), dim3((unsigned)a.nblocks), dim3(64 * NW), 0,
                       stream, a);
    return hipGetLastError();
}

template <int MODE, int SAVE = kSaveNone>
hipError_t launch_any(const FfnArgs& a, bool out_bf16, hipStream_t stream) {
    return out_bf16 ? launch<MODE, true, SAVE, 3, 3, 2, 2>(a, stream) : launch<MODE, false, SAVE, 3, 3, 2, 2>(a, stream);
}

}  // namespace

int64_t gated_fwd_blocks(int64_t M, int64_t N, int64_t G) {
    // of the 128-row tiles; the few-row form only takes grids near the chip's size
    return max_work_items(M, G < M ? G : M, 128) * ((N + 63) / 64);
}

int64_t ffn_dx_blocks(int64_t M, int64_t K, int64_t G) {
    return max_work_items(M, G < M ? G : M, 128) * ((K + 127) / 128);
}

int64_t ffn_dw_blocks(int64_t K, int64_t NN, int64_t G) { return G * ((K + 127) / 128) * ((NN + 127) / 128); }

// The few-row form is for grids that the 128-row tiles leave unfilled.  With
// B busy experts (at most min(G, M)) of few rows each, those tiles make B N/64
// workgroups, each streaming its columns of the weights alone; below one per
// CU the chip idles.  Measured at K = 2048, N = 512, cold weights (us, 128-row
// tiles / few rows): 1 expert 25.7 / 10.4, 8 experts (33 MB) 28.7 / 17.7, 32
// experts 37.5 / 39.4.  16 + 16 columns (8 waves) fill the chip from half as
// many experts as 32 + 32 (4 waves): 8 experts 17.7 against 18.8 us, 16
// experts (more workgroups than CUs) 29.4 against 20.7 us.
constexpr int kFewMaxRows = 64;   // mean rows an expert: up to 4 blocks of 16

template <bool OUT_BF16, int SAVE, int MB>
hipError_t launch_few_mb(const FfnArgs& a, int busy, hipStream_t stream) {
    if constexpr (SAVE != kSaveMx8)
        if ((int64_t)busy * (a.NN / 32) <= device_cus())
            return launch_few<OUT_BF16, SAVE, MB, 16, 8, MB == 4 ? 3 : 4>(a, stream);
    return launch_few<OUT_BF16, SAVE, MB, 32, 4, 3>(a, stream);
}

template <int SAVE, bool OUT_BF16>
hipError_t launch_gated(const FfnArgs& a, hipStream_t stream) {
    const int busy = a.G < a.M ? a.G : a.M, rows = (a.M + busy - 1) / busy;
    if (rows <= kFewMaxRows && (int64_t)busy * (a.NN / 128) < device_cus()) {
        if (rows <= 16) return launch_few_mb<OUT_BF16, SAVE, 1>(a, busy, stream);
        if (rows <= 32) return launch_few_mb<OUT_BF16, SAVE, 2>(a, busy, stream);
        return launch_few_mb<OUT_BF16, SAVE, 4>(a, busy, stream);
    }
    return launch<kGated, OUT_BF16, SAVE, 3, 3, 2, 2>(a, stream);
}

hipError_t launch_gated_fwd(const FfnArgs& a, bool out_bf16, hipStream_t stream) {
    if (a.gu_q != nullptr) return out_bf16 ? launch_gated<kSaveMx8, true>(a, stream) : launch_gated<kSaveMx8, false>(a, stream);
    if (a.gu != nullptr) return out_bf16 ? launch_gated<kSaveBf16, true>(a, stream) : launch_gated<kSaveBf16, false>(a, stream);
    return out_bf16 ? launch_gated<kSaveNone, true>(a, stream) : launch_gated<kSaveNone, false>(a, stream);
}

hipError_t launch_ffn_dx(const FfnArgs& a, bool out_bf16, hipStream_t stream) {
    return launch_any<kBwdX>(a, out_bf16, stream);
}

hipError_t launch_ffn_dw(const FfnArgs& a, bool out_bf16, hipStream_t stream) {
    return a.aq != nullptr ? launch_any<kBwdWQ>(a, out_bf16, stream) : launch_any<kBwdW>(a, out_bf16, stream);
}

}  // namespace gmm
