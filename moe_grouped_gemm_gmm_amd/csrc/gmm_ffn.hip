// Grouped products of the gated expert block for gfx950: its forward, and the
// products of its backward pass.
//
//   kGated   P = x . w[g],  h = silu(P[:, :N]) * P[:, N:]   (reduce over K)
//   kBwdX    dx = dP . w[g]^T                               (reduce over 2N)
//   kBwdW    dw[g] = x_g^T dP_g                             (reduce over rows)
//   kBwdWQ   the same with x from an 8-bit checkpoint
//
// In the gated forward a tile holds gate columns in its left half and the up
// columns of the same outputs in its right half, arranged so that gate and up
// of one output meet in one lane's accumulators: the activation, the product
// and the checkpoint of P are an epilogue on registers.
//
// Operands move from global memory to LDS with the load-to-LDS instructions
// (gmm_tile.hpp) and from there to 16 x 16 x 32 or 32 x 32 x 16 MFMAs, sums in
// fp32.  In the order they stand here:
//   ffn_kernel       128 x 128 or 128 x 256 tiles, every product
//   ffn_bwd_kernel   both products of a small backward pass in one launch
//   ffn_ws_kernel    160 x 256 tiles fed by load waves, forward and dX
//   gated_few_kernel the forward for few rows per expert, K split over waves
#include "gmm_launch.hpp"
#include "gmm_mx8.hpp"
#include "gmm_tile.hpp"

#include <cmath>
#include <type_traits>

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

// Work item of block b when every group's rows are cut into ceil(s / cap)
// items of equal height (to 16 rows; cap a multiple of 16): a group of just
// over cap rows gives two halves instead of a full item and a sliver.  Items
// are dealt to the XCDs as in balanced_work_item.
__device__ __forceinline__ WorkItem even_item(int g, int glo, int ghi, int idx, int cap) {
    const int n = (ghi - glo + cap - 1) / cap;
    const int h = ((ghi - glo + n - 1) / n + 15) & ~15;
    WorkItem it;
    it.g = g;
    it.tile = -1;
    it.lo = glo + idx * h;
    it.hi = min(ghi, it.lo + h);
    return it;
}

// The item of block b (g < 0: none) and its column tile for more than 256
// groups, in two passes over group_sizes.
__device__ inline WorkItem even_item_scan(const int32_t* __restrict__ group_sizes, int G, int M, int cap, int ntiles,
                                          int b, int& col) {
    int carry = 0, items = 0;
    for (int base = 0; base < G; base += 64) {
        const GroupChunk ch = group_chunk(group_sizes, G, M, base, carry);
        carry = ch.next_carry;
        items += lane_value(wave_incl_scan(group_items<true>(ch.lo, ch.hi, cap)), 63);
    }
    const int total = min(carry, M);
    const int L = xcd_balance(b, (items + tail_items<true>(total, M, cap)) * ntiles);
    if (L < 0) return WorkItem{-1, 0, 0, 0};
    const int w = L / ntiles;
    col = L % ntiles;
    if (w >= items) return tail_item<true>(G, M, total, items, cap, w);
    int first = 0;
    carry = 0;
    for (int base = 0; base < G; base += 64) {
        const GroupChunk ch = group_chunk(group_sizes, G, M, base, carry);
        carry = ch.next_carry;
        const int c = group_items<true>(ch.lo, ch.hi, cap), incl = wave_incl_scan(c), Wb = first + incl - c;
        const unsigned long long m = __ballot(c > 0 && w >= Wb && w < Wb + c);
        if (m) {
            const int src = __ffsll((long long)m) - 1;
            return even_item(base + src, lane_value(ch.lo, src), lane_value(ch.hi, src), w - lane_value(Wb, src), cap);
        }
        first += lane_value(incl, 63);
    }
    return WorkItem{-1, 0, 0, 0};   // not reached: w < items has an owner
}

// The items of a call, for one wave: up to 256 groups the clamped ranges and
// item offsets stay in registers, every load issued before the first scan;
// beyond, each item is found from group_sizes.
struct EvenItems {
    int lo[4], hi[4], cn[4], W[4], items, total;
    __device__ __forceinline__ void init(const int32_t* __restrict__ group_sizes, int G, int M, int cap) {
        if (G > 256) return;
        const int lane = lane_id();
        int raw[4], carry = 0;
        items = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) raw[k] = group_size_at(group_sizes, G, 64 * k + lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            lo[k] = hi[k] = cn[k] = W[k] = 0;
            if (64 * k < G) {
                const GroupChunk ch = group_chunk_of(raw[k], M, carry);
                lo[k] = ch.lo;
                hi[k] = ch.hi;
                carry = ch.next_carry;
                cn[k] = group_items<true>(ch.lo, ch.hi, cap);
                const int incl = wave_incl_scan(cn[k]);
                W[k] = items + incl - cn[k];
                items += lane_value(incl, 63);
            }
        }
        total = min(carry, M);
    }
    // the item of block b (g < 0: none) and its column tile
    __device__ __forceinline__ WorkItem find(const int32_t* __restrict__ group_sizes, int G, int M, int cap, int ntiles,
                                             int b, int& col) const {
        col = 0;
        if (G > 256) return even_item_scan(group_sizes, G, M, cap, ntiles, b, col);
        const int L = xcd_balance(b, (items + tail_items<true>(total, M, cap)) * ntiles);
        if (L < 0) return WorkItem{-1, 0, 0, 0};
        const int w = L / ntiles;
        col = L % ntiles;
        if (w >= items) return tail_item<true>(G, M, total, items, cap, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned long long m = __ballot(cn[k] > 0 && w >= W[k] && w < W[k] + cn[k]);
            if (m) {
                const int src = __ffsll((long long)m) - 1;
                return even_item(64 * k + src, lane_value(lo[k], src), lane_value(hi[k], src),
                                 w - lane_value(W[k], src), cap);
            }
        }
        return WorkItem{-1, 0, 0, 0};   // not reached: w < items has an owner
    }
};

// Work item of a workgroup; every mode's block 0 also writes the call's
// device status word.  TR x TC: tile rows (the most an item has) and columns of
// the product.
template <int MODE, int TR, int TC>
__device__ __forceinline__ bool ffn_item(const FfnArgs& a, int block, int* s_info, FfnItem& it) {
    const int lane = lane_id(), wave = threadIdx.x >> 6;
    if (wave == 1 && block == 0) {
        const int st = group_status(a.group_sizes, a.G, a.M);
        if (lane == 0) a.status[0] = st;
    }
    if constexpr (MODE == kBwdW || MODE == kBwdWQ) {
        if (wave == 0) {
            const TgmmTile tt = tgmm_tile(a.group_sizes, a.G, a.M, a.ntiles_r * a.ntiles_c,
                                          xcd_remap(block, a.nblocks), block, /*placement*/ 0);
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
            EvenItems items;
            items.init(a.group_sizes, a.G, a.M, TR);
            const WorkItem wi = items.find(a.group_sizes, a.G, a.M, TR, a.ntiles_c, block, col);
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

// Epilogue of the gated forward.  Fragments j < NJ / 2 of a lane's row are
// gate columns, j + NJ / 2 the same up columns; lane (lr, lg) holds columns
// 4lg .. +3 of each 16 and row lr of every other 16-row block.  Everything
// leaves through LDS (`sm`, idle by now) so that global stores cover whole row
// segments.
template <bool OUT_BF16, int SAVE, int NJ>
__device__ __forceinline__ void gated_epilogue(const FfnArgs& a, const FfnItem& it, v4f (&acc)[4][NJ], uint16_t* sm) {
    constexpr int TC = 32 * NJ, H = TC / 2, HJ = NJ / 2, NTHR = 256;
    const int tid = threadIdx.x, lane = lane_id();
    const int wm = tid >> 7, wn = (tid >> 6) & 1, lr = lane & 15, lg = lane >> 4;
    const int N = a.NN / 2, rows = it.hi - it.row0;
    const int r0 = 16 * wm + lr, hc = 16 * HJ * wn + 4 * lg;   // tile row of block 0, column of fragment 0
    if constexpr (SAVE == kSaveBf16) {
        constexpr int P = TC + 8;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                *reinterpret_cast<uint2*>(sm + (r0 + 32 * i) * P + (j < HJ ? 0 : H) + hc + 16 * (j % HJ)) =
                    make_uint2(pack_rne(acc[i][j][0], acc[i][j][1]), pack_rne(acc[i][j][2], acc[i][j][3]));
        __syncthreads();
        for (int e = tid; e < rows * (TC / 8); e += NTHR) {
            const int r = e / (TC / 8), c = (e % (TC / 8)) * 8;
            const int col = it.c0 + (c < H ? c : c - H);
            if (col < N)
                store_out(a.gu + (int64_t)(it.row0 + r) * a.NN + (c < H ? 0 : N) + col,
                          *reinterpret_cast<const uint4*>(sm + r * P + c));
        }
        __syncthreads();
    }
    if constexpr (SAVE == kSaveMx8) {
        // 32 gate (or up) columns of a row are one block: two fragments, spread
        // over the lanes lr, lr + 16, lr + 32, lr + 48
        constexpr int P = TC + 16, NS = TC / 32;
        uint8_t* cm = reinterpret_cast<uint8_t*>(sm);
        uint8_t* ss = cm + 128 * P;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < HJ; ++b) {   // HJ / 2 gate blocks, then as many up blocks
                const v4f v0 = acc[i][2 * b], v1 = acc[i][2 * b + 1];
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) m = max(m, max(abs_bits(v0[k]), abs_bits(v1[k])));
                const uint32_t c = mx8_scale_code(max_over_rows16(m));
                const float inv = mx8_inverse(c);
                const int r = r0 + 32 * i, col = (b < HJ / 2 ? 0 : H) + 32 * (b % (HJ / 2)) + hc;
                *reinterpret_cast<uint32_t*>(cm + r * P + col) =
                    e4m3x4(v0[0] * inv, v0[1] * inv, v0[2] * inv, v0[3] * inv);
                *reinterpret_cast<uint32_t*>(cm + r * P + col + 16) =
                    e4m3x4(v1[0] * inv, v1[1] * inv, v1[2] * inv, v1[3] * inv);
                if (lg == 0) ss[r * NS + (col >> 5)] = (uint8_t)c;
            }
        __syncthreads();
        for (int e = tid; e < rows * (TC / 16); e += NTHR) {
            const int r = e / (TC / 16), c = (e % (TC / 16)) * 16;
            const int col = it.c0 + (c < H ? c : c - H);
            if (col < N)
                store_out(a.gu_q + (int64_t)(it.row0 + r) * a.NN + (c < H ? 0 : N) + col,
                          *reinterpret_cast<const uint4*>(cm + r * P + c));
        }
        for (int e = tid; e < rows * (NS / 2); e += NTHR) {   // pairs of scale bytes: 64 columns
            const int r = e / (NS / 2), k = (e % (NS / 2)) * 2, up = k >= NS / 2;
            const int b = k - (up ? NS / 2 : 0);
            if (it.c0 + b * 32 < N)
                *reinterpret_cast<uint16_t*>(a.gu_s + (int64_t)(it.row0 + r) * (a.NN / 32) + ((up ? N : 0) + it.c0) / 32 + b) =
                    *reinterpret_cast<const uint16_t*>(ss + r * NS + k);
        }
        __syncthreads();
    }
    using V = typename std::conditional<OUT_BF16, uint2, float4>::type;   // four columns
    using E = typename std::conditional<OUT_BF16, uint16_t, float>::type;
    constexpr int P = H + 16 / (int)sizeof(E), C = 16 / (int)sizeof(E);
    E* om = reinterpret_cast<E*>(sm);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < HJ; ++j) {
            const v4f g = acc[i][j], u = acc[i][j + HJ];
            const float h0 = silu_mul(g[0], u[0]), h1 = silu_mul(g[1], u[1]), h2 = silu_mul(g[2], u[2]),
                        h3 = silu_mul(g[3], u[3]);
            V v;
            if constexpr (OUT_BF16) v = make_uint2(pack_rne(h0, h1), pack_rne(h2, h3));
            else v = make_float4(h0, h1, h2, h3);
            *reinterpret_cast<V*>(om + (r0 + 32 * i) * P + hc + 16 * j) = v;
        }
    __syncthreads();
    for (int e = tid; e < rows * (H / C); e += NTHR) {
        const int r = e / (H / C), c = (e % (H / C)) * C;
        if (it.c0 + c < N)
            store_out(reinterpret_cast<E*>(a.out) + (int64_t)(it.row0 + r) * N + it.c0 + c,
                      *reinterpret_cast<const uint4*>(om + r * P + c));
    }
}

// 32 bytes to LDS address p.  In asm because an LDS access that the compiler
// sees makes it wait for every load into LDS in flight; the barrier that
// publishes the data waits for the writes.
__device__ __forceinline__ void put32(unsigned p, const u32x4& l, const u32x4& h) {
    asm volatile("ds_write_b128 %0, %1\n\tds_write_b128 %0, %2 offset:16" : : "v"(p), "v"(l), "v"(h) : "memory");
}

// 16 E4M3 codes of one checkpoint block -> 16 bf16 values (exact).
__device__ __forceinline__ void mx8_expand16(const u32x4& codes, uint32_t scale_code, u32x4& lo, u32x4& hi) {
    // one instruction for two codes: values times 2^(c - 127), rounded to bf16
    // (exact); c = 0 stands for 2^-127, a subnormal scale
    const float s = mx8_scale(scale_code);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t p0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[d], s, false));
        const uint32_t p1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[d], s, true));
        if (d < 2) {
            lo[2 * d] = p0;
            lo[2 * d + 1] = p1;
        } else {
            hi[2 * d - 4] = p0;
            hi[2 * d - 3] = p1;
        }
    }
}

// ---- fragment reads of one 32-deep slice, one asm block and one wait each.
// A wave's four direct fragments of A sit 2048 bytes apart (every other 16 rows
// of 64 bytes, the same swizzle key), direct fragments of B 1024 bytes; a
// wave's transposed fragments j and j + 4 of B 256 bytes apart (columns 128
// apart: the key only permutes the low 3 bits of the 32-byte chunk); the second
// half of a transposed fragment HA / HB bytes on.

template <int HB>
__device__ __forceinline__ void read_direct_tr8(v8bf (&fa)[4], v8bf (&fb)[8], unsigned a, const unsigned (&b)[4]) {
    v4i d[4];
    u64 o[16];
    asm volatile(
        "ds_read_b128 %0, %20\n\t"
        "ds_read_b64_tr_b16 %4, %21\n\t"
        "ds_read_b64_tr_b16 %5, %21 offset:%25\n\t"
        "ds_read_b64_tr_b16 %6, %22\n\t"
        "ds_read_b64_tr_b16 %7, %22 offset:%25\n\t"
        "ds_read_b64_tr_b16 %8, %23\n\t"
        "ds_read_b64_tr_b16 %9, %23 offset:%25\n\t"
        "ds_read_b64_tr_b16 %10, %24\n\t"
        "ds_read_b64_tr_b16 %11, %24 offset:%25\n\t"
        "ds_read_b64_tr_b16 %12, %21 offset:256\n\t"
        "ds_read_b64_tr_b16 %13, %21 offset:%26\n\t"
        "ds_read_b64_tr_b16 %14, %22 offset:256\n\t"
        "ds_read_b64_tr_b16 %15, %22 offset:%26\n\t"
        "ds_read_b64_tr_b16 %16, %23 offset:256\n\t"
        "ds_read_b64_tr_b16 %17, %23 offset:%26\n\t"
        "ds_read_b64_tr_b16 %18, %24 offset:256\n\t"
        "ds_read_b64_tr_b16 %19, %24 offset:%26\n\t"
        "ds_read_b128 %1, %20 offset:2048\n\t"
        "ds_read_b128 %2, %20 offset:4096\n\t"
        "ds_read_b128 %3, %20 offset:6144\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]),
          "=&v"(o[4]), "=&v"(o[5]), "=&v"(o[6]), "=&v"(o[7]), "=&v"(o[8]), "=&v"(o[9]), "=&v"(o[10]), "=&v"(o[11]),
          "=&v"(o[12]), "=&v"(o[13]), "=&v"(o[14]), "=&v"(o[15])
        : "v"(a), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "i"(HB), "i"(HB + 256)
        : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) fa[i] = __builtin_bit_cast(v8bf, d[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) fb[i] = __builtin_bit_cast(v8bf, u64x2{o[2 * i], o[2 * i + 1]});
}

template <int NJ>
__device__ __forceinline__ void read_direct_direct(v8bf (&fa)[4], v8bf (&fb)[NJ], unsigned a, unsigned b) {
    v4i d[4], e[8];
    if constexpr (NJ == 8)
        asm volatile(
            "ds_read_b128 %0, %12\n\t"
            "ds_read_b128 %4, %13\n\t"
            "ds_read_b128 %5, %13 offset:1024\n\t"
            "ds_read_b128 %6, %13 offset:2048\n\t"
            "ds_read_b128 %7, %13 offset:3*1024\n\t"
            "ds_read_b128 %8, %13 offset:4096\n\t"
            "ds_read_b128 %9, %13 offset:5120\n\t"
            "ds_read_b128 %10, %13 offset:6144\n\t"
            "ds_read_b128 %11, %13 offset:7168\n\t"
            "ds_read_b128 %1, %12 offset:2048\n\t"
            "ds_read_b128 %2, %12 offset:4096\n\t"
            "ds_read_b128 %3, %12 offset:6144\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(e[0]), "=&v"(e[1]), "=&v"(e[2]), "=&v"(e[3]),
              "=&v"(e[4]), "=&v"(e[5]), "=&v"(e[6]), "=&v"(e[7])
            : "v"(a), "v"(b)
            : "memory");
    else
        asm volatile(
            "ds_read_b128 %0, %8\n\t"
            "ds_read_b128 %4, %9\n\t"
            "ds_read_b128 %5, %9 offset:1024\n\t"
            "ds_read_b128 %6, %9 offset:2048\n\t"
            "ds_read_b128 %7, %9 offset:3*1024\n\t"
            "ds_read_b128 %1, %8 offset:2048\n\t"
            "ds_read_b128 %2, %8 offset:4096\n\t"
            "ds_read_b128 %3, %8 offset:6144\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(e[0]), "=&v"(e[1]), "=&v"(e[2]), "=&v"(e[3])
            : "v"(a), "v"(b)
            : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) fa[i] = __builtin_bit_cast(v8bf, d[i]);
#pragma unroll
    for (int i = 0; i < NJ; ++i) fb[i] = __builtin_bit_cast(v8bf, e[i]);
}

template <int HA, int HB>
__device__ __forceinline__ void read_tr_tr8(v8bf (&fa)[4], v8bf (&fb)[8], const unsigned (&a)[4],
                                            const unsigned (&b)[4]) {
    u64 p[8], o[16];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %24\n\t"
        "ds_read_b64_tr_b16 %1, %24 offset:%32\n\t"
        "ds_read_b64_tr_b16 %8, %28\n\t"
        "ds_read_b64_tr_b16 %9, %28 offset:%33\n\t"
        "ds_read_b64_tr_b16 %10, %29\n\t"
        "ds_read_b64_tr_b16 %11, %29 offset:%33\n\t"
        "ds_read_b64_tr_b16 %12, %30\n\t"
        "ds_read_b64_tr_b16 %13, %30 offset:%33\n\t"
        "ds_read_b64_tr_b16 %14, %31\n\t"
        "ds_read_b64_tr_b16 %15, %31 offset:%33\n\t"
        "ds_read_b64_tr_b16 %16, %28 offset:256\n\t"
        "ds_read_b64_tr_b16 %17, %28 offset:%34\n\t"
        "ds_read_b64_tr_b16 %18, %29 offset:256\n\t"
        "ds_read_b64_tr_b16 %19, %29 offset:%34\n\t"
        "ds_read_b64_tr_b16 %20, %30 offset:256\n\t"
        "ds_read_b64_tr_b16 %21, %30 offset:%34\n\t"
        "ds_read_b64_tr_b16 %22, %31 offset:256\n\t"
        "ds_read_b64_tr_b16 %23, %31 offset:%34\n\t"
        "ds_read_b64_tr_b16 %2, %25\n\t"
        "ds_read_b64_tr_b16 %3, %25 offset:%32\n\t"
        "ds_read_b64_tr_b16 %4, %26\n\t"
        "ds_read_b64_tr_b16 %5, %26 offset:%32\n\t"
        "ds_read_b64_tr_b16 %6, %27\n\t"
        "ds_read_b64_tr_b16 %7, %27 offset:%32\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(p[0]), "=&v"(p[1]), "=&v"(p[2]), "=&v"(p[3]), "=&v"(p[4]), "=&v"(p[5]), "=&v"(p[6]), "=&v"(p[7]),
          "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]), "=&v"(o[4]), "=&v"(o[5]), "=&v"(o[6]), "=&v"(o[7]),
          "=&v"(o[8]), "=&v"(o[9]), "=&v"(o[10]), "=&v"(o[11]), "=&v"(o[12]), "=&v"(o[13]), "=&v"(o[14]), "=&v"(o[15])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "i"(HA), "i"(HB),
          "i"(HB + 256)
        : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) fa[i] = __builtin_bit_cast(v8bf, u64x2{p[2 * i], p[2 * i + 1]});
#pragma unroll
    for (int i = 0; i < 8; ++i) fb[i] = __builtin_bit_cast(v8bf, u64x2{o[2 * i], o[2 * i + 1]});
}

// Sizes of a tile of 128 x (32 NJ): 4 waves, 2 x 2, of 64 x (16 NJ).
template <int NJ>
struct FfnTile {
    static constexpr int kTR = 128, kTC = 32 * NJ, kS = 3, kRes = NJ == 8 ? 2 : 3;
    static constexpr int kSliceA = kTR * 32, kSliceB = kTC * 32, kStage = kSliceA + kSliceB;   // elements
    static constexpr int kNIB = NJ / 2;            // load-to-LDS instructions of B per wave and slice
    static_assert(kRes * kS * kStage * 2 <= 163840 - 1024, "the rings of kRes workgroups fit the LDS");
};

// Column of fragment j of wave column wn within the tile.  Direct B (dX):
// 16 NJ contiguous columns.  Transposed B: the tile's left and right half
// give NJ / 2 fragments each (gate and up, in the gated forward).
template <int MODE, int NJ>
__device__ __forceinline__ int frag_col(int wn, int j) {
    if constexpr (MODE == kBwdX) return 16 * (NJ * wn + j);
    return (j >= NJ / 2 ? 16 * NJ : 0) + 16 * ((NJ / 2) * wn + j % (NJ / 2));
}

// What one workgroup does: tile `block` of the product, the ring (S stages) in
// LDS.
template <int MODE, bool OUT_BF16, int SAVE, int NJ>
__device__ __forceinline__ void ffn_tile(const FfnArgs& a, int block, uint16_t* ring, int* s_info) {
    using T = FfnTile<NJ>;
    constexpr int S = T::kS, TR = T::kTR, TC = T::kTC, NTHR = 256, kSt = T::kStage, NIB = T::kNIB;
    constexpr bool kW = MODE == kBwdW || MODE == kBwdWQ;   // both operands transposed
    constexpr bool kSpread = kW;

    const int tid = threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    FfnItem it;
    if (!ffn_item<MODE, TR, TC>(a, block, s_info, it)) return;
    if (!kW && it.g == a.G) {
        zero_tail<MODE, OUT_BF16, SAVE, TC, NTHR>(a, it);
        return;
    }
    const int K = a.K, NN = a.NN, N = NN / 2;
    const int g = it.g, row0 = it.row0, hi = it.hi, c0 = it.c0, red_lo = it.red_lo, red_hi = it.red_hi;
    // 16-row blocks of the tile that hold rows, and those of this wave (the
    // wave rows take alternate blocks, so both have work in a short tile)
    const int blocks = (hi - row0 + 15) >> 4;
    const int wm = wave >> 1, wn = wave & 1;
    const int nb = kW ? min(4, max(0, blocks - 4 * wm)) : (blocks + 1 - wm) >> 1;

    // ---- global addresses of this lane's load-to-LDS instructions: two of A
    //      and NIB of B per wave and slice.  Rows and columns past the operand
    //      are clamped to its last ones (they only reach outputs that are not
    //      stored); a 16-row block of A without rows is not loaded.
    const int lda = MODE == kGated ? K : NN;
    const uint16_t* wg = a.b + (kW ? 0 : (int64_t)g * K * NN);
    const int na = MODE == kBwdWQ ? 0 : (kW ? 2 : (wave < blocks) + (wave + 4 < blocks));
    int64_t a_off[2], b_off[NIB];
    int a_row[2] = {0, 0}, b_row[NIB];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (kW) {
            const DmaLane d = dma_trans<kSpread, TR>(wave + 4 * i, lane);
            a_row[i] = d.row;
            a_off[i] = min(row0 + d.col, K - 8);
        } else {
            const DmaLane d = dma_direct<32, 4, 16>(wave + 4 * i, lane);
            a_off[i] = (int64_t)min(row0 + d.row, hi - 1) * lda + d.col;
        }
    }
#pragma unroll
    for (int i = 0; i < NIB; ++i) {
        if constexpr (MODE == kBwdX) {
            const DmaLane d = dma_direct<32, 4, 16>(wave + 4 * i, lane);
            b_row[i] = 0;
            b_off[i] = (int64_t)min(c0 + d.row, K - 1) * NN + d.col;
        } else {
            const DmaLane d = dma_trans<kSpread, TC>(wave + 4 * i, lane);
            b_row[i] = d.row;
            if constexpr (MODE == kGated)
                b_off[i] = d.col < TC / 2 ? min(c0 + d.col, N - 8) : N + min(c0 + d.col - TC / 2, N - 8);
            else
                b_off[i] = min(c0 + d.col, NN - 8);
        }
    }
    auto issue = [&](int t, int stage) {
        const int r0 = red_lo + t * 32;
        uint16_t* sa = ring + stage * kSt + 512 * wave;
        uint16_t* sb = sa + T::kSliceA;
#pragma unroll
        for (int i = 0; i < NIB; ++i) {
            const uint16_t* pb;
            if constexpr (kW)
                pb = a.b + (int64_t)min(r0 + b_row[i], red_hi - 1) * NN + b_off[i];
            else if constexpr (MODE == kGated)
                pb = wg + (int64_t)(r0 + b_row[i]) * NN + b_off[i];
            else
                pb = wg + b_off[i] + r0;
            __builtin_amdgcn_global_load_lds(pb, (GMM_LDS void*)(sb + 2048 * i), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i >= na) break;
            const uint16_t* pa;
            if constexpr (kW)
                pa = a.a + (int64_t)min(r0 + a_row[i], red_hi - 1) * K + a_off[i];
            else
                pa = a.a + a_off[i] + r0;
            __builtin_amdgcn_global_load_lds(pa, (GMM_LDS void*)(sa + 2048 * i), 16, 0, 0);
        }
    };
    const int nsl = (red_hi - red_lo + 31) >> 5;
    // this wave's share of slice t has landed when only the younger slices'
    // loads are outstanding
    static_assert(S == 3, "one younger slice");
    auto wait_slice = [&](int t) {
        if (t + 1 >= nsl) wait_vmem<0>();
        else if (MODE == kBwdWQ && t + 2 < nsl) wait_vmem<NIB + 2>();   // and the codes fetched with it
        else if (na == 2) wait_vmem<(NIB + 2) * (S - 2)>();
        else if (na == 1) wait_vmem<(NIB + 1) * (S - 2)>();
        else wait_vmem<NIB * (S - 2)>();
    };

    const unsigned ring_lds = (unsigned)(uintptr_t)(GMM_LDS uint16_t*)ring;
    // ---- checkpointed x: thread t takes the 16 codes of columns
    //      16 (t % 8) .. +15 of slice row t / 8, expands them and writes the
    //      32-byte chunk the transposed layout has there
    const int qrow = tid / 8, qchunk = tid % 8;
    const int qcol = min(row0 + 16 * qchunk, K - 16);
    // Two sets of registers: codes are fetched two steps before they are put,
    // so the wait for them leaves a whole step of loads in flight.
    u32x4 qd[2];
    uint32_t qs[2];
    auto fetch_codes = [&](int t, int set) {
        const int64_t m = min(red_lo + t * 32 + qrow, red_hi - 1);
        qd[set] = *reinterpret_cast<const u32x4*>(a.aq + m * K + qcol);
        qs[set] = a.as[m * (K >> 5) + (qcol >> 5)];
    };
    auto put_codes = [&](int t, int set, int stage) {
        u32x4 l, h;
        mx8_expand16(qd[set], qs[set], l, h);
        if (red_lo + t * 32 + qrow >= red_hi) l = h = u32x4{0u, 0u, 0u, 0u};
        put32(ring_lds + 2 * (unsigned)(stage * kSt + qrow * TR + 16 * (qchunk ^ trans_key<kSpread>(qrow))), l, h);
    };

    // ---- LDS addresses of this lane's fragments in stage 0
    const int lr = lane & 15, lg = lane >> 4;
    constexpr int kHalfA = 16 * TR * 2, kHalfB = (kSpread ? 16 : 4) * TC * 2;
    unsigned ra[4], rb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 16 * (2 * i + wm) + lr;   // interleaved blocks; only ra[0] with 2048-byte steps is used
        ra[i] = ring_lds + (kW ? tr_addr<true, TR>(lg, 64 * wm + 16 * i, lr)
                               : (unsigned)(2 * (row * 32 + 8 * (lg ^ direct_key<32>(row)))));
        const int br = 16 * NJ * wn + lr;
        rb[i] = ring_lds + 2 * T::kSliceA +
                (MODE == kBwdX ? (unsigned)(2 * (br * 32 + 8 * (lg ^ direct_key<32>(br))))
                               : tr_addr<kSpread, TC>(lg, frag_col<MODE, NJ>(wn, i), lr));
    }

    v4f acc[4][NJ];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    int stage = 0;
    // steady: at least S more slices follow (no conditions then, so that the
    // compiler's own count of the loads younger than the codes is exact)
    auto step = [&](int t, auto set_, auto steady_) __attribute__((always_inline)) {
        constexpr int set = decltype(set_)::value;   // t % 2, for the codes
        constexpr bool steady = decltype(steady_)::value;
        if constexpr (MODE == kBwdWQ)
            if (steady || t + 1 < nsl) put_codes(t + 1, set, stage == S - 1 ? 0 : stage + 1);
        if constexpr (steady && MODE == kBwdWQ) wait_vmem<NIB + 2>();
        else wait_slice(t);
        stage_barrier();
        if (steady || t + S - 1 < nsl) issue(t + S - 1, stage == 0 ? S - 1 : stage - 1);
        if constexpr (MODE == kBwdWQ)
            if (steady || t + S < nsl) fetch_codes(t + S, set);
        const unsigned so = (unsigned)(stage * kSt * 2);
        v8bf af[4], bf[NJ];
        if constexpr (MODE == kBwdX) {
            read_direct_direct<NJ>(af, bf, ra[0] + so, rb[0] + so);
        } else {
            const unsigned bd[4] = {rb[0] + so, rb[1] + so, rb[2] + so, rb[3] + so};
            if constexpr (kW) {
                const unsigned ad[4] = {ra[0] + so, ra[1] + so, ra[2] + so, ra[3] + so};
                if constexpr (NJ == 8) read_tr_tr8<kHalfA, kHalfB>(af, bf, ad, bd);
                else tr_slice_pair<kHalfA, kHalfB>(af, bf, ad, bd);
            } else if constexpr (NJ == 8) {
                read_direct_tr8<kHalfB>(af, bf, ra[0] + so, bd);
            } else {
                const unsigned ad[4] = {ra[0] + so, ra[1] + so, ra[2] + so, ra[3] + so};
                direct_tr_slice<kHalfB>(af, bf, ad, bd);
            }
        }
        if constexpr (kW) {   // rows past the group's end repeat its last row: dropped
            const int valid = red_hi - (red_lo + t * 32);
            if (valid < 32) {
#pragma unroll
                for (int i = 0; MODE == kBwdW && i < 4; ++i) af[i] = zero_rows_past<kSpread>(af[i], 0, lg, valid);
#pragma unroll
                for (int j = 0; j < NJ; ++j) bf[j] = zero_rows_past<kSpread>(bf[j], 0, lg, valid);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= nb) break;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    };
    constexpr std::integral_constant<int, 0> set0;
    constexpr std::integral_constant<int, 1> set1;
    if constexpr (MODE == kBwdWQ) {
        int t = 0;
        if (nsl > S + 1) {
            fetch_codes(0, 0);
            issue(0, 0);
            put_codes(0, 0, 0);
            fetch_codes(1, 0);
            issue(1, 1);
            fetch_codes(2, 1);
            do {
                step(t, set0, std::true_type{});
                step(t + 1, set1, std::true_type{});
                t += 2;
            } while (t + 1 + S < nsl);
        } else {
            if (nsl > 0) {
                fetch_codes(0, 0);
                issue(0, 0);
                put_codes(0, 0, 0);
            }
            if (nsl > 1) {
                fetch_codes(1, 0);
                issue(1, 1);
            }
            if (nsl > 2) fetch_codes(2, 1);
        }
        for (; t < nsl; t += 2) {
            step(t, set0, std::false_type{});
            if (t + 1 < nsl) step(t + 1, set1, std::false_type{});
        }
    } else {
#pragma unroll
        for (int t = 0; t < S - 1; ++t)
            if (t < nsl) issue(t, t);
        for (int t = 0; t < nsl; ++t) step(t, set0, std::false_type{});
    }
    __syncthreads();

    if constexpr (MODE == kGated) {
        gated_epilogue<OUT_BF16, SAVE, NJ>(a, it, acc, ring);
    } else {
        // each wave stages 64 rows x 64 columns at a time and stores whole row
        // segments; widths are multiples of 64, so a wave's 64 columns are all
        // inside or all outside
        const int ocols = MODE == kBwdX ? K : NN;
        const int64_t obase = kW ? (int64_t)g * K * NN : 0;
        auto tile_row = [&](int r) { return kW ? 64 * wm + r : 32 * (r >> 4) + 16 * wm + (r & 15); };
#pragma unroll
        for (int q = 0; q < NJ / 4; ++q) {
            if constexpr (OUT_BF16) {
                constexpr int kEpiRow = 64 + 8;
                static_assert(4 * 64 * kEpiRow <= S * kSt, "epilogue staging fits the ring");
                uint16_t* ep = ring + wave * 64 * kEpiRow;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const v4f v = acc[i][4 * q + j];
                        *reinterpret_cast<uint2*>(ep + (16 * i + lr) * kEpiRow + 16 * j + 4 * lg) =
                            make_uint2(pack_rne(v[0], v[1]), pack_rne(v[2], v[3]));
                    }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                const int orow = lane >> 3, ocol = (lane & 7) * 8;
                const int col = c0 + frag_col<MODE, NJ>(wn, 4 * q + ocol / 16) + ocol % 16;
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    const int r = 8 * p + orow;
                    const uint4 v = *reinterpret_cast<const uint4*>(ep + r * kEpiRow + ocol);
                    const int row = row0 + tile_row(r);
                    if (row < hi && col < ocols)
                        store_out(reinterpret_cast<uint16_t*>(a.out) + obase + (int64_t)row * ocols + col, v);
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row0 + tile_row(16 * i + lr);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int col = c0 + frag_col<MODE, NJ>(wn, 4 * q + j) + 4 * lg;
                        if (row < hi && col < ocols)
                            *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.out) + obase + (int64_t)row * ocols + col) =
                                acc[i][4 * q + j];
                    }
                }
            }
        }
    }
}

template <int MODE, bool OUT_BF16, int SAVE, int NJ>
__global__ __launch_bounds__(256, FfnTile<NJ>::kRes) void ffn_kernel(const FfnArgs a) {
    using T = FfnTile<NJ>;
    __shared__ __attribute__((aligned(1024))) uint16_t ring[T::kS * T::kStage];
    __shared__ int s_info[4];
    ffn_tile<MODE, OUT_BF16, SAVE, NJ>(a, blockIdx.x, ring, s_info);
}

// Both products of the backward pass in one grid (dX's blocks first, padded to
// a multiple of the XCDs): small problems wait for launches and for their
// last tiles, not for either product (301 rows, 5 experts, K = 512, 2N = 384, on
// the device: 15.6 us for the activation's gradient and two launches, 10.6 with
// one, 2.9 and 8.1 of it the two kernels).
template <bool X_BF16, bool W_BF16, bool MX8>
__global__ __launch_bounds__(256, FfnTile<4>::kRes) void ffn_bwd_kernel(const FfnArgs x, const FfnArgs w) {
    using T = FfnTile<4>;
    __shared__ __attribute__((aligned(1024))) uint16_t ring[T::kS * T::kStage];
    __shared__ int s_info[4];
    if ((int)blockIdx.x < x.nblocks)
        ffn_tile<kBwdX, X_BF16, kSaveNone, 4>(x, blockIdx.x, ring, s_info);
    else
        ffn_tile<MX8 ? kBwdWQ : kBwdW, W_BF16, kSaveNone, 4>(w, (int)blockIdx.x - x.nblocks, ring, s_info);
}

// Tiles of a's grid; false when it is too large.
template <int MODE, int NJ>
bool set_grid(FfnArgs& a) {
    using T = FfnTile<NJ>;
    int64_t nblocks;
    if constexpr (MODE == kBwdW || MODE == kBwdWQ) {
        a.ntiles_r = (a.K + T::kTR - 1) / T::kTR;
        a.ntiles_c = (a.NN + T::kTC - 1) / T::kTC;
        nblocks = (int64_t)a.G * a.ntiles_r * a.ntiles_c;
    } else {
        const int cols = MODE == kGated ? a.NN / 2 : a.K, tc = MODE == kGated ? T::kTC / 2 : T::kTC;
        a.ntiles_r = 0;
        a.ntiles_c = (cols + tc - 1) / tc;
        nblocks = max_work_items(a.M, a.G < a.M ? a.G : a.M, T::kTR) * a.ntiles_c;
    }
    a.nblocks = (int)nblocks;
    return nblocks < (int64_t)1 << 24;   // 2^32 threads
}

template <int MODE, bool OUT_BF16, int SAVE, int NJ>
hipError_t launch(FfnArgs a, hipStream_t stream) {
    if (!set_grid<MODE, NJ>(a)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((ffn_kernel<MODE, OUT_BF16, SAVE, NJ>), dim3((unsigned)a.nblocks), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <bool X_BF16, bool W_BF16>
hipError_t launch_both(FfnArgs x, FfnArgs w, hipStream_t stream) {
    if (!set_grid<kBwdX, 4>(x) || !set_grid<kBwdW, 4>(w)) return hipErrorInvalidConfiguration;
    x.nblocks = (x.nblocks + kNumXcd - 1) / kNumXcd * kNumXcd;
    const dim3 grid((unsigned)(x.nblocks + w.nblocks));
    if (w.aq != nullptr)
        hipLaunchKernelGGL((ffn_bwd_kernel<X_BF16, W_BF16, true>), grid, dim3(256), 0, stream, x, w);
    else
        hipLaunchKernelGGL((ffn_bwd_kernel<X_BF16, W_BF16, false>), grid, dim3(256), 0, stream, x, w);
    return hipGetLastError();
}

// ----------------------------------------- 160 x 256 tiles, load waves --
// The forward and dX on tiles of up to 160 rows x 256 columns, one workgroup
// per CU: 8 waves (2 x 4) multiply, each 80 x 64 in 32 x 32 x 16 MFMAs, and 4
// waves do nothing but issue the loads into a ring of 3 stages, 64 deep (156
// KB).  A load-to-LDS instruction that the memory system cannot take yet waits
// at issue, with the wave that issues it: in a wave that also multiplies the
// two times add up (8192 rows, 32 experts, K = 2048, 2N = 1024: forward 80 us
// on the smaller tiles, 57 on these).  By the counters the forward moves 32 GB/s
// a CU into LDS, with the matrix units 30 % and the LDS 25 % busy; dX 34 GB/s,
// 32 and 34 %.
// Direct rows are loaded 128 bytes at a time, whole cache lines (in 64-byte
// pieces, 32 deep, the rows of x cost the shard's forward 14 of its 56 us).
//
// With two multiplying waves per SIMD the LDS reads cannot hide behind other
// waves, so they are interleaved with the MFMAs of the quarter step before
// (ws_step).  One barrier a stage: at the barrier of step u the multiplying
// waves have read all of stage u and the load waves have waited for stage
// u + 1; after it stage u + 1 may be read and slice u + 3 loaded over slice u.
//
// A workgroup takes items until none is left.  After an item's slices one slot
// of the ring is skipped and serves to stage its results, while the load waves
// fill the two slots after it from the next item: the start of one item hides
// behind the end of the one before (dX of 65536 rows, 256 experts with the
// activation's gradient 462 -> 414 us).
//
// The wave rows take alternate 32-row blocks and a wave multiplies only its
// blocks that hold rows (a loop compiled for each count), so an item's cost
// follows its rows; 8 rows of A past the item's end are not loaded.
//
// LDS layout: direct operands as 128-byte rows, chunk c of row r at c ^ (r %
// 8); transposed B as two slices of 32 rows x 512 bytes, 32-byte chunk k of
// row r at k ^ (2 (r % 4)): one pass of a transposed read covers rows 4n ..
// 4n+3 of two neighbouring chunks.
typedef float v16f __attribute__((ext_vector_type(16)));

// One quarter step of a wave: the products of 16 reduction indices (NB 32-row
// blocks x 2 column blocks of 32 x 32 x 16) with the fragments already in
// registers, and between them the LDS reads of the next 16, all in one asm
// block that waits for its reads at its end, so that they take the matrix
// unit's time and no register is read before its load.  The compiler does not
// see the MFMAs, so the block also waits for their results itself: 12 wait
// states after the last one (s_nop 11, what the compiler keeps behind its own
// builtin before anything reads or overwrites the result), and two before the
// first for operands that vector instructions wrote.  Whatever register
// allocation places between two blocks or behind the last is then safe.  The
// wait falls into the time of the last MFMA (32 cycles, before which the next
// block's first cannot start).  A comes from NB direct fragments 8192 bytes
// apart; B from two transposed fragments 256 bytes apart, second halves 2048
// bytes on (BTR), or two direct ones 4096 bytes apart.  OB is added to
// transposed B's address.
template <int OB>
__device__ __forceinline__ void ws_step(std::integral_constant<int, 1>, std::integral_constant<bool, true>, v16f (&acc)[3][2],
                                         const v8bf (&fa)[3], const v8bf (&fb)[2], v8bf (&ga)[3], v8bf (&gb)[2], unsigned a,
                                         unsigned b) {
    v4i na0;
    u64 nb0, nb1, nb2, nb3;
    asm volatile(
        "s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %8, %7, %0\n\t"
        "ds_read_b64_tr_b16 %3, %11 offset:%12\n\t"
        "ds_read_b64_tr_b16 %4, %11 offset:%13\n\t"
        "ds_read_b64_tr_b16 %5, %11 offset:%14\n\t"
        "v_mfma_f32_32x32x16_bf16 %1, %9, %7, %1\n\t"
        "ds_read_b64_tr_b16 %6, %11 offset:%15\n\t"
        "ds_read_b128 %2, %10 offset:0\n\t"
        "s_nop 11\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "+v"(acc[0][0]), "+v"(acc[0][1]),
          "=&v"(na0), "=&v"(nb0), "=&v"(nb1), "=&v"(nb2), "=&v"(nb3)
        : "v"(fa[0]), "v"(fb[0]), "v"(fb[1]), "v"(a), "v"(b),
          "i"(OB), "i"(OB + 2048), "i"(OB + 256), "i"(OB + 2304)
        : "memory");
    ga[0] = __builtin_bit_cast(v8bf, na0);
    gb[0] = __builtin_bit_cast(v8bf, u64x2{nb0, nb1});
    gb[1] = __builtin_bit_cast(v8bf, u64x2{nb2, nb3});
}

template <int OB>
__device__ __forceinline__ void ws_step(std::integral_constant<int, 1>, std::integral_constant<bool, false>, v16f (&acc)[3][2],
                                         const v8bf (&fa)[3], const v8bf (&fb)[2], v8bf (&ga)[3], v8bf (&gb)[2], unsigned a,
                                         unsigned b) {
    v4i na0;
    v4i nb0, nb1;
    asm volatile(
        "s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %6, %5, %0\n\t"
        "ds_read_b128 %3, %9 offset:%10\n\t"
        "ds_read_b128 %4, %9 offset:%11\n\t"
        "v_mfma_f32_32x32x16_bf16 %1, %7, %5, %1\n\t"
        "ds_read_b128 %2, %8 offset:0\n\t"
        "s_nop 11\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "+v"(acc[0][0]), "+v"(acc[0][1]),
          "=&v"(na0), "=&v"(nb0), "=&v"(nb1)
        : "v"(fa[0]), "v"(fb[0]), "v"(fb[1]), "v"(a), "v"(b),
          "i"(0), "i"(4096)
        : "memory");
    ga[0] = __builtin_bit_cast(v8bf, na0);
    gb[0] = __builtin_bit_cast(v8bf, nb0);
    gb[1] = __builtin_bit_cast(v8bf, nb1);
}

template <int OB>
__device__ __forceinline__ void ws_step(std::integral_constant<int, 2>, std::integral_constant<bool, true>, v16f (&acc)[3][2],
                                         const v8bf (&fa)[3], const v8bf (&fb)[2], v8bf (&ga)[3], v8bf (&gb)[2], unsigned a,
                                         unsigned b) {
    v4i na0, na1;
    u64 nb0, nb1, nb2, nb3;
    asm volatile(
        "s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %12, %10, %0\n\t"
        "ds_read_b64_tr_b16 %6, %15 offset:%16\n\t"
        "ds_read_b64_tr_b16 %7, %15 offset:%17\n\t"
        "v_mfma_f32_32x32x16_bf16 %1, %13, %10, %1\n\t"
        "ds_read_b64_tr_b16 %8, %15 offset:%18\n\t"
        "ds_read_b64_tr_b16 %9, %15 offset:%19\n\t"
        "v_mfma_f32_32x32x16_bf16 %2, %12, %11, %2\n\t"
        "ds_read_b128 %4, %14 offset:0\n\t"
        "ds_read_b128 %5, %14 offset:8192\n\t"
        "v_mfma_f32_32x32x16_bf16 %3, %13, %11, %3\n\t"
        "s_nop 11\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "+v"(acc[0][0]), "+v"(acc[0][1]), "+v"(acc[1][0]), "+v"(acc[1][1]),
          "=&v"(na0), "=&v"(na1), "=&v"(nb0), "=&v"(nb1), "=&v"(nb2), "=&v"(nb3)
        : "v"(fa[0]), "v"(fa[1]), "v"(fb[0]), "v"(fb[1]), "v"(a), "v"(b),
          "i"(OB), "i"(OB + 2048), "i"(OB + 256), "i"(OB + 2304)
        : "memory");
    ga[0] = __builtin_bit_cast(v8bf, na0);
    ga[1] = __builtin_bit_cast(v8bf, na1);
    gb[0] = __builtin_bit_cast(v8bf, u64x2{nb0, nb1});
    gb[1] = __builtin_bit_cast(v8bf, u64x2{nb2, nb3});
}

template <int OB>
__device__ __forceinline__ void ws_step(std::integral_constant<int, 2>, std::integral_constant<bool, false>, v16f (&acc)[3][2],
                                         const v8bf (&fa)[3], const v8bf (&fb)[2], v8bf (&ga)[3], v8bf (&gb)[2], unsigned a,
                                         unsigned b) {
    v4i na0, na1;
    v4i nb0, nb1;
    asm volatile(
        "s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %10, %8, %0\n\t"
        "ds_read_b128 %6, %13 offset:%14\n\t"
        "v_mfma_f32_32x32x16_bf16 %1, %11, %8, %1\n\t"
        "ds_read_b128 %7, %13 offset:%15\n\t"
        "v_mfma_f32_32x32x16_bf16 %2, %10, %9, %2\n\t"
        "ds_read_b128 %4, %12 offset:0\n\t"
        "v_mfma_f32_32x32x16_bf16 %3, %11, %9, %3\n\t"
        "ds_read_b128 %5, %12 offset:8192\n\t"
        "s_nop 11\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "+v"(acc[0][0]), "+v"(acc[0][1]), "+v"(acc[1][0]), "+v"(acc[1][1]),
          "=&v"(na0), "=&v"(na1), "=&v"(nb0), "=&v"(nb1)
        : "v"(fa[0]), "v"(fa[1]), "v"(fb[0]), "v"(fb[1]), "v"(a), "v"(b),
          "i"(0), "i"(4096)
        : "memory");
    ga[0] = __builtin_bit_cast(v8bf, na0);
    ga[1] = __builtin_bit_cast(v8bf, na1);
    gb[0] = __builtin_bit_cast(v8bf, nb0);
    gb[1] = __builtin_bit_cast(v8bf, nb1);
}

template <int OB>
__device__ __forceinline__ void ws_step(std::integral_constant<int, 3>, std::integral_constant<bool, true>, v16f (&acc)[3][2],
                                         const v8bf (&fa)[3], const v8bf (&fb)[2], v8bf (&ga)[3], v8bf (&gb)[2], unsigned a,
                                         unsigned b) {
    v4i na0, na1, na2;
    u64 nb0, nb1, nb2, nb3;
    asm volatile(
        "s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %16, %13, %0\n\t"
        "ds_read_b64_tr_b16 %9, %19 offset:%20\n\t"
        "ds_read_b64_tr_b16 %10, %19 offset:%21\n\t"
        "v_mfma_f32_32x32x16_bf16 %1, %17, %13, %1\n\t"
        "ds_read_b64_tr_b16 %11, %19 offset:%22\n\t"
        "ds_read_b64_tr_b16 %12, %19 offset:%23\n\t"
        "v_mfma_f32_32x32x16_bf16 %2, %16, %14, %2\n\t"
        "ds_read_b128 %6, %18 offset:0\n\t"
        "ds_read_b128 %7, %18 offset:8192\n\t"
        "v_mfma_f32_32x32x16_bf16 %3, %17, %14, %3\n\t"
        "ds_read_b128 %8, %18 offset:16384\n\t"
        "v_mfma_f32_32x32x16_bf16 %4, %16, %15, %4\n\t"
        "v_mfma_f32_32x32x16_bf16 %5, %17, %15, %5\n\t"
        "s_nop 11\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "+v"(acc[0][0]), "+v"(acc[0][1]), "+v"(acc[1][0]), "+v"(acc[1][1]), "+v"(acc[2][0]), "+v"(acc[2][1]),
          "=&v"(na0), "=&v"(na1), "=&v"(na2), "=&v"(nb0), "=&v"(nb1), "=&v"(nb2), "=&v"(nb3)
        : "v"(fa[0]), "v"(fa[1]), "v"(fa[2]), "v"(fb[0]), "v"(fb[1]), "v"(a), "v"(b),
          "i"(OB), "i"(OB + 2048), "i"(OB + 256), "i"(OB + 2304)
        : "memory");
    ga[0] = __builtin_bit_cast(v8bf, na0);
    ga[1] = __builtin_bit_cast(v8bf, na1);
    ga[2] = __builtin_bit_cast(v8bf, na2);
    gb[0] = __builtin_bit_cast(v8bf, u64x2{nb0, nb1});
    gb[1] = __builtin_bit_cast(v8bf, u64x2{nb2, nb3});
}

template <int OB>
__device__ __forceinline__ void ws_step(std::integral_constant<int, 3>, std::integral_constant<bool, false>, v16f (&acc)[3][2],
                                         const v8bf (&fa)[3], const v8bf (&fb)[2], v8bf (&ga)[3], v8bf (&gb)[2], unsigned a,
                                         unsigned b) {
    v4i na0, na1, na2;
    v4i nb0, nb1;
    asm volatile(
        "s_nop 1\n\t"
        "v_mfma_f32_32x32x16_bf16 %0, %14, %11, %0\n\t"
        "ds_read_b128 %9, %17 offset:%18\n\t"
        "v_mfma_f32_32x32x16_bf16 %1, %15, %11, %1\n\t"
        "ds_read_b128 %10, %17 offset:%19\n\t"
        "v_mfma_f32_32x32x16_bf16 %2, %14, %12, %2\n\t"
        "ds_read_b128 %6, %16 offset:0\n\t"
        "v_mfma_f32_32x32x16_bf16 %3, %15, %12, %3\n\t"
        "ds_read_b128 %7, %16 offset:8192\n\t"
        "v_mfma_f32_32x32x16_bf16 %4, %14, %13, %4\n\t"
        "ds_read_b128 %8, %16 offset:16384\n\t"
        "v_mfma_f32_32x32x16_bf16 %5, %15, %13, %5\n\t"
        "s_nop 11\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "+v"(acc[0][0]), "+v"(acc[0][1]), "+v"(acc[1][0]), "+v"(acc[1][1]), "+v"(acc[2][0]), "+v"(acc[2][1]),
          "=&v"(na0), "=&v"(na1), "=&v"(na2), "=&v"(nb0), "=&v"(nb1)
        : "v"(fa[0]), "v"(fa[1]), "v"(fa[2]), "v"(fb[0]), "v"(fb[1]), "v"(a), "v"(b),
          "i"(0), "i"(4096)
        : "memory");
    ga[0] = __builtin_bit_cast(v8bf, na0);
    ga[1] = __builtin_bit_cast(v8bf, na1);
    ga[2] = __builtin_bit_cast(v8bf, na2);
    gb[0] = __builtin_bit_cast(v8bf, nb0);
    gb[1] = __builtin_bit_cast(v8bf, nb1);
}

// The reads alone, before the first quarter step (all three blocks of A).
template <bool BTR>
__device__ __forceinline__ void ws_read(v8bf (&ga)[3], v8bf (&gb)[2], unsigned a, unsigned b) {
    v4i d[3], e[2];
    u64 o[4];
    if constexpr (BTR) {
        asm volatile(
            "ds_read_b128 %0, %7\n\t"
            "ds_read_b128 %1, %7 offset:8192\n\t"
            "ds_read_b128 %2, %7 offset:16384\n\t"
            "ds_read_b64_tr_b16 %3, %8\n\t"
            "ds_read_b64_tr_b16 %4, %8 offset:2048\n\t"
            "ds_read_b64_tr_b16 %5, %8 offset:256\n\t"
            "ds_read_b64_tr_b16 %6, %8 offset:2304\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3])
            : "v"(a), "v"(b)
            : "memory");
        gb[0] = __builtin_bit_cast(v8bf, u64x2{o[0], o[1]});
        gb[1] = __builtin_bit_cast(v8bf, u64x2{o[2], o[3]});
    } else {
        asm volatile(
            "ds_read_b128 %0, %5\n\t"
            "ds_read_b128 %1, %5 offset:8192\n\t"
            "ds_read_b128 %2, %5 offset:16384\n\t"
            "ds_read_b128 %3, %6\n\t"
            "ds_read_b128 %4, %6 offset:4096\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(e[0]), "=&v"(e[1])
            : "v"(a), "v"(b)
            : "memory");
        gb[0] = __builtin_bit_cast(v8bf, e[0]);
        gb[1] = __builtin_bit_cast(v8bf, e[1]);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) ga[i] = __builtin_bit_cast(v8bf, d[i]);
}

constexpr int kWsRows = 160, kWsCols = 256, kWsStages = 3, kWsThreads = 768;
constexpr int kWsSliceA = kWsRows * 64, kWsSliceB = kWsCols * 64, kWsStage = kWsSliceA + kWsSliceB;   // elements
constexpr int kWsBytes = kWsStages * kWsStage * 2;
static_assert(kWsBytes <= 163840 - 1024, "the ring fits the LDS");

// Stages rows of E in one stage of the ring and stores them, RB 32-row blocks
// (of the item's five) a round, two barriers a round: VAL(i, b, q, v) gives the
// four values of the wave's row block i, columns 8q + 4 (lane / 32) .. +3 of
// its column block b of 32 (at column wcol + 32 b of the tile's WID).
template <typename E, int WID>
struct WsRounds {
    static constexpr int C = 16 / (int)sizeof(E), P = WID + C, kBlock = 32 * P * (int)sizeof(E);
    static constexpr int RB = 2 * kWsStage / kBlock, kRounds = (5 + RB - 1) / RB;
    static_assert(RB >= 1, "32 staged rows fit a stage");
};

// threadIdx.x as a value that the compiler takes for new: addresses made from
// it are made where they are used, at an item's end, instead of being held in
// registers over the items and their main loops (with fp32 results and P kept
// the kernel would spill 13 to 34 registers: the shard's forward with an 8-bit
// P 64.7 us, 57.5 without the spills).
__device__ __forceinline__ int fresh_tid() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

template <typename E, int WID, int NC, typename Val>
__device__ __forceinline__ void ws_store(int tid, E* out, int64_t ld, int row0, int rows, int col0, int cols,
                                          int wcol, uint16_t* sm, Val val) {
    using R = WsRounds<E, WID>;
    constexpr int C = R::C, P = R::P, RB = R::RB;
    const int lane = tid & 63, wm = __builtin_amdgcn_readfirstlane(tid >> 8);
    E* s = reinterpret_cast<E*>(sm);
#pragma unroll
    for (int k = 0; k < R::kRounds; ++k) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int blk = 2 * i + wm - k * RB;
            if (blk < 0 || blk >= RB || 2 * i + wm >= 5) continue;
#pragma unroll
            for (int b = 0; b < NC; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
                    val(i, b, q, v);
                    E* d = s + (32 * blk + (lane & 31)) * P + wcol + 32 * b + 8 * q + 4 * (lane >> 5);
                    if constexpr (sizeof(E) == 2)
                        *reinterpret_cast<uint2*>(d) = make_uint2(pack_rne(v[0], v[1]), pack_rne(v[2], v[3]));
                    else
                        *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
                }
        }
        stage_barrier();
        const int first = 32 * RB * k, n = min(rows - first, 32 * RB);
        for (int e = tid; e < n * (WID / C); e += 512) {
            const int r = e / (WID / C), c = (e % (WID / C)) * C;
            if (col0 + c < cols)
                store_out(out + (int64_t)(row0 + first + r) * ld + col0 + c, *reinterpret_cast<const uint4*>(s + r * P + c));
        }
        stage_barrier();
    }
}

template <int MODE, bool OUT_BF16, int SAVE>
__global__ __launch_bounds__(kWsThreads, 3) void ffn_ws_kernel(const FfnArgs a) {
    static_assert(MODE == kGated || MODE == kBwdX, "forward and dX");
    constexpr int S = kWsStages, kSt = kWsStage;
    constexpr bool kBTr = MODE == kGated;
    using E = typename std::conditional<OUT_BF16, uint16_t, float>::type;
    // barriers of an item's end
    constexpr int kEndBarriers = 2 * WsRounds<E, MODE == kGated ? 128 : 256>::kRounds +
                                 (SAVE == kSaveBf16 ? 4 * WsRounds<uint16_t, 128>::kRounds : SAVE == kSaveMx8 ? 2 : 0);
    __shared__ __attribute__((aligned(1024))) uint16_t ring[S * kSt];
    __shared__ __attribute__((aligned(16))) int s_info[8][4];   // items of the last rounds: g, first row, end, column tile
    const int tid = threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = a.K, NN = a.NN, N = NN / 2;
    const int nsl = (MODE == kGated ? K : NN) >> 6;
    constexpr int kItemCols = MODE == kGated ? kWsCols / 2 : kWsCols;
    if (wave == 1 && blockIdx.x == 0) {   // the call's device status word
        const int st = group_status(a.group_sizes, a.G, a.M);
        if (lane == 0) a.status[0] = st;
    }

    if (wave >= 8) {
        // ---- load waves, 1 KB an instruction: 8 rows of a direct operand or 2 of
        //      transposed B.  Wave p has A's instructions p, p + 4, .. (those that
        //      hold rows) and eight of B's 32.  The ring's slots go to the slices
        //      of one item after the other, with one slot after each item for its
        //      results; loading runs two slots ahead of the barriers, into the
        //      next item where this one ends.
        const int p = wave - 8, lda = MODE == kGated ? K : NN;
        EvenItems items;
        items.init(a.group_sizes, a.G, a.M, a.cap);
        const int64_t bstep = kBTr ? 64 * (int64_t)NN : 64;
        const uint16_t *pa[5], *pb[8];
        int na = 0, round = 0, t = 0, slot = 0, left = 0;   // of the item being loaded: slices left
        uint32_t is_item = 0, has_rows = 0;                 // of round r, at bit r % 32
        bool valid = true;
        auto next_item = [&]() {
            int col;
            const WorkItem wi = items.find(a.group_sizes, a.G, a.M, a.cap, a.ntiles_c,
                                           (int)(blockIdx.x + round * gridDim.x), col);
            if (p == 0) {   // in asm: an LDS write that the compiler sees would drain the ring
                const v4i info = {wi.g, wi.lo, wi.hi, col};
                const unsigned at = (unsigned)(uintptr_t)(GMM_LDS int*)s_info[round & 7];
                asm volatile("ds_write_b128 %0, %1" : : "v"(at), "v"(info) : "memory");
            }
            valid = wi.g >= 0;
            left = wi.g >= 0 && wi.g < a.G ? nsl : 0;
            const uint32_t bit = 1u << (round & 31);
            is_item = valid ? is_item | bit : is_item & ~bit;
            has_rows = left > 0 ? has_rows | bit : has_rows & ~bit;
            ++round;
            t = 0;
            if (left == 0) return;
            const uint16_t* wg = a.b + (int64_t)wi.g * K * NN;
            const int c0 = col * kItemCols, rows = wi.hi - wi.lo;
            na = 0;
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const DmaLane d = dma_direct<64, 8, 8>(p + 4 * i, lane);
                na += 8 * (p + 4 * i) < rows;
                pa[i] = a.a + (int64_t)min(wi.lo + d.row, wi.hi - 1) * lda + d.col;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = p + 4 * i;
                if constexpr (kBTr) {
                    const int r = 2 * j + (lane >> 5), c = (lane & 31) >> 1;   // row r of 64: slice r / 32
                    const int tc = 16 * (c ^ (2 * (r & 3))) + 8 * (lane & 1);
                    const int cc = tc < 128 ? min(c0 + tc, N - 8) : N + min(c0 + tc - 128, N - 8);
                    pb[i] = wg + (int64_t)r * NN + cc;
                } else {
                    const DmaLane d = dma_direct<64, 8, 8>(j, lane);
                    pb[i] = wg + (int64_t)min(c0 + d.row, K - 1) * NN + d.col;
                }
            }
        };
        // fills the next slot; returns the loads issued (none for results, or past the last item)
        auto advance = [&]() {
            if (!valid) return 0;
            uint16_t* sa = ring + slot * kSt + 512 * p;
            slot = slot == S - 1 ? 0 : slot + 1;
            if (left == 0) {   // the item's results go here
                next_item();
                return 0;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint16_t* q = pb[i] + bstep * t;
                __builtin_amdgcn_global_load_lds(q, (GMM_LDS void*)(sa + kWsSliceA + 2048 * i), 16, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                if (i >= na) break;
                const uint16_t* q = pa[i] + 64 * t;
                __builtin_amdgcn_global_load_lds(q, (GMM_LDS void*)(sa + 2048 * i), 16, 0, 0);
            }
            ++t;
            --left;
            return 8 + na;
        };
        // waits until only the n youngest loads are outstanding
        auto wait_younger = [&](int n) {
            switch (n) {
                case 13: wait_vmem<13>(); break;
                case 12: wait_vmem<12>(); break;
                case 11: wait_vmem<11>(); break;
                case 10: wait_vmem<10>(); break;
                case 9: wait_vmem<9>(); break;
                case 8: wait_vmem<8>(); break;
                default: wait_vmem<0>(); break;
            }
        };
        next_item();
        // slots 0 and 1; multiplying starts when slot 0 is in
        advance();
        int n1 = advance();   // loads of the youngest slot
        wait_younger(n1);
        stage_barrier();
        n1 = advance();
        for (int r = 0; is_item >> (r & 31) & 1u; ++r) {   // the item being multiplied (loading is at most three ahead)
            for (int l = has_rows >> (r & 31) & 1u ? nsl : 0; l > 0; --l) {
                wait_younger(n1);   // the next slot is in
                stage_barrier();    // this one has been read
                n1 = advance();
            }
            wait_younger(n1);
#pragma unroll
            for (int e = 0; e < kEndBarriers; ++e) stage_barrier();
            n1 = advance();
        }
        return;
    }

    // ---- multiplying waves
    const int wm = wave >> 2, wn = wave & 3, l32 = lane & 31, h = lane >> 5;
    const unsigned ring_lds = (unsigned)(uintptr_t)(GMM_LDS uint16_t*)ring;
    unsigned ra[4], rb[4];   // of the four quarter steps, slot 0
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int row = 32 * wm + l32;
        ra[s] = ring_lds + (unsigned)(128 * row + 16 * ((2 * s + h) ^ direct_key<64>(row)));
        if constexpr (kBTr) {
            const int r = 8 * h + ((lane & 15) >> 2);
            rb[s] = ring_lds + (unsigned)(2 * kWsSliceA + 512 * r + 32 * ((2 * wn + ((lane >> 4) & 1)) ^ (2 * (r & 3))) +
                                          8 * (lane & 3));
        } else {
            const int br = 64 * wn + l32;
            rb[s] = ring_lds + (unsigned)(2 * kWsSliceA + 128 * br + 16 * ((2 * s + h) ^ direct_key<64>(br)));
        }
    }
    int slot = 0;
    stage_barrier();   // slot 0 is in
    for (int round = 0;; ++round) {
        const int g = __builtin_amdgcn_readfirstlane(s_info[round & 7][0]);
        if (g < 0) break;
        FfnItem it;
        it.g = g;
        it.row0 = it.lo = __builtin_amdgcn_readfirstlane(s_info[round & 7][1]);
        it.hi = __builtin_amdgcn_readfirstlane(s_info[round & 7][2]);
        it.c0 = __builtin_amdgcn_readfirstlane(s_info[round & 7][3]) * kItemCols;
        const int row0 = it.row0, rows = it.hi - it.row0, c0 = it.c0;
        if (g == a.G) {
            zero_tail<MODE, OUT_BF16, SAVE, kWsCols, 512>(a, it);
#pragma unroll
            for (int e = 0; e < kEndBarriers; ++e) stage_barrier();
            slot = slot == S - 1 ? 0 : slot + 1;
            continue;
        }
        v16f acc[3][2];
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
        auto main_loop = [&](auto nbc) __attribute__((always_inline)) {
            constexpr int NB = decltype(nbc)::value;
            constexpr std::integral_constant<bool, kBTr> btr;
            v8bf fa[3], fb[2], ga[3], gb[2];
            if constexpr (NB > 0) ws_read<kBTr>(fa, fb, ra[0] + (unsigned)(slot * kSt * 2), rb[0] + (unsigned)(slot * kSt * 2));
            for (int t = 0; t < nsl; ++t) {
                const int next = slot == S - 1 ? 0 : slot + 1;
                const unsigned so = (unsigned)(slot * kSt * 2), so1 = (unsigned)(next * kSt * 2);
                if constexpr (NB > 0) {   // transposed B: 16 rows on, the second slice, its rows 16 on
                    ws_step<8192>(nbc, btr, acc, fa, fb, ga, gb, ra[1] + so, rb[1] + so);
                    ws_step<16384>(nbc, btr, acc, ga, gb, fa, fb, ra[2] + so, rb[2] + so);
                    ws_step<24576>(nbc, btr, acc, fa, fb, ga, gb, ra[3] + so, rb[3] + so);
                }
                stage_barrier();
                // past the last slice this reads a slot without using it
                if constexpr (NB > 0) ws_step<0>(nbc, btr, acc, ga, gb, fa, fb, ra[0] + so1, rb[0] + so1);
                slot = next;
            }
        };
        switch (((rows + 31) / 32 + 1 - wm) >> 1) {   // this wave's 32-row blocks that hold rows
            case 0: main_loop(std::integral_constant<int, 0>{}); break;
            case 1: main_loop(std::integral_constant<int, 1>{}); break;
            case 2: main_loop(std::integral_constant<int, 2>{}); break;
            default: main_loop(std::integral_constant<int, 3>{}); break;
        }

        uint16_t* sm = ring + slot * kSt;   // the item's slot for results
        slot = slot == S - 1 ? 0 : slot + 1;
        if constexpr (MODE == kGated) {
            if constexpr (SAVE == kSaveBf16) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    ws_store<uint16_t, 128, 1>(fresh_tid(), a.gu + p * N, NN, row0, rows, c0, N, 32 * wn, sm,
                                               [&](int i, int, int q, float (&v)[4]) {
#pragma unroll
                                                   for (int k = 0; k < 4; ++k) v[k] = acc[i][p][4 * q + k];
                                               });
            }
            if constexpr (SAVE == kSaveMx8) {
                // a wave's 32 gate (or up) columns of a row are one block, in lanes l and l + 32
                constexpr int P = 256 + 16;
                const int tid = fresh_tid(), l32 = tid & 31, h = (tid >> 5) & 1;
                uint8_t* cm = reinterpret_cast<uint8_t*>(sm);
                uint8_t* ss = cm + kWsRows * P;
                static_assert(kWsRows * (P + 8) <= 2 * kWsStage, "checkpoint staging fits a stage");
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    if (2 * i + wm >= 5) continue;
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        uint32_t m = 0;
#pragma unroll
                        for (int r = 0; r < 16; ++r) m = max(m, abs_bits(acc[i][p][r]));
                        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                        const u32x2 sw = __builtin_amdgcn_permlane32_swap(m, m, false, false);
                        const uint32_t c = mx8_scale_code(max(sw[0], sw[1]));
                        const float inv = mx8_inverse(c);
                        const int r = 64 * i + 32 * wm + l32;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<uint32_t*>(cm + r * P + 128 * p + 32 * wn + 8 * q + 4 * h) =
                                e4m3x4(acc[i][p][4 * q] * inv, acc[i][p][4 * q + 1] * inv, acc[i][p][4 * q + 2] * inv,
                                       acc[i][p][4 * q + 3] * inv);
                        if (h == 0) ss[r * 8 + 4 * p + wn] = (uint8_t)c;
                    }
                }
                stage_barrier();
                for (int e = tid; e < rows * 16; e += 512) {
                    const int r = e >> 4, c = (e & 15) * 16, col = c0 + (c & 127);
                    if (col < N)
                        store_out(a.gu_q + (int64_t)(row0 + r) * NN + (c < 128 ? 0 : N) + col,
                                  *reinterpret_cast<const uint4*>(cm + r * P + c));
                }
                for (int e = tid; e < rows * 4; e += 512) {   // pairs of scale bytes: 64 columns
                    const int r = e >> 2, p = (e >> 1) & 1, b = (e & 1) * 2;
                    if (c0 + 32 * b < N)
                        *reinterpret_cast<uint16_t*>(a.gu_s + (int64_t)(row0 + r) * (NN / 32) + (p * N + c0) / 32 + b) =
                            *reinterpret_cast<const uint16_t*>(ss + r * 8 + 4 * p + b);
                }
                stage_barrier();
            }
            // h over the gate sums, so that no second set of values is live
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][0][r] = silu_mul(acc[i][0][r], acc[i][1][r]);
            ws_store<E, 128, 1>(SAVE == kSaveNone ? tid : fresh_tid(), reinterpret_cast<E*>(a.out), N, row0, rows, c0, N, 32 * wn, sm,
                                [&](int i, int, int q, float (&v)[4]) {
#pragma unroll
                                    for (int k = 0; k < 4; ++k) v[k] = acc[i][0][4 * q + k];
                                });
        } else {
            ws_store<E, 256, 2>(tid, reinterpret_cast<E*>(a.out), K, row0, rows, c0, K, 64 * wn, sm,
                                [&](int i, int b, int q, float (&v)[4]) {
#pragma unroll
                                    for (int k = 0; k < 4; ++k) v[k] = acc[i][b][4 * q + k];
                                });
        }
    }
}

template <int MODE, bool OUT_BF16, int SAVE>
hipError_t launch_ws(FfnArgs a, int cap, hipStream_t stream) {
    const int cols = MODE == kGated ? a.NN / 2 : a.K, tc = MODE == kGated ? kWsCols / 2 : kWsCols;
    a.cap = cap;
    a.ntiles_r = 0;
    a.ntiles_c = (cols + tc - 1) / tc;
    a.nblocks = (int)(max_work_items(a.M, a.G < a.M ? a.G : a.M, cap) * a.ntiles_c);
    // one workgroup per CU, a multiple of the XCDs (the items' XCD placement counts on it)
    const int grid = (a.nblocks < device_cus() ? a.nblocks + kNumXcd - 1 : device_cus()) / kNumXcd * kNumXcd;
    hipLaunchKernelGGL((ffn_ws_kernel<MODE, OUT_BF16, SAVE>), dim3((unsigned)grid), dim3(kWsThreads), 0, stream, a);
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
// What bounds it: a pass over one token's 8 experts (33 MB) takes 18 us with cold
// weights, of which 3.4 us are launch and prologue; a bare read of as many cold
// bytes takes 10.4 us.  With 16 + 16 columns a row of weights is two pieces of 32
// bytes, so the L2s get four requests for each cache line (1.06 million in all).
// Deeper rings and more waves change nothing; weights that lie contiguously for
// each workgroup would (14 us), but the layout is the caller's.
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
    __shared__ int s_info[4];
    static_assert(NW * TR * kRow * 2 <= kRing, "the partial sums fit the rings");
    static_assert(kRing * 2 <= 163840 - 1024, "the rings fit the LDS");

    const int tid = threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    FfnItem it;
    if (!ffn_item<kGated, TR, 2 * CT>(a, blockIdx.x, s_info, it)) return;
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

// 256 columns a tile or 128.  The wide tile reads its rows half as often and
// feeds each MFMA from fewer LDS reads, but two workgroups fill a CU instead
// of three smaller ones: it pays once the narrow tiles would need more than
// one round of the chip (three a CU) and the columns do not leave more than a
// sixth of it unused.  Measured (us, 128 / 256 columns; shard: 8192 rows, 32
// experts, K = 2048, 2N = 1024; production: 65536 rows, 256 experts): forward
// shard 73.7 / 75.9, production 465 / 385; dX 73.9 / 72.4, 502 / 461; weight
// gradient 63.0 / 60.3, 607 / 522 (dX and the gradient with the 11 and 75 us
// of the activation's gradient in both figures).
bool wide_tiles(int64_t row_tiles, int64_t cols) {
    const int64_t wide = (cols + 255) / 256;
    return row_tiles * ((cols + 127) / 128) > 3 * device_cus() && wide * 256 * 5 <= cols * 6;
}

// Rows an item of the 160 x 256 tiles may have, or 0 where the smaller tiles
// are taken.  One workgroup fills a CU, so the grid should be one round of the
// chip at least three quarters full.  Two such rounds pay for dX where the
// groups are small enough (two items) for the weights to be most of what is
// read, and for the forward where besides the rows of x lie a multiple of 4 KB
// apart: the smaller tiles read those rows 64 bytes at a time and run into one
// set of memory channels (8192 rows, 32 experts, 2N = 1024: K = 1536 47 us, K =
// 2048 80).  Over more rounds dX still gains (`many`: the largest cap), the
// forward does not.  Of the caps that fit, the cheapest: rounds x (the weights'
// columns + the products of the item's rows), measured as 2 : rows / 160.  Not
// on short reductions, nor (forward) on groups of few rows.  The rows of an
// item are estimated from the mean and spread of evenly routed groups.
// Measured (us, smaller tiles / these; dX with the activation's gradient; rows,
// experts, K, 2N):
//   one round: 8192, 32, 2048, 1024 forward 80.3 / 57.0; 16384, 64, 1024, 512
//   36.9 / 30.5; 8192, 32, 768, 512 20.2 / 19.2; 8192, 16, 1024, 640 23.3 /
//   24.3; dX 4096, 32, 2048, 1024 54.2 / 38.3; 8192, 16, 1024, 640 29.1 / 24.5;
//   8192, 32, 768, 512 19.6 / 19.7
//   two: 16384, 64, 2048, 1024 forward 122 / 104, dX 123 / 107; forward with
//   other pitches 12000, 60, 1024, 1024 51.0 / 55.6; 10000, 64, 1536, 1024 66.1
//   / 74.6; with three items a group 6000, 20, 2048, 1280 53.6 / 61.4; less
//   than three quarters full: dX 5000, 12, 2048, 1024 39.5 / 46.0
//   more: 65536, 256, 2048, 1024 dX 456 / 403, forward 385 / 377 (Zipf 390 /
//   394); 24000, 64, 2048, 1024 dX 161 / 151; 16384, 1, 4096, 1024 forward 119 /
//   145
//   short or few: forward 3000, 8, 512, 2048 17.1 / 18.1; 2048, 32, 2048, 1024
//   34.8 / 41.7
//   odd sizes: 1777, 13, 1088, 1408 forward 22.7 / 21.1 (a third of the experts
//   empty: 21.1 / 21.1), dX 25.8 / 23.8; 2000, 11, 1536, 1280 forward 26.5 / 24.6
// Under skewed (Zipf) routing, which the host does not see, the forward of 8192
// rows loses, 79.0 / 88.8; its dX does not, 75.0 / 72.8.
int ws_cap(int M, int G, int red, int tiles, int min_red, double min_mean, bool many) {
    const int64_t busy = G < M ? G : M, cus = device_cus();
    const double mean = (double)M / (double)busy, high = mean + 2.0 * sqrt(mean);
    if (red < min_red || mean < min_mean) return 0;
    const auto full = [&](int64_t wgs, int64_t r) { return 4 * wgs >= 3 * r * cus; };
    int best = 0;
    double cost = 0.0;
    for (int cap = 64; cap <= kWsRows; cap += 32) {
        const int64_t n = (int64_t)ceil(high / cap), wgs = busy * n * tiles, r = (wgs + cus - 1) / cus;
        if (!full(wgs, r) || r > ((many ? mean <= 2 * kWsRows : n <= 2 && red % 2048 == 0) ? 2 : 1)) continue;
        const double c = (double)r * (2.0 + mean / (double)n / 160.0);
        if (best == 0 || c < cost) {
            best = cap;
            cost = c;
        }
    }
    if (best == 0 && many) {
        const int64_t wgs = busy * (int64_t)ceil(high / kWsRows) * tiles, r = (wgs + cus - 1) / cus;
        if (r > 1 && full(wgs, r)) return kWsRows;
    }
    return best;
}

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
hipError_t launch_few_mb(const FfnArgs& a, const FfnChoice& c, hipStream_t stream) {
    if constexpr (SAVE != kSaveMx8)
        if (c.cols == 32) return launch_few<OUT_BF16, SAVE, MB, 16, 8, MB == 4 ? 3 : 4>(a, stream);
    return launch_few<OUT_BF16, SAVE, MB, 32, 4, 3>(a, stream);
}

template <int SAVE, bool OUT_BF16>
hipError_t launch_gated(const FfnArgs& a, hipStream_t stream) {
    const FfnChoice c = gated_fwd_choice(a.M, a.K, a.NN, a.G, SAVE == kSaveMx8);
    if (c.kernel == kFfnFewRows) {
        if (c.rows == 16) return launch_few_mb<OUT_BF16, SAVE, 1>(a, c, stream);
        if (c.rows == 32) return launch_few_mb<OUT_BF16, SAVE, 2>(a, c, stream);
        return launch_few_mb<OUT_BF16, SAVE, 4>(a, c, stream);
    }
    if (c.kernel == kFfnLoadWaves) return launch_ws<kGated, OUT_BF16, SAVE>(a, c.rows, stream);
    return c.cols == 256 ? launch<kGated, OUT_BF16, SAVE, 8>(a, stream) : launch<kGated, OUT_BF16, SAVE, 4>(a, stream);
}

template <int MODE>
hipError_t launch_bwd(const FfnArgs& a, const FfnChoice& c, bool out_bf16, hipStream_t stream) {
    if constexpr (MODE == kBwdX)
        if (c.kernel == kFfnLoadWaves)
            return out_bf16 ? launch_ws<MODE, true, kSaveNone>(a, c.rows, stream)
                            : launch_ws<MODE, false, kSaveNone>(a, c.rows, stream);
    if (c.cols == 256)
        return out_bf16 ? launch<MODE, true, kSaveNone, 8>(a, stream) : launch<MODE, false, kSaveNone, 8>(a, stream);
    return out_bf16 ? launch<MODE, true, kSaveNone, 4>(a, stream) : launch<MODE, false, kSaveNone, 4>(a, stream);
}

}  // namespace

FfnChoice gated_fwd_choice(int M, int K, int NN, int G, bool keep_mx8) {
    const int busy = G < M ? G : M, rows = (M + busy - 1) / busy;
    if (rows <= kFewMaxRows && (int64_t)busy * (NN / 128) < device_cus()) {
        // a checkpoint's block is 32 columns of one row: the wider tile's
        const bool narrow = !keep_mx8 && (int64_t)busy * (NN / 32) <= device_cus();
        return {kFfnFewRows, narrow ? 8 : 4, rows <= 16 ? 16 : (rows <= 32 ? 32 : 64), narrow ? 32 : 64};
    }
    const int cap = ws_cap(M, G, K, (NN + 255) / 256, 768, 96.0, false);
    if (cap > 0) return {kFfnLoadWaves, 12, cap, 256};
    return {kFfnTiles, 4, 128, wide_tiles(max_work_items(M, busy, 128), NN) ? 256 : 128};
}

FfnChoice ffn_dx_choice(int M, int K, int NN, int G) {
    const int cap = ws_cap(M, G, NN, (K + 255) / 256, 512, 48.0, true);
    if (cap > 0) return {kFfnLoadWaves, 12, cap, 256};
    return {kFfnTiles, 4, 128, wide_tiles(max_work_items(M, G < M ? G : M, 128), K) ? 256 : 128};
}

FfnChoice ffn_dw_choice(int K, int NN, int G) {
    return {kFfnTiles, 4, 128, wide_tiles((int64_t)G * ((K + 127) / 128), NN) ? 256 : 128};
}

FfnChoice ffn_bwd_choice(int M, int K, int NN, int G) {
    FfnChoice c = ffn_dx_choice(M, K, NN, G);
    if (c.kernel == kFfnTiles && c.cols == 128 && ffn_dw_choice(K, NN, G).cols == 128) c.kernel = kFfnBoth;
    return c;
}

int64_t gated_fwd_blocks(int64_t M, int64_t N, int64_t G) {
    // of the 128-row tiles; the few-row form only takes grids near the chip's size
    return max_work_items(M, G < M ? G : M, 128) * ((N + 63) / 64);
}

int64_t ffn_dx_blocks(int64_t M, int64_t K, int64_t G) {
    return max_work_items(M, G < M ? G : M, 128) * ((K + 127) / 128);
}

int64_t ffn_dw_blocks(int64_t K, int64_t NN, int64_t G) { return G * ((K + 127) / 128) * ((NN + 127) / 128); }

hipError_t launch_gated_fwd(const FfnArgs& a, bool out_bf16, hipStream_t stream) {
    if (a.gu_q != nullptr) return out_bf16 ? launch_gated<kSaveMx8, true>(a, stream) : launch_gated<kSaveMx8, false>(a, stream);
    if (a.gu != nullptr) return out_bf16 ? launch_gated<kSaveBf16, true>(a, stream) : launch_gated<kSaveBf16, false>(a, stream);
    return out_bf16 ? launch_gated<kSaveNone, true>(a, stream) : launch_gated<kSaveNone, false>(a, stream);
}

hipError_t launch_ffn_dx(const FfnArgs& a, bool out_bf16, hipStream_t stream) {
    return launch_bwd<kBwdX>(a, ffn_dx_choice(a.M, a.K, a.NN, a.G), out_bf16, stream);
}

hipError_t launch_ffn_dw(const FfnArgs& a, bool out_bf16, hipStream_t stream) {
    const FfnChoice c = ffn_dw_choice(a.K, a.NN, a.G);
    return a.aq != nullptr ? launch_bwd<kBwdWQ>(a, c, out_bf16, stream) : launch_bwd<kBwdW>(a, c, out_bf16, stream);
}

hipError_t launch_ffn_bwd(const FfnArgs& x, bool x_bf16, const FfnArgs& w, bool w_bf16, hipStream_t stream) {
    if (ffn_bwd_choice(x.M, x.K, x.NN, x.G).kernel != kFfnBoth) {
        const hipError_t e = launch_ffn_dx(x, x_bf16, stream);
        return e != hipSuccess ? e : launch_ffn_dw(w, w_bf16, stream);
    }
    if (x_bf16) return w_bf16 ? launch_both<true, true>(x, w, stream) : launch_both<true, false>(x, w, stream);
    return w_bf16 ? launch_both<false, true>(x, w, stream) : launch_both<false, false>(x, w, stream);
}

}  // namespace gmm
