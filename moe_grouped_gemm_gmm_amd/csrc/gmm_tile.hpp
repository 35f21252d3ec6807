// Device helpers shared by the load-to-LDS grouped kernels (gmm_bf16.hip and
// the gated-block kernels): tgmm work placement, the XOR-swizzled LDS slice
// layouts, their fragment reads and the global addresses the load-to-LDS
// instructions take.
#pragma once

#include "gmm_device.hpp"

namespace gmm {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// tgmm work placement.  A tgmm workgroup owns one 128 x 128 tile of one
// group's dW and walks all of that group's rows, so its cost is the group's
// size.  Blocks run on XCD b % 8 in the order of b.  By default logical ids
// are remapped so that each XCD takes a contiguous run of groups in index
// order, all T tiles of a group on one XCD (its rows of X and dY then fill
// one L2).  Under a skewed routing (the largest group holding more than four
// times the mean rows, e.g. Zipf-popular experts) that leaves some XCD with
// far more rows than the others (1.4x the mean for the production routing),
// so there
//  - every group's T tiles are spread evenly over the 8 XCDs (XCD x takes
//    tiles x*T/8 .. (x+1)*T/8 - 1: with N/128 column tiles per K tile a
//    contiguous band of K tiles, so each column of X is still read by one
//    XCD), and each XCD carries exactly an eighth of the work;
//  - within an XCD, groups go in decreasing size class (>= 2048, >= 512,
//    >= 128 rows, the rest; index order within a class), an approximation of
//    longest-processing-time-first: each freed slot takes the next block, so
//    long tiles started last would set the finishing time.
// Every workgroup derives the same choice and the same order from
// group_sizes alone (a size class depends only on the group's own size), so
// both mappings are bijections from blocks to (group, tile).
__device__ __forceinline__ int tgmm_size_class(int s) {
    return s >= 2048 ? 0 : (s >= 512 ? 1 : (s >= 128 ? 2 : 3));
}

struct TgmmTile {
    int g, t, row_lo, row_hi;
};

// The r-th group of size class cls (cls < 0: of all groups) in index order
// among one chunk of 64 groups, whose clamped row ranges the caller
// supplies (lane i: group base + i); true when found (r is decremented past
// each chunk).
__device__ __forceinline__ bool tgmm_pick(int base, int G, int lo, int hi, int cls, int& r,
                                          TgmmTile& out) {
    const int lane = lane_id();
    const bool in = base + lane < G && (cls < 0 || tgmm_size_class(hi - lo) == cls);
    const unsigned long long mask = __ballot(in);
    const int n = __popcll(mask);
    if (r < n) {
        const unsigned long long sel = __ballot(in && __popcll(mask & ((1ull << lane) - 1ull)) == r);
        const int src = __ffsll((long long)sel) - 1;
        out.g = base + src;
        out.row_lo = lane_value(lo, src);
        out.row_hi = lane_value(hi, src);
        return true;
    }
    r -= n;
    return false;
}

// One wave; every lane gets the result.  T = tiles per group, L = the
// block's id after the default XCD remap (block: before it).  A group's rows are its clamped
// range (group_chunk: a negative size reads as 0, rows stop at M).  Up to
// 256 groups the ranges stay in registers (one load and one scan per 64
// groups); beyond, the second pass reads and scans them again.
__device__ inline TgmmTile tgmm_tile(const int32_t* __restrict__ group_sizes, int G, int M, int T,
                                     int L, int block, int placement) {
    const bool inreg = G <= 256;
    int glo[4], ghi[4];
    // pass 1: clamped ranges, class counts and the total
    int cnt0 = 0, cnt1 = 0, cnt2 = 0, carry = 0;
    auto count = [&](int base, int sz) {
        const int c = base + lane_id() < G ? tgmm_size_class(sz) : 4;
        cnt0 += __popcll(__ballot(c == 0));
        cnt1 += __popcll(__ballot(c == 1));
        cnt2 += __popcll(__ballot(c == 2));
    };
    if (inreg) {
        // all four loads issued before the first scan: a chain of dependent
        // load round trips is what this prologue would otherwise wait on
        int raw[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) raw[c] = group_size_at(group_sizes, G, 64 * c + lane_id());
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            glo[c] = ghi[c] = 0;
            if (64 * c < G) {
                const GroupChunk ch = group_chunk_of(raw[c], M, carry);
                glo[c] = ch.lo;
                ghi[c] = ch.hi;
                carry = ch.next_carry;
                count(64 * c, ch.hi - ch.lo);
            }
        }
    } else {
        for (int base = 0; base < G; base += 64) {
            const GroupChunk ch = group_chunk(group_sizes, G, M, base, carry);
            carry = ch.next_carry;
            count(base, ch.hi - ch.lo);
        }
    }
    const int tot = min(carry, M);
    // skewed: some group holds more than four times the mean (placement 0);
    // placement 1 / 2 force the contiguous / spread mapping (the host checks
    // that spreading has a multiple of 8 tiles per group)
    const bool skewed = placement == 2 || (placement == 0 && T % kNumXcd == 0 && [&] {
        bool big = false;
        if (inreg) {
#pragma unroll
            for (int c = 0; c < 4; ++c) big = big || (int64_t)(ghi[c] - glo[c]) * G > 4 * (int64_t)tot;
        } else {
            int cr = 0;
            for (int base = 0; base < G; base += 64) {
                const GroupChunk ch = group_chunk(group_sizes, G, M, base, cr);
                cr = ch.next_carry;
                big = big || (int64_t)(ch.hi - ch.lo) * G > 4 * (int64_t)tot;
            }
        }
        return __ballot(big) != 0ull;
    }());
    TgmmTile out;
    out.g = -1;   // stays so only for blocks >= G * T (none are launched)
    out.row_lo = out.row_hi = 0;
    int r, cls = -1;   // cls < 0: index order
    if (skewed) {
        const int tx = T / kNumXcd, i = block / kNumXcd;
        r = i / tx;
        out.t = (block % kNumXcd) * tx + i % tx;
        cls = 0;
        if (r >= cnt0) { r -= cnt0; cls = 1;
            if (r >= cnt1) { r -= cnt1; cls = 2;
                if (r >= cnt2) { r -= cnt2; cls = 3; } } }
    } else {
        r = L / T;
        out.t = L % T;
        if (inreg) {   // group r itself: its rows from the ranges in registers
            const int c = r >> 6, l = r & 63;
            const int lo = c == 0 ? glo[0] : (c == 1 ? glo[1] : (c == 2 ? glo[2] : glo[3]));
            const int hi = c == 0 ? ghi[0] : (c == 1 ? ghi[1] : (c == 2 ? ghi[2] : ghi[3]));
            out.g = r;
            out.row_lo = lane_value(lo, l);
            out.row_hi = lane_value(hi, l);
            return out;
        }
    }
    // pass 2: the group at that position and its rows
    if (inreg) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (64 * c < G && tgmm_pick(64 * c, G, glo[c], ghi[c], cls, r, out)) break;
    } else {
        int cr = 0;
        for (int base = 0; base < G; base += 64) {
            const GroupChunk ch = group_chunk(group_sizes, G, M, base, cr);
            cr = ch.next_carry;
            if (tgmm_pick(base, G, ch.lo, ch.hi, cls, r, out)) break;
        }
    }
    return out;
}

// Sizes of a ring of S stages of (64 WM) x (64 WN) tiles, RES rings per CU.
template <int S, int RES, int WM, int WN>
struct DmaShape {
    static constexpr int kTR = 64 * WM;                  // tile rows (the A operand's dimension)
    static constexpr int kTC = 64 * WN;                  // tile columns (the B operand's)
    static constexpr int kWaves = WM * WN;
    static constexpr int kStage64 = (kTR + kTC) * 64 * 2;   // bytes of a 64-deep stage
    static constexpr int kRD = RES * S * kStage64 <= 163840 - 1024 ? 64 : 32;   // slice depth
    static constexpr int kSliceA = kTR * kRD;            // bf16 elements of A's slice
    static constexpr int kSliceB = kTC * kRD;            // of B's
    static constexpr int kStage = kSliceA + kSliceB;
    static constexpr int kInstrA = kSliceA * 2 / 1024 / kWaves;   // load-to-LDS instructions per wave
    static constexpr int kInstrB = kSliceB * 2 / 1024 / kWaves;
    static constexpr int kChunks = kRD / 8;              // 16-byte chunks per direct row
    static constexpr int kRows = 64 / kChunks;           // direct rows per instruction
};

template <bool kSpread>
__device__ __forceinline__ int trans_key(int r) {
    return kSpread ? (r & 7) : ((r & 3) | ((r >> 1) & 4));
}

template <int RD>
__device__ __forceinline__ int direct_key(int R) {
    return RD == 64 ? (R & 7) : ((R >> 1) & 3);
}

// Direct fragment: 8 reduction values at chunk `chunk` of row `row`.
template <int RD>
__device__ __forceinline__ v8bf swz_read_direct(const uint16_t* tile, int row, int chunk) {
    return *reinterpret_cast<const v8bf*>(tile + row * RD + 8 * (chunk ^ direct_key<RD>(row)));
}

// The transposed reads of one operand's slice: fragments i = 0..3 of NB
// 32-deep blocks, two ds_read_b64_tr_b16 each, as read_tr lays them out.
// addr[i] is the LDS byte address of fragment i's first read in block 0;
// the second read sits HALF bytes on (rows +4 natural, +16 spread: the same
// key, so the same swizzled chunk), block 1 BLK bytes on (rows +32).  One
// asm block that waits for its own reads before it ends (the
// ds_read_b64_tr_b16 builtin makes the compiler drain every load-to-LDS load
// in flight before it, which would flatten the ring).
typedef unsigned long long u64;
typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
template <int NB, int HALF, int BLK>
__device__ __forceinline__ void tr_slice(v8bf (&f)[2][4], const unsigned (&addr)[4]) {
    if constexpr (NB == 2) {
        u64 o[16];
        asm volatile(
            "ds_read_b64_tr_b16 %0, %16\n\t"
            "ds_read_b64_tr_b16 %1, %16 offset:%20\n\t"
            "ds_read_b64_tr_b16 %2, %16 offset:%21\n\t"
            "ds_read_b64_tr_b16 %3, %16 offset:%22\n\t"
            "ds_read_b64_tr_b16 %4, %17\n\t"
            "ds_read_b64_tr_b16 %5, %17 offset:%20\n\t"
            "ds_read_b64_tr_b16 %6, %17 offset:%21\n\t"
            "ds_read_b64_tr_b16 %7, %17 offset:%22\n\t"
            "ds_read_b64_tr_b16 %8, %18\n\t"
            "ds_read_b64_tr_b16 %9, %18 offset:%20\n\t"
            "ds_read_b64_tr_b16 %10, %18 offset:%21\n\t"
            "ds_read_b64_tr_b16 %11, %18 offset:%22\n\t"
            "ds_read_b64_tr_b16 %12, %19\n\t"
            "ds_read_b64_tr_b16 %13, %19 offset:%20\n\t"
            "ds_read_b64_tr_b16 %14, %19 offset:%21\n\t"
            "ds_read_b64_tr_b16 %15, %19 offset:%22\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]), "=&v"(o[4]), "=&v"(o[5]), "=&v"(o[6]),
              "=&v"(o[7]), "=&v"(o[8]), "=&v"(o[9]), "=&v"(o[10]), "=&v"(o[11]), "=&v"(o[12]), "=&v"(o[13]),
              "=&v"(o[14]), "=&v"(o[15])
            : "v"(addr[0]), "v"(addr[1]), "v"(addr[2]), "v"(addr[3]), "i"(HALF), "i"(BLK), "i"(BLK + HALF)
            : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[0][i] = __builtin_bit_cast(v8bf, u64x2{o[4 * i], o[4 * i + 1]});
            f[1][i] = __builtin_bit_cast(v8bf, u64x2{o[4 * i + 2], o[4 * i + 3]});
        }
    } else {
        u64 o[8];
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8\n\t"
            "ds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
            "ds_read_b64_tr_b16 %2, %9\n\t"
            "ds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
            "ds_read_b64_tr_b16 %4, %10\n\t"
            "ds_read_b64_tr_b16 %5, %10 offset:%12\n\t"
            "ds_read_b64_tr_b16 %6, %11\n\t"
            "ds_read_b64_tr_b16 %7, %11 offset:%12\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]), "=&v"(o[4]), "=&v"(o[5]), "=&v"(o[6]),
              "=&v"(o[7])
            : "v"(addr[0]), "v"(addr[1]), "v"(addr[2]), "v"(addr[3]), "i"(HALF)
            : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) f[0][i] = __builtin_bit_cast(v8bf, u64x2{o[2 * i], o[2 * i + 1]});
    }
}

// Both operands' transposed reads of a 32-deep slice (tgmm) in one asm
// block, so the slice waits on the LDS once: fragments i = 0..3 of A at
// aa[i] (second read HALF_A bytes on) and of B at ba[i] (HALF_B on).
template <int HALF_A, int HALF_B>
__device__ __forceinline__ void tr_slice_pair(v8bf (&fa)[4], v8bf (&fb)[4], const unsigned (&aa)[4],
                                              const unsigned (&ba)[4]) {
    u64 o[16];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %16\n\t"
        "ds_read_b64_tr_b16 %1, %16 offset:%24\n\t"
        "ds_read_b64_tr_b16 %2, %17\n\t"
        "ds_read_b64_tr_b16 %3, %17 offset:%24\n\t"
        "ds_read_b64_tr_b16 %4, %18\n\t"
        "ds_read_b64_tr_b16 %5, %18 offset:%24\n\t"
        "ds_read_b64_tr_b16 %6, %19\n\t"
        "ds_read_b64_tr_b16 %7, %19 offset:%24\n\t"
        "ds_read_b64_tr_b16 %8, %20\n\t"
        "ds_read_b64_tr_b16 %9, %20 offset:%25\n\t"
        "ds_read_b64_tr_b16 %10, %21\n\t"
        "ds_read_b64_tr_b16 %11, %21 offset:%25\n\t"
        "ds_read_b64_tr_b16 %12, %22\n\t"
        "ds_read_b64_tr_b16 %13, %22 offset:%25\n\t"
        "ds_read_b64_tr_b16 %14, %23\n\t"
        "ds_read_b64_tr_b16 %15, %23 offset:%25\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]), "=&v"(o[4]), "=&v"(o[5]), "=&v"(o[6]),
          "=&v"(o[7]), "=&v"(o[8]), "=&v"(o[9]), "=&v"(o[10]), "=&v"(o[11]), "=&v"(o[12]), "=&v"(o[13]),
          "=&v"(o[14]), "=&v"(o[15])
        : "v"(aa[0]), "v"(aa[1]), "v"(aa[2]), "v"(aa[3]), "v"(ba[0]), "v"(ba[1]), "v"(ba[2]), "v"(ba[3]),
          "i"(HALF_A), "i"(HALF_B)
        : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        fa[i] = __builtin_bit_cast(v8bf, u64x2{o[2 * i], o[2 * i + 1]});
        fb[i] = __builtin_bit_cast(v8bf, u64x2{o[8 + 2 * i], o[8 + 2 * i + 1]});
    }
}

// The forward's reads of a 32-deep slice in one asm block (one wait): A's
// four direct fragments (16 bytes at da[i]) and B's transposed ones (at
// ba[i], second read HALF_B bytes on).
template <int HALF_B>
__device__ __forceinline__ void direct_tr_slice(v8bf (&fa)[4], v8bf (&fb)[4], const unsigned (&da)[4],
                                                const unsigned (&ba)[4]) {
    v4i d0, d1, d2, d3;
    u64 o[8];
    asm volatile(
        "ds_read_b128 %0, %12\n\t"
        "ds_read_b128 %1, %13\n\t"
        "ds_read_b128 %2, %14\n\t"
        "ds_read_b128 %3, %15\n\t"
        "ds_read_b64_tr_b16 %4, %16\n\t"
        "ds_read_b64_tr_b16 %5, %16 offset:%20\n\t"
        "ds_read_b64_tr_b16 %6, %17\n\t"
        "ds_read_b64_tr_b16 %7, %17 offset:%20\n\t"
        "ds_read_b64_tr_b16 %8, %18\n\t"
        "ds_read_b64_tr_b16 %9, %18 offset:%20\n\t"
        "ds_read_b64_tr_b16 %10, %19\n\t"
        "ds_read_b64_tr_b16 %11, %19 offset:%20\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(d0), "=&v"(d1), "=&v"(d2), "=&v"(d3), "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]),
          "=&v"(o[4]), "=&v"(o[5]), "=&v"(o[6]), "=&v"(o[7])
        : "v"(da[0]), "v"(da[1]), "v"(da[2]), "v"(da[3]), "v"(ba[0]), "v"(ba[1]), "v"(ba[2]), "v"(ba[3]),
          "i"(HALF_B)
        : "memory");
    fa[0] = __builtin_bit_cast(v8bf, d0);
    fa[1] = __builtin_bit_cast(v8bf, d1);
    fa[2] = __builtin_bit_cast(v8bf, d2);
    fa[3] = __builtin_bit_cast(v8bf, d3);
#pragma unroll
    for (int i = 0; i < 4; ++i) fb[i] = __builtin_bit_cast(v8bf, u64x2{o[2 * i], o[2 * i + 1]});
}

// LDS byte address (relative to the slice) of the first read of the
// transposed fragment at columns c0 .. c0+15 in block 0, for this lane, in
// a slice of PITCH-element rows.
template <bool kSpread, int PITCH>
__device__ __forceinline__ unsigned tr_addr(int lg, int c0, int lr) {
    const int r = (kSpread ? 4 : 8) * lg + (lr >> 2);
    return (unsigned)(2 * (r * PITCH + 16 * ((c0 >> 4) ^ trans_key<kSpread>(r)) + (lr & 3) * 4));
}

// A transposed fragment of block s with the reduction rows at or past
// `valid` zeroed (element e holds row r + e for e < 4 and r1 + e - 4 after,
// as read).
template <bool kSpread>
__device__ __forceinline__ v8bf zero_rows_past(v8bf v, int s, int lg, int valid) {
    const int r = s * 32 + (kSpread ? 4 : 8) * lg;
    const int r1 = r + (kSpread ? 16 : 4);
    u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int row = (q < 2 ? r : r1) + 2 * (q & 1);
        w[q] &= (row < valid ? 0x0000FFFFu : 0u) | (row + 1 < valid ? 0xFFFF0000u : 0u);
    }
    return __builtin_bit_cast(v8bf, w);
}

// Where a lane's load-to-LDS instruction j of one operand's slice reads
// from, relative to the slice's first reduction index.  The instruction
// fills LDS bytes [1024 j, 1024 (j + 1)) of the slice; lane l's 16 bytes go
// to byte 16 l of that kilobyte.
//  direct (rows of 2 RD bytes): kRows rows per instruction, kChunks lanes
//    per row; lane l writes row kRows j + l / kChunks at chunk position
//    l % kChunks, so it loads chunk (l % kChunks) ^ dkey(row): `row` and
//    the element offset `col` of that chunk within the row.
//  transposed (rows of 2 PITCH bytes): 512 / PITCH rows per instruction,
//    PITCH / 8 lanes per row; lane l writes row (512 / PITCH) j + l / (PITCH
//    / 8) at 32-byte position p = (l % (PITCH / 8)) / 2, half l % 2, so it
//    loads 32-byte chunk p ^ key(row), half l % 2: `row` (a reduction index
//    within the slice) and `col`, the element offset within the tile.
struct DmaLane {
    int row, col;
};
template <int RD, int CHUNKS, int ROWS>
__device__ __forceinline__ DmaLane dma_direct(int j, int lane) {
    const int R = ROWS * j + lane / CHUNKS;
    return DmaLane{R, 8 * ((lane % CHUNKS) ^ direct_key<RD>(R))};
}
template <bool kSpread, int PITCH>
__device__ __forceinline__ DmaLane dma_trans(int j, int lane) {
    constexpr int kLanesPerRow = PITCH / 8;
    const int r = (512 / PITCH) * j + lane / kLanesPerRow;
    const int p = (lane % kLanesPerRow) >> 1;
    return DmaLane{r, 16 * (p ^ trans_key<kSpread>(r)) + 8 * (lane & 1)};
}

}  // namespace gmm
