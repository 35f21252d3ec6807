// Gradient of the plain grouped product's epilogue: dpre = dout * act'(pre),
// the operand of the two products that follow, and db[g], the column sums of
// dpre over the rows of group g.
//
// One pass over dout and pre, bound by memory.  A workgroup takes an item, up to
// 32 or 128 rows of one group, and a strip of columns, eight a lane; a lane adds
// its rows' dpre in fp32 before they are rounded, the lanes of a column meet in
// LDS, and the item's sums go to a row of `part`.  A second launch adds each
// group's items.  No atomics: the order of every sum is that of the rows and
// items.
#include "gmm_launch.hpp"
#include "gmm_linear.hpp"

namespace gmm {

namespace {

constexpr int kStripLanes = 16;   // lanes across a strip at most: 128 columns

// Rows of an item: 32 to fill the chip, 128 once that gives enough workgroups
// (fewer partial sums to write and add: 65536 rows, 256 groups, N = 2048, no
// activation 82 -> 56 us).
int item_rows(int64_t M, int64_t N) { return M * N >= (int64_t(1) << 25) ? 128 : 32; }

struct GradArgs {
    const uint16_t *dout, *pre;
    const int32_t* group_sizes;
    int M, N, G, act, strips, lanes, item_rows;   // lanes across a strip
    uint16_t* dpre;
    float* part;                       // [item, N], or NULL: db is not wanted
    int32_t* status;
};

__global__ __launch_bounds__(256) void linear_grad_kernel(const GradArgs a) {
    __shared__ float sums[256 * 8];
    __shared__ int s_info[3];
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
    const int w = (int)(blockIdx.x / a.strips), strip = (int)(blockIdx.x % a.strips);
    if (wave == 1 && blockIdx.x == 0) {
        const int st = group_status(a.group_sizes, a.G, a.M);
        if (lane == 0) a.status[0] = st;
    }
    if (wave == 0) {
        const WorkItem it = find_work_item<true>(a.group_sizes, a.G, a.M, a.item_rows, w);
        if (lane == 0) { s_info[0] = it.g; s_info[1] = it.lo; s_info[2] = it.hi; }
    }
    __syncthreads();
    const int g = s_info[0], lo = s_info[1], hi = s_info[2];
    if (g < 0 || g == a.G) return;   // rows past the total: their dpre is never read
    const int across = tid % a.lanes, down = 256 / a.lanes, r0 = tid / a.lanes;
    const int col = (strip * a.lanes + across) * 8;
    const bool in = r0 < down && col < a.N;
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    if (in) {
        for (int row = lo + r0; row < hi; row += down) {
            const int64_t e = (int64_t)row * a.N + col;
            float d[8];
            load_n<8>(a.dout, true, e, d);
            if (a.act != kActNone) {
                float z[8];
                load_n<8>(a.pre, true, e, z);
                with_act(a.act, [&](auto act) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] *= act_slope<decltype(act)::value>(z[i]);
                });
                if (a.dpre != nullptr)
                    *reinterpret_cast<uint4*>(a.dpre + e) =
                        make_uint4(pack_rne(d[0], d[1]), pack_rne(d[2], d[3]), pack_rne(d[4], d[5]), pack_rne(d[6], d[7]));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += d[i];
        }
    }
    if (a.part == nullptr) return;   // the whole grid
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[8 * tid + i] = s[i];
    __syncthreads();
    for (int c = tid; c < a.lanes * 8; c += 256) {
        if (strip * a.lanes * 8 + c >= a.N) break;
        float t = 0.0f;
        for (int r = 0; r < down; ++r) t += sums[r * a.lanes * 8 + c];
        a.part[(int64_t)w * a.N + strip * a.lanes * 8 + c] = t;
    }
}

// db[g, 64 columns]: the sum of the group's items, sixteen threads to four
// columns, each every sixteenth item (20000 rows of one group, N = 1024, both
// launches: 179 us with a thread adding all items, 17.5 so).
template <bool OUT_BF16>
__global__ __launch_bounds__(256) void linear_db_kernel(const int32_t* __restrict__ group_sizes, int M, int N, int G,
                                                        int item_rows, const float* __restrict__ part,
                                                        void* __restrict__ db) {
    __shared__ int s_first, s_count;
    __shared__ v4f sums[16][16];
    const int g = blockIdx.y, across = threadIdx.x & 15, down = threadIdx.x >> 4;
    if (threadIdx.x < 64) {   // items of earlier groups, and of this one
        int carry = 0, items = 0;
        for (int base = 0; base <= g; base += 64) {
            const GroupChunk ch = group_chunk(group_sizes, G, M, base, carry);
            carry = ch.next_carry;
            const int c = group_items<true>(ch.lo, ch.hi, item_rows), incl = wave_incl_scan(c);
            if (g < base + 64 && lane_id() == g - base) { s_first = items + incl - c; s_count = c; }
            items += lane_value(incl, 63);
        }
    }
    __syncthreads();
    const int col = blockIdx.x * 64 + 4 * across;   // N is a multiple of 64
    const float* p = part + (int64_t)s_first * N + col;
    const int n = s_count;
    v4f s = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int i = down; i < n; i += 16) s += *reinterpret_cast<const v4f*>(p + (int64_t)i * N);
    sums[down][across] = s;
    __syncthreads();
    if (down != 0) return;
#pragma unroll
    for (int d = 1; d < 16; ++d) s += sums[d][across];
    const float v[4] = {s[0], s[1], s[2], s[3]};
    store_n<OUT_BF16, 4>(db, (int64_t)g * N + col, v);
}

int64_t grad_items(int64_t M, int64_t N, int64_t G) { return max_work_items(M, G < M ? G : M, item_rows(M, N)); }

}  // namespace

int64_t linear_part_words(int64_t M, int64_t N, int64_t G) { return M > 0 && N > 0 && G > 0 ? grad_items(M, N, G) * N : 0; }

int64_t linear_db_blocks(int64_t N, int64_t G) { return N / 64 * G; }

hipError_t launch_linear_grad(const void* dout, const void* pre, int act, const int32_t* group_sizes, int M, int N, int G,
                              void* dpre, void* db, bool db_bf16, float* part, int32_t* status, hipStream_t stream) {
    if (M > 0 && ((act != kActNone && dpre != nullptr) || db != nullptr)) {
        GradArgs a = {};
        a.dout = static_cast<const uint16_t*>(dout);
        a.pre = static_cast<const uint16_t*>(pre);
        a.group_sizes = group_sizes;
        a.M = M;
        a.N = N;
        a.G = G;
        a.act = act;
        a.strips = (N / 8 + kStripLanes - 1) / kStripLanes;
        a.lanes = (N / 8 + a.strips - 1) / a.strips;
        a.item_rows = item_rows(M, N);
        a.dpre = static_cast<uint16_t*>(dpre);
        a.part = db != nullptr ? part : nullptr;
        a.status = status;
        const int64_t blocks = grad_items(M, N, G) * a.strips;
        if (blocks >= int64_t(1) << 24) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL(linear_grad_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (db == nullptr) return hipSuccess;
    const dim3 grid((unsigned)(N / 64), (unsigned)G);
    const int rows = item_rows(M, N);
    if (db_bf16)
        hipLaunchKernelGGL((linear_db_kernel<true>), grid, dim3(256), 0, stream, group_sizes, M, N, G, rows, part, db);
    else
        hipLaunchKernelGGL((linear_db_kernel<false>), grid, dim3(256), 0, stream, group_sizes, M, N, G, rows, part, db);
    return hipGetLastError();
}

}  // namespace gmm
