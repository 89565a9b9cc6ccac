// etp_group_rows.hip -- rows grouped by a type id: a stable counting sort.
//
// A row's key is its id, or n_groups where the id is none of them, so that rows
// without a group come last. Keys of up to 8 bits take one pass, of up to 16 two
// (least significant digit first, each pass stable). A pass counts digits per
// workgroup, turns the counts into places, and places the rows: within a wave a
// row's rank among equal digits comes from ballots over the digit's bits, waves
// and tiles follow each other in row order, and a tile's rows are put in order in
// LDS first, so that rows of one digit are written side by side. No result
// depends on the order of an atomic.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "etp_dense.hpp"

namespace etp {

constexpr int kDigits = 256;
constexpr int kItems = 16;           // rows a lane of a tile
constexpr int kMostBlocks = 2048;    // workgroups that share the rows (and sets of counts)

struct GroupRowsArgs {
    int64_t M;
    int G;
    const int *ids;
    const int *from;  // rows in the order of the pass before, or null
    int *ptr, *order; // group_ptr (last pass of one), and where the rows go
    int *counts;      // [kDigits][blocks], then [kDigits] totals
    int shift;        // of the digit
    int64_t per;      // rows of a workgroup, whole tiles
};

__device__ __forceinline__ int key_of(const GroupRowsArgs &a, int row)
{
    const int id = a.ids[row];
    return static_cast<unsigned>(id) < static_cast<unsigned>(a.G) ? id : a.G;
}

// Exclusive sums over 256 values, one a thread of the first four waves; every
// thread of the workgroup calls it.
__device__ __forceinline__ int scan_digits(int v, int *waves)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int sum = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int t = __shfl_up(sum, d, 64);
        sum += lane >= d ? t : 0;
    }
    if (lane == 63 && w < 4)
        waves[w] = sum;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        before += k < w ? waves[k] : 0;
    __syncthreads();
    return before + sum - v;
}

// Places the tile's rows: W waves, each kItems / W * 4 times 64 consecutive rows.
// base: where each digit's next row goes.
template <int W>
struct TileSort {
    static constexpr int kLaneItems = kItems * 4 / W, kTile = 64 * W * kLaneItems;
    int count[W][kDigits];
    int base[kDigits], waves[4];
    int rows[kTile];
    uint8_t digit[kTile];

    __device__ __forceinline__ void place(const GroupRowsArgs &a, int64_t row0, int n)
    {
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
        for (int i = threadIdx.x; i < W * kDigits; i += 64 * W)
            (&count[0][0])[i] = 0;
        __syncthreads();
        int row[kLaneItems], rank[kLaneItems], dig[kLaneItems];
#pragma unroll
        for (int i = 0; i < kLaneItems; ++i) {
            const int at = (w * kLaneItems + i) * 64 + lane;
            row[i] = at < n ? (a.from ? a.from[row0 + at] : static_cast<int>(row0 + at)) : -1;
        }
#pragma unroll
        for (int i = 0; i < kLaneItems; ++i)
            dig[i] = row[i] >= 0 ? key_of(a, row[i]) >> a.shift & (kDigits - 1) : -1;
#pragma unroll
        for (int i = 0; i < kLaneItems; ++i) {
            uint64_t same = __ballot(dig[i] >= 0);
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                const uint64_t set = __ballot(dig[i] >> b & 1);
                same &= dig[i] >> b & 1 ? set : ~set;
            }
            // (lanes without a row have every bit set: they match no lane with one)
            const int below = __popcll(same & ((1ull << lane) - 1)), lead = __ffsll(static_cast<long long>(same)) - 1;
            int had = 0;
            if (dig[i] >= 0 && below == 0)
                had = atomicAdd(&count[w][dig[i]], __popcll(same));
            rank[i] = __shfl(had, lead & 63, 64) + below;
        }
        __syncthreads();
        const int d = threadIdx.x & (kDigits - 1);
        int sum = 0;
        if (threadIdx.x < kDigits)
            for (int k = 0; k < W; ++k)
                sum += count[k][d];
        const int start = scan_digits(threadIdx.x < kDigits ? sum : 0, waves);
        if (threadIdx.x < kDigits) {
            int at = start;
            for (int k = 0; k < W; ++k) {
                const int c = count[k][d];
                count[k][d] = at;
                at += c;
            }
            base[d] -= start;  // a row at place p of the tile goes to base + p
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kLaneItems; ++i)
            if (row[i] >= 0) {
                const int at = count[w][dig[i]] + rank[i];
                rows[at] = row[i];
                digit[at] = static_cast<uint8_t>(dig[i]);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += 64 * W)
            a.order[base[digit[i]] + i] = rows[i];
        __syncthreads();
        if (threadIdx.x < kDigits)
            base[d] += start + sum;
        __syncthreads();
    }
};

__global__ void __launch_bounds__(256) group_count_kernel(const GroupRowsArgs a)
{
    __shared__ int count[4][kDigits];
    for (int i = threadIdx.x; i < 4 * kDigits; i += 256)
        (&count[0][0])[i] = 0;
    __syncthreads();
    const int w = threadIdx.x >> 6;
    const int64_t first = blockIdx.x * a.per, last = first + a.per < a.M ? first + a.per : a.M;
    for (int64_t i = first + threadIdx.x; i < last; i += 256) {
        const int row = a.from ? a.from[i] : static_cast<int>(i);
        atomicAdd(&count[w][key_of(a, row) >> a.shift & (kDigits - 1)], 1);
    }
    __syncthreads();
    const int d = threadIdx.x;
    a.counts[static_cast<int64_t>(d) * gridDim.x + blockIdx.x] = count[0][d] + count[1][d] + count[2][d] + count[3][d];
}

// One digit's counts of all workgroups into exclusive sums, and its total.
__global__ void __launch_bounds__(256) group_scan_kernel(int *counts, const int blocks)
{
    __shared__ int waves[4], carry;
    int *c = counts + static_cast<int64_t>(blockIdx.x) * blocks;
    int before = 0;
    for (int i0 = 0; i0 < blocks; i0 += 256) {
        const int i = i0 + threadIdx.x, v = i < blocks ? c[i] : 0;
        const int at = scan_digits(v, waves);
        if (i < blocks)
            c[i] = before + at;
        if (threadIdx.x == 255)
            carry = at + v;
        __syncthreads();
        before += carry;
        __syncthreads();
    }
    if (threadIdx.x == 0)
        counts[static_cast<int64_t>(kDigits) * blocks + blockIdx.x] = before;
}

__global__ void __launch_bounds__(256) group_place_kernel(const GroupRowsArgs a)
{
    __shared__ TileSort<4> t;
    const int d = threadIdx.x;
    const int start = scan_digits(a.counts[kDigits * static_cast<int64_t>(gridDim.x) + d], t.waves);
    t.base[d] = start + a.counts[static_cast<int64_t>(d) * gridDim.x + blockIdx.x];
    if (a.ptr && blockIdx.x == 0 && d <= a.G)
        a.ptr[d] = start;
    const int64_t first = blockIdx.x * a.per, last = first + a.per < a.M ? first + a.per : a.M;
    for (int64_t r = first; r < last; r += t.kTile)
        t.place(a, r, last - r < t.kTile ? static_cast<int>(last - r) : t.kTile);
}

// group_ptr from sorted keys: a slot writes the starts of the groups behind the
// key before it up to its own.
__device__ __forceinline__ void starts_at(const GroupRowsArgs &a, int64_t slot)
{
    const int was = slot > 0 ? key_of(a, a.order[slot - 1]) : -1;
    const int key = slot < a.M ? key_of(a, a.order[slot]) : a.G;
    for (int g = was + 1; g <= key; ++g)
        a.ptr[g] = static_cast<int>(slot);
}

__global__ void __launch_bounds__(256) group_starts_kernel(const GroupRowsArgs a)
{
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i <= a.M; i += gridDim.x * 256ll)
        starts_at(a, i);
}

// All passes of few rows in one workgroup: one launch instead of three or seven.
__global__ void __launch_bounds__(1024) group_small_kernel(GroupRowsArgs a, int *between)
{
    __shared__ TileSort<16> t;
    const int passes = a.G < kDigits ? 1 : 2;
    int *const order = a.order;
    for (int p = 0; p < passes; ++p) {
        a.shift = 8 * p;
        a.from = p ? between : nullptr;
        a.order = p + 1 < passes ? between : order;
        if (threadIdx.x < kDigits)
            t.base[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < a.M; i += 1024)
            atomicAdd(&t.base[key_of(a, a.from ? a.from[i] : i) >> a.shift & (kDigits - 1)], 1);
        __syncthreads();
        const int start = scan_digits(threadIdx.x < kDigits ? t.base[threadIdx.x] : 0, t.waves);
        if (threadIdx.x < kDigits) {
            t.base[threadIdx.x] = start;
            if (passes == 1 && static_cast<int>(threadIdx.x) <= a.G)
                a.ptr[threadIdx.x] = start;
        }
        __syncthreads();
        for (int r = 0; r < a.M; r += t.kTile)
            t.place(a, r, a.M - r < t.kTile ? static_cast<int>(a.M - r) : t.kTile);
        __threadfence_block();
        __syncthreads();
    }
    if (passes > 1)
        for (int64_t i = threadIdx.x; i <= a.M; i += 1024)
            starts_at(a, i);
}

constexpr int64_t kSmallRows = 16384;

struct GroupRowsCut {
    int blocks, passes;
    int64_t per;
};

static GroupRowsCut group_rows_cut(int64_t M, int G)
{
    constexpr int64_t tile = TileSort<4>::kTile;
    GroupRowsCut c;
    const int64_t tiles = (M + tile - 1) / tile;
    c.per = (tiles + kMostBlocks - 1) / kMostBlocks * tile;
    c.blocks = static_cast<int>(M > 0 ? (M + c.per - 1) / c.per : 0);
    c.passes = G < kDigits ? 1 : 2;
    return c;
}

size_t group_rows_workspace_bytes(int64_t M, int G)
{
    if (M == 0)
        return 0;
    const GroupRowsCut c = group_rows_cut(M, G);
    const size_t counts = M <= kSmallRows ? 0 : sizeof(int) * kDigits * (static_cast<size_t>(c.blocks) + 1);
    return counts + (c.passes > 1 ? sizeof(int) * static_cast<size_t>(M) : 0);
}

hipError_t launch_group_rows(int64_t M, int G, const int *ids, int *ptr, int *order, void *ws, hipStream_t stream)
{
    GroupRowsArgs a{M, G, ids, nullptr, ptr, order, static_cast<int *>(ws), 0, 0};
    if (M <= kSmallRows) {
        hipLaunchKernelGGL(group_small_kernel, dim3(1), dim3(1024), 0, stream, a, static_cast<int *>(ws));
        return hipGetLastError();
    }
    const GroupRowsCut c = group_rows_cut(M, G);
    a.per = c.per;
    int *between = a.counts + kDigits * (static_cast<size_t>(c.blocks) + 1);
    hipError_t e = hipSuccess;
    for (int p = 0; p < c.passes; ++p) {
        a.shift = 8 * p;
        a.from = p ? between : nullptr;
        a.order = p + 1 < c.passes ? between : order;
        a.ptr = c.passes == 1 ? ptr : nullptr;
        hipLaunchKernelGGL(group_count_kernel, dim3(c.blocks), dim3(256), 0, stream, a);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        hipLaunchKernelGGL(group_scan_kernel, dim3(kDigits), dim3(256), 0, stream, a.counts, c.blocks);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        hipLaunchKernelGGL(group_place_kernel, dim3(c.blocks), dim3(256), 0, stream, a);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    if (c.passes > 1) {
        a.ptr = ptr;
        const int64_t blocks = M / 256 + 1;
        hipLaunchKernelGGL(group_starts_kernel, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0,
                           stream, a);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace etp
