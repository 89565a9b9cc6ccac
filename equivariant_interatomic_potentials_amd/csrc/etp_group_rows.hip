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
constexpr int kItems = 16;  // rows a lane of a tile
constexpr int kMostBlocks = 2048;  // workgroups that share the rows (and sets of counts)
constexpr int kSmallRows = 8192;   // rows that one workgroup sorts in its LDS

struct GroupRowsArgs {
    int64_t M;
    int G;
    const int *ids;
    const int *from;   // rows in the order of the pass before, or null
    int *ptr, *order;  // group_ptr (where one pass gives it), and where the rows go
    int *counts;       // [kDigits][blocks], then [kDigits] totals
    int shift, bits;   // of the digit
    int64_t per;       // rows of a workgroup, whole tiles
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

// W waves, each Items times 64 consecutive rows: the place of every row among the
// tile's.
template <int W, int Items>
struct TileSort {
    static constexpr int kTile = 64 * W * Items;
    int count[W][kDigits];
    int waves[4];

    // dig: the rows' digits, -1 past the end. at: where they belong in the tile.
    // start and sum: of the thread's digit, the first 256 threads each one.
    __device__ __forceinline__ void rank(const int (&dig)[Items], int bits, int (&at)[Items], int &start, int &sum)
    {
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
        for (int i = threadIdx.x; i < W * kDigits; i += 64 * W)
            (&count[0][0])[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < Items; ++i) {
            uint64_t same = __ballot(dig[i] >= 0);
            for (int b = 0; b < bits; ++b) {
                const bool set = dig[i] >> b & 1;
                const uint64_t with = __ballot(set);
                same &= set ? with : ~with;
            }
            // (a lane without a row gets a place that is not used)
            const int below = __popcll(same & ((1ull << lane) - 1)), lead = __ffsll(static_cast<long long>(same)) - 1;
            int had = 0;
            if (dig[i] >= 0 && below == 0)
                had = atomicAdd(&count[w][dig[i]], __popcll(same));
            at[i] = __shfl(had, lead & 63, 64) + below;
        }
        __syncthreads();
        const int d = threadIdx.x & (kDigits - 1);
        sum = 0;
        if (threadIdx.x < kDigits)
            for (int k = 0; k < W; ++k) {
                const int c = count[k][d];
                count[k][d] = sum;
                sum += c;
            }
        start = scan_digits(sum, waves);
        if (threadIdx.x < kDigits)
            for (int k = 0; k < W; ++k)
                count[k][d] += start;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < Items; ++i)
            at[i] += dig[i] >= 0 ? count[w][dig[i]] : 0;
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
    for (int64_t i0 = first; i0 < last; i0 += 256 * kItems) {
        int key[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int64_t i = i0 + 256 * k + threadIdx.x;
            key[k] = i < last ? key_of(a, a.from ? a.from[i] : static_cast<int>(i)) : -1;
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k)
            if (key[k] >= 0)
                atomicAdd(&count[w][key[k] >> a.shift & (kDigits - 1)], 1);
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
    constexpr int kEach = kMostBlocks / 256;
    int v[kEach], sum = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int i = threadIdx.x * kEach + k;
        v[k] = i < blocks ? c[i] : 0;
        sum += v[k];
    }
    int at = scan_digits(sum, waves);
    if (threadIdx.x == 255)
        carry = at + sum;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int i = threadIdx.x * kEach + k;
        if (i < blocks)
            c[i] = at;
        at += v[k];
    }
    __syncthreads();
    if (threadIdx.x == 0)
        counts[static_cast<int64_t>(kDigits) * blocks + blockIdx.x] = carry;
}

// Places the rows, tile by tile: a tile's rows are put in order in LDS first, so
// that the rows of one digit are written side by side.
__global__ void __launch_bounds__(256) group_place_kernel(const GroupRowsArgs a)
{
    using Sort = TileSort<4, kItems>;
    __shared__ Sort t;
    __shared__ int base[kDigits], rows[Sort::kTile];
    __shared__ uint8_t digit[Sort::kTile];
    const int d = threadIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int next = scan_digits(a.counts[kDigits * static_cast<int64_t>(gridDim.x) + d], t.waves);
    if (a.ptr && blockIdx.x == 0 && d <= a.G)
        a.ptr[d] = next;
    next += a.counts[static_cast<int64_t>(d) * gridDim.x + blockIdx.x];
    const int64_t first = blockIdx.x * a.per, last = first + a.per < a.M ? first + a.per : a.M;
    for (int64_t r = first; r < last; r += Sort::kTile) {
        const int n = last - r < Sort::kTile ? static_cast<int>(last - r) : Sort::kTile;
        int row[kItems], dig[kItems], at[kItems], start, sum;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int p = (w * kItems + i) * 64 + lane;
            row[i] = p < n ? (a.from ? a.from[r + p] : static_cast<int>(r + p)) : -1;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            dig[i] = row[i] >= 0 ? key_of(a, row[i]) >> a.shift & (kDigits - 1) : -1;
        t.rank(dig, a.bits, at, start, sum);
        base[d] = next - start;  // a row at place p of the tile goes to base + p
        next += sum;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (row[i] >= 0) {
                rows[at[i]] = row[i];
                digit[at[i]] = static_cast<uint8_t>(dig[i]);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += 256)
            a.order[base[digit[i]] + i] = rows[i];
        __syncthreads();
    }
}

// group_ptr from sorted keys: a slot writes the starts of the groups behind the
// key before it up to its own.
__global__ void __launch_bounds__(256) group_starts_kernel(const GroupRowsArgs a)
{
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i <= a.M; i += gridDim.x * 256ll) {
        const int was = i > 0 ? key_of(a, a.order[i - 1]) : -1, key = i < a.M ? key_of(a, a.order[i]) : a.G;
        for (int g = was + 1; g <= key; ++g)
            a.ptr[g] = static_cast<int>(i);
    }
}

// Few rows: all passes in one workgroup and one launch.
template <int Items>
__global__ void __launch_bounds__(1024) group_small_kernel(const GroupRowsArgs a)
{
    using Sort = TileSort<16, Items>;
    __shared__ Sort t;
    __shared__ int rows[Sort::kTile];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, M = static_cast<int>(a.M);
    const bool twice = a.G >= kDigits;
    int row[Items], key[Items], dig[Items], at[Items], start, sum;
#pragma unroll
    for (int i = 0; i < Items; ++i) {
        row[i] = (w * Items + i) * 64 + lane;
        key[i] = row[i] < M ? key_of(a, row[i]) : -1;
        dig[i] = key[i] >= 0 ? key[i] & (kDigits - 1) : -1;
    }
    t.rank(dig, twice ? 8 : a.bits, at, start, sum);
    if (!twice) {
        if (static_cast<int>(threadIdx.x) <= a.G && threadIdx.x < kDigits)
            a.ptr[threadIdx.x] = start;
#pragma unroll
        for (int i = 0; i < Items; ++i)
            if (key[i] >= 0)
                a.order[at[i]] = row[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < Items; ++i)
        if (key[i] >= 0)
            rows[at[i]] = row[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < Items; ++i) {
        const int p = (w * Items + i) * 64 + lane;
        row[i] = p < M ? rows[p] : -1;
        key[i] = p < M ? key_of(a, row[i]) : -1;
        dig[i] = key[i] >= 0 ? key[i] >> 8 : -1;
    }
    __syncthreads();  // the ranks below reuse the counts, the keys the rows
    t.rank(dig, a.bits, at, start, sum);
#pragma unroll
    for (int i = 0; i < Items; ++i)
        if (key[i] >= 0) {
            a.order[at[i]] = row[i];
            rows[at[i]] = key[i];
        }
    __syncthreads();
    for (int i = threadIdx.x; i <= M; i += 1024) {
        const int was = i > 0 ? rows[i - 1] : -1, is = i < M ? rows[i] : a.G;
        for (int g = was + 1; g <= is; ++g)
            a.ptr[g] = i;
    }
}

struct GroupRowsCut {
    int blocks, passes;
    int64_t per;
};

static GroupRowsCut group_rows_cut(int64_t M, int G)
{
    constexpr int64_t tile = 256 * kItems;
    GroupRowsCut c;
    const int64_t tiles = (M + tile - 1) / tile;
    c.per = (tiles + kMostBlocks - 1) / kMostBlocks * tile;
    c.blocks = static_cast<int>(M > 0 ? (M + c.per - 1) / c.per : 0);
    c.passes = G < kDigits ? 1 : 2;
    return c;
}

size_t group_rows_workspace_bytes(int64_t M, int G)
{
    if (M <= kSmallRows)
        return 0;
    const GroupRowsCut c = group_rows_cut(M, G);
    return sizeof(int) * kDigits * (static_cast<size_t>(c.blocks) + 1) +
           (c.passes > 1 ? sizeof(int) * static_cast<size_t>(M) : 0);
}

static int bits_of(int most)
{
    int b = 0;
    while (most >> b)
        ++b;
    return b;
}

hipError_t launch_group_rows(int64_t M, int G, const int *ids, int *ptr, int *order, void *ws, hipStream_t stream)
{
    GroupRowsArgs a{M, G, ids, nullptr, ptr, order, static_cast<int *>(ws), 0, 0, 0};
    if (M <= kSmallRows) {
        a.bits = bits_of(G < kDigits ? G : G >> 8);
        const auto kernel = M <= kSmallRows / 8 ? group_small_kernel<1> : group_small_kernel<8>;
        hipLaunchKernelGGL(kernel, dim3(1), dim3(1024), 0, stream, a);
        return hipGetLastError();
    }
    const GroupRowsCut c = group_rows_cut(M, G);
    a.per = c.per;
    int *between = a.counts + kDigits * (static_cast<size_t>(c.blocks) + 1);
    hipError_t e = hipSuccess;
    for (int p = 0; p < c.passes; ++p) {
        a.shift = 8 * p;
        a.bits = bits_of(c.passes == 1 ? G : p ? G >> 8 : kDigits - 1);
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
