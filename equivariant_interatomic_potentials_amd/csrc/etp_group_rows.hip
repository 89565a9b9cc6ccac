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
//
// 5172508 rows in 100 groups: 38 us (counting 9, sums 2, placing 28), of which the 41
// MB that have to move take 8. Counting waits for its one-word loads and LDS atomics
// (waves wait for 68% of their cycles). In the placing 10.9 million vector instructions
// (43 of 86 thousand cycles), LDS (31) and a chain of barriers for each tile of 4096 rows
// take turns; fewer instructions or other shapes of the tile changed the one for the
// other. 5184 rows: one launch, 5.6 us.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "etp_dense.hpp"

namespace etp {

constexpr int kDigits = 256;
constexpr int kItems = 4;          // rows a lane of a tile
constexpr int kWaves = 16;         // waves that place a tile
constexpr int kMostBlocks = 2048;  // workgroups that share the rows (and sets of counts)
constexpr int kRun = 32;           // workgroups whose counts are added up for the others
constexpr int kFewBlocks = 96;     // so many add all counts themselves
constexpr int kSmallRows = 8192;   // rows that one workgroup sorts in its LDS

struct GroupRowsArgs {
    int64_t M;
    int G;
    const int *ids;
    const int *from;   // rows in the order of the pass before, and their keys; or null
    const uint16_t *from_key;
    int *ptr, *order;  // group_ptr (where one pass gives it), and where the rows go
    uint16_t *key;     // where their keys go, or null
    int *counts;       // [blocks][kDigits], then the sums of runs [runs][kDigits]
    int shift, bits;   // of the digit
    int runs;          // of kRun workgroups, 0 where there are few workgroups
    int64_t per;       // rows of a workgroup, whole tiles
};

__device__ __forceinline__ int key_of(const GroupRowsArgs &a, int64_t row)
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

    // key: the rows' keys, -1 past the end. at: where they belong in the tile.
    // start and sum: of the thread's digit, the first 256 threads each one.
    __device__ __forceinline__ void rank(const int (&key)[Items], int shift, int bits, int (&at)[Items], int &start, int &sum)
    {
        const int w = threadIdx.x >> 6;
        for (int i = threadIdx.x; i < W * kDigits; i += 64 * W)
            (&count[0][0])[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < Items; ++i) {
            // the lanes that agree in every bit
            const uint64_t same = __ballot(key[i] >= 0);
            const int dig = key[i] >> shift & (kDigits - 1);
            uint32_t lo = static_cast<uint32_t>(same), hi = static_cast<uint32_t>(same >> 32);
#pragma unroll
            for (int b = 0; b < 8; ++b)
                if (b < bits) {
                    const int bit = __builtin_amdgcn_sbfe(dig, b, 1);  // 0 or -1
                    const uint64_t with = __ballot(bit != 0);
                    lo &= ~(static_cast<uint32_t>(with) ^ bit);
                    hi &= ~(static_cast<uint32_t>(with >> 32) ^ bit);
                }
            // a lane without a row gets a place that is not used; the first of the
            // others moves the count on, which the wave reads again only after that
            const int below = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
            int *const c = &count[w][dig];
            const int had = *c;
            __builtin_amdgcn_wave_barrier();
            if (key[i] >= 0 && below == 0)
                *c = had + __builtin_popcount(lo) + __builtin_popcount(hi);
            __builtin_amdgcn_wave_barrier();
            at[i] = had + below;
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
            at[i] += count[w][key[i] >> shift & (kDigits - 1)];
    }
};

__global__ void __launch_bounds__(64 * kWaves) group_count_kernel(const GroupRowsArgs a)
{
    __shared__ int count[kWaves][kDigits];
    for (int i = threadIdx.x; i < kWaves * kDigits; i += 64 * kWaves)
        (&count[0][0])[i] = 0;
    __syncthreads();
    const int w = threadIdx.x >> 6;
    const int64_t first = blockIdx.x * a.per, last = first + a.per < a.M ? first + a.per : a.M;
    for (int64_t i0 = first; i0 < last; i0 += 64 * kWaves * kItems) {
        int key[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int64_t i = i0 + 64 * kWaves * k + threadIdx.x;
            key[k] = i < last ? (a.from ? a.from_key[i] : key_of(a, i)) : -1;
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k)
            if (key[k] >= 0)
                atomicAdd(&count[w][key[k] >> a.shift & (kDigits - 1)], 1);
    }
    __syncthreads();
    const int d = threadIdx.x;
    if (d < kDigits) {
        int sum = 0;
#pragma unroll
        for (int k = 0; k < kWaves; ++k)
            sum += count[k][d];
        a.counts[static_cast<int64_t>(blockIdx.x) * kDigits + d] = sum;
    }
}

// The counts of every kRun workgroups added up: what the placing workgroups, of
// which each adds all counts before its own, read instead of them. (Sums written back
// for each workgroup would share lines between the digits' writers: 7 to 15 us for
// 1263 workgroups, this 4.)
__global__ void __launch_bounds__(1024) group_sum_kernel(int *counts, const int blocks)
{
    __shared__ int sums[4][kDigits];
    const int d = threadIdx.x & (kDigits - 1), way = threadIdx.x / kDigits;
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kRun / 4; ++k) {
        const int b = blockIdx.x * kRun + way * (kRun / 4) + k;
        sum += b < blocks ? counts[static_cast<int64_t>(b) * kDigits + d] : 0;
    }
    sums[way][d] = sum;
    __syncthreads();
    if (way == 0)
        counts[(static_cast<int64_t>(blocks) + blockIdx.x) * kDigits + d] = sums[0][d] + sums[1][d] + sums[2][d] + sums[3][d];
}

// Places the rows, tile by tile: a tile's rows are put in order in LDS first (place
// in the tile and key in one word), so that the rows of one digit are written side by
// side.
__global__ void __launch_bounds__(64 * kWaves) group_place_kernel(const GroupRowsArgs a)
{
    using Sort = TileSort<kWaves, kItems>;
    static_assert(Sort::kTile <= 1 << 16);
    __shared__ Sort t;
    __shared__ int base[kDigits];
    __shared__ __attribute__((aligned(16))) uint32_t rows[Sort::kTile];
    const int d = threadIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t first = blockIdx.x * a.per, last = first + a.per < a.M ? first + a.per : a.M;
    int key[kItems];
    auto load = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int64_t p = r + (w * kItems + i) * 64 + lane;
            key[i] = p < last ? (a.from ? a.from_key[p] : key_of(a, p)) : -1;
        }
    };
    load(first);
    // the digit's rows in all, and of the workgroups before
    int all = 0, before = 0;
    {
        constexpr int kWays = 8;  // of four digits a thread
        static_assert(64 * kWaves >= kWays * kDigits / 4 && sizeof(rows) >= kWays * 2 * kDigits * sizeof(int));
        const int way = d / (kDigits / 4), col = d % (kDigits / 4), blocks = gridDim.x, me = blockIdx.x;
        const int run = a.runs ? me / kRun : 0;
        const int4 *counts = reinterpret_cast<const int4 *>(a.counts) + col, *sums = counts + static_cast<int64_t>(blocks) * (kDigits / 4);
        int4 sum = {0, 0, 0, 0}, own = {0, 0, 0, 0};
        auto add = [](int4 &o, const int4 &v, bool on) {
            o.x += on ? v.x : 0;
            o.y += on ? v.y : 0;
            o.z += on ? v.z : 0;
            o.w += on ? v.w : 0;
        };
#pragma unroll 2
        for (int s = way; s < (way < kWays ? a.runs : 0); s += kWays) {
            const int4 v = sums[s * (kDigits / 4)];
            add(sum, v, true);
            add(own, v, s < run);
        }
#pragma unroll 2
        for (int b = run * kRun + way; b < (way < kWays ? a.runs ? me : blocks : 0); b += kWays) {
            const int4 v = counts[static_cast<int64_t>(b) * (kDigits / 4)];
            add(sum, v, !a.runs);
            add(own, v, b < me);
        }
        int4(*shared)[2][kDigits / 4] = reinterpret_cast<int4(*)[2][kDigits / 4]>(rows);
        if (way < kWays) {
            shared[way][0][col] = sum;
            shared[way][1][col] = own;
        }
        __syncthreads();
        if (d < kDigits)
            for (int k = 0; k < kWays; ++k) {
                all += reinterpret_cast<const int *>(shared[k][0])[d];
                before += reinterpret_cast<const int *>(shared[k][1])[d];
            }
    }
    int next = scan_digits(all, t.waves);
    if (a.ptr && blockIdx.x == 0 && d < kDigits && d <= a.G)
        a.ptr[d] = next;
    next += before;
    for (int64_t r = first; r < last; r += Sort::kTile) {
        const int n = last - r < Sort::kTile ? static_cast<int>(last - r) : Sort::kTile;
        int at[kItems], start, sum;
        if (r > first)
            load(r);
        t.rank(key, a.shift, a.bits, at, start, sum);
        if (d < kDigits) {
            base[d] = next - start;  // a row at place p of the tile goes to base + p
            next += sum;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (key[i] >= 0)
                rows[at[i]] = ((w * kItems + i) * 64 + lane) << 16 | key[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int p = 64 * kWaves * i + threadIdx.x;
            if (p < n) {
                const uint32_t u = rows[p];
                const int64_t row = r + (u >> 16);
                const int to = base[u >> a.shift & (kDigits - 1)] + p;
                a.order[to] = a.from ? a.from[row] : static_cast<int>(row);
                if (a.key)
                    a.key[to] = static_cast<uint16_t>(u);
            }
        }
        __syncthreads();
    }
}

// Start i of the groups behind `was` up to `key`, lane by lane; called by whole waves.
// A lane writes a few itself, the whole wave more (where one lane wrote them all, 65534
// empty groups in a row took 1.7 ms).
__device__ __forceinline__ void write_starts(int *ptr, int was, int key, int i)
{
    constexpr int kFew = 4;
    if (key - was <= kFew)
        for (int g = was + 1; g <= key; ++g)
            ptr[g] = i;
    for (uint64_t more = __ballot(key - was > kFew); more; more &= more - 1) {
        const int l = __builtin_ctzll(more);
        const int from = __builtin_amdgcn_readlane(was, l) + 1, to = __builtin_amdgcn_readlane(key, l);
        const int start = __builtin_amdgcn_readlane(i, l);
        for (int g = from + (threadIdx.x & 63); g <= to; g += 64)
            ptr[g] = start;
    }
}

// group_ptr from sorted keys: a slot writes the starts of the groups behind the
// key before it up to its own.
__global__ void __launch_bounds__(256) group_starts_kernel(const GroupRowsArgs a)
{
    for (int64_t i0 = blockIdx.x * 256ll; i0 <= a.M; i0 += gridDim.x * 256ll) {
        const int64_t i = i0 + threadIdx.x;
        const int was = i > 0 && i <= a.M ? a.from_key[i - 1] : -1;
        write_starts(a.ptr, was, i > a.M ? was : i < a.M ? a.from_key[i] : a.G, static_cast<int>(i));
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
    int row[Items], key[Items], at[Items], start, sum;
#pragma unroll
    for (int i = 0; i < Items; ++i) {
        row[i] = (w * Items + i) * 64 + lane;
        key[i] = row[i] < M ? key_of(a, row[i]) : -1;
    }
    t.rank(key, 0, twice ? 8 : a.bits, at, start, sum);
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
    }
    __syncthreads();  // the ranks below reuse the counts, the keys the rows
    t.rank(key, 8, a.bits, at, start, sum);
#pragma unroll
    for (int i = 0; i < Items; ++i)
        if (key[i] >= 0) {
            a.order[at[i]] = row[i];
            rows[at[i]] = key[i];
        }
    __syncthreads();
    for (int i0 = 0; i0 <= M; i0 += 1024) {
        const int i = i0 + threadIdx.x, was = i > 0 && i <= M ? rows[i - 1] : -1;
        write_starts(a.ptr, was, i > M ? was : i < M ? rows[i] : a.G, i);
    }
}

struct GroupRowsCut {
    int blocks, runs, passes;
    int64_t per;
};

static GroupRowsCut group_rows_cut(int64_t M, int G)
{
    constexpr int64_t tile = 64 * kWaves * kItems;
    GroupRowsCut c;
    const int64_t tiles = (M + tile - 1) / tile;
    c.per = (tiles + kMostBlocks - 1) / kMostBlocks * tile;
    c.blocks = static_cast<int>(M > 0 ? (M + c.per - 1) / c.per : 0);
    c.runs = c.blocks > kFewBlocks ? (c.blocks + kRun - 1) / kRun : 0;
    c.passes = G < kDigits ? 1 : 2;
    return c;
}

size_t group_rows_workspace_bytes(int64_t M, int G)
{
    if (M <= kSmallRows)
        return 0;
    const GroupRowsCut c = group_rows_cut(M, G);
    return sizeof(int) * kDigits * (static_cast<size_t>(c.blocks) + c.runs) +
           (c.passes > 1 ? (sizeof(int) + 2 * sizeof(uint16_t)) * static_cast<size_t>(M) : 0);
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
    GroupRowsArgs a{M, G, ids, nullptr, nullptr, ptr, order, nullptr, static_cast<int *>(ws), 0, 0, 0, 0};
    if (M <= kSmallRows) {
        a.bits = bits_of(G < kDigits ? G : G >> 8);
        const auto kernel = M <= kSmallRows / 8 ? group_small_kernel<1> : group_small_kernel<8>;
        hipLaunchKernelGGL(kernel, dim3(1), dim3(1024), 0, stream, a);
        return hipGetLastError();
    }
    const GroupRowsCut c = group_rows_cut(M, G);
    a.per = c.per;
    a.runs = c.runs;
    // of two passes: the rows in the order of the first, and the keys after each
    int *between = a.counts + kDigits * (static_cast<size_t>(c.blocks) + c.runs);
    uint16_t *keys = reinterpret_cast<uint16_t *>(between + (c.passes > 1 ? M : 0));
    hipError_t e = hipSuccess;
    for (int p = 0; p < c.passes; ++p) {
        a.shift = 8 * p;
        a.bits = bits_of(c.passes == 1 ? G : p ? G >> 8 : kDigits - 1);
        a.from = p ? between : nullptr;
        a.from_key = keys;
        a.order = p + 1 < c.passes ? between : order;
        a.key = c.passes == 1 ? nullptr : keys + p * M;
        a.ptr = c.passes == 1 ? ptr : nullptr;
        hipLaunchKernelGGL(group_count_kernel, dim3(c.blocks), dim3(64 * kWaves), 0, stream, a);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        if (a.runs) {
            hipLaunchKernelGGL(group_sum_kernel, dim3(a.runs), dim3(1024), 0, stream, a.counts, c.blocks);
            if ((e = hipGetLastError()) != hipSuccess)
                return e;
        }
        hipLaunchKernelGGL(group_place_kernel, dim3(c.blocks), dim3(64 * kWaves), 0, stream, a);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    if (c.passes > 1) {
        a.ptr = ptr;
        a.from_key = keys + M;
        const int64_t blocks = M / 256 + 1;
        hipLaunchKernelGGL(group_starts_kernel, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0,
                           stream, a);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace etp
