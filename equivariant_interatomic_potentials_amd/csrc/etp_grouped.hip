// etp_grouped.hip -- the linear layer with a matrix for each group of rows (an
// element, a pair of elements, an expert), forward and input gradient.
#include "etp_grouped.hpp"

namespace etp {

// The product of one group: its matrix and bias.
template <typename T>
__device__ __forceinline__ ProductArgs product_of_group(const GroupedProductArgs &a, int g)
{
    ProductArgs p = a.p;
    p.W = static_cast<const T *>(p.W) + static_cast<int64_t>(g) * p.KD * p.ND;
    if (p.bias)
        p.bias += static_cast<int64_t>(g) * p.ND;
    return p;
}

// Few rows a group: a workgroup owns 16 rows of one group and 64 columns, its
// four waves take every fourth chunk of the contraction straight from memory, and
// the partial tiles are added in wave order through LDS. Bound by latency: the
// group, then the rows' indexes, then rows and matrix, one after the other (21 rows in
// 64 groups, 128 x 128 float: 7.4 us in a trace; a call is bound by the host, 8.2).
constexpr int kThinRows = 32768;  // of the grid's second dimension
template <typename T, Dense D>
__global__ void __launch_bounds__(256) grouped_thin_kernel(const GroupedProductArgs ga, const int tiles)
{
    __shared__ f32x4 part[3][4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int tile = blockIdx.z * kThinRows + blockIdx.y, n0 = blockIdx.x * 64;
    if (tile >= tiles)
        return;  // the whole workgroup
    TileWalk at;
    at.start(ga.gr, 4, tile, tile + 1);
    if (at.n == 0)
        return;  // the whole workgroup: a number that stands for nothing
    const ProductArgs a = product_of_group<T>(ga, at.g);
    const int own = row_of_slot(ga.gr, at.slot + c, c < at.n);
    const int64_t row = own < 0 ? a.M : own, rc = own < 0 ? 0 : own;
    f32x4 acc[4][1];
#pragma unroll
    for (int t = 0; t < 4; ++t)
        acc[t][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 32 * wave; k < a.KD; k += 128) {
        RowChunk<T, D> x;
        x.load(a, rc, k + 8 * q);
        MatrixColumn<T, D> w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)  // this lane's column of tile t: the one whose entry is c
            w[t].load(a, k + 8 * q, n0 + (sizeof(T) == 4 ? 16 * t + c
                                                         : 32 * (t >> 1) + 8 * (c >> 2) + 4 * (t & 1) + (c & 3)));
        const Frag<kRowParts<T, D>> xf[1] = {x.frag(a)};
        const Frag<kParts<T>> wf[4] = {w[0].frag(), w[1].frag(), w[2].frag(), w[3].frag()};
        mma(wf, xf, acc);
    }
    if (wave > 0) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            part[wave - 1][t][lane] = acc[t][0];
    }
    lds_barrier();
    if (wave > 0)
        return;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int w = 0; w < 3; ++w)
            acc[t][0] += part[w][t][lane];
        const int j = n0 + col_of_quarter<T>(t, q);
        if (D == Dense::Fwd && a.bias) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[t][0][i] += j + i < a.ND ? a.bias[j + i] : 0.f;
        }
    }
    float add[sizeof(T) == 4 ? 4 : 2][8];
    load_group_addend<T, D>(a, row, n0, q, add);
    store_group<T, D>(a, row, n0, q, acc, add);
}

// Contraction of at most 128: a team of workgroups owns a run of consecutive
// 16-row tiles and takes them in turn, each workgroup nb columns (a multiple of 64)
// of as many tiles as it has waves. It keeps its columns of one group's matrix in
// LDS while its waves walk that group's tiles, each on its own; at the next group
// the matrix is laid out anew, between two barriers. The next tile's rows are in
// flight during this one's products, and the row indexes of the one after it. HBM
// bounds it: 441172 x 64 x 64 float in 4 groups with residual and z 111 us, 4.1 TB/s
// through an order, 107 us where the rows lie in groups (a large copy: 5.0 TB/s).
// Waves a SIMD that its registers allow: the rows in flight and their parts grow
// with the contraction (a kernel that takes a few registers more than 128 or 168
// runs a wave less, and the last workgroups in a second round). Two are held to that by
// a few registers in scratch memory: float forward of 33 to 64 entries, 28 bytes a lane,
// and of 97 to 128, 36.
template <typename T, Dense D, int KC>
constexpr int kResidentWaves = sizeof(T) == 4 ? (D == Dense::Gx ? (KC == 1 ? 4 : KC == 2 ? 3 : 2) : KC <= 2 ? 4 : 3)
                                              : (D == Dense::Gx && KC > 2 ? 3 : 4);

template <typename T, Dense D, int KC>
__global__ void __launch_bounds__((256 * kResidentWaves<T, D, KC>), (kResidentWaves<T, D, KC>))
    grouped_resident_kernel(const GroupedProductArgs ga, const int nb, const int nsplit, const int tiles, const int per,
                            const int team)
{
    using Mx = MatrixLds<T, D>;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    bf16bits *matrix = reinterpret_cast<bf16bits *>(smem);  // [KC] chunks
    float *bias = reinterpret_cast<float *>(matrix + KC * Mx::chunk(nb));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int c = lane & 15, q = lane >> 4;
    // the column blocks of a workgroup's tiles and its team share an XCD
    const int each = gridDim.x >> 3, id = (blockIdx.x & 7) * each + (blockIdx.x >> 3);
    const int n0 = (id % nsplit) * nb, member = id / nsplit % team * waves, stride = team * waves;
    const int from = id / nsplit / team * per, stop = from + per < tiles ? from + per : tiles;
    if (from >= tiles)
        return;  // the whole workgroup
    TileWalk at;
    at.start(ga.gr, 4, from, stop);
    bool first = true;
    while (at.n > 0) {
        const ProductArgs a = product_of_group<T>(ga, at.g);
        const int t0 = at.tile, s0 = at.slot, end = at.end;
        const int t1 = at.last_tile(4) + 1 < stop ? at.last_tile(4) + 1 : stop;
        auto row_of = [&](int tile) {
            const int64_t s = s0 + (static_cast<int64_t>(tile - t0) << 4) + c;
            return row_of_slot(ga.gr, static_cast<int>(s), tile < t1 && s < end);
        };
        RowChunk<T, D> next[KC];
        auto fetch = [&](int row) {
#pragma unroll
            for (int kc = 0; kc < KC; ++kc)
                next[kc].load(a, row < 0 ? 0 : row, 32 * kc + 8 * q);
        };
        // where the workgroup's next tiles lie: at t0 + ahead, and the same modulo stride
        const int ahead = (member - (t0 - from) % stride + stride) % stride;
        if (ahead < t1 - t0 || ahead + waves > stride) {
            int tile = t0 + (ahead + wave) % stride;
            int own = row_of(tile), then = row_of(tile + stride);
            if (tile < t1)
                fetch(own);
            if (!first)
                lds_barrier();  // every wave is done with the group before
            first = false;
            for (int i = threadIdx.x; i < KC * Mx::pieces(nb); i += blockDim.x) {
                const int kc = i / Mx::pieces(nb), j = i % Mx::pieces(nb);
                Raw8<T> v;
                Mx::load(a, j, nb, 32 * kc, n0, v);
                Mx::store(matrix + kc * Mx::chunk(nb), j, nb, v);
            }
            for (int i = threadIdx.x; i < nb; i += blockDim.x)
                bias[i] = a.bias && n0 + i < a.ND ? a.bias[n0 + i] : 0.f;
            lds_barrier();
            for (; tile < t1; tile += stride) {
                Frag<kRowParts<T, D>> xf[KC][1];
#pragma unroll
                for (int kc = 0; kc < KC; ++kc)
                    xf[kc][0] = next[kc].frag(a);
                const int64_t row = own < 0 ? a.M : own;
                if (tile + stride < t1) {
                    own = then;
                    fetch(own);
                    then = row_of(tile + 2 * stride);
                }
                for (int g = 0; g < nb / 64 && n0 + 64 * g < a.ND; ++g) {
                    float add[sizeof(T) == 4 ? 4 : 2][8];
                    load_group_addend<T, D>(a, row, n0 + 64 * g, q, add);
                    f32x4 acc[4][1];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        acc[t][0] = *reinterpret_cast<const f32x4 *>(bias + 64 * g + col_of_quarter<T>(t, q));
#pragma unroll
                    for (int kc = 0; kc < KC; ++kc) {
#pragma unroll
                        for (int t = 0; t < 4; t += 2) {
                            const bf16bits *m = matrix + kc * Mx::chunk(nb);
                            const Frag<kParts<T>> w[2] = {Mx::tile(m, 4 * g + t, nb, lane), Mx::tile(m, 4 * g + t + 1, nb, lane)};
                            mma(w, xf[kc], acc, t);
                        }
                    }
                    store_group<T, D>(a, row, n0 + 64 * g, q, acc, add);
                }
            }
        }
        // the run's next group
        at.tile = t1 - 1;
        at.next(ga.gr, 4, stop);
    }
}

// Longer contractions: a workgroup of four waves owns a tile of 32 RT rows of one
// group and 128 columns (64 or 32 where the result has no more, the waves one
// below the other) and takes the contraction in chunks of 64 (32 where the rows
// have three parts), rows and matrix through LDS, one chunk there while the next
// is on its way in registers. 32768 x 512 x 512 bf16 in 64 groups: 45 us without
// activation and z, 61 with GELU and z. No unit is full: of 160 thousand cycles LDS is
// busy for 61 (22 of them bank conflicts), vector instructions for 54, matrix ones for
// 17, and 541 MB pass L2 (8.5 TB/s, 75% hits); waves wait for 47% of theirs, since a
// workgroup's loads, barriers, products and epilogue take turns and the few workgroups
// of a compute unit overlap them in part only. Tried, and no faster: 128-row tiles (2.3 rounds of workgroups; 71 us), operands straight into LDS
// without registers (62), the same through several tiles as one sequence (70: two
// workgroups a compute unit are too few for the epilogue).
template <typename T, Dense D, int RT, int kCols>
__global__ void __launch_bounds__(256, kCols == 128 ? 2 : kCols == 64 ? 3 : 4)
    grouped_stream_kernel(const GroupedProductArgs ga, const int ncol, const int tiles)
{
    using Mx = MatrixLds<T, D>;
    using Piece = RowPiece<T, D>;
    constexpr int PR = kRowParts<T, D>, SUB = kStreamSub<T, D>, kRows = 32 * RT, kShift = RT == 4 ? 7 : 6;
    static_assert(kRows == 1 << kShift);
    constexpr int WC = kCols == 128 ? 2 : 1, RW = RT * WC / 2, TW = kCols / 16 / WC;  // waves across, a wave's tiles
    constexpr int SR = 32 * SUB + 8, kPlane = kRows * SR;  // LDS rows (elements), a part
    constexpr int kItems = (Mx::pieces(kCols) + 255) / 256;  // matrix pieces per thread and 32 of the contraction
    const bool lays = Mx::pieces(kCols) % 256 == 0 || threadIdx.x < Mx::pieces(kCols);
    constexpr int RP = 32 * SUB / Piece::V, kRowItems = kRows * RP / 256;  // pieces of a row; per thread
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    bf16bits *rows = reinterpret_cast<bf16bits *>(smem), *matrix = rows + PR * kPlane;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    // the column blocks of a tile, and the tiles next to it (which read the same
    // matrix), share an XCD
    const int each = gridDim.x >> 3, id = (blockIdx.x & 7) * each + (blockIdx.x >> 3);
    if (id / ncol >= tiles)
        return;  // the whole workgroup
    TileWalk at;
    at.start(ga.gr, kShift, id / ncol, id / ncol + 1);
    if (at.n == 0)
        return;  // a number that stands for nothing
    const ProductArgs a = product_of_group<T>(ga, at.g);
    const int n0 = (id % ncol) * kCols, wr = wave / WC * 16 * RW, wt = wave % WC * TW;  // this wave's rows, tiles
    int from[kRowItems];
#pragma unroll
    for (int n = 0; n < kRowItems; ++n) {
        const int r = (threadIdx.x + 256 * n) / RP, row = row_of_slot(ga.gr, at.slot + r, r < at.n);
        from[n] = row < 0 ? 0 : row;  // (what a row of no slot gives is not stored)
    }
    int to[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r)
        to[r] = row_of_slot(ga.gr, at.slot + wr + 16 * r + c, wr + 16 * r + c < at.n);

    f32x4 acc[TW][RW];
#pragma unroll
    for (int t = 0; t < TW; ++t) {
        const int j = n0 + col_of_quarter<T>(wt + t, q);
        f32x4 b = {0.f, 0.f, 0.f, 0.f};
        if (D == Dense::Fwd && a.bias) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = j + i < a.ND ? a.bias[j + i] : 0.f;
        }
#pragma unroll
        for (int r = 0; r < RW; ++r)
            acc[t][r] = b;
    }
    const int nk = (a.KD + 32 * SUB - 1) / (32 * SUB);
    Piece xn[kRowItems];
    Raw8<T> wn[SUB][kItems];
    auto fetch = [&](int it) {
#pragma unroll
        for (int n = 0; n < kRowItems; ++n)
            xn[n].load(a, from[n], it * 32 * SUB + (threadIdx.x + 256 * n) % RP * Piece::V);
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int n = 0; n < kItems; ++n)
                if (lays)
                    Mx::load(a, threadIdx.x + 256 * n, kCols, (it * SUB + u) * 32, n0, wn[u][n]);
    };
    fetch(0);
    for (int it = 0; it < nk; ++it) {
        if (it > 0)
            lds_barrier();  // the last chunk has been read
#pragma unroll
        for (int n = 0; n < kRowItems; ++n) {
            const int i = threadIdx.x + 256 * n;
            xn[n].store(a, rows + i / RP * SR + i % RP * Piece::V, kPlane);
        }
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int n = 0; n < kItems; ++n)
                if (lays)
                    Mx::store(matrix + u * Mx::chunk(kCols), threadIdx.x + 256 * n, kCols, wn[u][n]);
        if (it + 1 < nk)
            fetch(it + 1);
        lds_barrier();
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            Frag<PR> xf[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r)
#pragma unroll
                for (int p = 0; p < PR; ++p)
                    xf[r].p[p] =
                        *reinterpret_cast<const bf16x8 *>(rows + p * kPlane + (wr + 16 * r + c) * SR + 32 * u + 8 * q);
#pragma unroll
            for (int t = 0; t < TW; t += 2) {
                const bf16bits *m = matrix + u * Mx::chunk(kCols);
                const Frag<kParts<T>> w[2] = {Mx::tile(m, wt + t, kCols, lane), Mx::tile(m, wt + t + 1, kCols, lane)};
                mma(w, xf, acc, t);
            }
        }
    }
    const int j0 = n0 + 16 * wt;
    if (j0 >= a.ND)
        return;
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const int64_t row = to[r] < 0 ? a.M : to[r];
        float add[sizeof(T) == 4 ? 4 : 2][8];
        load_group_addend<T, D>(a, row, j0, q, add);
        f32x4 v[4][1] = {};  // 32 columns: the others are past ND
#pragma unroll
        for (int t = 0; t < TW; ++t)
            v[t][0] = acc[t][r];
        store_group<T, D>(a, row, j0, q, v, add);
    }
}

template <typename T, Dense D, int KC>
static hipError_t launch_resident(const GroupedProductArgs &a, dim3 grid, dim3 block, size_t lds, int nb, int nsplit,
                                  int tiles, int per, int team, hipStream_t stream)
{
    if (lds > 64 * 1024) {
        const hipError_t e =
            hipFuncSetAttribute(reinterpret_cast<const void *>(&grouped_resident_kernel<T, D, KC>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL((grouped_resident_kernel<T, D, KC>), grid, block, lds, stream, a, nb, nsplit, tiles, per, team);
    return hipGetLastError();
}

// As many workgroups as LDS and 16 waves a compute unit let run at once.
template <typename T, Dense D>
static hipError_t launch_resident_product(const GroupedProductArgs &a, hipStream_t stream)
{
    const int kc = (a.p.KD + 31) / 32;
    const int nb = a.p.ND <= 64 ? 64 : 128, nsplit = (a.p.ND + nb - 1) / nb;
    const size_t lds = sizeof(bf16bits) * kc * MatrixLds<T, D>::chunk(nb) + nb * sizeof(float);
    const int room = kc == 1 ? kResidentWaves<T, D, 1> : kc == 2 ? kResidentWaves<T, D, 2> : kc == 3 ? kResidentWaves<T, D, 3>
                                                                                             : kResidentWaves<T, D, 4>;
    // whole waves a SIMD for each workgroup: one of 5 waves puts two on one SIMD, and
    // the third such workgroup finds no registers there
    const int fit = static_cast<int>(160 * 1024 / lds);
    int per_cu = fit < room ? fit : room;
    while (room % per_cu)
        --per_cu;
    const int waves = 4 * room / per_cu;
    const int tiles = static_cast<int>((a.p.M >> 4) + a.gr.n);
    int runs = (tiles + waves - 1) / waves;
    const int most = kComputeUnits * per_cu / nsplit;
    runs = runs < most ? runs : most < 1 ? 1 : most;
    // few groups: large teams, whose tiles lie side by side at any time, at the price
    // of a matrix laid out by every workgroup of a team (441172 x 64 x 64 float in 4
    // groups: 107 us in 8 teams, 115 in 64; in 1: 104 and 110); many: each on its own
    // (in 1000 groups: 215 us in 8 teams, 128 in 1024; in 64 to 100 both alike)
    int teams = a.gr.n <= 32 ? 8 : runs;
    teams = teams < runs ? teams : runs;
    const int team = runs / teams;
    const int per = (tiles + teams - 1) / teams;
    teams = (tiles + per - 1) / per;
    runs = team * teams;
    const dim3 grid(static_cast<unsigned>((runs * static_cast<int64_t>(nsplit) + 7) / 8 * 8)), block(64 * waves);
    switch (kc) {
    case 1: return launch_resident<T, D, 1>(a, grid, block, lds, nb, nsplit, tiles, per, team, stream);
    case 2: return launch_resident<T, D, 2>(a, grid, block, lds, nb, nsplit, tiles, per, team, stream);
    case 3: return launch_resident<T, D, 3>(a, grid, block, lds, nb, nsplit, tiles, per, team, stream);
    default: return launch_resident<T, D, 4>(a, grid, block, lds, nb, nsplit, tiles, per, team, stream);
    }
}

template <typename T, Dense D, int RT, int kCols>
static hipError_t launch_stream(const GroupedProductArgs &a, hipStream_t stream)
{
    constexpr int SUB = kStreamSub<T, D>;
    constexpr size_t lds = sizeof(bf16bits) * (kRowParts<T, D> * 32 * RT * (32 * SUB + 8) + SUB * MatrixLds<T, D>::chunk(kCols));
    static_assert(lds <= 64 * 1024);
    const int ncol = (a.p.ND + kCols - 1) / kCols, tiles = static_cast<int>((a.p.M / (32 * RT)) + a.gr.n);
    hipLaunchKernelGGL((grouped_stream_kernel<T, D, RT, kCols>),
                       dim3(static_cast<unsigned>((static_cast<int64_t>(tiles) * ncol + 7) / 8 * 8)), dim3(256), lds,
                       stream, a, ncol, tiles);
    return hipGetLastError();
}

// The forms and where they change places, both sides measured (forward, SiLU; us):
// thin up to 2048 workgroups of contractions of at most 128 (16000 x 128 x 128 in 64
// groups: float 18, resident 22; bf16 15 and 17; 32000 rows: 27 and 27, 24 and 20) and
// where groups are small (64 rows of each of 1000 groups: float 65 and 76, bf16 53 and
// 33; 32 rows: 38 and 67, 34 and 30); of longer ones for small float groups (4000 x
// 512 x 512 in 64: 40 as 64-row tiles 38; 2000: 27 and 37) and the smallest bf16 calls
// (64 x 512 x 512 in 8: 11 and 13; 21 in 64: 14 and 11). Tiles of 128 rows pay for
// large float groups only (65536 x 512 x 512 in 8: 266 and 272, in bf16 118 and 102).
template <typename T, Dense D>
hipError_t launch_grouped_product(const GroupedProductArgs &a, hipStream_t stream)
{
    const int64_t rows = a.p.M / a.gr.n;  // of a group, on average
    const int64_t tiles = (a.p.M >> 4) + a.gr.n, nc = (a.p.ND + 63) / 64;
    const bool is_float = sizeof(T) == 4, lies = a.p.KD <= 128;
    if (tiles * nc <= (lies ? 2048 : 128) || rows < (lies ? (is_float ? 64 : 32) : (is_float ? 48 : 0))) {
        const dim3 grid(static_cast<unsigned>(nc), static_cast<unsigned>(tiles < kThinRows ? tiles : kThinRows),
                        static_cast<unsigned>((tiles + kThinRows - 1) / kThinRows));
        hipLaunchKernelGGL((grouped_thin_kernel<T, D>), grid, dim3(256), 0, stream, a, static_cast<int>(tiles));
        return hipGetLastError();
    }
    // (d is kept for layers of more than 128 inputs and outputs only)
    if constexpr (D != Dense::GxD) {
        if (lies)
            return launch_resident_product<T, D>(a, stream);
        if (a.p.ND <= 32)
            return launch_stream<T, D, 2, 32>(a, stream);
        if (a.p.ND <= 64)
            return launch_stream<T, D, 2, 64>(a, stream);
    }
    if constexpr (sizeof(T) == 4)
        if (rows >= 4096)
            return launch_stream<T, D, 4, 128>(a, stream);
    return launch_stream<T, D, 2, 128>(a, stream);
}

template hipError_t launch_grouped_product<float, Dense::Gx>(const GroupedProductArgs &, hipStream_t);
template hipError_t launch_grouped_product<float, Dense::GxD>(const GroupedProductArgs &, hipStream_t);
template hipError_t launch_grouped_product<float, Dense::GxPlain>(const GroupedProductArgs &, hipStream_t);
template hipError_t launch_grouped_product<bf16bits, Dense::Gx>(const GroupedProductArgs &, hipStream_t);
template hipError_t launch_grouped_product<bf16bits, Dense::GxD>(const GroupedProductArgs &, hipStream_t);
template hipError_t launch_grouped_product<bf16bits, Dense::GxPlain>(const GroupedProductArgs &, hipStream_t);

hipError_t launch_grouped_linear(const GroupedLinearArgs &ga, hipStream_t stream)
{
    const LinearArgs &a = ga.l;
    if (a.M == 0)
        return hipSuccess;
    const GroupedProductArgs g{{a.M, a.K, a.N, a.x, a.ldx, nullptr, 0, a.W, a.bias, a.act, a.res, a.ldr, a.y, a.ldy,
                                a.z, a.ldz, false},
                               {ga.group_ptr, ga.order, ga.n_groups, static_cast<int>(a.M)}};
    return a.bf16 ? launch_grouped_product<bf16bits, Dense::Fwd>(g, stream) : launch_grouped_product<float, Dense::Fwd>(g, stream);
}

}  // namespace etp
