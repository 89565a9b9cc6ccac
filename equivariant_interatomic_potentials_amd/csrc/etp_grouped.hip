// etp_grouped.hip -- the linear layer with a matrix for each group of rows (an
// element, a pair of elements, an expert), and its VJP.
#include "etp_dense_product.hpp"
#include "etp_groups_of_rows.hpp"

namespace etp {

struct GroupedProductArgs {
    ProductArgs p;  // W and bias of group 0
    Groups gr;
};

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
// the partial tiles are added in wave order through LDS. Bound by the latency of
// its few loads.
template <typename T, Dense D>
__global__ void __launch_bounds__(256) grouped_thin_kernel(const GroupedProductArgs ga, const int ncol)
{
    __shared__ f32x4 part[3][4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x / ncol, n0 = (blockIdx.x % ncol) * 64;
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

// Contraction of at most 128: a workgroup owns a run of consecutive 16-row tiles
// and nb columns (a multiple of 64). It keeps its columns of one group's matrix in
// LDS while its waves walk that group's tiles of the run, each on its own; at the
// next group the matrix is laid out anew, between two barriers. The next tile's
// rows are in flight during this one's products, and the row indexes of the one
// after it.
template <typename T, Dense D, int KC>
__global__ void __launch_bounds__(512)
    grouped_resident_kernel(const GroupedProductArgs ga, const int nb, const int nsplit, const int tiles, const int per)
{
    using Mx = MatrixLds<T, D>;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    bf16bits *matrix = reinterpret_cast<bf16bits *>(smem);  // [KC] chunks
    float *bias = reinterpret_cast<float *>(matrix + KC * Mx::chunk(nb));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int c = lane & 15, q = lane >> 4;
    // the column blocks of a run, and the runs next to it, share an XCD
    const int each = gridDim.x >> 3, id = (blockIdx.x & 7) * each + (blockIdx.x >> 3);
    const int n0 = (id % nsplit) * nb;
    const int from = id / nsplit * per, stop = from + per < tiles ? from + per : tiles;
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
        int tile = t0 + wave;
        int own = row_of(tile), then = row_of(tile + waves);
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
        for (; tile < t1; tile += waves) {
            Frag<kRowParts<T, D>> xf[KC][1];
#pragma unroll
            for (int kc = 0; kc < KC; ++kc)
                xf[kc][0] = next[kc].frag(a);
            const int64_t row = own < 0 ? a.M : own;
            if (tile + waves < t1) {
                own = then;
                fetch(own);
                then = row_of(tile + 2 * waves);
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
        // the run's next group
        at.tile = t1 - 1;
        at.next(ga.gr, 4, stop);
    }
}

// Longer contractions: a workgroup of four waves owns a tile of 32 RT rows of one
// group and 128 columns (64 or 32 where the result has no more, the waves one
// below the other) and takes the contraction in chunks of 64 (32 where the rows
// have three parts), rows and matrix through LDS, one chunk there while the next
// is on its way in registers.
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
                                  int tiles, int per, hipStream_t stream)
{
    if (lds > 64 * 1024) {
        const hipError_t e =
            hipFuncSetAttribute(reinterpret_cast<const void *>(&grouped_resident_kernel<T, D, KC>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL((grouped_resident_kernel<T, D, KC>), grid, block, lds, stream, a, nb, nsplit, tiles, per);
    return hipGetLastError();
}

// As many workgroups as LDS and 16 waves a compute unit let run at once.
template <typename T, Dense D>
static hipError_t launch_resident_product(const GroupedProductArgs &a, hipStream_t stream)
{
    const int kc = (a.p.KD + 31) / 32;
    const int nb = a.p.ND <= 64 ? 64 : 128, nsplit = (a.p.ND + nb - 1) / nb;
    const size_t lds = sizeof(bf16bits) * kc * MatrixLds<T, D>::chunk(nb) + nb * sizeof(float);
    const int waves = lds <= 40 * 1024 ? 4 : 8;
    const int fit = static_cast<int>(160 * 1024 / lds), per_cu = fit < 16 / waves ? fit : 16 / waves;
    const int tiles = static_cast<int>((a.p.M >> 4) + a.gr.n);
    int runs = (tiles + waves - 1) / waves;
    const int most = kComputeUnits * per_cu / nsplit;
    runs = runs < most ? runs : most < 1 ? 1 : most;
    const int per = (tiles + runs - 1) / runs;
    runs = (tiles + per - 1) / per;
    const dim3 grid(static_cast<unsigned>((runs * static_cast<int64_t>(nsplit) + 7) / 8 * 8)), block(64 * waves);
    switch (kc) {
    case 1: return launch_resident<T, D, 1>(a, grid, block, lds, nb, nsplit, tiles, per, stream);
    case 2: return launch_resident<T, D, 2>(a, grid, block, lds, nb, nsplit, tiles, per, stream);
    case 3: return launch_resident<T, D, 3>(a, grid, block, lds, nb, nsplit, tiles, per, stream);
    default: return launch_resident<T, D, 4>(a, grid, block, lds, nb, nsplit, tiles, per, stream);
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

template <typename T, Dense D>
static hipError_t launch_product(const GroupedProductArgs &a, hipStream_t stream)
{
    const int64_t rows = a.p.M / a.gr.n;  // of a group, on average
    if (rows < 32) {
        const int64_t tiles = (a.p.M >> 4) + a.gr.n;
        const int nc = (a.p.ND + 63) / 64;
        hipLaunchKernelGGL((grouped_thin_kernel<T, D>), dim3(static_cast<unsigned>(tiles * nc)), dim3(256), 0, stream, a,
                           nc);
        return hipGetLastError();
    }
    // (d is kept for layers of more than 128 inputs and outputs only)
    if constexpr (D != Dense::GxD) {
        if (a.p.KD <= 128)
            return launch_resident_product<T, D>(a, stream);
    }
    const bool small = rows < 256 || (a.p.M + 127) / 128 * ((a.p.ND + 127) / 128) < 2 * kComputeUnits;
    if constexpr (D != Dense::GxD) {
        if (a.p.ND <= 32)
            return small ? launch_stream<T, D, 2, 32>(a, stream) : launch_stream<T, D, 4, 32>(a, stream);
        if (a.p.ND <= 64)
            return small ? launch_stream<T, D, 2, 64>(a, stream) : launch_stream<T, D, 4, 64>(a, stream);
    }
    return small ? launch_stream<T, D, 2, 128>(a, stream) : launch_stream<T, D, 4, 128>(a, stream);
}

// ---------------------------------------------------------------------------
// The VJP over panels of rows of one group. A workgroup owns a run of
// consecutive tiles (panels) and a block of at most 128 x 128 of the matrices:
// d and x of a panel are formed in registers from one read of gy, z and x, cut
// into bf16 parts and put into LDS row by row; then
//   gx = d W^T (where one block holds the whole matrix): fragments of d are read
//     as they lie, W_g's columns stay in a wave's registers for the group;
//   gW_g += x^T d: the contraction runs along the rows; the transposing LDS read
//     hands a lane four rows of one column, and the result stays in the
//     accumulators until the group ends.
// A group that lies in one run is written straight to gW and gb. Of one that
// crosses runs each leaves a partial set, at most two a run: set 2 s of what began
// in an earlier run, set 2 s + 1 of what goes on in the next; they are added in
// that order by grouped_join_kernel.
struct GroupedPanelArgs {
    LinearVjpArgs v;  // W, gW, gb of group 0
    Groups gr;
    const float *d;  // d [rows][N], or null: from gy and z
    int tiles, per;  // tile numbers, and how many of them a run has
    int runs;
    int nkb, blocks;  // blocks along K, and in all
    int64_t set;      // floats of a partial set: gW, then gb, of those that are wanted
};

// Parts of x and d, waves, LDS rows (elements), buffers, panel rows, LDS bytes
// and workgroups of a compute unit. The rules are the linear layer's.
struct GroupedShape {
    int px, pd, waves, sx, sd, bufs, rows, shift, lds, per_cu;
    constexpr GroupedShape(bool bf16, int kc, int nc, bool plain)
        : px(bf16 ? 1 : 3), pd(bf16 && plain ? 1 : 3),
          waves(bf16 ? (kc == 4 && nc > 1 ? 8 : 4) : (kc == 4 || nc == 4 ? 8 : 4)), sx(32 * kc + 8), sd(32 * nc + 8),
          bufs(waves == 8 && !(bf16 && nc == 2) ? 2 : 1),
          rows(2 * bufs * 64 * (px * sx + pd * sd) <= 144 * 1024 ? 64 : 32), shift(rows == 64 ? 6 : 5),
          lds(2 * bufs * rows * (px * sx + pd * sd)),
          per_cu(waves == 8 ? 3 - bufs : 160 * 1024 / lds < 3 ? 160 * 1024 / lds : 3)
    {
    }
};
template <typename T, int KC, int NC, bool Plain>
constexpr GroupedShape kGroupedShape{sizeof(T) == 2, KC, NC, Plain};

template <typename T, int KC, int NC, bool Plain, bool FromD>
__global__ void __launch_bounds__((64 * kGroupedShape<T, KC, NC, Plain>.waves),
                                  (kGroupedShape<T, KC, NC, Plain>.waves / 4 * kGroupedShape<T, KC, NC, Plain>.per_cu))
    grouped_panel_kernel(const GroupedPanelArgs p)
{
    static_assert(!(Plain && FromD), "without an activation d is gy");
    constexpr GroupedShape S = kGroupedShape<T, KC, NC, Plain>;
    constexpr int PX = S.px, PD = S.pd, W = S.waves, SX = S.sx, SD = S.sd, kRows = S.rows;
    constexpr int kBuf = kRows * (PX * SX + PD * SD);  // elements of one panel
    constexpr Cut C = kCut<T>;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    bf16bits *const lds = reinterpret_cast<bf16bits *>(smem);  // [bufs] of d [PD][kRows][SD], x [PX][kRows][SX]
    const LinearVjpArgs &a = p.v;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    // workgroup i runs on XCD i % 8: the blocks of one run, which read the same
    // rows, and the runs next to it, which read the same matrices, share one
    const int total = p.runs * p.blocks, each = (total + 7) / 8;
    const int id = (blockIdx.x & 7) * each + (blockIdx.x >> 3);
    if (id >= total || static_cast<int>(blockIdx.x >> 3) >= each)
        return;
    const int s = id / p.blocks, blk = id % p.blocks;
    const int k0 = (blk % p.nkb) * 32 * KC, j0 = (blk / p.nkb) * 32 * NC;
    const int K = a.K, N = a.N;
    const bool want_gx = a.gx != nullptr, want_gw = a.gW != nullptr, want_gb = a.gb != nullptr && k0 == 0;
    const int from = s * p.per, stop = from + p.per < p.tiles ? from + p.per : p.tiles;

    // loads: a thread takes 16 bytes of the same columns in every RD-th (RX-th)
    // row of the panel, so that a wave covers whole rows
    using Src = std::conditional_t<FromD, float, T>;
    constexpr int kTiles = kRows / 16, VD = kVec<Src>, VX = kVec<T>;
    constexpr int DP = 32 * NC / VD, XP = 32 * KC / VX;  // pieces of a row
    constexpr int RD = 64 * W / DP, RX = 64 * W / XP;    // rows at a time
    constexpr int ND = (kRows + RD - 1) / RD, NX = (kRows + RX - 1) / RX;
    const int drow = threadIdx.x / DP, dcol = threadIdx.x % DP * VD;
    const int xrow = threadIdx.x / XP, xcol = threadIdx.x % XP * VX;
    RawVec<Src> gn[ND];
    RawVec<T> zn[Plain || FromD ? 1 : ND], xn[NX];
    // rows: the panel's, lane by lane; those of no row read nothing and are zero
    auto fetch = [&](int rows) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < ND; ++n) {
            const int at = drow + RD * n;
            const int r = __shfl(rows, at & 63, 64);
            const bool live = r >= 0 && (kRows % RD == 0 || at < kRows);
            const int64_t rc = live ? r : 0;
            const int valid = live ? N - j0 - dcol : 0;
            if constexpr (FromD) {
                gn[n].load(p.d + rc * N + j0 + dcol, valid);
            } else {
                gn[n].load(static_cast<const T *>(a.gy) + rc * a.ldgy + j0 + dcol, valid);
                if constexpr (!Plain)
                    zn[n].load(static_cast<const T *>(a.z) + rc * a.ldz + j0 + dcol, valid);
            }
        }
        if (want_gw) {
#pragma unroll
            for (int n = 0; n < NX; ++n) {
                const int at = xrow + RX * n;
                const int r = __shfl(rows, at & 63, 64);
                const bool live = r >= 0 && (kRows % RX == 0 || at < kRows);
                xn[n].load(static_cast<const T *>(a.x) + static_cast<int64_t>(live ? r : 0) * a.ldx + k0 + xcol,
                           live ? K - k0 - xcol : 0);
            }
        }
    };

    // gx: a wave owns G column tiles (a pair for bf16, whose lanes store eight
    // columns) and RT of the row tiles
    constexpr int G = sizeof(T) == 4 ? 1 : 2, groups = 2 * KC / G, RS0 = W / groups, RS = RS0 < kTiles ? RS0 : kTiles;
    static_assert(RS >= 1, "too few waves for the columns of gx");
    constexpr int RT = kTiles / RS;
    const int grp = wave % groups, rt0 = (wave / groups) * RT;
    const bool gx_wave = want_gx && wave / groups < RS;
    Frag<PX> wf[NC][G];
    // gW: waves as WK x WN, each KT x JT tiles of 16 x 16
    constexpr int WN = W == 4 || NC == 1 ? 2 : 4, WK = W / WN, KT = 2 * KC / WK, JT = 2 * NC / WN;
    const int kt0 = (wave / WN) * KT, jt0 = (wave % WN) * JT;
    f32x4 acc[KT][JT];
    float gb[VD];

    // the fetched panel's parts into LDS
    auto put = [&](bf16bits *dl) __attribute__((always_inline)) {
        bf16bits *xl = dl + PD * kRows * SD;
#pragma unroll
        for (int n = 0; n < ND; ++n) {
            const int row = drow + RD * n;
            if (kRows % RD && row >= kRows)
                continue;
            float d[VD];
#pragma unroll
            for (int i = 0; i < VD; ++i) {
                d[i] = gn[n].get(i);
                if constexpr (!FromD && !Plain)
                    d[i] *= act_slope(a.act, zn[n].get(i));
                gb[i] += d[i];
            }
            if constexpr (PD == 1)
                *reinterpret_cast<u32x4 *>(dl + row * SD + dcol) = gn[n].v;
            else
                put_parts<PD, C>(dl + row * SD + dcol, kRows * SD, d);
        }
        if (want_gw) {
#pragma unroll
            for (int n = 0; n < NX; ++n) {
                const int row = xrow + RX * n;
                if (kRows % RX && row >= kRows)
                    continue;
                if constexpr (PX == 1) {
                    *reinterpret_cast<u32x4 *>(xl + row * SX + xcol) = xn[n].v;
                } else {
                    float x[VX];
#pragma unroll
                    for (int i = 0; i < VX; ++i)
                        x[i] = xn[n].get(i);
                    put_parts<PX>(xl + row * SX + xcol, kRows * SX, x);
                }
            }
        }
    };

    // what the panel in LDS adds: gx of its rows, and its share of gW
    auto products = [&](const bf16bits *dl, int rows) __attribute__((always_inline)) {
        const bf16bits *xl = dl + PD * kRows * SD;
        if (gx_wave) {
            f32x4 o[G][RT];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    o[g][r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                Frag<PD> df[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int t = 0; t < PD; ++t)
                        df[r].p[t] = *reinterpret_cast<const bf16x8 *>(
                            dl + (t * kRows + 16 * (rt0 + r) + c) * SD + 32 * n + 8 * q);
                mma(wf[n], df, o);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int row = __shfl(rows, 16 * (rt0 + r) + c, 64);
                const int k = sizeof(T) == 4 ? 16 * grp + 4 * q : 32 * grp + 8 * q;
                if (row >= 0 && k < K) {
                    T *dst = static_cast<T *>(a.gx) + static_cast<int64_t>(row) * a.ldgx + k;
                    float v[8];
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[4 * g + i] = o[g][r][i];
                    if (a.accumulate) {
                        float was[8];
                        load_n<4 * G>(dst, K - k, was);
#pragma unroll
                        for (int i = 0; i < 4 * G; ++i)
                            v[i] += was[i];
                    }
                    store_n<4 * G>(dst, K - k, v);
                }
            }
        }
        if (want_gw) {
#pragma unroll
            for (int st = 0; st < kRows / 32; ++st) {
                Frag<PD> df[JT];
#pragma unroll
                for (int j = 0; j < JT; ++j)
#pragma unroll
                    for (int t = 0; t < PD; ++t)
                        df[j].p[t] = read_transposed(dl + t * kRows * SD, SD, st, 16 * (jt0 + j), lane);
                constexpr int KS = KT < 2 ? KT : 2;  // row tiles at a time
#pragma unroll
                for (int i = 0; i < KT; i += KS) {
                    Frag<PX> xf[KS];
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int t = 0; t < PX; ++t)
                            xf[k].p[t] = read_transposed(xl + t * kRows * SX, SX, st, 16 * (kt0 + i + k), lane);
                    mma(xf, df, acc, i);
                }
            }
        }
    };

    TileWalk at;
    at.start(p.gr, S.shift, from, stop);
    if (at.n == 0)
        return;  // the whole workgroup
    int rows = row_of_slot(p.gr, at.slot + lane, lane < at.n);
    fetch(rows);
    // the panel after it: its rows' indexes are on their way one panel ahead
    TileWalk then = at;
    then.next(p.gr, S.shift, stop);
    int rows_then = row_of_slot(p.gr, then.slot + lane, lane < then.n);
    while (at.n > 0) {
        const int g = at.g;
        const bool whole = at.first_tile(S.shift) >= from && at.last_tile(S.shift) < stop;
        const int set = 2 * s + (at.first_tile(S.shift) >= from ? 1 : 0);
        if (gx_wave) {
#pragma unroll
            for (int h = 0; h < G; ++h)
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    const int k = sizeof(T) == 4 ? 16 * grp + c : 32 * grp + 8 * (c >> 2) + 4 * h + (c & 3);
                    const int j = 32 * n + 8 * q;
                    Raw8<T> raw;
                    raw.load(static_cast<const T *>(a.W) + (static_cast<int64_t>(g) * K + (k < K ? k : 0)) * N + j,
                             k < K ? N - j : 0);
                    wf[n][h] = raw.template frag<PX>();
                }
        }
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int j = 0; j < JT; ++j)
                acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < VD; ++i)
            gb[i] = 0.f;
        int buf = 0;
        if constexpr (S.bufs == 2) {
            lds_barrier();  // of the group before: its sums or its last panel
            put(lds);
        }
        for (;;) {
            // `rows` names the panel in LDS (or about to be), `rows_then` the next
            const bool more = then.n > 0, same = more && then.g == g;
            int rows_last = rows_then;
            if constexpr (S.bufs == 1)
                put(lds);
            if (more) {
                fetch(rows_then);
                at = then;
                then.next(p.gr, S.shift, stop);
                rows_then = row_of_slot(p.gr, then.slot + lane, lane < then.n);
            } else {
                at.n = 0;
            }
            lds_barrier();  // the panel's parts are seen by every wave
            products(lds + buf * kBuf, rows);
            rows = rows_last;
            if constexpr (S.bufs == 2) {
                if (same) {
                    buf ^= 1;
                    put(lds + buf * kBuf);  // was last read before this panel's barrier
                }
            } else {
                lds_barrier();  // the next panel overwrites the rows
            }
            if (!same)
                break;
        }
        // the group's sums
        float *gw = nullptr, *gbias = nullptr;
        bool add = false;
        if (whole) {
            gw = want_gw ? a.gW + static_cast<int64_t>(g) * K * N : nullptr;
            gbias = want_gb ? a.gb + static_cast<int64_t>(g) * N : nullptr;
            add = a.accumulate;
        } else {
            float *part = static_cast<float *>(a.ws) + set * p.set;
            gw = part;
            gbias = part + p.set - N;
        }
        if (want_gw) {
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    const int jj = j0 + 16 * (jt0 + j) + c;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int k = k0 + 16 * (kt0 + i) + 4 * q + r;
                        if (k < K && jj < N) {
                            float *o = gw + static_cast<int64_t>(k) * N + jj;
                            *o = add ? *o + acc[i][j][r] : acc[i][j][r];
                        }
                    }
                }
        }
        if (want_gb) {
            // the threads that share columns, through LDS, in row order
            float *sums = reinterpret_cast<float *>(smem);  // [RD][32 NC]
            static_assert(RD * 32 * NC * sizeof(float) <= static_cast<size_t>(S.lds));
            if constexpr (S.bufs == 2)
                lds_barrier();  // the last panel has been read
#pragma unroll
            for (int i = 0; i < VD; ++i)
                sums[drow * 32 * NC + dcol + i] = gb[i];
            lds_barrier();
            for (int j = threadIdx.x; j < 32 * NC; j += 64 * W) {
                float v = 0.f;
                for (int r = 0; r < RD; ++r)
                    v += sums[r * 32 * NC + j];
                if (j0 + j < N)
                    gbias[j0 + j] = add ? gbias[j0 + j] + v : v;
            }
            if constexpr (S.bufs == 1)
                lds_barrier();  // the next group's panel overwrites the sums
        }
    }
}

// The groups that cross runs: boundary b = 1 .. runs - 1 (blockIdx.y < runs - 1)
// adds the parts of the group that crosses it, if it is the first one that the
// group crosses, 64 entries a workgroup by 4 threads each, every one its parts in
// order. The other rows of workgroups zero the gradients of groups without rows.
__global__ void __launch_bounds__(256) grouped_join_kernel(const GroupedPanelArgs p, const int shift)
{
    __shared__ float lds[4][65];
    const LinearVjpArgs &a = p.v;
    const int64_t nw = a.gW ? static_cast<int64_t>(a.K) * a.N : 0;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 64 + tx;
    if (static_cast<int>(blockIdx.y) >= p.runs - 1) {
        const int rest = gridDim.y - (p.runs - 1);
        for (int g = blockIdx.y - (p.runs - 1) + ty * rest; g < p.gr.n; g += 4 * rest) {
            const int begin = group_start(p.gr, g);
            if (group_start(p.gr, g + 1) > begin || i >= p.set)
                continue;
            if (i < nw)
                a.gW[g * nw + i] = 0.f;
            else
                a.gb[static_cast<int64_t>(g) * a.N + i - nw] = 0.f;
        }
        return;
    }
    const int b = blockIdx.y + 1, edge = b * p.per;
    const int g = group_of_tile(p.gr, shift, edge);
    const int begin = group_start(p.gr, g), end = group_start(p.gr, g + 1);
    const int first = (begin >> shift) + g, last = first + ((end - begin - 1) >> shift);
    if (first >= edge || last < edge || first < edge - p.per)
        return;
    const int run1 = last / p.per;
    const float *part = static_cast<const float *>(a.ws);
    float v = 0.f;
    if (i < p.set)
        for (int r = b - 1 + ty; r <= run1; r += 4)
            v += part[(2 * static_cast<int64_t>(r) + (r == b - 1 ? 1 : 0)) * p.set + i];
    lds[ty][tx] = v;
    lds_barrier();
    if (ty > 0 || i >= p.set)
        return;
    v = (lds[0][tx] + lds[1][tx]) + (lds[2][tx] + lds[3][tx]);
    float *o = i < nw ? a.gW + g * nw + i : a.gb + static_cast<int64_t>(g) * a.N + i - nw;
    *o = a.accumulate ? *o + v : v;
}

// How a VJP call is cut: as the linear layer's, in one panel kernel where K and N
// are at most 128, else gx as a product and gW in blocks of up to 128 x 128, with
// d made once before both where K and N are above 128 and there is an activation.
struct GroupedCut {
    bool fused, keep_d;
    int kc, nc, nkb, nnb;
    int shift, tiles, per, runs;
    size_t d_bytes, part_bytes;
};

static GroupedCut grouped_cut(int64_t M, int G, int K, int N, bool bf16, bool plain)
{
    GroupedCut v{};
    auto chunks = [](int n) { return n <= 32 ? 1 : n <= 64 ? 2 : 4; };
    v.kc = chunks(K);
    v.nc = chunks(N);
    v.nkb = (K + 127) / 128;
    v.nnb = (N + 127) / 128;
    v.fused = K <= 128 && N <= 128;
    const GroupedShape shape(bf16, v.kc, v.nc, plain);
    v.shift = shape.shift;
    v.tiles = static_cast<int>((M >> v.shift) + G);
    // as many runs as run at once (one more would double the time), or over up to
    // four rounds where that fills them better by a tenth
    const int64_t blocks = static_cast<int64_t>(v.nkb) * v.nnb, room = static_cast<int64_t>(kComputeUnits) * shape.per_cu;
    int64_t s = 0, rounds = 1;
    for (int64_t n = 1; n <= 4; ++n) {
        const int64_t t = n * room / blocks;
        if (s == 0 ? t > 0 : 10 * n * s < 9 * rounds * t) {
            s = t;
            rounds = n;
        }
    }
    s = s < v.tiles ? s : v.tiles;
    s = s < 1 ? 1 : s;
    v.per = static_cast<int>((v.tiles + s - 1) / s);
    v.runs = (v.tiles + v.per - 1) / v.per;
    v.keep_d = K > 128 && N > 128 && !plain;
    v.d_bytes = v.keep_d ? (sizeof(float) * static_cast<size_t>(M) * N + 15) / 16 * 16 : 0;
    v.part_bytes = sizeof(float) * 2 * static_cast<size_t>(v.runs) * (static_cast<size_t>(K) + 1) * N;
    v.part_bytes = (v.part_bytes + 15) / 16 * 16;
    return v;
}

size_t grouped_linear_vjp_workspace_bytes(int64_t M, int G, int K, int N, bool bf16)
{
    if (M == 0)
        return 0;
    size_t most = 0;
    for (const bool plain : {false, true}) {
        const GroupedCut v = grouped_cut(M, G, K, N, bf16, plain);
        const size_t all = v.d_bytes + v.part_bytes, bias = grouped_cut(M, G, 1, N, bf16, plain).part_bytes;
        most = all > most ? all : most;
        most = bias > most ? bias : most;
    }
    return most;
}

template <typename T, int KC, int NC, bool Plain, bool FromD>
static hipError_t launch_panel(const GroupedPanelArgs &p, hipStream_t stream)
{
    constexpr GroupedShape S = kGroupedShape<T, KC, NC, Plain>;
    if (S.lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(
            reinterpret_cast<const void *>(&grouped_panel_kernel<T, KC, NC, Plain, FromD>),
            hipFuncAttributeMaxDynamicSharedMemorySize, S.lds);
        if (e != hipSuccess)
            return e;
    }
    const int64_t total = static_cast<int64_t>(p.runs) * p.blocks;
    hipLaunchKernelGGL((grouped_panel_kernel<T, KC, NC, Plain, FromD>), dim3(static_cast<unsigned>((total + 7) / 8 * 8)),
                       dim3(64 * S.waves), S.lds, stream, p);
    return hipGetLastError();
}

template <typename T, bool Plain>
static hipError_t panel_by_shape(const GroupedPanelArgs &p, const GroupedCut &v, hipStream_t stream)
{
    if constexpr (!Plain)
        if (p.d)
            return launch_panel<T, 4, 4, false, true>(p, stream);
    switch (v.kc * 8 + v.nc) {
    case 9: return launch_panel<T, 1, 1, Plain, false>(p, stream);
    case 10: return launch_panel<T, 1, 2, Plain, false>(p, stream);
    case 12: return launch_panel<T, 1, 4, Plain, false>(p, stream);
    case 17: return launch_panel<T, 2, 1, Plain, false>(p, stream);
    case 18: return launch_panel<T, 2, 2, Plain, false>(p, stream);
    case 20: return launch_panel<T, 2, 4, Plain, false>(p, stream);
    case 33: return launch_panel<T, 4, 1, Plain, false>(p, stream);
    case 34: return launch_panel<T, 4, 2, Plain, false>(p, stream);
    default: return launch_panel<T, 4, 4, Plain, false>(p, stream);
    }
}

// d = gy act'(z) in float, dense rows
template <typename T>
__global__ void __launch_bounds__(256) grouped_slope_kernel(const LinearVjpArgs a, float *__restrict__ d)
{
    const int nv = (a.N + 7) / 8;
    const int64_t count = a.M * nv;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < count; i += gridDim.x * 256ll) {
        const int64_t r = i / nv;
        const int j = static_cast<int>(i - r * nv) * 8;
        float g[8], z[8];
        load8(static_cast<const T *>(a.gy) + r * a.ldgy + j, a.N - j, g);
        load8(static_cast<const T *>(a.z) + r * a.ldz + j, a.N - j, z);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            g[k] *= act_slope(a.act, z[k]);
        store8(d + r * a.N + j, a.N - j, g);
    }
}

template <typename T>
static hipError_t grouped_vjp(const GroupedLinearVjpArgs &ga, hipStream_t stream)
{
    const LinearVjpArgs &a = ga.v;
    const Groups gr{ga.group_ptr, ga.order, ga.n_groups, static_cast<int>(a.M)};
    const bool plain = a.act == kActNone, bf16 = sizeof(T) == 2;
    const int64_t set = (a.gW ? static_cast<int64_t>(a.K) * a.N : 0) + (a.gb ? a.N : 0);
    hipError_t e = hipSuccess;
    GroupedCut v{};
    GroupedPanelArgs p{a, gr, nullptr, 0, 1, 1, 1, 1, set};
    if (a.M > 0) {
        v = grouped_cut(a.M, gr.n, a.K, a.N, bf16, plain);
        if (!a.gW && !(v.fused && a.gx)) {
            v = grouped_cut(a.M, gr.n, 1, a.N, bf16, plain);
            v.fused = false;
        }
        p.tiles = v.tiles;
        p.per = v.per;
        p.runs = v.runs;
        p.nkb = v.nkb;
        p.blocks = v.nkb * v.nnb;
        if (!v.fused || set == 0) {
            // without the sums there is no workspace either: d as the product goes
            if (set > 0 && v.keep_d) {
                float *d = reinterpret_cast<float *>(static_cast<unsigned char *>(a.ws) + v.part_bytes);
                const int64_t blocks = (a.M * ((a.N + 7) / 8) + 255) / 256;
                hipLaunchKernelGGL(grouped_slope_kernel<T>, dim3(static_cast<unsigned>(blocks < 16384 ? blocks : 16384)),
                                   dim3(256), 0, stream, a, d);
                if ((e = hipGetLastError()) != hipSuccess)
                    return e;
                p.d = d;
            }
            if (a.gx) {
                const GroupedProductArgs g{{a.M, a.N, a.K, p.d ? p.d : a.gy, p.d ? a.N : a.ldgy, a.z, a.ldz, a.W,
                                            nullptr, a.act, nullptr, 0, a.gx, a.ldgx, nullptr, 0, a.accumulate},
                                           gr};
                e = p.d ? launch_product<T, Dense::GxD>(g, stream)
                    : plain ? launch_product<T, Dense::GxPlain>(g, stream)
                            : launch_product<T, Dense::Gx>(g, stream);
                if (e != hipSuccess)
                    return e;
            }
            p.v.gx = nullptr;
        }
        if (set > 0)
            e = plain ? panel_by_shape<T, true>(p, v, stream) : panel_by_shape<T, false>(p, v, stream);
    }
    if (e != hipSuccess || set == 0)
        return e;
    // groups without rows are zeroed by up to 1024 rows of workgroups
    const int rest = a.accumulate ? 0 : gr.n < 4096 ? (gr.n + 3) / 4 : 1024;
    if (p.runs - 1 + rest == 0)
        return hipSuccess;
    hipLaunchKernelGGL(grouped_join_kernel, dim3(static_cast<unsigned>((set + 63) / 64), p.runs - 1 + rest), dim3(256), 0,
                       stream, p, v.shift);
    return hipGetLastError();
}

hipError_t launch_grouped_linear(const GroupedLinearArgs &ga, hipStream_t stream)
{
    const LinearArgs &a = ga.l;
    if (a.M == 0)
        return hipSuccess;
    const GroupedProductArgs g{{a.M, a.K, a.N, a.x, a.ldx, nullptr, 0, a.W, a.bias, a.act, a.res, a.ldr, a.y, a.ldy,
                                a.z, a.ldz, false},
                               {ga.group_ptr, ga.order, ga.n_groups, static_cast<int>(a.M)}};
    return a.bf16 ? launch_product<bf16bits, Dense::Fwd>(g, stream) : launch_product<float, Dense::Fwd>(g, stream);
}

hipError_t launch_grouped_linear_vjp(const GroupedLinearVjpArgs &a, hipStream_t stream)
{
    return a.v.bf16 ? grouped_vjp<bf16bits>(a, stream) : grouped_vjp<float>(a, stream);
}

}  // namespace etp
