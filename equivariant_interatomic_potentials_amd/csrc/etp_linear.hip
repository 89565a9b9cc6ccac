// etp_linear.hip -- the linear layer with bias, activation and residual, and
// its VJP.
#include "etp_dense_product.hpp"

namespace etp {

// ---------------------------------------------------------------------------
// y = act(x W + bias) + res (forward) and gx = d W^T, d = gy act'(z) (input
// gradient) are one product: rows r of [M][KD] times a [KD][ND] matrix in
// float accumulators, with another first operand and another epilogue.
//
// Operands are swapped: the matrix is the first operand of the instruction
// and the rows are the second, so that a lane ends with consecutive columns
// of one row and stores them as one vector, and loads its eight consecutive
// k of a row straight from memory (each row of x is needed by one wave only;
// only the matrix goes through LDS, in fragment order: a lane's 16 bytes next
// to its neighbours').

// Contraction of at most 128: the workgroup keeps its columns of the matrix
// (nb, a multiple of 64) in LDS and its waves walk 16-row tiles, each on its
// own, without another barrier. The column blocks of a row range run side by
// side on one XCD (workgroups b and b + 8 share one), so that the rows are
// read from memory once. The products are a quarter of the time that the rows
// take to come and go, so what counts is loads ahead (the next tile's are in
// flight during this one's products) and whole 64-byte stores: 441172 x 64 x 64
// float with residual and z 105 us, 4.3 TB/s (a large copy: 5.0); 32768 x 128
// x 512 bf16 with z 25.5 us, 3.0 TB/s, of which 5 us are the launch's start and
// the matrix's way into LDS. grad_x alone, 441172 x 64 x 64: float 85 us, 4.0
// TB/s, bf16 33 us.
template <typename T, Dense D, int KC>
__global__ void __launch_bounds__(512) product_resident_kernel(const ProductArgs a, const int nb, const int nsplit)
{
    using Mx = MatrixLds<T, D>;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    bf16bits *matrix = reinterpret_cast<bf16bits *>(smem);  // [KC] chunks
    float *bias = reinterpret_cast<float *>(matrix + KC * Mx::chunk(nb));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int c = lane & 15, q = lane >> 4;
    const int b8 = blockIdx.x >> 3, s = b8 % nsplit;
    const int64_t stream = static_cast<int64_t>(b8 / nsplit) * 8 + (blockIdx.x & 7);
    const int64_t nstream = gridDim.x / nsplit, ntile = (a.M + 15) / 16;
    if (stream * waves >= ntile)
        return;  // the whole workgroup: padding of the last group of 8
    const int n0 = s * nb;
    RowChunk<T, D> next[KC];
    auto fetch = [&](int64_t tile) {
        const int64_t row = tile * 16 + c, rc = row < a.M ? row : a.M - 1;
#pragma unroll
        for (int kc = 0; kc < KC; ++kc)
            next[kc].load(a, rc, 32 * kc + 8 * q);
    };
    // the first rows are on their way while the matrix is laid out
    int64_t tile = stream * waves + wave;
    if (tile < ntile)
        fetch(tile);
    for (int i = threadIdx.x; i < KC * Mx::pieces(nb); i += blockDim.x) {
        const int kc = i / Mx::pieces(nb), j = i % Mx::pieces(nb);
        Raw8<T> v;
        Mx::load(a, j, nb, 32 * kc, n0, v);
        Mx::store(matrix + kc * Mx::chunk(nb), j, nb, v);
    }
    for (int i = threadIdx.x; i < nb; i += blockDim.x)
        bias[i] = a.bias && n0 + i < a.ND ? a.bias[n0 + i] : 0.f;
    lds_barrier();
    for (; tile < ntile; tile += nstream * waves) {
        Frag<kRowParts<T, D>> xf[KC][1];
#pragma unroll
        for (int kc = 0; kc < KC; ++kc)
            xf[kc][0] = next[kc].frag(a);
        if (tile + nstream * waves < ntile)
            fetch(tile + nstream * waves);
        const int64_t row = tile * 16 + c;
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

// Longer contractions: a workgroup of four waves (2 x 2) owns 32 RT rows and
// 128 columns and takes the contraction in chunks of 64 (32 where the rows
// have three parts), rows and matrix through LDS: whole rows per wave on the way in (a wave that loads
// 16 rows of 64 bytes each takes about three times as long as for 1 KiB
// without a gap), and each operand's parts formed once. One chunk lies in LDS
// while the next is on its way in registers; the workgroups that share a
// compute unit fill each other's barriers. RT = 2 is for grids that would
// leave compute units without work. Narrow results take 64 or 32 columns, the
// waves one below the other, where 128 would mostly multiply zeros: 441172 x
// 256 x 8 float 176 -> 98 us, 4.9 TB/s, x 64 bf16 129 -> 78 us, 4.3 TB/s. Wide
// ones are bound by LDS reads and matrix instructions taking turns: 32768 x
// 512 x 512 forward float 113 to 130 us (a library's float product of that
// size: 115 at its best rate), bf16 42 to 47 us.
template <typename T, Dense D, int RT, int kCols>
__global__ void __launch_bounds__(256, kCols == 128 ? 2 : kCols == 64 ? 3 : 4) product_stream_kernel(const ProductArgs a, const int ncol)
{
    using Mx = MatrixLds<T, D>;
    using Piece = RowPiece<T, D>;
    constexpr int PR = kRowParts<T, D>, SUB = kStreamSub<T, D>, kRows = 32 * RT;
    constexpr int WC = kCols == 128 ? 2 : 1, RW = RT * WC / 2, TW = kCols / 16 / WC;  // waves across, a wave's tiles
    constexpr int SR = 32 * SUB + 8, kPlane = kRows * SR;  // LDS rows (elements), a part
    constexpr int kItems = (Mx::pieces(kCols) + 255) / 256;  // matrix pieces per thread and 32 of the contraction
    const bool lays = Mx::pieces(kCols) % 256 == 0 || threadIdx.x < Mx::pieces(kCols);
    constexpr int RP = 32 * SUB / Piece::V, kRowItems = kRows * RP / 256;  // pieces of a row; per thread
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    bf16bits *rows = reinterpret_cast<bf16bits *>(smem), *matrix = rows + PR * kPlane;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    // the column blocks of a row block run side by side on one XCD
    const int b8 = blockIdx.x >> 3;
    const int64_t row0 = (static_cast<int64_t>(b8 / ncol) * 8 + (blockIdx.x & 7)) * kRows;
    if (row0 >= a.M)
        return;  // the whole workgroup
    const int n0 = (b8 % ncol) * kCols, wr = wave / WC * 16 * RW, wt = wave % WC * TW;  // this wave's rows, tiles

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
        for (int n = 0; n < kRowItems; ++n) {
            const int i = threadIdx.x + 256 * n;
            const int64_t row = row0 + i / RP;
            xn[n].load(a, row < a.M ? row : a.M - 1, it * 32 * SUB + i % RP * Piece::V);
        }
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
        const int64_t row = row0 + wr + 16 * r + c;
        float add[sizeof(T) == 4 ? 4 : 2][8];
        load_group_addend<T, D>(a, row, j0, q, add);
        f32x4 v[4][1] = {};  // 32 columns: the others are past ND
#pragma unroll
        for (int t = 0; t < TW; ++t)
            v[t][0] = acc[t][r];
        store_group<T, D>(a, row, j0, q, v, add);
    }
}

// Few rows and a long contraction: a workgroup owns 16 rows and 64 columns,
// its four waves take every fourth chunk of the contraction straight from
// memory (nothing of the matrix is shared within the workgroup), and the
// partial tiles are added in wave order through LDS. Taken where 64-row tiles
// would leave compute units without work; bound by the latency of its few
// loads.
template <typename T, Dense D>
__global__ void __launch_bounds__(256) product_thin_kernel(const ProductArgs a, const int ncol)
{
    __shared__ f32x4 part[3][4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int n0 = (blockIdx.x % ncol) * 64;
    const int64_t row = static_cast<int64_t>(blockIdx.x / ncol) * 16 + c, rc = row < a.M ? row : a.M - 1;
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

// Dynamic LDS beyond the runtime's default limit of 64 KiB has to be asked
// for, on the device at hand.
template <typename T, Dense D, int KC>
static hipError_t launch_resident(const ProductArgs &a, dim3 grid, dim3 block, size_t lds, int nb, int nsplit,
                                  hipStream_t stream)
{
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(
            reinterpret_cast<const void *>(&product_resident_kernel<T, D, KC>),
            hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL((product_resident_kernel<T, D, KC>), grid, block, lds, stream, a, nb, nsplit);
    return hipGetLastError();
}

// As many workgroups as LDS and 16 waves a compute unit let run at once, in
// eighths of the chip. (Kernels of more than 128 registers, most input gradients
// and the float forwards of more than 64 inputs, run 8 or 12 of those waves and
// leave the last workgroups to a second round.)
template <typename T, Dense D>
static hipError_t launch_resident_product(const ProductArgs &a, hipStream_t stream)
{
    const int kc = (a.KD + 31) / 32;
    const int nb = a.ND <= 64 ? 64 : 128, nsplit = (a.ND + nb - 1) / nb;
    const size_t lds = sizeof(bf16bits) * kc * MatrixLds<T, D>::chunk(nb) + nb * sizeof(float);
    const int waves = lds <= 40 * 1024 ? 4 : 8;
    const int per_cu = static_cast<int>(160 * 1024 / lds) < 16 / waves ? static_cast<int>(160 * 1024 / lds)
                                                                        : 16 / waves;
    int64_t streams = ((a.M + 15) / 16 + waves - 1) / waves;
    const int64_t most = kComputeUnits * per_cu / nsplit / 8 * 8;
    streams = (streams + 7) / 8 * 8;
    streams = streams < most ? streams : most < 8 ? 8 : most;
    const dim3 grid(static_cast<unsigned>(streams * nsplit)), block(64 * waves);
    switch (kc) {
    case 1: return launch_resident<T, D, 1>(a, grid, block, lds, nb, nsplit, stream);
    case 2: return launch_resident<T, D, 2>(a, grid, block, lds, nb, nsplit, stream);
    case 3: return launch_resident<T, D, 3>(a, grid, block, lds, nb, nsplit, stream);
    default: return launch_resident<T, D, 4>(a, grid, block, lds, nb, nsplit, stream);
    }
}

template <typename T, Dense D, int RT, int kCols>
static hipError_t launch_stream(const ProductArgs &a, int ncol, hipStream_t stream)
{
    constexpr int SUB = kStreamSub<T, D>;
    constexpr size_t lds = sizeof(bf16bits) * (kRowParts<T, D> * 32 * RT * (32 * SUB + 8) + SUB * MatrixLds<T, D>::chunk(kCols));
    static_assert(lds <= 64 * 1024);
    const int64_t blocks = (a.M + 32 * RT - 1) / (32 * RT);
    hipLaunchKernelGGL((product_stream_kernel<T, D, RT, kCols>), dim3(static_cast<unsigned>((blocks + 7) / 8 * 8 * ncol)),
                       dim3(256), lds, stream, a, ncol);
    return hipGetLastError();
}

template <typename T, Dense D>
static hipError_t launch_product(const ProductArgs &a, hipStream_t stream)
{
    const int64_t ntile = (a.M + 15) / 16;
    // (d is kept for layers of more than 128 inputs and outputs only)
    if constexpr (D != Dense::GxD) {
        if (a.KD <= 128)
            return launch_resident_product<T, D>(a, stream);
    }
    const int ncol = (a.ND + 127) / 128;
    const int64_t wide = (a.M + 127) / 128 * ncol, half = (a.M + 63) / 64 * ncol;
    if (half < kComputeUnits) {
        const int nc = (a.ND + 63) / 64;
        hipLaunchKernelGGL((product_thin_kernel<T, D>), dim3(static_cast<unsigned>(ntile * nc)), dim3(256), 0, stream,
                           a, nc);
        return hipGetLastError();
    }
    if constexpr (D != Dense::GxD) {
        if (a.ND <= 32)
            return wide < 2 * kComputeUnits ? launch_stream<T, D, 2, 32>(a, 1, stream)
                                            : launch_stream<T, D, 4, 32>(a, 1, stream);
        if (a.ND <= 64)
            return wide < 2 * kComputeUnits ? launch_stream<T, D, 2, 64>(a, 1, stream)
                                            : launch_stream<T, D, 4, 64>(a, 1, stream);
    }
    return wide < 2 * kComputeUnits ? launch_stream<T, D, 2, 128>(a, ncol, stream)
                                    : launch_stream<T, D, 4, 128>(a, ncol, stream);
}

// ---------------------------------------------------------------------------
// The VJP over panels of rows. A workgroup walks its panels: d and x are
// formed in registers from one read of gy, z and x, cut into bf16 parts and
// put into LDS row by row; then
//   gx = d W^T: the contraction runs along a row, so fragments of d are read
//     from LDS as they lie, and each wave keeps its columns of W in registers
//     for all panels;
//   gW += x^T d: the contraction runs along the rows; the transposing LDS
//     read (ds_read_b64_tr_b16) hands a lane four rows of one column, and the
//     result stays in the accumulators until the last panel.
// So each input is read once and only gx and one partial gW per workgroup are
// written (added by sum_parts_kernel in a fixed order). gb is summed in
// registers from d itself. With K and N above 128 the same kernel forms a 128
// x 128 block of gW per workgroup (no gx) from d made once by slope_kernel.
//
// With narrow layers HBM bounds it (5172508 x 64 x 64 bf16: 549 us, 4.8 TB/s).
// 131072 x 64 x 128 float: 55 us, 3.6 TB/s; of 100 thousand cycles the vector
// units (forming the parts) are busy for 49, LDS for 29, matrix instructions for
// 25, overlapped in part by the eight waves of the one workgroup a compute unit
// (two would fit LDS, but not the registers: 128 a lane, and spill). In 128 x
// 128 blocks (32768 x 512 x 512 bf16: 78 of the call's 156 us) it is 69, 57 and
// 49 of 151 thousand, again with one workgroup a compute unit; two would spill.
struct PanelArgs {
    LinearVjpArgs v;
    const float *d;   // d [M][N], or null: from gy and z
    int64_t npanel;
    int nsplit;       // workgroups along the panels
    int nkb;          // blocks of 32 KC along K (1 with gx)
    int blocks;       // of gW
    int64_t set;      // floats of a partial set: gW, then gb, of those that are wanted
};

// With eight waves and one workgroup a compute unit, two panels' parts lie in
// LDS, and while one feeds the products the next is formed and written: one
// barrier a panel, of 64 rows, or 32 where two of 64 do not fit. Otherwise one
// panel of 64 rows, so that several workgroups share a compute unit and fill
// each other's waits: for bf16 wherever their accumulators fit the registers
// (200000 x 128 x 64 takes 13% longer with one workgroup of two buffers; 128 x
// 128 would spill, 78 -> 132 us), for float up to 64 x 64.
struct PanelShape {
    int px, waves, sx, sd, bufs, rows, lds, per_cu;  // parts of x, row strides (elements), workgroups that fit
    constexpr PanelShape(bool bf16, int kc, int nc)
        : px(bf16 ? 1 : 3), waves(bf16 ? (kc == 4 && nc > 1 ? 8 : 4) : (kc == 4 || nc == 4 ? 8 : 4)), sx(32 * kc + 8), sd(32 * nc + 8),
          bufs(waves == 8 && !(bf16 && nc == 2) ? 2 : 1), rows(2 * bufs * 64 * (px * sx + 3 * sd) <= 144 * 1024 ? 64 : 32),
          lds(2 * bufs * rows * (px * sx + 3 * sd)),
          per_cu(waves == 8 ? 3 - bufs : 160 * 1024 / lds < 3 ? 160 * 1024 / lds : 3)
    {
    }
};
template <typename T, int KC, int NC>
constexpr PanelShape kPanelShape{sizeof(T) == 2, KC, NC};

template <typename T, int KC, int NC, bool FromD>
__global__ void __launch_bounds__((64 * kPanelShape<T, KC, NC>.waves),
                                  (kPanelShape<T, KC, NC>.waves / 4 * kPanelShape<T, KC, NC>.per_cu)) panel_kernel(const PanelArgs p)
{
    constexpr PanelShape S = kPanelShape<T, KC, NC>;
    constexpr int PX = S.px, W = S.waves, SX = S.sx, SD = S.sd, kRows = S.rows;
    constexpr int kBuf = kRows * (PX * SX + 3 * SD);  // elements of one panel
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    bf16bits *const lds = reinterpret_cast<bf16bits *>(smem);  // [bufs] of d [3][kRows][SD], x [PX][kRows][SX]
    const LinearVjpArgs &a = p.v;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    // workgroup i runs on XCD i % 8: the blocks that read the same panels run
    // on one of them, so that its L2 serves all but the first (with the splits
    // cut to one round it saved a quarter of 20000 x 384 x 1024 bf16). A
    // single block has nothing to share and walks in step (by XCD 5172508 x 64
    // x 64 bf16 takes 2.6% longer).
    const int total = p.nsplit * p.blocks, each = (total + 7) / 8;
    const int id = p.blocks > 1 ? (blockIdx.x & 7) * each + (blockIdx.x >> 3) : blockIdx.x;
    if (id >= total)
        return;
    const int s = id / p.blocks, blk = id % p.blocks;
    const int k0 = (blk % p.nkb) * 32 * KC, j0 = (blk / p.nkb) * 32 * NC;
    const int K = a.K, N = a.N;
    const bool want_gx = a.gx != nullptr, want_gw = a.gW != nullptr, want_gb = a.gb != nullptr && k0 == 0;

    // loads: a thread takes 16 bytes of the same columns in every ND-th (NX-th)
    // row of the panel, so that a wave covers whole rows (half the width a row
    // and wave costs a quarter of the bandwidth)
    using Src = std::conditional_t<FromD, float, T>;
    constexpr int kTiles = kRows / 16, VD = kVec<Src>, VX = kVec<T>;
    constexpr int DP = 32 * NC / VD, XP = 32 * KC / VX;   // pieces of a row
    constexpr int RD = 64 * W / DP, RX = 64 * W / XP;      // rows at a time
    constexpr int ND = (kRows + RD - 1) / RD, NX = (kRows + RX - 1) / RX;
    const int drow = threadIdx.x / DP, dcol = threadIdx.x % DP * VD;
    const int xrow = threadIdx.x / XP, xcol = threadIdx.x % XP * VX;
    RawVec<Src> gn[ND];
    RawVec<T> zn[ND], xn[NX];
    auto fetch = [&](int64_t panel) {
#pragma unroll
        for (int n = 0; n < ND; ++n) {
            const int64_t r = panel * kRows + drow + RD * n, rc = r < a.M ? r : a.M - 1;
            const int valid = N - j0 - dcol;
            if constexpr (FromD) {
                gn[n].load(p.d + rc * N + j0 + dcol, valid);
            } else {
                gn[n].load(static_cast<const T *>(a.gy) + rc * a.ldgy + j0 + dcol, valid);
                if (a.act != kActNone)
                    zn[n].load(static_cast<const T *>(a.z) + rc * a.ldz + j0 + dcol, valid);
            }
        }
        if (want_gw) {
#pragma unroll
            for (int n = 0; n < NX; ++n) {
                const int64_t r = panel * kRows + xrow + RX * n, rc = r < a.M ? r : a.M - 1;
                xn[n].load(static_cast<const T *>(a.x) + rc * a.ldx + k0 + xcol, K - k0 - xcol);
            }
        }
    };

    // gx: a wave owns G column tiles (a pair for bf16, whose lanes store eight
    // columns) and RT of the row tiles
    constexpr int G = sizeof(T) == 4 ? 1 : 2, groups = 2 * KC / G, RS0 = W / groups, RS = RS0 < kTiles ? RS0 : kTiles;
    constexpr int RT = kTiles / RS;
    const int grp = wave % groups, rt0 = (wave / groups) * RT;
    const bool gx_wave = want_gx && wave / groups < RS;
    Frag<PX> wf[NC][G];
    if (gx_wave) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const int k = sizeof(T) == 4 ? 16 * grp + c : 32 * grp + 8 * (c >> 2) + 4 * g + (c & 3);
                const int j = 32 * n + 8 * q;
                Raw8<T> raw;
                raw.load(static_cast<const T *>(a.W) + static_cast<int64_t>(k < K ? k : 0) * N + j,
                         k < K ? N - j : 0);
                wf[n][g] = raw.template frag<PX>();
            }
    }

    // gW: waves as WK x WN, each KT x JT tiles of 16 x 16
    constexpr int WN = W == 4 || NC == 1 ? 2 : 4, WK = W / WN, KT = 2 * KC / WK, JT = 2 * NC / WN;
    const int kt0 = (wave / WN) * KT, jt0 = (wave % WN) * JT;
    f32x4 acc[KT][JT];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int j = 0; j < JT; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    float gb[VD];
#pragma unroll
    for (int i = 0; i < VD; ++i)
        gb[i] = 0.f;

    // the fetched panel's parts into LDS
    auto put = [&](int64_t panel, bf16bits *dl) __attribute__((always_inline)) {
        bf16bits *xl = dl + 3 * kRows * SD;
#pragma unroll
        for (int n = 0; n < ND; ++n) {
            const int row = drow + RD * n;
            if (kRows % RD && row >= kRows)
                continue;
            const bool live = panel * kRows + row < a.M;
            float d[VD];
#pragma unroll
            for (int i = 0; i < VD; ++i) {
                d[i] = gn[n].get(i);
                if (!FromD && a.act != kActNone)
                    d[i] *= act_slope(a.act, zn[n].get(i));
                d[i] = live ? d[i] : 0.f;
                gb[i] += d[i];
            }
            put_parts<3, kCut<T>>(dl + row * SD + dcol, kRows * SD, d);
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

    if (s < p.npanel) {
        fetch(s);
        if (S.bufs == 2) {
            put(s, lds);
            if (s + p.nsplit < p.npanel)
                fetch(s + p.nsplit);
        }
    }
    int buf = 0;
    for (int64_t panel = s; panel < p.npanel; panel += p.nsplit, buf ^= S.bufs - 1) {
        if (S.bufs == 1) {
            put(panel, lds);
            if (panel + p.nsplit < p.npanel)
                fetch(panel + p.nsplit);
        }
        // the panel's parts are seen by every wave; of two buffers the one
        // written next was last read before this barrier
        lds_barrier();
        const bf16bits *dl = lds + buf * kBuf, *xl = dl + 3 * kRows * SD;
        if (S.bufs == 2 && panel + p.nsplit < p.npanel) {
            put(panel + p.nsplit, lds + (buf ^ 1) * kBuf);
            if (panel + 2 * p.nsplit < p.npanel)
                fetch(panel + 2 * p.nsplit);
        }
        if (gx_wave) {
            f32x4 o[G][RT];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    o[g][r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                Frag<3> df[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int t = 0; t < 3; ++t)
                        df[r].p[t] = *reinterpret_cast<const bf16x8 *>(
                            dl + (t * kRows + 16 * (rt0 + r) + c) * SD + 32 * n + 8 * q);
                mma(wf[n], df, o);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int64_t row = panel * kRows + 16 * (rt0 + r) + c;
                const int k = sizeof(T) == 4 ? 16 * grp + 4 * q : 32 * grp + 8 * q;
                if (row < a.M && k < K) {
                    T *dst = static_cast<T *>(a.gx) + row * a.ldgx + k;
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
                Frag<3> df[JT];
#pragma unroll
                for (int j = 0; j < JT; ++j)
#pragma unroll
                    for (int t = 0; t < 3; ++t)
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
        if (S.bufs == 1)
            lds_barrier();  // the next panel overwrites the rows
    }
    if (S.bufs == 2)
        lds_barrier();  // the sums below reuse the space

    float *part = static_cast<float *>(a.ws) + s * p.set;
    if (want_gw) {
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                const int jj = j0 + 16 * (jt0 + j) + c;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int k = k0 + 16 * (kt0 + i) + 4 * q + r;
                    if (k < K && jj < N)
                        part[static_cast<int64_t>(k) * N + jj] = acc[i][j][r];
                }
            }
    }
    if (want_gb) {
        // the threads that share columns, through LDS, in row order
        float *sums = reinterpret_cast<float *>(smem);  // [RD][32 NC]
        static_assert(RD * 32 * NC * sizeof(float) <= static_cast<size_t>(S.lds));
#pragma unroll
        for (int i = 0; i < VD; ++i)
            sums[drow * 32 * NC + dcol + i] = gb[i];
        lds_barrier();
        for (int j = threadIdx.x; j < 32 * NC; j += 64 * W) {
            float v = 0.f;
            for (int r = 0; r < RD; ++r)
                v += sums[r * 32 * NC + j];
            if (j0 + j < N)
                part[p.set - N + j0 + j] = v;
        }
    }
}

// d = gy act'(z) in float, dense rows: 32768 x 512 bf16, 27 us at 4.9 TB/s.
// (Kept as three bf16 parts instead, the blocks' vector work shrinks and their
// reads grow by half: the call of 32768 x 512 x 512 took 1% less for bf16 and 3%
// more for float.)
template <typename T>
__global__ void __launch_bounds__(256) slope_kernel(const LinearVjpArgs a, float *__restrict__ d)
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

// out0, out1 (+)= the sums over n sets of n0 + n1 partial values: Cols columns
// of Ways threads a workgroup; a thread adds every Ways-th set in order, then
// the Ways sums are added as a tree (short chains keep a long sum's rounding
// down and its reads in flight together). Ways = 64 for more than 64 sets: 5 us
// for 512 sets of 64 x 65.
template <int Cols, int Ways>
__global__ void __launch_bounds__(Cols * Ways) sum_parts_kernel(const int64_t n0, float *out0, const int64_t n1,
                                                                float *out1, const int n,
                                                                const float *__restrict__ part, const int accumulate)
{
    __shared__ float lds[Ways][Cols + 1];
    const int tx = threadIdx.x % Cols, ty = threadIdx.x / Cols;
    const int64_t count = n0 + n1, i = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * Cols + tx;
    float v = 0.f;
    if (i < count) {
        int s = ty;
        for (; s + 3 * Ways < n; s += 4 * Ways) {
            float u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                u[k] = part[(s + k * Ways) * count + i];
            v += (u[0] + u[1]) + (u[2] + u[3]);
        }
        for (; s < n; s += Ways)
            v += part[s * count + i];
    }
    lds[ty][tx] = v;
    for (int d = Ways / 2; d; d >>= 1) {
        lds_barrier();
        if (ty < d)
            lds[ty][tx] += lds[ty + d][tx];
    }
    if (ty > 0 || i >= count)
        return;
    float *o = i < n0 ? out0 : out1;
    if (!o)
        return;
    o += i < n0 ? i : i - n0;
    *o = accumulate ? *o + lds[0][tx] : lds[0][tx];
}

hipError_t launch_sum_parts(int64_t n0, float *out0, int64_t n1, float *out1, int n, const float *part,
                            bool accumulate, hipStream_t stream)
{
    const int64_t count = n0 + n1;
    auto grid = [count](int cols) {  // a launch takes fewer than 2^32 threads along x
        const int64_t blocks = (count + cols - 1) / cols, x = blocks < (1 << 20) ? blocks : 1 << 20;
        return dim3(static_cast<unsigned>(x), static_cast<unsigned>((blocks + x - 1) / x));
    };
    if (n > 64)
        hipLaunchKernelGGL((sum_parts_kernel<16, 64>), grid(16), dim3(1024), 0,
                           stream, n0, out0, n1, out1, n, part, accumulate ? 1 : 0);
    else
        hipLaunchKernelGGL((sum_parts_kernel<64, 4>), grid(64), dim3(256), 0,
                           stream, n0, out0, n1, out1, n, part, accumulate ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_linear(const LinearArgs &a, hipStream_t stream)
{
    if (a.M == 0)
        return hipSuccess;
    const ProductArgs p{a.M, a.K, a.N, a.x, a.ldx, nullptr, 0, a.W, a.bias, a.act, a.res, a.ldr,
                        a.y, a.ldy, a.z, a.ldz, false};
    return a.bf16 ? launch_product<bf16bits, Dense::Fwd>(p, stream) : launch_product<float, Dense::Fwd>(p, stream);
}

// How a VJP call is cut: all in one panel kernel where K and N are at most
// 128, else gx as a product and gW in blocks of up to 128 x 128, with d made
// once before both where K and N are above 128 (where only one is, forming d
// again costs less than keeping it). gb without gW needs the blocks along N
// only, as if there were one input (gx is a product of its own then, unless
// the one panel kernel forms it on the way).
struct VjpCut {
    bool fused, keep_d;  // one kernel for all; d made once
    int kc, nc;          // chunks of 32 of a block: 1, 2 or 4
    int nkb, nnb;        // blocks along K and N
    int64_t npanel;
    int nsplit;          // panel streams, and partial sets
    size_t d_bytes, part_bytes;
};

static VjpCut vjp_cut(int64_t M, int K, int N, bool bf16)
{
    VjpCut v{};
    auto chunks = [](int n) { return n <= 32 ? 1 : n <= 64 ? 2 : 4; };
    v.kc = chunks(K);
    v.nc = chunks(N);
    v.nkb = (K + 127) / 128;
    v.nnb = (N + 127) / 128;
    v.fused = K <= 128 && N <= 128;
    const PanelShape shape(bf16, v.kc, v.nc);
    v.npanel = (M + shape.rows - 1) / shape.rows;
    // as many splits as run at once (one more would double the time), or over
    // up to four rounds where that fills them better by a tenth
    const int64_t blocks = static_cast<int64_t>(v.nkb) * v.nnb, room = static_cast<int64_t>(kComputeUnits) * shape.per_cu;
    int64_t s = 0, rounds = 1;
    for (int64_t n = 1; n <= 4; ++n) {
        const int64_t t = n * room / blocks;
        if (s == 0 ? t > 0 : 10 * n * s < 9 * rounds * t) {
            s = t;
            rounds = n;
        }
    }
    s = s < v.npanel ? s : v.npanel;
    v.nsplit = static_cast<int>(s < 1 ? 1 : s);
    v.keep_d = K > 128 && N > 128;
    v.d_bytes = v.keep_d ? (sizeof(float) * static_cast<size_t>(M) * N + 15) / 16 * 16 : 0;
    v.part_bytes = sizeof(float) * static_cast<size_t>(v.nsplit) * (static_cast<size_t>(K) + 1) * N;
    return v;
}

size_t linear_vjp_workspace_bytes(int64_t M, int K, int N, bool bf16)
{
    if (M == 0)
        return 0;
    const VjpCut v = vjp_cut(M, K, N, bf16);
    const size_t all = v.d_bytes + v.part_bytes, bias = vjp_cut(M, 1, N, bf16).part_bytes;
    return all > bias ? all : bias;
}

template <typename T, int KC, int NC, bool FromD>
static hipError_t launch_panel(const PanelArgs &p, hipStream_t stream)
{
    constexpr PanelShape S = kPanelShape<T, KC, NC>;
    if (S.lds > 64 * 1024) {
        const hipError_t e =
            hipFuncSetAttribute(reinterpret_cast<const void *>(&panel_kernel<T, KC, NC, FromD>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, S.lds);
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL((panel_kernel<T, KC, NC, FromD>), dim3(static_cast<unsigned>((p.nsplit * p.blocks + 7) / 8 * 8)),
                       dim3(64 * S.waves), S.lds, stream, p);
    return hipGetLastError();
}

template <typename T>
static hipError_t panel_by_shape(const PanelArgs &p, const VjpCut &v, hipStream_t stream)
{
    if (p.d)
        return launch_panel<T, 4, 4, true>(p, stream);
    switch (v.kc * 8 + v.nc) {
    case 9: return launch_panel<T, 1, 1, false>(p, stream);
    case 10: return launch_panel<T, 1, 2, false>(p, stream);
    case 12: return launch_panel<T, 1, 4, false>(p, stream);
    case 17: return launch_panel<T, 2, 1, false>(p, stream);
    case 18: return launch_panel<T, 2, 2, false>(p, stream);
    case 20: return launch_panel<T, 2, 4, false>(p, stream);
    case 33: return launch_panel<T, 4, 1, false>(p, stream);
    case 34: return launch_panel<T, 4, 2, false>(p, stream);
    default: return launch_panel<T, 4, 4, false>(p, stream);
    }
}

template <typename T>
static hipError_t linear_vjp(const LinearVjpArgs &a, const VjpCut &v, int64_t set, hipStream_t stream)
{
    const bool sums = set > 0;
    PanelArgs p{a, nullptr, v.npanel, v.nsplit, v.nkb, v.nkb * v.nnb, set};
    hipError_t e = hipSuccess;
    if (!v.fused || !sums) {
        // without the sums there is no workspace either: d as the product goes
        if (sums && v.keep_d && a.act != kActNone) {
            float *d = reinterpret_cast<float *>(static_cast<unsigned char *>(a.ws) + v.part_bytes);
            const int64_t blocks = (a.M * ((a.N + 7) / 8) + 255) / 256;
            hipLaunchKernelGGL(slope_kernel<T>, dim3(static_cast<unsigned>(blocks < 16384 ? blocks : 16384)),
                               dim3(256), 0, stream, a, d);
            if ((e = hipGetLastError()) != hipSuccess)
                return e;
            p.d = d;
        }
        if (a.gx) {
            const ProductArgs g{a.M, a.N, a.K, p.d ? p.d : a.gy, p.d ? a.N : a.ldgy, a.z, a.ldz, a.W, nullptr, a.act,
                                nullptr, 0, a.gx, a.ldgx, nullptr, 0, a.accumulate};
            e = p.d ? launch_product<T, Dense::GxD>(g, stream) : launch_product<T, Dense::Gx>(g, stream);
        }
        p.v.gx = nullptr;
    }
    return e == hipSuccess && sums ? panel_by_shape<T>(p, v, stream) : e;
}

hipError_t launch_linear_vjp(const LinearVjpArgs &a, hipStream_t stream)
{
    const int64_t n0 = a.gW ? static_cast<int64_t>(a.K) * a.N : 0, n1 = a.gb ? a.N : 0;
    hipError_t e = hipSuccess;
    int nsplit = 0;
    if (a.M > 0) {
        VjpCut v = vjp_cut(a.M, a.K, a.N, a.bf16);
        if (!a.gW && !(v.fused && a.gx)) {
            v = vjp_cut(a.M, 1, a.N, a.bf16);
            v.fused = false;
        }
        nsplit = v.nsplit;
        e = a.bf16 ? linear_vjp<bf16bits>(a, v, n0 + n1, stream) : linear_vjp<float>(a, v, n0 + n1, stream);
    }
    if (e == hipSuccess && n0 + n1 > 0)
        e = launch_sum_parts(n0, a.gW, n1, a.gb, nsplit, static_cast<const float *>(a.ws), a.accumulate, stream);
    return e;
}

}  // namespace etp
