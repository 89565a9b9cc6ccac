// etp_grouped_vjp.hip -- the VJP of the linear layer with a matrix for each group
// of rows.
#include "etp_grouped.hpp"

namespace etp {

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
// that order by grouped_join_kernel. (Runs of whole panels, not of whole groups: ends
// moved to the nearer group's end save the parts and lose as much to uneven runs.)
//
// The sums of a long group are no one chain of float additions: the matrix instruction
// drops what lies below its accumulator's last place, always to the same side, so that
// 100000 rows in one accumulator were 8e-4 of the result off where all terms are alike
// (the atoms of a crystal). After `fold` panels they are added to the sums so far, and
// parts are joined in double: 1.7e-5 at any number of rows.
//
// 5172508 x 64 x 64 bf16 in 16 groups without activation: 411 us, 4.8 TB/s, a copy's
// rate. 131072 x 64 x 128 float in 25 groups: 66 us, 3.1 TB/s; of 162 thousand cycles
// vector instructions take 48, LDS 36 and matrix instructions 25, and waves wait for 45%
// of theirs: forming the parts, storing them and the products of one workgroup a compute
// unit take turns. 32768 x 512 x 512 bf16 in 64 groups with SiLU: d 29, gx 73, gW 119 us
// and the join 19. gW and gx have three products a term, 13 us each at the matrix rate;
// in gW's 280 thousand cycles LDS is busy for 107, vector instructions for 74 and matrix
// ones for 52, again in turns (waves wait for 45%); in gx' 165 LDS for 103, vector
// instructions for 61, matrix ones for 52. (d kept as parts and brought straight into
// LDS: gW 103, but gx 88 and d 31.)
//
// No instance spills vector registers. (The masks and places of a block's entries, which
// the compiler forms before the panels if it can, once took 20 to 40 of them.)
struct GroupedPanelArgs {
    LinearVjpArgs v;  // W, gW, gb of group 0
    Groups gr;
    const float *d;  // d [rows][N], or null: from gy and z
    int tiles, per;  // tile numbers, and how many of them a run has
    int runs;
    int nkb, blocks;  // blocks along K, and in all
    int64_t set;      // floats of a partial set: gW, then gb, of those that are wanted
    int fold;         // panels of a chain
};

// Parts of x and d, waves, LDS rows (elements), buffers, panel rows, LDS bytes
// and workgroups of a compute unit. The rules are the linear layer's.
struct GroupedShape {
    int px, pd, waves, sx, sd, bufs, rows, shift, lds, per_cu;
    constexpr GroupedShape(bool bf16, int kc, int nc, bool plain)
        : px(bf16 ? 1 : 3), pd(bf16 && plain ? 1 : 3),
          waves(bf16 ? (kc == 4 && nc > 1 ? 8 : 4) : (kc == 4 || (nc == 4 && !plain) ? 8 : 4)), sx(32 * kc + 8), sd(32 * nc + 8),
          bufs(waves == 8 ? 2 : 1),
          rows(!bf16 && waves == 4 && nc == 4 ? 32 : 2 * bufs * 64 * (px * sx + pd * sd) <= 144 * 1024 ? 64 : 32), shift(rows == 64 ? 6 : 5),
          lds(2 * bufs * rows * (px * sx + pd * sd)),
          per_cu(waves == 8 ? 1 : (bf16 && kc == 4) || nc == 4 ? 2 : 160 * 1024 / lds < 3 ? 160 * 1024 / lds : 3)
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
    // (d is kept where gx is a product of its own)
    const bool want_gx = !FromD && a.gx != nullptr, want_gw = a.gW != nullptr, want_gb = a.gb != nullptr && k0 == 0;
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
    // The chains of a group are added up in registers where a block is 128 x 128 (two waves
    // a SIMD; through memory 65536 x 512 x 512 float in 8 groups takes 607 us, so 594), else
    // where the group's sums go (in registers 441172 x 64 x 64 bf16 takes 78 us, so 74).
    constexpr bool kHolds = KC == 4 && NC == 4;
    f32x4 acc[KT][JT], held[kHolds ? KT : 1][kHolds ? JT : 1];
    float gb[VD], gb_held[VD];
    auto end_chain = [&](bool first) __attribute__((always_inline)) {
        if constexpr (kHolds) {
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    held[i][j] = first ? acc[i][j] : held[i][j] + acc[i][j];
                    acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
#pragma unroll
            for (int i = 0; i < VD; ++i) {
                gb_held[i] = first ? gb[i] : gb_held[i] + gb[i];
                gb[i] = 0.f;
            }
        }
    };

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

    // the panel whose products come next, and the two after it; rows name their rows.
    // Values are fetched one panel ahead (two with two buffers), indexes one more
    TileWalk at, then, after;
    at.start(p.gr, S.shift, from, stop);
    if (at.n == 0)
        return;  // the whole workgroup
    auto rows_of = [&](const TileWalk &w) { return row_of_slot(p.gr, w.slot + lane, lane < w.n); };
    int rows = rows_of(at);
    fetch(rows);
    then = at;
    then.next(p.gr, S.shift, stop);
    int rows_then = rows_of(then);
    after = then;
    if (then.n > 0)
        after.next(p.gr, S.shift, stop);
    int rows_after = rows_of(after);
    bool begun = false;  // the group has sums in memory
    while (at.n > 0) {   // a group, or a chain of it; the registers hold the first panel
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
        end_chain(true);
        int buf = 0, left = p.fold;
        if constexpr (S.bufs == 2) {
            lds_barrier();  // of the group before: its sums or its last panel
            put(lds);
            if (then.n > 0)
                fetch(rows_then);
        }
        for (bool same = true; same;) {
            same = then.n > 0 && then.g == g && (kHolds || left > 1);
            if constexpr (S.bufs == 1) {
                put(lds);
                if (then.n > 0)
                    fetch(rows_then);
            }
            lds_barrier();  // the panel's parts are seen by every wave
            if constexpr (S.bufs == 2) {
                // the other buffer was last read before this barrier
                if (same) {
                    put(lds + (buf ^ 1) * kBuf);
                    if (after.n > 0)
                        fetch(rows_after);
                }
            }
            products(lds + buf * kBuf, rows);
            buf ^= S.bufs - 1;
            if (--left == 0) {
                end_chain(false);
                left = p.fold;
            }
            at = then;
            rows = rows_then;
            then = after;
            rows_then = rows_after;
            if (then.n > 0) {
                after.next(p.gr, S.shift, stop);
                rows_after = rows_of(after);
            }
            if constexpr (S.bufs == 1)
                lds_barrier();  // the next panel overwrites the rows
        }
        // the group's sums, or what they grow by
        if constexpr (kHolds) {
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int j = 0; j < JT; ++j)
                    acc[i][j] += held[i][j];
#pragma unroll
            for (int i = 0; i < VD; ++i)
                gb[i] += gb_held[i];
        }
        float *gw = nullptr, *gbias = nullptr;
        bool add = begun;
        if (whole) {
            gw = want_gw ? a.gW + static_cast<int64_t>(g) * K * N : nullptr;
            gbias = want_gb ? a.gb + static_cast<int64_t>(g) * N : nullptr;
            add |= a.accumulate;
        } else {
            float *part = static_cast<float *>(a.ws) + set * p.set;
            gw = part;
            gbias = part + p.set - N;
        }
        if (want_gw) {
            // the lane's first entry, opaque: else the places and masks of all its entries are
            // formed once for all groups and held in registers through the panels (441172 x
            // 64 x 64 bf16 with SiLU 79 us, so 74)
            int kl = k0 + 16 * kt0 + 4 * q, jl = j0 + 16 * jt0 + c;
            asm volatile("" : "+v"(kl), "+v"(jl));
            if (add) {
                // read together, a row of tiles at a time; past the matrix anything (not stored)
#pragma unroll
                for (int i = 0; i < KT; ++i) {
                    float was[JT][4];
#pragma unroll
                    for (int j = 0; j < JT; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int k = kl + 16 * i + r, jj = jl + 16 * j;
                            was[j][r] = gw[k < K && jj < N ? static_cast<int64_t>(k) * N + jj : 0];
                        }
#pragma unroll
                    for (int j = 0; j < JT; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[i][j][r] += was[j][r];
                }
            }
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int j = 0; j < JT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int k = kl + 16 * i + r, jj = jl + 16 * j;
                        if (k < K && jj < N)
                            gw[static_cast<int64_t>(k) * N + jj] = acc[i][j][r];
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
        begun = !kHolds && at.n > 0 && at.g == g;
    }
}

// Four entries from i of a group's sums: its gradients of W, then of the bias.
__device__ __forceinline__ void store_sums(const GroupedPanelArgs &p, int64_t g, int64_t i, const float (&v)[4], bool add)
{
    const LinearVjpArgs &a = p.v;
    const int64_t nw = p.set - (a.gb ? a.N : 0);
    if (i + 4 <= nw) {
        float *o = a.gW + g * nw + i, sum[8] = {v[0], v[1], v[2], v[3]};
        if (add) {
            float was[8];
            load_n<4>(o, 4, was);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sum[k] += was[k];
        }
        store_n<4>(o, 4, sum);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (i + k < p.set) {
            float *o = i + k < nw ? a.gW + g * nw + i + k : a.gb + g * a.N + (i + k - nw);
            *o = add ? *o + v[k] : v[k];
        }
}

// Adds the parts of the groups that cross runs, `span` entries a workgroup, four a
// lane at a time, every wave a quarter of the parts in order, in double (there may be
// thousands); and zeroes the gradients of groups without rows. Where there are few groups, row y of the grid is
// group y; else rows up to runs - 1 are the boundaries between runs, and a boundary
// stands for the group that crosses it if that crosses no earlier one, and the other
// rows look for groups without rows (25 groups in 512 runs by boundaries: 18 us, of
// which most find their group and leave; by groups 5).
__global__ void __launch_bounds__(256) grouped_join_kernel(const GroupedPanelArgs p, const int shift, const int by_group, const int span)
{
    __shared__ double lds[3][64][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t from = static_cast<int64_t>(blockIdx.x) * span, stop = from + span < p.set ? from + span : p.set;
    auto zero = [&](int g) {
        const float none[4] = {0.f, 0.f, 0.f, 0.f};
        for (int64_t i = from + 4 * threadIdx.x; i < stop; i += 1024)
            store_sums(p, g, i, none, false);
    };
    int g = blockIdx.y;
    if (!by_group) {
        const int bounds = p.runs - 1, y = blockIdx.y;
        if (y >= bounds) {
            for (g = y - bounds; g < p.gr.n; g += gridDim.y - bounds)
                if (group_start(p.gr, g + 1) <= group_start(p.gr, g))
                    zero(g);
            return;
        }
        g = group_of_tile(p.gr, shift, (y + 1) * p.per);
    }
    const int begin = group_start(p.gr, g), end = group_start(p.gr, g + 1);
    if (end <= begin) {
        if (by_group && !p.v.accumulate)
            zero(g);
        return;
    }
    const int first = (begin >> shift) + g, last = first + ((end - begin - 1) >> shift);
    const int run0 = first / p.per, run1 = last / p.per;
    if (run0 == run1 || (!by_group && run0 != static_cast<int>(blockIdx.y)))
        return;
    for (int64_t i0 = from; i0 < stop; i0 += 256) {
        const int64_t i = i0 + 4 * lane;
        const float *part = static_cast<const float *>(p.v.ws) + i;
        const int valid = stop - i < 4 ? static_cast<int>(stop - i) : 4;
        double v[4] = {0.0, 0.0, 0.0, 0.0};
        if (valid > 0) {
#pragma unroll 4
            for (int r = run0 + wave; r <= run1; r += 4) {
                float u[8];
                load_n<4>(part + (2 * static_cast<int64_t>(r) + (r == run0 ? 1 : 0)) * p.set, valid, u);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] += u[k];
            }
        }
        if (i0 > from)
            lds_barrier();  // the sums before have been read
        if (wave > 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                lds[wave - 1][lane][k] = v[k];
        }
        lds_barrier();
        if (wave == 0 && valid > 0) {
            float sum[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sum[k] = static_cast<float>((v[k] + lds[0][lane][k]) + (lds[1][lane][k] + lds[2][lane][k]));
            store_sums(p, g, i, sum, p.v.accumulate);
        }
    }
}

// How a VJP call is cut: as the linear layer's, in one panel kernel where K and N
// are at most 128, else gx as a product and gW in blocks of up to 128 x 128, with
// d made once before both where K and N are above 128 and there is an activation.
struct GroupedCut {
    bool fused, keep_d;
    int kc, nc, nkb, nnb;
    int shift, tiles, per, runs, fold;
    size_t d_bytes, part_bytes;
};

// Panels of a chain: at most 256 results of matrix instructions on top of each other
// (32 rows take six in a float layer, three in a bf16 one, one without an activation).
// Shorter ones cost: with half of it 5172508 x 64 x 64 bf16 takes 8 us more.
static int chain_panels(bool bf16, bool plain, int shift)
{
    return (!bf16 ? 1344 : plain ? 8192 : 2688) >> shift;
}
constexpr int kChains = 32;  // of a group in one run

// Runs for a tile size and a number of workgroups that run at once: as many as those
// (one more would double the time), or over up to four rounds where that fills them
// better by a tenth; more where one would take a group in more than kChains chains.
static void cut_runs(GroupedCut &v, int64_t M, int G, int K, int N, int shift, int per_cu, int chain)
{
    v.shift = shift;
    v.tiles = static_cast<int>((M >> shift) + G);
    const int64_t blocks = static_cast<int64_t>(v.nkb) * v.nnb, room = static_cast<int64_t>(kComputeUnits) * per_cu;
    int64_t s = 0, rounds = 1;
    for (int64_t n = 1; n <= 4; ++n) {
        const int64_t t = n * room / blocks;
        if (s == 0 ? t > 0 : 10 * n * s < 9 * rounds * t) {
            s = t;
            rounds = n;
        }
    }
    // panels that one group may have, and in a run of as many chains as may be
    const int most = static_cast<int>((M - 1) >> shift) + 1, run = kChains * chain;
    const int64_t least = most > run ? (v.tiles + run - 1) / run : 1;
    s = s < least ? least : s;
    s = s < v.tiles ? s : v.tiles;
    v.per = static_cast<int>((v.tiles + s - 1) / s);
    v.runs = (v.tiles + v.per - 1) / v.per;
    // chains of like length
    const int longest = v.per < most ? v.per : most, chains = (longest + chain - 1) / chain;
    v.fold = (longest + chains - 1) / chains;
    // (of one run every group's sums go straight to the gradients)
    const size_t sets = v.runs > 1 ? 2 * static_cast<size_t>(v.runs) : 0;
    v.part_bytes = sizeof(float) * sets * (static_cast<size_t>(K) + 1) * N;
    v.part_bytes = (v.part_bytes + 15) / 16 * 16;
}

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
    cut_runs(v, M, G, K, N, shape.shift, shape.per_cu, chain_panels(bf16, plain, shape.shift));
    v.keep_d = K > 128 && N > 128 && !plain;
    v.d_bytes = v.keep_d ? (sizeof(float) * static_cast<size_t>(M) * N + 15) / 16 * 16 : 0;
    return v;
}

size_t grouped_linear_vjp_workspace_bytes(int64_t M, int G, int K, int N, bool bf16)
{
    if (M == 0)
        return 0;
    size_t most = 0;
    auto take = [&](const GroupedCut &v) { most = v.d_bytes + v.part_bytes > most ? v.d_bytes + v.part_bytes : most; };
    for (const bool plain : {false, true}) {
        take(grouped_cut(M, G, K, N, bf16, plain));
        take(grouped_cut(M, G, 1, N, bf16, plain));  // the bias gradient alone
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

static hipError_t launch_join(const GroupedPanelArgs &p, int shift, hipStream_t stream)
{
    const int n = p.gr.n;
    const bool by_group = n <= 4 * p.runs;
    // groups without rows are looked for by up to 1024 rows of workgroups
    const int rest = p.v.accumulate ? 0 : n < 1024 ? n : 1024;
    const int rows = by_group ? n : p.runs - 1 + rest;
    if (rows == 0)
        return hipSuccess;
    // (more entries a workgroup where most workgroups would only find nothing to do)
    const int span = p.set * rows <= (1 << 22) ? 256 : 1024;
    hipLaunchKernelGGL(grouped_join_kernel, dim3(static_cast<unsigned>((p.set + span - 1) / span), rows), dim3(256), 0,
                       stream, p, shift, by_group ? 1 : 0, span);
    return hipGetLastError();
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
    GroupedPanelArgs p{a, gr, nullptr, 0, 1, 1, 1, 1, set, 1};
    if (a.M > 0) {
        v = grouped_cut(a.M, gr.n, a.K, a.N, bf16, plain);
        if (!a.gW && !(v.fused && a.gx)) {
            v = grouped_cut(a.M, gr.n, 1, a.N, bf16, plain);
            v.fused = false;
        }
        p.tiles = v.tiles;
        p.per = v.per;
        p.runs = v.runs;
        p.fold = v.fold;
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
                e = p.d ? launch_grouped_product<T, Dense::GxD>(g, stream)
                    : plain ? launch_grouped_product<T, Dense::GxPlain>(g, stream)
                            : launch_grouped_product<T, Dense::Gx>(g, stream);
                if (e != hipSuccess)
                    return e;
            }
            p.v.gx = nullptr;
        }
        if (set > 0)
            e = plain ? panel_by_shape<T, true>(p, v, stream) : panel_by_shape<T, false>(p, v, stream);
    }
    return e == hipSuccess && set > 0 ? launch_join(p, v.shift, stream) : e;
}

hipError_t launch_grouped_linear_vjp(const GroupedLinearVjpArgs &a, hipStream_t stream)
{
    return a.v.bf16 ? grouped_vjp<bf16bits>(a, stream) : grouped_vjp<float>(a, stream);
}

}  // namespace etp
