// etp_orth.hip -- the orthogonalised update: Newton-Schulz steps
// X <- a X + (b A + c A^2) X, A = X X^T, on X / (|X|_F + eps). Everywhere X is
// n x m with n <= m (a tall matrix is read and written transposed).
//
// All products run on the matrix cores on three bf16 parts
// (etp_dense_mma.hpp): the steps amplify small singular values by up to a^5, so
// that every product has to be of float quality, also for bf16 matrices (with
// two parts one strong direction over a floor of 10^-3 comes out wrong by 10^-3
// before the result is rounded, with three by 2 10^-5). A and P = b A + c A^2
// are symmetric: only tiles on one side of the diagonal are formed.
//
//  * n <= 128: orth_strip_kernel, a workgroup per 16 W <= 128 columns. The
//    strip of X stays in registers for all steps (a wave holds 16 columns, all
//    n rows, in accumulator layout, which is also the operand layout of P X);
//    LDS holds the parts of X^T, then of A, then of P in the same space. With
//    one strip (m <= 128) all steps are one launch: a matrix has one compute
//    unit, whose matrix instructions are busy 38% of the time and LDS 58%, in
//    turns (34 of 128 x 128: 76 us, five steps; spread over more units with a
//    launch a step it took a fifth longer). Wider matrices take one launch per
//    step: each strip adds the strips' partial A in order, forms P
//    for itself, updates its columns and leaves its part of the next A.
//  * larger: three products a step over the parts in global memory, 64 x 64
//    tiles (orth_product_kernel). 15 launches that wait for each other, each of
//    12 to 17 us, of which a unit's loads at 64 bytes a cycle are a third (two of
//    512 x 1024: 220 us).
#include <type_traits>

#include "etp_dense_mma.hpp"

namespace etp {

constexpr int kOrthParts = 3;

// ------------------------------------------------------------------- norms

constexpr int kNormParts = 64;  // partial sums of squares per matrix

// part[b][p] = sum of squares of slice p of matrix b (whole 16-byte vectors,
// the odd end in the last slice), in double
template <typename T>
__global__ void __launch_bounds__(256) orth_norm_kernel(const T *__restrict__ G, const int64_t count,
                                                        double *__restrict__ part)
{
    __shared__ double lds[256];
    constexpr int V = kVec<T>;
    const T *g = G + blockIdx.y * count;
    const int64_t nv = count / V;
    const int64_t i0 = nv * blockIdx.x / kNormParts, i1 = nv * (blockIdx.x + 1) / kNormParts;
    double s = 0.0;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += 256) {
        RawVec<T> v;
        v.load(g + i * V, V);
#pragma unroll
        for (int k = 0; k < V; ++k)
            s = __builtin_fma(static_cast<double>(v.get(k)), static_cast<double>(v.get(k)), s);
    }
    if (blockIdx.x == kNormParts - 1 && threadIdx.x < count % V) {
        const double v = to_f32(g[nv * V + threadIdx.x]);
        s = __builtin_fma(v, v, s);
    }
    lds[threadIdx.x] = s;
    for (int d = 128; d; d >>= 1) {
        lds_barrier();
        if (threadIdx.x < d)
            lds[threadIdx.x] += lds[threadIdx.x + d];
    }
    if (threadIdx.x == 0)
        part[blockIdx.y * kNormParts + blockIdx.x] = lds[0];
}

// 1 / (|G|_F + eps) as m 2^e: it can pass a float on either side (a zero matrix
// and a small eps; entries near the largest float, whose norm is larger than
// any), an entry times it cannot.
struct OrthScale {
    float m;
    int e;
    __device__ __forceinline__ OrthScale(double squares, float eps)
    {
        const double v = 1.0 / (sqrt(squares) + eps);
        m = static_cast<float>(__builtin_amdgcn_frexp_mant(v));
        e = __builtin_amdgcn_frexp_exp(v);
    }
    __device__ __forceinline__ float operator()(float v) const { return m * __builtin_amdgcn_ldexpf(v, e); }
};

// the sum of squares of matrix b from its partial sums, in every lane
__device__ __forceinline__ double orth_squares(const double *part, int b)
{
    double s = part[b * kNormParts + (threadIdx.x & 63)];
#pragma unroll
    for (int m = 32; m; m >>= 1)
        s += __shfl_xor(s, m);
    return s;
}

// ------------------------------------------------------------------ strips

struct StripArgs {
    OrthArgs o;
    int n, m, tall;
    int strips;          // workgroups per matrix
    int step;            // -1: first launch of several (scale, partial A); else the step; all steps if strips = 1
    const double *norm;  // partial sums of squares, or null: summed by the strip kernel
    const float *x_in;   // X between launches, in register order
    float *x_out;
    const float *a_in;   // partial A of this launch's X, in register order
    float *a_out;
};

template <int P>
__device__ __forceinline__ void put4(bf16bits *at, int plane, f32x4 v)
{
    put_parts<P>(at, plane, {v[0], v[1], v[2], v[3]});
}

// One tile (four of the eight slots) of a fragment of rows 16 r .. + 15 of a
// symmetric matrix, contraction over its column tile k: read as it lies, or,
// where only the mirror tile is stored, read transposed from there.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ s16x4 symmetric_half(const bf16bits *m, int stride, int r, int k, bool stored, int lane)
{
    typedef __attribute__((address_space(3))) s16x4 *lds4;
    const int c = lane & 15, q = lane >> 4;
    if (stored)
        return *reinterpret_cast<const s16x4 *>(m + (16 * r + c) * stride + 16 * k + 4 * q);
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds4)(m + (16 * k + 4 * q + (c >> 2)) * stride + 16 * r + 4 * (c & 3)));
}

// NT tiles of 16 rows, W waves of 16 columns; NT <= W.
template <typename T, int NT, int W>
__global__ void __launch_bounds__(64 * W) orth_strip_kernel(const StripArgs s)
{
    // LDS row stride (elements): rows start 4 or more banks apart, so neither
    // 16 rows of 8 bytes nor 4 rows of 32 collide
    constexpr int P = kOrthParts, SN = 16 * NT + 24;
    constexpr int kPlane = 16 * W * SN;  // X^T: 16 W rows; A, P: 16 NT rows
    constexpr int NH = W / NT, OMAX = (NT / 2 + NH) / NH;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    bf16bits *pl = reinterpret_cast<bf16bits *>(smem);  // [P][kPlane]
    __shared__ double red[W];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int b = blockIdx.y, g = blockIdx.x;
    const int64_t id = static_cast<int64_t>(b) * s.strips + g;
    const int n = s.n, m = s.m, col = 16 * W * g + 16 * wave + c;
    const int64_t nm = static_cast<int64_t>(n) * m;
    const float ca = s.o.coef[0], cb = s.o.coef[1], cc = s.o.coef[2];

    // this wave's tiles of A: column tile tj, row tiles tj + o for every NH-th
    // offset o up to half way round (mod NT): each pair of tiles once, those
    // half way round twice. Tile (tj + o, tj) is stored as row tile tj, column
    // tile tj + o: rows r hold the columns up to half way round after r.
    int tj = wave % NT;
    const int th = wave / NT;
    auto mine = [&](int o) { return NH == 1 || o % NH == th; };
    auto around = [&](int o) { return (tj + o) % NT; };

    // the strip: x[i][r] = X[16 i + 4 q + r][col]
    f32x4 x[NT];
    const float *xs = s.x_in + (id * W + wave) * NT * 256 + lane * 4;
    float *xs_out = s.x_out + (id * W + wave) * NT * 256 + lane * 4;
    if (s.strips == 1 || s.step < 0) {
        const T *G = static_cast<const T *>(s.o.G) + b * nm;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * i + 4 * q + r;
                x[i][r] = row < n && col < m
                              ? to_f32(G[s.tall ? static_cast<int64_t>(col) * n + row
                                                : static_cast<int64_t>(row) * m + col])
                              : 0.f;
            }
        double t = 0.0;
        if (s.norm) {
            t = orth_squares(s.norm, b);
        } else {
            // all of the matrix by every workgroup of it
            for (int64_t i = threadIdx.x; i < nm; i += 64 * W) {
                const double v = to_f32(G[i]);
                t = __builtin_fma(v, v, t);
            }
#pragma unroll
            for (int d = 32; d; d >>= 1)
                t += __shfl_xor(t, d);
            if (lane == 0)
                red[wave] = t;
            lds_barrier();
            t = red[0];
#pragma unroll
            for (int w = 1; w < W; ++w)
                t += red[w];
        }
        const OrthScale scale(t, s.o.eps);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[i][r] = scale(x[i][r]);
    } else {
#pragma unroll
        for (int i = 0; i < NT; ++i)
            x[i] = *reinterpret_cast<const f32x4 *>(xs + i * 256);
    }

    f32x4 acc[OMAX][1];  // offset o at o / NH
    // acc = this strip's part of A = X X^T
    auto gram = [&]() __attribute__((always_inline)) {
        // the tiles' LDS addresses are worked out anew in every step: kept over
        // the steps they would take a register each, and spill
        asm volatile("" : "+s"(tj));
#pragma unroll
        for (int i = 0; i < NT; ++i)
            put4<P>(pl + (16 * wave + c) * SN + 16 * i + 4 * q, kPlane, x[i]);
        lds_barrier();
#pragma unroll
        for (int k = 0; k < OMAX; ++k)
            acc[k][0] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ch = 0; ch < W / 2; ++ch) {
            Frag<P> fj[1], fi[OMAX];
#pragma unroll
            for (int p = 0; p < P; ++p)
                fj[0].p[p] = read_transposed(pl + p * kPlane, SN, ch, 16 * tj, lane);
#pragma unroll
            for (int k = 0; k < OMAX; ++k)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    fi[k].p[p] = NH == 1 && k == 0
                                     ? fj[0].p[p]
                                     : read_transposed(pl + p * kPlane, SN, ch, 16 * around(NH * k + th), lane);
            mma(fi, fj, acc);
            __builtin_amdgcn_sched_barrier(0);  // one chunk's fragments at a time are what the registers hold
        }
        lds_barrier();
    };
    auto put_tiles = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int o = 0; o <= NT / 2; ++o)
            if (mine(o))
                put4<P>(pl + (16 * tj + c) * SN + 16 * around(o) + 4 * q, kPlane, acc[o / NH][0]);
        lds_barrier();
    };
    // X <- a X + (b A + c A^2) X, with A's tiles in acc
    auto update = [&]() __attribute__((always_inline)) {
        asm volatile("" : "+s"(tj));
        put_tiles();
        f32x4 sq[OMAX][1];
#pragma unroll
        for (int k = 0; k < OMAX; ++k)
            sq[k][0] = f32x4{0.f, 0.f, 0.f, 0.f};
        // the contraction goes round from tj, so that what is stored and what
        // is mirrored is known here
        auto half = [&](int o, int k, int p) __attribute__((always_inline)) {  // row tile tj + o, column tile tj + k
            return symmetric_half(pl + p * kPlane, SN, around(o), around(k), (k - o + NT) % NT <= NT / 2, lane);
        };
#pragma unroll
        for (int k = 0; k < NT; k += 2) {
            Frag<P> fj[1];
#pragma unroll
            for (int p = 0; p < P; ++p)
                fj[0].p[p] = __builtin_bit_cast(
                    bf16x8, __builtin_shufflevector(half(0, k, p), half(0, k + 1, p), 0, 1, 2, 3, 4, 5, 6, 7));
            if constexpr (NH == 1) {
                Frag<P> fi[OMAX];
                fi[0] = fj[0];
#pragma unroll
                for (int o = 1; o <= NT / 2; ++o)
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        fi[o].p[p] = __builtin_bit_cast(
                            bf16x8, __builtin_shufflevector(half(o, k, p), half(o, k + 1, p), 0, 1, 2, 3, 4, 5, 6, 7));
                mma(fi, fj, sq);
                __builtin_amdgcn_sched_barrier(0);
            } else {
#pragma unroll
                for (int o = 0; o <= NT / 2; ++o)
                    if (mine(o)) {
                        Frag<P> fi[1];
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            fi[0].p[p] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(half(o, k, p), half(o, k + 1, p),
                                                                                            0, 1, 2, 3, 4, 5, 6, 7));
                        mma(fi, fj, sq, o / NH);
                    }
            }
        }
        lds_barrier();
#pragma unroll
        for (int k = 0; k < OMAX; ++k)
            acc[k][0] = cb * acc[k][0] + cc * sq[k][0];
        put_tiles();
        Frag<P> fx[NT / 2][1];
#pragma unroll
        for (int ch = 0; ch < NT / 2; ++ch) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = x[2 * ch + (i >> 2)][i & 3];
            fx[ch][0] = split8<P>(v);
        }
        constexpr int R = NT < 4 ? NT : 4;  // row tiles at a time
#pragma unroll
        for (int i = 0; i < NT; i += R) {
            f32x4 y[R][1];
#pragma unroll
            for (int r = 0; r < R; ++r)
                y[r][0] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ch = 0; ch < NT / 2; ++ch) {
                Frag<P> fp[R];
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        s16x4 h[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            h[u] = symmetric_half(pl + p * kPlane, SN, i + r, 2 * ch + u,
                                                  (2 * ch + u - i - r + NT) % NT <= NT / 2, lane);
                        fp[r].p[p] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
                    }
                mma(fp, fx[ch], y);
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
                x[i + r] = ca * x[i + r] + y[r][0];  // one rounding at the size of X, not one per product
        }
        lds_barrier();
    };

    // one strip: all steps; else the launch's part of one: (the strips' sum of
    // A, update,) partial A of what X now is
    const bool one = s.strips == 1;
    const int64_t set = static_cast<int64_t>(W) * OMAX * 256;  // a strip's partial A
    const int64_t own = (static_cast<int64_t>(wave) * OMAX * 64 + lane) * 4;
    bool form = one || s.step < 0;
    for (int k = one ? 0 : s.step;;) {
        if (form) {
            if (!one) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    *reinterpret_cast<f32x4 *>(xs_out + i * 256) = x[i];
            }
            gram();
            if (!one) {
                float *out = s.a_out + id * set + own;
#pragma unroll
                for (int i = 0; i < OMAX; ++i)
                    *reinterpret_cast<f32x4 *>(out + i * 256) = acc[i][0];
                return;
            }
        } else {
#pragma unroll
            for (int i = 0; i < OMAX; ++i)
                acc[i][0] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int p = 0; p < s.strips; p += 4) {  // four sets in flight, added in order
                f32x4 in[4][OMAX];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int64_t at = static_cast<int64_t>(b) * s.strips + (p + u < s.strips ? p + u : p);
#pragma unroll
                    for (int i = 0; i < OMAX; ++i)
                        in[u][i] = *reinterpret_cast<const f32x4 *>(s.a_in + at * set + own + i * 256);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (p + u < s.strips) {
#pragma unroll
                        for (int i = 0; i < OMAX; ++i)
                            acc[i][0] += in[u][i];
                    }
            }
        }
        update();
        if (++k == s.o.steps)
            break;
        form = true;
    }
    T *X = static_cast<T *>(s.o.X) + b * nm;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * i + 4 * q + r;
            if (row < n && col < m)
                X[s.tall ? static_cast<int64_t>(col) * n + row : static_cast<int64_t>(row) * m + col] =
                    from_f32<T>(x[i][r]);
        }
}

// ---------------------------------------------------------- large matrices

// A matrix [rows][cols] as bf16 parts in global memory, rows and columns
// padded with zeros to multiples of 64, each part of a matrix in fragment
// order: 16 rows by 32 columns together, as the 64 lanes hold them, so that a
// wave's fragment is 1 KiB without a gap (16 rows of 64 bytes each take about
// three times as long to load). Place of entry (row, col) of a part, col a
// multiple of eight:
__device__ __forceinline__ int64_t part_place(int row, int col, int cols)
{
    return (static_cast<int64_t>(row >> 4) * (cols >> 5) + (col >> 5)) * 512 + (((col >> 3) & 3) * 16 + (row & 15)) * 8;
}

enum class OrthOp { Gram, Poly, Apply };

struct OrthProductArgs {
    int rows, cols, depth;     // padded sizes of the result and the contraction
    int tiles, mats;           // per matrix, matrices
    const bf16bits *A, *B;     // [rows][depth], [cols][depth]
    const bf16bits *D;         // added with weight beta: A itself (Poly), X (Apply)
    float alpha, beta;
    bf16bits *out, *out_t;     // result and its transpose as parts
    void *last;                // result of the last step, in the caller's layout
    int n, m, tall;
};

constexpr int kOT = 64;  // tile

// Results are alpha A B^T + beta D in 64 x 64 tiles. Both operands lie along
// the contraction (X^T is kept beside X, and A, P are symmetric). There are a
// few hundred tiles at most, so a tile takes a whole compute unit: its four
// waves each form all of it over every fourth chunk of 32 of the contraction,
// with fragments straight from memory into registers (nothing is shared
// before the end, so nothing goes through LDS and no wave waits for another;
// one wave to a SIMD has the registers for the next chunk's 24 KiB while it
// works on this one), and the four are added in wave order. The tile leaves
// through LDS, so that it can be written along its rows and along its columns.
constexpr int kOrthOut = kOT + 4;  // LDS row stride of the tile (floats)

template <typename T, OrthOp Op>
__global__ void __launch_bounds__(256, 1) orth_product_kernel(const OrthProductArgs a)
{
    constexpr int P = kOrthParts, SO = kOrthOut;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    float *tile = reinterpret_cast<float *>(smem);  // [4][64][SO]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    // workgroups b and b + 8 run on the same XCD: each XCD takes a run of
    // consecutive tiles, so that it fetches few rows of the operands into its
    // L2
    const int w = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
    if (w >= a.tiles * a.mats)
        return;  // the whole workgroup: padding to a multiple of 8
    const int b = w / a.tiles, t = w - b * a.tiles;
    int ti, tj;
    if constexpr (Op == OrthOp::Apply) {
        ti = t % (a.rows / kOT);
        tj = t / (a.rows / kOT);
    } else {  // tiles on and above the diagonal: tj (tj + 1) / 2 + ti
        tj = 0;
        ti = t;
        while (ti > tj)
            ti -= ++tj;
    }
    const int r0 = ti * kOT, c0 = tj * kOT;
    const int64_t pa = static_cast<int64_t>(a.rows) * a.depth, pb = static_cast<int64_t>(a.cols) * a.depth;  // a part
    const int64_t band = static_cast<int64_t>(a.depth) * 16;                                              // 16 rows
    const bf16bits *A = a.A + b * P * pa + (r0 >> 4) * band + lane * 8;
    const bf16bits *B = a.B + b * P * pb + (c0 >> 4) * band + lane * 8;

    Frag<P> fa[2][4], fb[2][4];  // [buffer][tile]
    auto fetch = [&](int ch, int buf) __attribute__((always_inline)) {
        if (32 * ch >= a.depth)
            return;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                fa[buf][i].p[p] = *reinterpret_cast<const bf16x8 *>(A + p * pa + i * band + ch * 512);
                fb[buf][i].p[p] = *reinterpret_cast<const bf16x8 *>(B + p * pb + i * band + ch * 512);
            }
    };
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    fetch(wave, 0);
    for (int ch = wave; 32 * ch < a.depth; ch += 8) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (32 * (ch + 4 * u) >= a.depth)
                break;
            fetch(ch + 4 * u + 4, u ^ 1);
            mma(fa[u], fb[u], acc);
        }
    }
    float *mine = tile + wave * kOT * SO;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                mine[(16 * i + 4 * q + r) * SO + 16 * j + c] = acc[i][j][r];
    lds_barrier();
    // thread: rows orow + 32 h, eight columns from oc of the tile
    const int orow = threadIdx.x >> 3, oc = (threadIdx.x & 7) * 8;
    const bool last = Op == OrthOp::Apply && a.last;
    // out [rows][cols], and out_t [cols][rows] (for a symmetric result the
    // same matrix)
    auto put = [&](bf16bits *o, int row, int col, int R, int C, const float (&v)[8]) {
        const Frag<P> f = split8<P>(v);
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<bf16x8 *>(o + (static_cast<int64_t>(b) * P + p) * R * C + part_place(row, col, C)) = f.p[p];
    };
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = orow + 32 * h;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float *t = tile + row * SO + oc + i;
            v[h][i] = a.alpha * ((t[0] + t[kOT * SO]) + (t[2 * kOT * SO] + t[3 * kOT * SO]));
        }
        if (Op != OrthOp::Gram) {
#pragma unroll
            for (int p = P - 1; p >= 0; --p) {
                float f[8];
                load8(a.D + (static_cast<int64_t>(b) * P + p) * a.rows * a.cols + part_place(r0 + row, c0 + oc, a.cols), 8, f);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[h][i] = __builtin_fmaf(a.beta, f[i], v[h][i]);
            }
        }
        if (!last)
            put(a.out, r0 + row, c0 + oc, a.rows, a.cols, v[h]);
        else if (!a.tall && r0 + row < a.n)
            store8(static_cast<T *>(a.last) + (static_cast<int64_t>(b) * a.n + r0 + row) * a.m + c0 + oc, a.m - c0 - oc,
                   v[h]);
    }
    if (last ? !a.tall : Op != OrthOp::Apply && ti == tj)
        return;
    // back through the tile for the transpose (with what was added)
    lds_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            tile[(orow + 32 * h) * SO + oc + i] = v[h][i];
    lds_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = orow + 32 * h;
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = tile[(oc + i) * SO + row];
        if (!last)
            put(a.out_t, c0 + row, r0 + oc, a.cols, a.rows, w);
        else if (c0 + row < a.m)
            store8(static_cast<T *>(a.last) + (static_cast<int64_t>(b) * a.m + c0 + row) * a.n + r0 + oc, a.n - r0 - oc, w);
    }
}

// X = G scale as parts, and X^T: a 64 x 64 tile of X per workgroup, eight
// values a thread and store
template <typename T>
__global__ void __launch_bounds__(512) orth_split_kernel(const T *__restrict__ G, const double *__restrict__ norm,
                                                         const float eps, const int n, const int m, const int tall,
                                                         const int np, const int mp, bf16bits *__restrict__ X,
                                                         bf16bits *__restrict__ XT)
{
    constexpr int P = kOrthParts;
    __shared__ float tile[kOT][kOT + 1];  // as G lies: rows of X, or rows of X^T when tall
    const int b = blockIdx.y, rt = np / kOT, r0 = (blockIdx.x % rt) * kOT, c0 = (blockIdx.x / rt) * kOT;
    const int row = threadIdx.x >> 3, col = (threadIdx.x & 7) * 8;
    const int gr0 = tall ? c0 : r0, gc0 = tall ? r0 : c0, gr = tall ? m : n, gc = tall ? n : m;
    const int valid = gr0 + row < gr ? gc - gc0 - col : 0;
    float v[8];
    load8(G + (static_cast<int64_t>(b) * gr + (valid > 0 ? gr0 + row : 0)) * gc + (valid > 0 ? gc0 + col : 0), valid, v);
    const OrthScale scale(orth_squares(norm, b), eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = scale(v[i]);
        tile[row][col + i] = v[i];
    }
    auto put = [&](bf16bits *o, int R, int C, int o0, int o1) {
        const Frag<P> f = split8<P>(v);
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<bf16x8 *>(o + (static_cast<int64_t>(b) * P + p) * R * C + part_place(o0 + row, o1 + col, C)) =
                f.p[p];
    };
    if (tall)
        put(XT, mp, np, c0, r0);
    else
        put(X, np, mp, r0, c0);
    lds_barrier();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = tile[col + i][row];
    if (tall)
        put(X, np, mp, r0, c0);
    else
        put(XT, mp, np, c0, r0);
}

// ---------------------------------------------------------------- dispatch

struct OrthCut {
    int n, m, tall;
    int nt, w, strips;        // strip kernel (n <= 128)
    bool own_norm;            // the strip kernel sums the squares itself
    int np, mp;               // padded sizes (larger)
    size_t norm, xs, as;      // bytes of the workspace's pieces
    size_t x, a;
};

static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

static OrthCut orth_cut(int B, int rows, int cols)
{
    OrthCut c{};
    c.tall = rows > cols;
    c.n = c.tall ? cols : rows;
    c.m = c.tall ? rows : cols;
    const size_t b = static_cast<size_t>(B);
    c.norm = up256(b * kNormParts * sizeof(double));
    if (c.n <= 128) {
        auto tiles = [](int v) { return v <= 32 ? 2 : v <= 64 ? 4 : 8; };
        c.nt = tiles(c.n);
        c.w = tiles(c.m);
        c.strips = (c.m + 127) / 128;
        c.own_norm = static_cast<int64_t>(c.n) * c.m <= 32768;
        if (c.strips > 1) {
            const int nh = c.w / c.nt, omax = (c.nt / 2 + nh) / nh;
            c.xs = up256(b * c.strips * c.w * c.nt * 256 * sizeof(float));
            c.as = up256(b * c.strips * c.w * omax * 256 * sizeof(float));
        }
        return c;
    }
    c.np = (c.n + kOT - 1) / kOT * kOT;
    c.mp = (c.m + kOT - 1) / kOT * kOT;
    c.x = up256(b * kOrthParts * c.np * c.mp * sizeof(bf16bits));
    c.a = up256(b * kOrthParts * c.np * c.np * sizeof(bf16bits));
    return c;
}

size_t orthogonalize_workspace_bytes(int B, int rows, int cols)
{
    const OrthCut c = orth_cut(B, rows, cols);
    return c.norm + 2 * c.xs + 2 * c.as + 4 * c.x + 2 * c.a;
}

template <typename T, int NT, int W>
static hipError_t launch_strips(const StripArgs &s, hipStream_t stream)
{
    constexpr size_t lds = sizeof(bf16bits) * kOrthParts * 16 * W * (16 * NT + 24);
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&orth_strip_kernel<T, NT, W>),
                                                        hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL((orth_strip_kernel<T, NT, W>), dim3(s.strips, s.o.B), dim3(64 * W), lds,
                       stream, s);
    return hipGetLastError();
}

template <typename T>
static hipError_t strips_by_shape(const StripArgs &s, const OrthCut &c, hipStream_t stream)
{
    switch (c.nt * 10 + c.w) {
    case 22: return launch_strips<T, 2, 2>(s, stream);
    case 24: return launch_strips<T, 2, 4>(s, stream);
    case 28: return launch_strips<T, 2, 8>(s, stream);
    case 44: return launch_strips<T, 4, 4>(s, stream);
    case 48: return launch_strips<T, 4, 8>(s, stream);
    default: return launch_strips<T, 8, 8>(s, stream);
    }
}

template <typename T, OrthOp Op>
static hipError_t launch_orth_product(const OrthProductArgs &a, hipStream_t stream)
{
    constexpr size_t lds = 4 * kOT * kOrthOut * sizeof(float);
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&orth_product_kernel<T, Op>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess)
        return e;
    const int64_t work = static_cast<int64_t>(a.tiles) * a.mats;
    if (work > 0x7FFFFFF0)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((orth_product_kernel<T, Op>), dim3(static_cast<unsigned>((work + 7) / 8 * 8)), dim3(256), lds,
                       stream, a);
    return hipGetLastError();
}

template <typename T>
static hipError_t orthogonalize(const OrthArgs &o, hipStream_t stream)
{
    const OrthCut c = orth_cut(o.B, o.rows, o.cols);
    unsigned char *ws = static_cast<unsigned char *>(o.ws);
    double *norm = reinterpret_cast<double *>(ws);
    ws += c.norm;
    const T *G = static_cast<const T *>(o.G);
    hipError_t e = hipSuccess;
    if (!c.own_norm) {
        hipLaunchKernelGGL(orth_norm_kernel<T>, dim3(kNormParts, o.B), dim3(256), 0, stream, G,
                           static_cast<int64_t>(c.n) * c.m, norm);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    if (c.nt) {
        StripArgs s{o, c.n, c.m, c.tall, c.strips, c.strips == 1 ? 0 : -1, c.own_norm ? nullptr : norm, nullptr, nullptr,
                    nullptr, nullptr};
        if (c.strips == 1)
            return strips_by_shape<T>(s, c, stream);
        // each launch reads one set of X and partial sums and writes the other
        float *xs[2] = {reinterpret_cast<float *>(ws), reinterpret_cast<float *>(ws + c.xs)};
        float *as[2] = {reinterpret_cast<float *>(ws + 2 * c.xs), reinterpret_cast<float *>(ws + 2 * c.xs + c.as)};
        for (; s.step < o.steps && e == hipSuccess; ++s.step) {
            const int i = s.step & 1;
            s.x_in = xs[i];
            s.x_out = xs[i ^ 1];
            s.a_in = as[i];
            s.a_out = as[i ^ 1];
            e = strips_by_shape<T>(s, c, stream);
        }
        return e;
    }
    bf16bits *X[2] = {reinterpret_cast<bf16bits *>(ws), reinterpret_cast<bf16bits *>(ws + c.x)};
    bf16bits *XT[2] = {reinterpret_cast<bf16bits *>(ws + 2 * c.x), reinterpret_cast<bf16bits *>(ws + 3 * c.x)};
    bf16bits *A = reinterpret_cast<bf16bits *>(ws + 4 * c.x), *Q = reinterpret_cast<bf16bits *>(ws + 4 * c.x + c.a);
    const unsigned rt = c.np / kOT, ct = c.mp / kOT;
    hipLaunchKernelGGL(orth_split_kernel<T>, dim3(rt * ct, o.B), dim3(512), 0, stream, G, norm, o.eps, c.n, c.m,
                       c.tall, c.np, c.mp, X[0], XT[0]);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    const int sym = static_cast<int>(rt * (rt + 1) / 2), all = static_cast<int>(rt * ct);
    for (int k = 0; k < o.steps; ++k) {
        const int i = k & 1;
        const OrthProductArgs ga{c.np, c.np, c.mp, sym, o.B, X[i], X[i], nullptr, 1.f, 0.f, A, A, nullptr, c.n, c.m, c.tall};
        const OrthProductArgs gp{c.np, c.np, c.np, sym, o.B, A, A, A, o.coef[2], o.coef[1], Q, Q, nullptr, c.n, c.m, c.tall};
        const OrthProductArgs gx{c.np, c.mp, c.np, all, o.B, Q, XT[i], X[i], 1.f, o.coef[0], X[i ^ 1], XT[i ^ 1],
                                 k + 1 == o.steps ? o.X : nullptr, c.n, c.m, c.tall};
        if ((e = launch_orth_product<T, OrthOp::Gram>(ga, stream)) != hipSuccess ||
            (e = launch_orth_product<T, OrthOp::Poly>(gp, stream)) != hipSuccess ||
            (e = launch_orth_product<T, OrthOp::Apply>(gx, stream)) != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_orthogonalize(const OrthArgs &a, hipStream_t stream)
{
    if (a.B == 0)
        return hipSuccess;
    return a.bf16 ? orthogonalize<bf16bits>(a, stream) : orthogonalize<float>(a, stream);
}

}  // namespace etp
