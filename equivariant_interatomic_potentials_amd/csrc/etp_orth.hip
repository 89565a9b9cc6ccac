// etp_orth.hip -- the orthogonalised update: Newton-Schulz steps
// X <- a X + (b A + c A^2) X, A = X X^T, on X / (|X|_F + eps). Everywhere X is
// n x m with n <= m (a tall matrix is read and written transposed).
//
// All products run on the matrix cores on bf16 parts (etp_dense_mma.hpp): three
// for float matrices, whose small singular values the steps amplify by up to
// a^5, so that every product has to be of float quality; two (2^-16) for bf16
// ones, whose result is rounded to 2^-8. A and P = b A + c A^2 are symmetric:
// the tiles on and above the diagonal are formed and mirrored.
//
//  * n <= 128: orth_strip_kernel, a workgroup per 16 W <= 128 columns. The
//    strip of X stays in registers for all steps (a wave holds 16 columns, all
//    n rows, in accumulator layout, which is also the operand layout of P X);
//    LDS holds the parts of X^T, then of A, then of P in the same space. With
//    one strip (m <= 128) all steps are one launch. Wider matrices take one
//    launch per step: each strip adds the strips' partial A in order, forms P
//    for itself, updates its columns and leaves its part of the next A.
//  * larger: three products a step over the parts in global memory, 64 x 64
//    tiles (orth_product_kernel).
#include <type_traits>

#include "etp_dense_mma.hpp"

namespace etp {

template <typename T>
constexpr int kOrthParts = sizeof(T) == 4 ? 3 : 2;

// ------------------------------------------------------------------- norms

constexpr int kNormParts = 64;  // partial sums of squares per matrix

// part[b][p] = sum of squares of slice p of matrix b, in double
template <typename T>
__global__ void __launch_bounds__(256) orth_norm_kernel(const T *__restrict__ G, const int64_t count,
                                                        double *__restrict__ part)
{
    __shared__ double lds[256];
    const T *g = G + blockIdx.y * count;
    const int64_t i0 = count * blockIdx.x / kNormParts, i1 = count * (blockIdx.x + 1) / kNormParts;
    double s = 0.0;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += 256) {
        const double v = to_f32(g[i]);
        s = __builtin_fma(v, v, s);
    }
    lds[threadIdx.x] = s;
    for (int d = 128; d; d >>= 1) {
        __syncthreads();
        if (threadIdx.x < d)
            lds[threadIdx.x] += lds[threadIdx.x + d];
    }
    if (threadIdx.x == 0)
        part[blockIdx.y * kNormParts + blockIdx.x] = lds[0];
}

// 1 / (|G_b|_F + eps) from the partial sums, in every lane
__device__ __forceinline__ float orth_scale(const double *part, int b, float eps)
{
    double s = part[b * kNormParts + (threadIdx.x & 63)];
#pragma unroll
    for (int m = 32; m; m >>= 1)
        s += __shfl_xor(s, m);
    return static_cast<float>(1.0 / (sqrt(s) + eps));
}

// ------------------------------------------------------------------ strips

struct StripArgs {
    OrthArgs o;
    int n, m, tall;
    int strips;          // workgroups per matrix
    int step;            // -1: first launch of several (scale, partial A); else the step; all steps if strips = 1
    const double *norm;  // partial sums of squares (strips > 1)
    float *xs;           // X between launches, in register order
    const float *a_in;   // partial A of this launch's X, in register order
    float *a_out;
};

// Four floats as P parts at consecutive places of P planes.
template <int P>
__device__ __forceinline__ void put4(bf16bits *at, int plane, f32x4 v)
{
    float w[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int p = 0; p < P; ++p) {
        uint2 u;
        u.x = take_pair(w[0], w[1]);
        u.y = take_pair(w[2], w[3]);
        *reinterpret_cast<uint2 *>(at + p * plane) = u;
    }
}

// Place of column j of A and P within an LDS row: in each 32 columns, the four
// from 4 q and the four from 16 + 4 q lie together, as the eight contraction
// slots that a lane of quarter q holds (of X in registers, and so of A).
__device__ __forceinline__ int slot_of(int j) { return (j & ~31) + 8 * ((j >> 2) & 3) + 4 * ((j >> 4) & 1) + (j & 3); }

// NT tiles of 16 rows, W waves of 16 columns; NT <= W.
template <typename T, int NT, int W>
__global__ void __launch_bounds__(64 * W) orth_strip_kernel(const StripArgs s)
{
    constexpr int P = kOrthParts<T>, SN = 16 * NT + 16;  // LDS row stride (elements)
    constexpr int kPlane = 16 * W * SN;                  // X^T: 16 W rows; A, P: 16 NT rows
    constexpr int NH = W / NT, OMAX = (NT / 2 + NH) / NH;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    bf16bits *pl = reinterpret_cast<bf16bits *>(smem);  // [P][kPlane]
    __shared__ double red[W];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int b = blockIdx.x / s.strips, g = blockIdx.x % s.strips;
    const int n = s.n, m = s.m, col = 16 * W * g + 16 * wave + c;
    const int64_t nm = static_cast<int64_t>(n) * m;
    const float ca = s.o.coef[0], cb = s.o.coef[1], cc = s.o.coef[2];

    // this wave's tiles of A: column tile j, row tiles j + o for every NH-th
    // offset o up to half way round (each pair of tiles once)
    const int tj = wave % NT, th = wave / NT;
    auto row_tile = [&](int k) { return (tj + th + NH * k) % NT; };
    // (an offset past that is computed like the others, and not used)
    auto has = [&](int k) {
        const int o = th + NH * k;
        return o <= NT / 2 && !(2 * o == NT && 2 * tj >= NT);
    };

    // the strip: x[i][r] = X[16 i + 4 q + r][col]
    f32x4 x[NT];
    float *xs = s.xs + (static_cast<int64_t>(blockIdx.x) * W + wave) * NT * 256 + lane * 4;
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
        float scale;
        if (s.strips == 1) {
            double t = 0.0;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    t = __builtin_fma(static_cast<double>(x[i][r]), static_cast<double>(x[i][r]), t);
#pragma unroll
            for (int d = 32; d; d >>= 1)
                t += __shfl_xor(t, d);
            if (lane == 0)
                red[wave] = t;
            __syncthreads();
            t = red[0];
#pragma unroll
            for (int w = 1; w < W; ++w)
                t += red[w];
            scale = static_cast<float>(1.0 / (sqrt(t) + s.o.eps));
        } else {
            scale = orth_scale(s.norm, b, s.o.eps);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
            x[i] *= scale;
    } else {
#pragma unroll
        for (int i = 0; i < NT; ++i)
            x[i] = *reinterpret_cast<const f32x4 *>(xs + i * 256);
    }

    f32x4 acc[OMAX][1];
    // acc = this strip's part of A = X X^T
    auto gram = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
            put4<P>(pl + (16 * wave + c) * SN + 16 * i + 4 * q, kPlane, x[i]);
        __syncthreads();
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
                    fi[k].p[p] = NH == 1 && k == 0 ? fj[0].p[p]
                                                   : read_transposed(pl + p * kPlane, SN, ch, 16 * row_tile(k), lane);
            mma(fi, fj, acc);
        }
        __syncthreads();
    };
    // the tiles of a symmetric matrix (and their mirror images) into LDS
    auto put_tiles = [&](const f32x4 (&t)[OMAX][1]) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < OMAX; ++k)
            if (has(k)) {
                const int i = row_tile(k);
                put4<P>(pl + (16 * tj + c) * SN + slot_of(16 * i + 4 * q), kPlane, t[k][0]);
                if (i != tj) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float v = t[k][0][r];
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            const bf16bits u = from_f32<bf16bits>(v);
                            pl[p * kPlane + (16 * i + 4 * q + r) * SN + slot_of(16 * tj + c)] = u;
                            v -= to_f32(u);
                        }
                    }
                }
            }
        __syncthreads();
    };
    // X <- a X + (b A + c A^2) X, with A's tiles in acc
    auto update = [&]() __attribute__((always_inline)) {
        put_tiles(acc);
        f32x4 sq[OMAX][1];
#pragma unroll
        for (int k = 0; k < OMAX; ++k)
            sq[k][0] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ch = 0; ch < NT / 2; ++ch) {
            Frag<P> fj[1], fi[OMAX];
#pragma unroll
            for (int p = 0; p < P; ++p)
                fj[0].p[p] = *reinterpret_cast<const bf16x8 *>(pl + p * kPlane + (16 * tj + c) * SN + 32 * ch + 8 * q);
#pragma unroll
            for (int k = 0; k < OMAX; ++k)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    fi[k].p[p] = NH == 1 && k == 0
                                     ? fj[0].p[p]
                                     : *reinterpret_cast<const bf16x8 *>(
                                           pl + p * kPlane + (16 * row_tile(k) + c) * SN + 32 * ch + 8 * q);
            mma(fi, fj, sq);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < OMAX; ++k)
            acc[k][0] = cb * acc[k][0] + cc * sq[k][0];
        put_tiles(acc);
        Frag<P> fx[NT / 2][1];
#pragma unroll
        for (int ch = 0; ch < NT / 2; ++ch) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = x[2 * ch + (i >> 2)][i & 3];
            fx[ch][0] = split8_rounded<P>(v);
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
                    for (int p = 0; p < P; ++p)
                        fp[r].p[p] = *reinterpret_cast<const bf16x8 *>(pl + p * kPlane + (16 * (i + r) + c) * SN +
                                                                       32 * ch + 8 * q);
                mma(fp, fx[ch], y);
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
                x[i + r] = ca * x[i + r] + y[r][0];  // one rounding at the size of X, not one per product
        }
        __syncthreads();
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
                    *reinterpret_cast<f32x4 *>(xs + i * 256) = x[i];
            }
            gram();
            if (!one) {
                float *out = s.a_out + static_cast<int64_t>(blockIdx.x) * set + own;
#pragma unroll
                for (int i = 0; i < OMAX; ++i)
                    *reinterpret_cast<f32x4 *>(out + i * 256) = acc[i][0];
                return;
            }
        } else {
#pragma unroll
            for (int i = 0; i < OMAX; ++i)
                acc[i][0] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int p = 0; p < s.strips; ++p) {
                const float *in = s.a_in + (static_cast<int64_t>(b) * s.strips + p) * set + own;
#pragma unroll
                for (int i = 0; i < OMAX; ++i)
                    acc[i][0] += *reinterpret_cast<const f32x4 *>(in + i * 256);
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
// padded with zeros to multiples of 64: part p of element (r, c) of matrix b
// at ((b P + p) rows + r) cols + c.

enum class OrthOp { Gram, Poly, Apply };

struct OrthProductArgs {
    int rows, cols, depth;     // padded sizes of the result and the contraction
    const bf16bits *A, *B;     // [rows][depth], [cols][depth]
    const bf16bits *D;         // added with weight beta: A itself (Poly), X (Apply)
    float alpha, beta;
    bf16bits *out, *out_t;     // result and its transpose as parts
    void *last;                // result of the last step, in the caller's layout
    int n, m, tall;
};

constexpr int kOT = 64;  // tile

// Results are alpha A B^T + beta D in 64 x 64 tiles. Both operands lie along
// the contraction (X^T is kept beside X, and A, P are symmetric). Two groups
// of four waves (32 x 32 each) take alternate chunks of 32 of the contraction
// through their own double-buffered LDS tiles, a 16-byte load per thread and
// part, and are added at the end: a few hundred tiles are all there are, so
// the compute unit's second set of waves has to come from the same tile. The
// tile leaves through LDS, so that it can be written along its rows and along
// its columns.
template <typename T, OrthOp Op>
__global__ void __launch_bounds__(512) orth_product_kernel(const OrthProductArgs a)
{
    constexpr int P = kOrthParts<T>, SK = 40, SO = kOT + 4;
    constexpr int kBuf = P * kOT * SK;  // elements of one operand's chunk
    static_assert(8 * kBuf * sizeof(bf16bits) >= 2 * kOT * SO * sizeof(float));
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    bf16bits *la = reinterpret_cast<bf16bits *>(smem) + grp * 4 * kBuf, *lb = la + 2 * kBuf;  // [2][P][64][SK] each
    float *tile = reinterpret_cast<float *>(smem);                                            // [2][64][SO]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4, b = blockIdx.y;
    int ti, tj;
    if constexpr (Op == OrthOp::Apply) {
        ti = blockIdx.x % (a.rows / kOT);
        tj = blockIdx.x / (a.rows / kOT);
    } else {  // tiles on and above the diagonal: tj (tj + 1) / 2 + ti
        tj = 0;
        ti = blockIdx.x;
        while (ti > tj)
            ti -= ++tj;
    }
    const int r0 = ti * kOT, c0 = tj * kOT;
    const bf16bits *A = a.A + static_cast<int64_t>(b) * P * a.rows * a.depth;
    const bf16bits *B = a.B + static_cast<int64_t>(b) * P * a.cols * a.depth;
    const int lr = (threadIdx.x >> 2) & 63, lk = (threadIdx.x & 3) * 8;

    u32x4 na[P], nb[P];
    auto fetch = [&](int k) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            na[p] = *reinterpret_cast<const u32x4 *>(A + (static_cast<int64_t>(p) * a.rows + r0 + lr) * a.depth + k + lk);
            nb[p] = *reinterpret_cast<const u32x4 *>(B + (static_cast<int64_t>(p) * a.cols + c0 + lr) * a.depth + k + lk);
        }
    };
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int wr = ((wave >> 1) & 1) * 32, wc = (wave & 1) * 32;
    fetch(32 * grp);
    for (int k = 32 * grp, buf = 0; k < a.depth; k += 64, buf ^= 1) {  // depth is a multiple of 64
#pragma unroll
        for (int p = 0; p < P; ++p) {
            *reinterpret_cast<u32x4 *>(la + buf * kBuf + (p * kOT + lr) * SK + lk) = na[p];
            *reinterpret_cast<u32x4 *>(lb + buf * kBuf + (p * kOT + lr) * SK + lk) = nb[p];
        }
        __syncthreads();
        if (k + 64 < a.depth)
            fetch(k + 64);
        Frag<P> fa[2], fb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                fa[i].p[p] = *reinterpret_cast<const bf16x8 *>(la + buf * kBuf + (p * kOT + wr + 16 * i + c) * SK + 8 * q);
                fb[i].p[p] = *reinterpret_cast<const bf16x8 *>(lb + buf * kBuf + (p * kOT + wc + 16 * i + c) * SK + 8 * q);
            }
        mma(fa, fb, acc);
    }
    __syncthreads();
    float *mine = tile + grp * kOT * SO;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                mine[(wr + 16 * i + 4 * q + r) * SO + wc + 16 * j + c] = acc[i][j][r];
    __syncthreads();
    // thread: row orow, eight columns from oc of the tile
    const int orow = threadIdx.x >> 3, oc = (threadIdx.x & 7) * 8;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = a.alpha * (tile[orow * SO + oc + i] + tile[kOT * SO + orow * SO + oc + i]);
    if (Op != OrthOp::Gram) {
#pragma unroll
        for (int p = P - 1; p >= 0; --p) {
            const bf16bits *d = a.D + ((static_cast<int64_t>(b) * P + p) * a.rows + r0 + orow) * a.cols + c0 + oc;
            float f[8];
            load8(d, 8, f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = __builtin_fmaf(a.beta, f[i], v[i]);
        }
    }
    const bool last = Op == OrthOp::Apply && a.last;
    if (last && !a.tall) {
        if (r0 + orow < a.n)
            store8(static_cast<T *>(a.last) + (static_cast<int64_t>(b) * a.n + r0 + orow) * a.m + c0 + oc,
                   a.m - c0 - oc, v);
        return;
    }
    // out [rows][cols], and out_t [cols][rows] (for a symmetric result the
    // same matrix)
    auto put = [&](bf16bits *o, int row, int col, int R, int C) {
        const Frag<P> f = split8_rounded<P>(v);
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<bf16x8 *>(o + ((static_cast<int64_t>(b) * P + p) * R + row) * C + col) = f.p[p];
    };
    if (!last)
        put(a.out, r0 + orow, c0 + oc, a.rows, a.cols);
    if (Op != OrthOp::Apply && ti == tj)
        return;
    // back through the tile for the transpose (with what was added)
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        tile[orow * SO + oc + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = tile[(oc + i) * SO + orow];
    if (!last)
        put(a.out_t, c0 + orow, r0 + oc, a.cols, a.rows);
    else if (c0 + orow < a.m)
        store8(static_cast<T *>(a.last) + (static_cast<int64_t>(b) * a.m + c0 + orow) * a.n + r0 + oc, a.n - r0 - oc, v);
}

// X = G scale as parts, and X^T: a 64 x 64 tile of X per workgroup
template <typename T>
__global__ void __launch_bounds__(256) orth_split_kernel(const T *__restrict__ G, const double *__restrict__ norm,
                                                         const float eps, const int n, const int m, const int tall,
                                                         const int np, const int mp, bf16bits *__restrict__ X,
                                                         bf16bits *__restrict__ XT)
{
    constexpr int P = kOrthParts<T>;
    __shared__ float tile[kOT][kOT + 1];  // as G lies: rows of X, or rows of X^T when tall
    const int b = blockIdx.y, rt = np / kOT, r0 = (blockIdx.x % rt) * kOT, c0 = (blockIdx.x / rt) * kOT;
    const float scale = orth_scale(norm, b, eps);
    const T *g = G + static_cast<int64_t>(b) * n * m;
    const int gr0 = tall ? c0 : r0, gc0 = tall ? r0 : c0, gr = tall ? m : n, gc = tall ? n : m;
    for (int i = threadIdx.x; i < kOT * kOT; i += 256) {
        const int r = i >> 6, c = i & 63;
        tile[r][c] = gr0 + r < gr && gc0 + c < gc ? to_f32(g[static_cast<int64_t>(gr0 + r) * gc + gc0 + c]) * scale
                                                  : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {  // X, then X^T
        const bool turn = (k == 1) != (tall != 0);
        bf16bits *o = k ? XT : X;
        const int R = k ? mp : np, C = k ? np : mp, o0 = k ? c0 : r0, o1 = k ? r0 : c0;
        for (int i = threadIdx.x; i < kOT * kOT; i += 256) {
            const int r = i >> 6, c = i & 63;
            float v = turn ? tile[c][r] : tile[r][c];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                o[((static_cast<int64_t>(b) * P + p) * R + o0 + r) * C + o1 + c] =
                    from_f32<bf16bits>(v);
                v -= to_f32(from_f32<bf16bits>(v));
            }
        }
    }
}

// ---------------------------------------------------------------- dispatch

struct OrthCut {
    int n, m, tall;
    int nt, w, strips;        // strip kernel (n <= 128)
    int np, mp;               // padded sizes (larger)
    size_t norm, xs, as;      // bytes of the workspace's pieces
    size_t x, a;
};

static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

static OrthCut orth_cut(int B, int rows, int cols, bool bf16)
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
        if (c.strips > 1) {
            const int nh = c.w / c.nt, omax = (c.nt / 2 + nh) / nh;
            c.xs = up256(b * c.strips * c.w * c.nt * 256 * sizeof(float));
            c.as = up256(b * c.strips * c.w * omax * 256 * sizeof(float));
        }
        return c;
    }
    c.np = (c.n + kOT - 1) / kOT * kOT;
    c.mp = (c.m + kOT - 1) / kOT * kOT;
    const size_t parts = bf16 ? kOrthParts<bf16bits> : kOrthParts<float>;
    c.x = up256(b * parts * c.np * c.mp * sizeof(bf16bits));
    c.a = up256(b * parts * c.np * c.np * sizeof(bf16bits));
    return c;
}

size_t orthogonalize_workspace_bytes(int B, int rows, int cols, bool bf16)
{
    const OrthCut c = orth_cut(B, rows, cols, bf16);
    return c.norm + c.xs + 2 * c.as + 4 * c.x + 2 * c.a;
}

template <typename T, int NT, int W>
static hipError_t launch_strips(const StripArgs &s, hipStream_t stream)
{
    constexpr size_t lds = sizeof(bf16bits) * kOrthParts<T> * 16 * W * (16 * NT + 16);
    if (lds > 64 * 1024) {
        static const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&orth_strip_kernel<T, NT, W>),
                                                        hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL((orth_strip_kernel<T, NT, W>), dim3(static_cast<unsigned>(s.o.B) * s.strips), dim3(64 * W), lds,
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
static hipError_t launch_orth_product(const OrthProductArgs &a, dim3 grid, hipStream_t stream)
{
    constexpr size_t lds = 8 * kOrthParts<T> * kOT * 40 * sizeof(bf16bits);
    if (lds > 64 * 1024) {
        static const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&orth_product_kernel<T, Op>),
                                                        hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL((orth_product_kernel<T, Op>), grid, dim3(512), lds, stream, a);
    return hipGetLastError();
}

template <typename T>
static hipError_t orthogonalize(const OrthArgs &o, hipStream_t stream)
{
    const OrthCut c = orth_cut(o.B, o.rows, o.cols, o.bf16);
    unsigned char *ws = static_cast<unsigned char *>(o.ws);
    double *norm = reinterpret_cast<double *>(ws);
    ws += c.norm;
    const T *G = static_cast<const T *>(o.G);
    hipError_t e = hipSuccess;
    if (c.nt && c.strips == 1) {
        const StripArgs s{o, c.n, c.m, c.tall, 1, 0, nullptr, nullptr, nullptr, nullptr};
        return strips_by_shape<T>(s, c, stream);
    }
    hipLaunchKernelGGL(orth_norm_kernel<T>, dim3(kNormParts, o.B), dim3(256), 0, stream, G,
                       static_cast<int64_t>(c.n) * c.m, norm);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    if (c.nt) {
        StripArgs s{o, c.n, c.m, c.tall, c.strips, -1, norm, reinterpret_cast<float *>(ws), nullptr, nullptr};
        float *as[2] = {reinterpret_cast<float *>(ws + c.xs), reinterpret_cast<float *>(ws + c.xs + c.as)};
        for (; s.step < o.steps && e == hipSuccess; ++s.step) {  // reads one set of partial sums, writes the other
            s.a_in = as[s.step & 1];
            s.a_out = as[(s.step + 1) & 1];
            e = strips_by_shape<T>(s, c, stream);
        }
        return e;
    }
    bf16bits *X[2] = {reinterpret_cast<bf16bits *>(ws), reinterpret_cast<bf16bits *>(ws + c.x)};
    bf16bits *XT[2] = {reinterpret_cast<bf16bits *>(ws + 2 * c.x), reinterpret_cast<bf16bits *>(ws + 3 * c.x)};
    bf16bits *A = reinterpret_cast<bf16bits *>(ws + 4 * c.x), *Q = reinterpret_cast<bf16bits *>(ws + 4 * c.x + c.a);
    const unsigned rt = c.np / kOT, ct = c.mp / kOT;
    hipLaunchKernelGGL(orth_split_kernel<T>, dim3(rt * ct, o.B), dim3(256), 0, stream, G, norm, o.eps, c.n, c.m,
                       c.tall, c.np, c.mp, X[0], XT[0]);
    const dim3 sym(rt * (rt + 1) / 2, o.B), all(rt * ct, o.B);
    for (int k = 0; k < o.steps; ++k) {
        const int i = k & 1;
        const OrthProductArgs ga{c.np, c.np, c.mp, X[i], X[i], nullptr, 1.f, 0.f, A, A, nullptr, c.n, c.m, c.tall};
        const OrthProductArgs gp{c.np, c.np, c.np, A, A, A, o.coef[2], o.coef[1], Q, Q, nullptr, c.n, c.m, c.tall};
        const OrthProductArgs gx{c.np, c.mp, c.np, Q, XT[i], X[i], 1.f, o.coef[0], X[i ^ 1], XT[i ^ 1],
                                 k + 1 == o.steps ? o.X : nullptr, c.n, c.m, c.tall};
        if ((e = launch_orth_product<T, OrthOp::Gram>(ga, sym, stream)) != hipSuccess ||
            (e = launch_orth_product<T, OrthOp::Poly>(gp, sym, stream)) != hipSuccess ||
            (e = launch_orth_product<T, OrthOp::Apply>(gx, all, stream)) != hipSuccess)
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
