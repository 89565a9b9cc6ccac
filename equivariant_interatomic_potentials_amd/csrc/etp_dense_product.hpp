// etp_dense_product.hpp -- the pieces of a product of rows with a matrix that
// the linear layer's kernels and the grouped layer's are made of: row operands
// and the matrix on their way into fragments, and the epilogue.
#pragma once
#include <type_traits>

#include "etp_dense_mma.hpp"

namespace etp {

constexpr int kComputeUnits = 256;

// Fwd: rows are x; Gx: rows are gy and z; GxD: rows are d, in float; GxPlain: rows
// are gy as stored, which without an activation is d.
enum class Dense { Fwd, Gx, GxD, GxPlain };

struct ProductArgs {
    int64_t M;
    int KD, ND;      // contraction, output columns
    const void *A;   // rows: x, gy, or d
    int64_t lda;
    const void *Z;   // pre-activation (Gx with an activation)
    int64_t ldz;
    const void *W;   // [n_in][n_out]: [KD][ND] (Fwd) or [ND][KD] (Gx)
    const float *bias;
    int act;
    const void *res;
    int64_t ldr;
    void *out;
    int64_t ldo;
    void *zout;
    int64_t ldzo;
    bool accumulate;
};

// Parts of the row operand, which hold it exactly: a stored value, or d, which
// is a float also in a bf16 layer (with two of its parts terms that cancel
// would leave grad_x wrong by up to 2^-15 of each).
template <typename T, Dense D>
constexpr int kRowParts = D == Dense::Fwd || D == Dense::GxPlain ? kParts<T> : 3;

// Chunks of 32 of the contraction that a tile of a long one takes at a time:
// two, but one where the rows have three parts, so that more workgroups share a
// compute unit (grad_x alone, 200000 x 128 x 300 bf16: 130 us with one, 136 with
// two; 20000 x 384 x 1024: 74 and 87).
template <typename T, Dense D>
constexpr int kStreamSub = kRowParts<T, D> == 3 ? 1 : 2;

// Eight entries of a row as loaded, and as matrix-core parts.
template <typename T, Dense D>
struct RowChunk {
    Raw8<T> v;
    __device__ __forceinline__ void load(const ProductArgs &a, int64_t row, int k)
    {
        v.load(static_cast<const T *>(a.A) + row * a.lda + k, a.KD - k);
    }
    __device__ __forceinline__ Frag<kParts<T>> frag(const ProductArgs &) const
    {
        return v.template frag<kParts<T>>();
    }
};

template <typename T>
struct RowChunk<T, Dense::Gx> {
    Raw8<T> g, z;
    __device__ __forceinline__ void load(const ProductArgs &a, int64_t row, int k)
    {
        g.load(static_cast<const T *>(a.A) + row * a.lda + k, a.KD - k);
        if (a.act != kActNone)
            z.load(static_cast<const T *>(a.Z) + row * a.ldz + k, a.KD - k);
    }
    __device__ __forceinline__ Frag<kRowParts<T, Dense::Gx>> frag(const ProductArgs &a) const
    {
        float d[8];
        g.get(d);
        if (a.act != kActNone) {
            float zv[8];
            z.get(zv);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] *= act_slope(a.act, zv[i]);
        }
        return split8<kRowParts<T, Dense::Gx>, kCut<T>>(d);
    }
};

template <typename T>
struct RowChunk<T, Dense::GxD> {
    Raw8<float> d;
    __device__ __forceinline__ void load(const ProductArgs &a, int64_t row, int k)
    {
        d.load(static_cast<const float *>(a.A) + row * a.lda + k, a.KD - k);
    }
    __device__ __forceinline__ Frag<kRowParts<T, Dense::GxD>> frag(const ProductArgs &) const
    {
        return d.template frag<kRowParts<T, Dense::GxD>, kCut<T>>();
    }
};

// A lane's result columns: a float lane stores four columns of a 16-column
// tile (64 contiguous bytes a row for the wave); a bf16 lane stores eight
// columns out of a pair of tiles (again 64 bytes), which are interleaved for
// that: entry c of tile t is column 32 (t / 2) + 8 (c / 4) + 4 (t % 2) + c % 4.
template <typename T>
__device__ __forceinline__ int tile_of_col(int j)
{
    return sizeof(T) == 4 ? j >> 4 : 2 * (j >> 5) + ((j >> 2) & 1);
}
template <typename T>
__device__ __forceinline__ int entry_of_col(int j)
{
    return sizeof(T) == 4 ? j & 15 : 4 * ((j >> 3) & 3) + (j & 3);
}
// first of the four consecutive columns that quarter q of tile t holds
template <typename T>
__device__ __forceinline__ int col_of_quarter(int t, int q)
{
    return sizeof(T) == 4 ? 16 * t + 4 * q : 32 * (t >> 1) + 8 * q + 4 * (t & 1);
}

// The matrix in LDS, in chunks of 32 of the contraction by nb columns, parts
// apart. Forward: W's rows run along the columns, so it lies row by row as in
// memory (16-byte loads and stores) and the transposing read hands a lane its
// eight k of a column; LDS row 4 q + i (16 + 4 q + i) of a chunk holds k = 8 q +
// i (8 q + 4 + i), the slots that read takes, and the columns of a pair of
// tiles are interleaved as the result wants them. Input gradient: W's rows run
// along the contraction and lie in fragment order.
template <typename T, Dense D>
struct MatrixLds {
    static constexpr int P = kParts<T>;
    static constexpr bool kRows = D == Dense::Fwd;
    // elements of one chunk of nb columns
    static __host__ __device__ constexpr int chunk(int nb) { return kRows ? P * 32 * (nb + 8) : P * 32 * nb; }
    // pieces of eight elements of one chunk
    static __host__ __device__ constexpr int pieces(int nb) { return 4 * nb; }
    // place of quarter q of column c in a tile: columns one after the other,
    // their quarters turned so that neither the stores (a column's four
    // quarters by consecutive threads) nor the reads (a quarter of 16 columns)
    // collide: 32768 x 512 x 512 bf16 grad_x, 50.1 -> 47.8 us
    static __device__ __forceinline__ int swizzled(int c, int q) { return 4 * c + (q ^ ((c >> 2) & 3)); }

    // piece i of the chunk from k0: consecutive threads along W's rows
    static __device__ __forceinline__ void load(const ProductArgs &a, int i, int nb, int k0, int n0, Raw8<T> &v)
    {
        const T *W = static_cast<const T *>(a.W);
        int row, col, valid;
        if constexpr (kRows) {
            row = k0 + i / (nb / 8);
            col = n0 + i % (nb / 8) * 8;
            valid = row < a.KD ? a.ND - col : 0;
        } else {
            row = n0 + i / 4;
            col = k0 + i % 4 * 8;
            valid = row < a.ND ? a.KD - col : 0;
        }
        v.load(W + (valid > 0 ? static_cast<int64_t>(row) * (kRows ? a.ND : a.KD) + col : 0), valid);
    }
    static __device__ __forceinline__ void store(bf16bits *m, int i, int nb, const Raw8<T> &v)
    {
        const Frag<P> f = v.template frag<P>();
        if constexpr (kRows) {
            const int k = i / (nb / 8), j = i % (nb / 8) * 8, r = 16 * ((k >> 2) & 1) + 4 * (k >> 3) + (k & 3);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                bf16bits *at = m + (p * 32 + r) * (nb + 8);
                if constexpr (sizeof(T) == 4) {
                    *reinterpret_cast<bf16x8 *>(at + j) = f.p[p];
                } else {  // columns 32 g + 8 q .. + 3 and .. + 7: entries 4 q .. + 3 of tiles 2 g and 2 g + 1
                    const u32x4 u = __builtin_bit_cast(u32x4, f.p[p]);
                    at += (j & ~31) + ((j & 31) >> 1);
                    *reinterpret_cast<uint2 *>(at) = uint2{u[0], u[1]};
                    *reinterpret_cast<uint2 *>(at + 16) = uint2{u[2], u[3]};
                }
            }
        } else {
            const int j = i / 4, q = i % 4;
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<bf16x8 *>(
                    m + ((tile_of_col<T>(j) * P + p) * 64 + swizzled(entry_of_col<T>(j), q)) * 8) = f.p[p];
        }
    }
    static __device__ __forceinline__ Frag<P> tile(const bf16bits *m, int t, int nb, int lane)
    {
        Frag<P> f;
#pragma unroll
        for (int p = 0; p < P; ++p)
            f.p[p] = kRows ? read_transposed(m + p * 32 * (nb + 8), nb + 8, 0, 16 * t, lane)
                           : *reinterpret_cast<const bf16x8 *>(m + ((t * P + p) * 64 + swizzled(lane & 15, lane >> 4)) * 8);
        return f;
    }
};

// A lane's eight k of one column straight from memory.
template <typename T, Dense D>
struct MatrixColumn {
    T v[8];
    __device__ __forceinline__ void load(const ProductArgs &a, int k, int j)
    {
        const T *W = static_cast<const T *>(a.W);
        if constexpr (D == Dense::Fwd) {
            const T *p = W + static_cast<int64_t>(k) * a.ND + j;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = k + i < a.KD && j < a.ND ? p[static_cast<int64_t>(i) * a.ND] : T(0);
        } else {
            const T *p = W + static_cast<int64_t>(j < a.ND ? j : 0) * a.KD + k;
            const int valid = j < a.ND ? a.KD - k : 0;
            if constexpr (sizeof(T) == 4)
                load8(p, valid, v);
            else
                *reinterpret_cast<u32x4_any *>(v) = load8(p, valid);
        }
    }
    __device__ __forceinline__ Frag<kParts<T>> frag() const
    {
        if constexpr (sizeof(T) == 4) {
            return split8<3>(v);
        } else {
            u32x4 u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = v[2 * i] | static_cast<uint32_t>(v[2 * i + 1]) << 16;
            return {{__builtin_bit_cast(bf16x8, u)}};
        }
    }
};

// Epilogue: NV consecutive columns from j of one row (4 float, 8 bf16).
template <typename T, Dense D, int NV>
__device__ __forceinline__ void store_cols(const ProductArgs &a, int64_t row, int j, float (&v)[8], const float (&r)[8])
{
    const int valid = a.ND - j;
    if (valid <= 0)
        return;
    if constexpr (D == Dense::Fwd) {
        if (a.zout)
            store_n<NV>(static_cast<T *>(a.zout) + row * a.ldzo + j, valid, v);
        if (a.act != kActNone) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                v[i] = act_value(a.act, v[i]);
        }
        if (a.res) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                v[i] += r[i];
        }
    } else if (a.accumulate) {  // input gradients
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] += r[i];
    }
    store_n<NV>(static_cast<T *>(a.out) + row * a.ldo + j, valid, v);
}

// What the epilogue adds: the residual (Fwd), or the output itself (Gx).
template <typename T, Dense D, int NV>
__device__ __forceinline__ void load_addend(const ProductArgs &a, int64_t row, int j, float (&r)[8])
{
    const int valid = a.ND - j;
    if constexpr (D == Dense::Fwd) {
        if (a.res && valid > 0)
            load_n<NV>(static_cast<const T *>(a.res) + row * a.ldr + j, valid, r);
    } else {
        if (a.accumulate && valid > 0)
            load_n<NV>(static_cast<const T *>(a.out) + row * a.ldo + j, valid, r);
    }
}

// The four tiles acc of a 64-column group from column j0 (tile 0's first) of
// row `row`: epilogue and stores.
template <typename T, Dense D>
__device__ __forceinline__ void store_group(const ProductArgs &a, int64_t row, int j0, int q, const f32x4 (&acc)[4][1],
                                            const float (&add)[sizeof(T) == 4 ? 4 : 2][8])
{
    if (row >= a.M)
        return;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f32x4 u = acc[t][0];
            float v[8] = {u[0], u[1], u[2], u[3]};
            store_cols<T, D, 4>(a, row, j0 + col_of_quarter<T>(t, q), v, add[t]);
        }
    } else {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const f32x4 u = acc[2 * t][0], w = acc[2 * t + 1][0];
            float v[8] = {u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]};
            store_cols<T, D, 8>(a, row, j0 + col_of_quarter<T>(2 * t, q), v, add[t]);
        }
    }
}

template <typename T, Dense D>
__device__ __forceinline__ void load_group_addend(const ProductArgs &a, int64_t row, int j0, int q,
                                                  float (&add)[sizeof(T) == 4 ? 4 : 2][8])
{
    const int64_t rc = row < a.M ? row : a.M - 1;
#pragma unroll
    for (int t = 0; t < (sizeof(T) == 4 ? 4 : 2); ++t)
        load_addend<T, D, sizeof(T) == 4 ? 4 : 8>(a, rc, j0 + col_of_quarter<T>(sizeof(T) == 4 ? t : 2 * t, q),
                                                  add[t]);
}

// Sixteen bytes of a row operand's source as loaded, and into LDS as parts.
template <typename T, Dense D>
struct RowPiece {
    using Src = std::conditional_t<D == Dense::GxD, float, T>;
    static constexpr int V = kVec<Src>;
    RawVec<Src> v;
    RawVec<T> z;  // Gx
    __device__ __forceinline__ void load(const ProductArgs &a, int64_t row, int k)
    {
        const int valid = a.KD - k;
        v.load(static_cast<const Src *>(a.A) + row * a.lda + k, valid);
        if (D == Dense::Gx && a.act != kActNone)
            z.load(static_cast<const T *>(a.Z) + row * a.ldz + k, valid);
    }
    __device__ __forceinline__ void store(const ProductArgs &a, bf16bits *at, int plane) const
    {
        if constexpr (sizeof(Src) == 2 && (D == Dense::Fwd || D == Dense::GxPlain)) {
            *reinterpret_cast<u32x4 *>(at) = v.v;
        } else {
            float f[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[i] = v.get(i);
                if (D == Dense::Gx && a.act != kActNone)
                    f[i] *= act_slope(a.act, z.get(i));
            }
            put_parts<kRowParts<T, D>, kCut<T>>(at, plane, f);
        }
    }
};

}  // namespace etp
