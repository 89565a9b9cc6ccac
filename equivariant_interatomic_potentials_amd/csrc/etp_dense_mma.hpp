// etp_dense_mma.hpp -- matrix-core fragments of the dense operators.
//
// Every product runs on v_mfma_f32_16x16x32_bf16: lane (c = lane % 16,
// q = lane / 16) holds entries k = 8 q .. 8 q + 7 of row c of the first and of
// column c of the second operand, and rows 4 q .. 4 q + 3 of column c of the
// float result. A float operand is cut exactly into three bf16 parts
// (v = p0 + p1 + p2, rounded to nearest, so |p1| <= 2^-8 |v| and |p2| <=
// 2^-17 |v|), and the six products of parts i, j with i + j <= 2 are added in
// float: the dropped ones are at most 2^-24 of |v w| and of either sign, a float
// product's own rounding, at six bf16 instructions of 16 cycles for 8192
// products where the fp32 instruction takes 256 cycles.
#pragma once
#include "etp_dense.hpp"

namespace etp {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// the same with the element's alignment only (global memory takes any)
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// bf16 parts that hold a stored value of T exactly
template <typename T>
constexpr int kParts = sizeof(T) == 4 ? 3 : 1;

template <int P>
struct Frag {
    bf16x8 p[P];
};

// How a part is taken from a float. Round: to the nearest bf16, which leaves a
// remainder of either sign and half the size, so that the dropped products are
// small and have no bias. Chop: the upper half of the bits, for products against
// an operand of one part, of which none is dropped; fewer instructions (VJP
// 441172 x 64 x 64 bf16: 51 us, 53 rounded; grad_x 32768 x 512 x 512: 90 and 93).
enum class Cut { Round, Chop };
template <typename T>
constexpr Cut kCut = kParts<T> == 1 ? Cut::Chop : Cut::Round;  // against a stored T

// The next part of a and b, and what remains of them. The first rounded part of
// values above the largest bf16 (3.39e38) is that one, not infinity. (A NaN's
// first part may be a number; its second is a NaN.)
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <Cut C, bool First>
__device__ __forceinline__ uint32_t take_pair(float &a, float &b)
{
    uint32_t u;
    if constexpr (C == Cut::Chop) {
        u = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    } else {
        constexpr float kMost = 0x1.fep127f;
        u = __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(First ? __builtin_amdgcn_fmed3f(a, -kMost, kMost) : a),
                                                static_cast<__bf16>(First ? __builtin_amdgcn_fmed3f(b, -kMost, kMost) : b)});
    }
    a -= __uint_as_float(u << 16);
    b -= __uint_as_float(u & 0xFFFF0000u);
    return u;
}

// N floats as pairs of P bf16 parts; three hold them exactly (below 2^-110, where
// the last is subnormal, to 2^-134).
template <int P, Cut C, int N>
__device__ __forceinline__ void take_parts(const float (&v)[N], uint32_t (&u)[P][N / 2])
{
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        float a = v[2 * i], b = v[2 * i + 1];
        u[0][i] = take_pair<C, true>(a, b);
#pragma unroll
        for (int p = 1; p < P; ++p)
            u[p][i] = take_pair<C, false>(a, b);
    }
}

template <int P, Cut C = Cut::Round>
__device__ __forceinline__ Frag<P> split8(const float (&v)[8])
{
    Frag<P> f;
    uint32_t u[P][4];
    take_parts<P, C>(v, u);
#pragma unroll
    for (int p = 0; p < P; ++p)
        f.p[p] = __builtin_bit_cast(bf16x8, u32x4{u[p][0], u[p][1], u[p][2], u[p][3]});
    return f;
}

// A workgroup barrier for what goes through LDS: it orders LDS accesses only,
// so that loads from memory that were asked for ahead stay in flight across it.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Eight consecutive stored values, the ones from `valid` on zero (not read).
__device__ __forceinline__ void load8(const float *p, int valid, float (&v)[8])
{
    if (valid >= 8) {
        const f32x4 a = *reinterpret_cast<const f32x4_any *>(p), b = *reinterpret_cast<const f32x4_any *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = i < valid ? p[i] : 0.f;
    }
}

__device__ __forceinline__ u32x4 load8(const bf16bits *p, int valid)
{
    if (valid >= 8)
        return *reinterpret_cast<const u32x4_any *>(p);
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        h[i] = i < valid ? p[i] : 0u;
    return u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
}

__device__ __forceinline__ void load8(const bf16bits *p, int valid, float (&v)[8])
{
    const u32x4 u = load8(p, valid);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

// Eight stored values as loaded, turned into floats where they are used (so
// that nothing waits for the load before that).
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
    float v[8];
    __device__ __forceinline__ void load(const float *p, int valid) { load8(p, valid, v); }
    __device__ __forceinline__ void get(float (&o)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = v[i];
    }
    template <int P, Cut C = Cut::Round>
    __device__ __forceinline__ Frag<P> frag() const
    {
        return split8<P, C>(v);
    }
};
template <>
struct Raw8<bf16bits> {
    u32x4 v;
    __device__ __forceinline__ void load(const bf16bits *p, int valid) { v = load8(p, valid); }
    __device__ __forceinline__ void get(float (&o)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(v[i] << 16);
            o[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        }
    }
    template <int P>
    __device__ __forceinline__ Frag<P> frag() const
    {
        static_assert(P == 1, "a bf16 value is one part");
        return {{__builtin_bit_cast(bf16x8, v)}};
    }
};

// Writes eight consecutive values, the first `valid` of them.
__device__ __forceinline__ void store8(float *p, int valid, const float (&v)[8])
{
    if (valid >= 8) {
        *reinterpret_cast<f32x4_any *>(p) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4_any *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid)
                p[i] = v[i];
    }
}

__device__ __forceinline__ void store8(bf16bits *p, int valid, const float (&v)[8])
{
    if (valid >= 8) {
        u32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = from_f32<bf16bits>(v[2 * i]) | static_cast<uint32_t>(from_f32<bf16bits>(v[2 * i + 1])) << 16;
        *reinterpret_cast<u32x4_any *>(p) = u;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid)
                p[i] = from_f32<bf16bits>(v[i]);
    }
}

// Four or eight consecutive values (v holds eight).
template <int N, typename T>
__device__ __forceinline__ void load_n(const T *p, int valid, float (&v)[8])
{
    if constexpr (N == 8) {
        load8(p, valid, v);
    } else if (valid >= 4) {
        const f32x4 a = *reinterpret_cast<const f32x4_any *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = a[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = i < valid ? p[i] : 0.f;
    }
}

template <int N, typename T>
__device__ __forceinline__ void store_n(T *p, int valid, const float (&v)[8])
{
    if constexpr (N == 8) {
        store8(p, valid, v);
    } else if (valid >= 4) {
        *reinterpret_cast<f32x4_any *>(p) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < valid)
                p[i] = v[i];
    }
}

// Sixteen bytes of stored values (four floats, eight bf16) as loaded.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));
template <typename T>
struct RawVec;
template <>
struct RawVec<float> {
    float v[8];
    __device__ __forceinline__ void load(const float *p, int valid) { load_n<4>(p, valid, v); }
    __device__ __forceinline__ float get(int i) const { return v[i]; }
};
template <>
struct RawVec<bf16bits> {
    u32x4 v;
    __device__ __forceinline__ void load(const bf16bits *p, int valid) { v = load8(p, valid); }
    __device__ __forceinline__ float get(int i) const
    {
        return __uint_as_float(i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
    }
};

// N floats (four or eight) as P parts at consecutive places of P planes `plane`
// elements apart.
template <int P, Cut C = Cut::Round, int N>
__device__ __forceinline__ void put_parts(bf16bits *at, int plane, const float (&v)[N])
{
    uint32_t u[P][N / 2];
    take_parts<P, C>(v, u);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if constexpr (N == 8)
            *reinterpret_cast<u32x4 *>(at + p * plane) = u32x4{u[p][0], u[p][1], u[p][2], u[p][3]};
        else
            *reinterpret_cast<uint2 *>(at + p * plane) = uint2{u[p][0], u[p][1]};
    }
}

// acc[i0 + i][j] += a[i] b[j] for all i and j: the products of part u of a and
// v of b up to order u + v = most parts - 1 (three parts: six products; two:
// three; one against P: P), the smallest first, each over all i and j before
// the next, so that instructions that follow each other do not wait for each
// other's result.
template <int PA, int PB, int NA, int NB, int N>
__device__ __forceinline__ void mma(const Frag<PA> (&a)[NA], const Frag<PB> (&b)[NB], f32x4 (&acc)[N][NB], int i0 = 0)
{
#pragma unroll
    for (int s = (PA > PB ? PA : PB) - 1; s >= 0; --s)
#pragma unroll
        for (int u = 0; u < PA; ++u)
            if (s - u >= 0 && s - u < PB) {
#pragma unroll
                for (int i = 0; i < NA; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[i0 + i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i].p[u], b[j].p[s - u],
                                                                                 acc[i0 + i][j], 0, 0, 0);
            }
}

// Fragment of a contraction that runs along the rows of a row-major bf16
// matrix in LDS, rows 32 step .. + 31, columns col0 .. + 15: the transposing
// read hands a lane four rows of its column. Slots 0 .. 3 of quarter q are rows
// 4 q .. + 3 of the step, slots 4 .. 7 the rows 16 below (both operands alike:
// the order within a contraction is free). Rows of 16 bytes more than a
// multiple of 64 are best: 5.6 cycles a read, against 6.9 with 32 bytes more
// (two reads make what one 16-byte read of a row brings in 8.2).
__device__ __forceinline__ bf16x8 read_transposed(const bf16bits *rows, int stride, int step, int col0, int lane)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 *lds4;
    const int q = lane >> 4, l = lane & 15;
    const bf16bits *p = rows + (32 * step + 4 * q + (l >> 2)) * stride + col0 + 4 * (l & 3);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 16 * stride));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

}  // namespace etp
