// etp_layer_norm.hip -- the layer norm over the columns of each row, and its
// VJP with the weights' gradients.
//
// Both are one pass over the data, bound by HBM. LPR lanes (a power of two up
// to the wave) own a row and hold it in registers, 16 bytes a load, so that
// mean, variance (from the differences) and the result come from one read;
// sums over the row are exchanges between the LPR lanes. The mean is taken
// twice, of the row and of the differences from that, so that rows with a
// common offset (constant ones among them) keep the digits of their spread
// (32768 x 512 bf16 12.4 -> 12.7 us). A lane keeps the same columns for every
// row it meets, so gamma and beta are read once and the VJP's column sums grow
// in registers; waves walk the rows with the grid's stride and load the next
// row while they work on the present one. Rows of more than 2048 columns take a
// workgroup each and read the row again (from cache) for every sum.
//
// Measured: forward 32768 x 512 bf16 12.7 us (5.3 TB/s, part of it from
// cache); VJP 441172 x 64 float 66 us (5.2 TB/s), 5184 x 777 bf16 16 us (1.5
// TB/s: two launches, and rows of 1554 bytes on any alignment), 50000 x 2000
// float 240 us (5.0 TB/s).
#include "etp_dense_mma.hpp"

namespace etp {

template <int Ctrl>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), Ctrl, 0xF, 0xF, true));
}

// Sum over aligned groups of N lanes, in every lane of the group.
template <int N>
__device__ __forceinline__ float group_sum(float v)
{
    if constexpr (N >= 2)
        v = dpp_add<0xB1>(v);  // quad_perm 1,0,3,2
    if constexpr (N >= 4)
        v = dpp_add<0x4E>(v);  // quad_perm 2,3,0,1
    if constexpr (N >= 8)
        v = dpp_add<0x141>(v);  // row_half_mirror
    if constexpr (N >= 16)
        v = dpp_add<0x140>(v);  // row_mirror
    if constexpr (N >= 32) {  // rows of 16 lanes with their neighbours, then the wave's halves
        const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(w[0]) + __uint_as_float(w[1]);
    }
    if constexpr (N >= 64) {
        const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(w[0]) + __uint_as_float(w[1]);
    }
    return v;
}

// s / c from inv = 1 / c with one correction, so that a quotient that is a
// float comes out exactly.
__device__ __forceinline__ float quotient(float s, float c, float inv)
{
    const float m = s * inv;
    return __builtin_fmaf(__builtin_fmaf(-m, c, s), inv, m);
}

// The columns of lane l of a row's LPR lanes: vector n holds kVec columns
// from col[n], its own ones the entries [lo[n], hi). The last vector of a
// ragged row is moved back to end at the row's end (its first entries belong
// to the vector before it), so that every load is a whole vector; only rows
// shorter than a vector are loaded by parts.
template <typename T, int LPR, int NI, bool RAG>
struct Columns {
    int col[NI], lo[NI], hi;
    __device__ __forceinline__ Columns(int l, int C)
    {
        constexpr int V = kVec<T>;
        hi = RAG && C < V ? C : V;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int want = (n * LPR + l) * V;
            const int last = C > V ? C - V : 0;
            col[n] = RAG && want > last ? last : want;
            lo[n] = RAG ? (want - col[n] < V ? want - col[n] : V) : 0;
        }
    }
    __device__ __forceinline__ bool own(int n, int i) const { return !RAG || (i >= lo[n] && i < hi); }
    // row: the row's first element; entries that are not own hold anything
    __device__ __forceinline__ void load(const T *row, int n, RawVec<T> &v) const { v.load(row + col[n], hi); }
    __device__ __forceinline__ void store(T *row, int n, const float (&v)[8]) const
    {
        constexpr int V = kVec<T>;
        if (!RAG || (lo[n] == 0 && hi == V)) {
            store_n<V>(row + col[n], V, v);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (own(n, i))
                    row[col[n] + i] = from_f32<T>(v[i]);
        }
    }
    // the columns' entries of a weight vector, `none` where there is no vector
    __device__ __forceinline__ void weights(const float *w, int n, float none, float (&v)[kVec<T>]) const
    {
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u[i] = none;
        if (w)
            load_n<kVec<T>>(w + col[n], hi, u);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            v[i] = u[i];
    }
};

template <typename T, int LPR, int NI, bool RAG>
__global__ void __launch_bounds__(256) layer_norm_kernel(const NormArgs a)
{
    constexpr int V = kVec<T>, RPW = 64 / LPR;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Columns<T, LPR, NI, RAG> cs(lane % LPR, a.C);
    float gamma[NI][V], beta[NI][V];
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        cs.weights(a.gamma, n, 1.f, gamma[n]);
        cs.weights(a.beta, n, 0.f, beta[n]);
    }
    const float inv = 1.f / static_cast<float>(a.C);
    const int64_t step = static_cast<int64_t>(gridDim.x) * 4 * RPW;
    int64_t r = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * RPW + lane / LPR;
    float x[NI][V];
    RawVec<T> nx[NI];
    auto fetch = [&](int64_t row) {
        const T *p = static_cast<const T *>(a.x) + (row < a.M ? row : a.M - 1) * a.ldx;
#pragma unroll
        for (int n = 0; n < NI; ++n)
            cs.load(p, n, nx[n]);
    };
    fetch(r);
    for (int64_t r0 = r - lane / LPR; r0 < a.M; r0 += step, r += step) {
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[n][i] = nx[n].get(i);
        if (r0 + step < a.M)
            fetch(r + step);
        float s = 0.f;
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i)
                s += cs.own(n, i) ? x[n][i] : 0.f;
        float mean = quotient(group_sum<LPR>(s), static_cast<float>(a.C), inv);
        // the row's sum has rounded at the size of its values: the differences,
        // at the size of their spread, give what the mean is off by
        s = 0.f;
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[n][i] = cs.own(n, i) ? x[n][i] - mean : 0.f;
                s += x[n][i];
            }
        const float off = group_sum<LPR>(s) * inv;
        mean += off;
        float v = 0.f;
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[n][i] = cs.own(n, i) ? x[n][i] - off : 0.f;
                v = __builtin_fmaf(x[n][i], x[n][i], v);
            }
        const float rstd = 1.f / sqrtf(__builtin_fmaf(group_sum<LPR>(v), inv, a.eps));
        if (r >= a.M)
            continue;
        T *y = static_cast<T *>(a.y) + r * a.ldy;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            float o[8];
#pragma unroll
            for (int i = 0; i < V; ++i)
                o[i] = __builtin_fmaf(x[n][i] * rstd, gamma[n][i], beta[n][i]);
            cs.store(y, n, o);
        }
        if (lane % LPR == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
    }
}

constexpr int kVjpWaves = 8;

// Input gradient and this workgroup's column sums, part[b][0][c] = sum gy h,
// part[b][1][c] = sum gy over its rows: lanes, then the wave's row groups,
// then the waves in turn.
template <typename T, int LPR, int NI, bool RAG>
__global__ void __launch_bounds__(64 * kVjpWaves) layer_norm_vjp_kernel(const NormVjpArgs a)
{
    constexpr int V = kVec<T>, RPW = 64 / LPR;
    __shared__ float sums[2][LPR * NI * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Columns<T, LPR, NI, RAG> cs(lane % LPR, a.C);
    float gamma[NI][V], gg[NI][V], gb[NI][V];
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        cs.weights(a.gamma, n, 1.f, gamma[n]);
#pragma unroll
        for (int i = 0; i < V; ++i)
            gg[n][i] = gb[n][i] = 0.f;
    }
    const float inv = 1.f / static_cast<float>(a.C);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kVjpWaves * RPW;
    int64_t r = (static_cast<int64_t>(blockIdx.x) * kVjpWaves + wave) * RPW + lane / LPR;
    RawVec<T> nx[NI], ng[NI];
    float nmean, nrstd;
    auto fetch = [&](int64_t row) {
        const int64_t rc = row < a.M ? row : a.M - 1;
        const T *p = static_cast<const T *>(a.x) + rc * a.ldx, *g = static_cast<const T *>(a.gy) + rc * a.ldgy;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            cs.load(p, n, nx[n]);
            cs.load(g, n, ng[n]);
        }
        nmean = a.mean[rc];
        nrstd = a.rstd[rc];
    };
    // 32 floats a lane leave no registers for a row ahead
    constexpr bool kAhead = !(sizeof(T) == 4 && NI == 8);
    if (kAhead)
        fetch(r);
    for (int64_t r0 = r - lane / LPR; r0 < a.M; r0 += step, r += step) {
        if (!kAhead)
            fetch(r);
        float h[NI][V], g[NI][V];
        const float mean = nmean, rstd = nrstd;
        const bool live = r < a.M;
        float s = 0.f, t = 0.f;
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool own = live && cs.own(n, i);
                g[n][i] = own ? ng[n].get(i) : 0.f;
                h[n][i] = own ? (nx[n].get(i) - mean) * rstd : 0.f;
            }
        if (kAhead && r0 + step < a.M)
            fetch(r + step);
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                gg[n][i] = __builtin_fmaf(g[n][i], h[n][i], gg[n][i]);
                gb[n][i] += g[n][i];
                g[n][i] *= gamma[n][i];
                s += g[n][i];
                t = __builtin_fmaf(g[n][i], h[n][i], t);
            }
        if (!a.gx)
            continue;
        s = group_sum<LPR>(s) * inv;
        t = group_sum<LPR>(t) * inv;
        if (!live)
            continue;
        T *gx = static_cast<T *>(a.gx) + r * a.ldgx;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            float o[8];
            RawVec<T> was;
            if (a.accumulate)
                cs.load(gx, n, was);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                o[i] = rstd * (g[n][i] - s - h[n][i] * t);
                if (a.accumulate)
                    o[i] += was.get(i);
            }
            cs.store(gx, n, o);
        }
    }
    if (!a.ws)
        return;
#pragma unroll
    for (int n = 0; n < NI; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int m = LPR; m < 64; m <<= 1) {
                gg[n][i] += __shfl_xor(gg[n][i], m);
                gb[n][i] += __shfl_xor(gb[n][i], m);
            }
        }
    for (int w = 0; w < kVjpWaves; ++w) {
        if (wave == w && lane < LPR) {
#pragma unroll
            for (int n = 0; n < NI; ++n)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = (n * V + i) * LPR + lane;
                    sums[0][e] = w ? sums[0][e] + gg[n][i] : gg[n][i];
                    sums[1][e] = w ? sums[1][e] + gb[n][i] : gb[n][i];
                }
        }
        __syncthreads();
    }
    float *part = static_cast<float *>(a.ws) + static_cast<int64_t>(blockIdx.x) * 2 * a.C;
    for (int k = threadIdx.x; k < 2 * LPR * NI * V; k += 64 * kVjpWaves) {
        const int w = k >= LPR * NI * V, e = k - w * LPR * NI * V;  // e: column order
        const int vec = e / V, i = e % V, want = vec * V, last = a.C > V ? a.C - V : 0;
        const int c = (RAG && want > last ? last : want) + i;  // the vector's column (Columns)
        if (c >= want && c < a.C)
            part[w * a.C + c] = sums[w][(vec / LPR * V + i) * LPR + vec % LPR];
    }
}

// --------------------------------------------------------------- long rows

__device__ __forceinline__ float wave_sum(float v) { return group_sum<64>(v); }
__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int m = 32; m; m >>= 1)
        v += __shfl_xor(v, m);
    return v;
}

// sum over the workgroup's 256 threads, in every thread
template <typename S>
__device__ __forceinline__ S block_sum(S v, S *lds)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

template <typename T>
__global__ void __launch_bounds__(256) layer_norm_long_kernel(const NormArgs a)
{
    __shared__ float lds[4];
    __shared__ double wide[4];
    const float inv = 1.f / static_cast<float>(a.C);
    for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + r * a.ldx;
        // the mean as a float and what that is off by, from a double sum (another
        // pass over the differences, as for short rows, took 15 to 30% longer)
        double s = 0.0;
        for (int c = threadIdx.x; c < a.C; c += 256)
            s += to_f32(x[c]);
        s = block_sum(s, wide) / a.C;
        const float mean = static_cast<float>(s), off = static_cast<float>(s - mean);
        float q = 0.f;
        for (int c = threadIdx.x; c < a.C; c += 256) {
            const float d = to_f32(x[c]) - mean - off;
            q = __builtin_fmaf(d, d, q);
        }
        const float rstd = 1.f / sqrtf(__builtin_fmaf(block_sum(q, lds), inv, a.eps));
        T *y = static_cast<T *>(a.y) + r * a.ldy;
        for (int c = threadIdx.x; c < a.C; c += 256)
            y[c] = from_f32<T>(__builtin_fmaf((to_f32(x[c]) - mean - off) * rstd, a.gamma ? a.gamma[c] : 1.f,
                                              a.beta ? a.beta[c] : 0.f));
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) layer_norm_long_gx_kernel(const NormVjpArgs a)
{
    __shared__ float lds[4];
    const float inv = 1.f / static_cast<float>(a.C);
    for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + r * a.ldx, *gy = static_cast<const T *>(a.gy) + r * a.ldgy;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s = 0.f, t = 0.f;
        for (int c = threadIdx.x; c < a.C; c += 256) {
            const float h = (to_f32(x[c]) - mean) * rstd, d = to_f32(gy[c]) * (a.gamma ? a.gamma[c] : 1.f);
            s += d;
            t = __builtin_fmaf(d, h, t);
        }
        s = block_sum(s, lds) * inv;
        t = block_sum(t, lds) * inv;
        T *gx = static_cast<T *>(a.gx) + r * a.ldgx;
        for (int c = threadIdx.x; c < a.C; c += 256) {
            const float h = (to_f32(x[c]) - mean) * rstd, d = to_f32(gy[c]) * (a.gamma ? a.gamma[c] : 1.f);
            const float g = rstd * (d - s - h * t);
            gx[c] = from_f32<T>(a.accumulate ? to_f32(gx[c]) + g : g);
        }
    }
}

// part[s][0][c] = sum over the rows of split s of gy h, part[s][1][c] of gy
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_long_gw_kernel(const NormVjpArgs a, const int nsplit)
{
    const int c = blockIdx.x * 256 + threadIdx.x, s = blockIdx.y;
    if (c >= a.C)
        return;
    const int64_t r0 = a.M * s / nsplit, r1 = a.M * (s + 1) / nsplit;
    float gg = 0.f, gb = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float g = to_f32(static_cast<const T *>(a.gy)[r * a.ldgy + c]);
        const float h = (to_f32(static_cast<const T *>(a.x)[r * a.ldx + c]) - a.mean[r]) * a.rstd[r];
        gg = __builtin_fmaf(g, h, gg);
        gb += g;
    }
    float *part = static_cast<float *>(a.ws) + static_cast<int64_t>(s) * 2 * a.C;
    part[c] = gg;
    part[a.C + c] = gb;
}

// ----------------------------------------------------------------- dispatch

constexpr int kLongRow = 2048;

// How rows of C <= 2048 columns lie in a wave: lanes per row and vectors per
// lane. Several rows a wave and sums within 16 lanes come first; the forward
// holds up to 32 columns a lane, the VJP, which needs six registers a column,
// 16 where the row allows it.
struct NormShape {
    int lpr, ni;
};

static constexpr NormShape norm_shape(int C, int V, bool vjp)
{
    const int vecs = (C + V - 1) / V, most = vjp && V == 8 ? 2 : 4;
    int lpr = 1;
    while (lpr < 16 && lpr < vecs)
        lpr *= 2;
    int ni = 1;
    while (ni < most && lpr * ni < vecs)
        ni *= 2;
    while (lpr < 64 && lpr * ni < vecs)
        lpr *= 2;
    while (lpr * ni < vecs)
        ni *= 2;
    return {lpr, ni};
}

// Calls f(LPR, NI, RAG) for rows of C columns in vectors of V; only shapes that
// some row has are compiled.
template <int V, bool Vjp, int LPR, int NI>
constexpr bool norm_shape_taken()
{
    constexpr NormShape s = norm_shape(LPR * NI * V, V, Vjp);  // (a shape's longest row is a full one)
    return LPR * NI * V <= kLongRow && s.lpr == LPR && s.ni == NI;
}

template <int V, bool Vjp, typename F>
static hipError_t by_shape(int C, F &&f)
{
    const NormShape s = norm_shape(C, V, Vjp);
#define ETP_NORM_CASE(L, N)                                                                                   \
    if constexpr (norm_shape_taken<V, Vjp, L, N>())                                                           \
        if (s.lpr == L && s.ni == N)                                                                          \
            return C == L * N * V ? f(std::integral_constant<int, L>{}, std::integral_constant<int, N>{},     \
                                      std::false_type{})                                                      \
                                  : f(std::integral_constant<int, L>{}, std::integral_constant<int, N>{},     \
                                      std::true_type{});
    ETP_NORM_CASE(1, 1)
    ETP_NORM_CASE(2, 1)
    ETP_NORM_CASE(4, 1)
    ETP_NORM_CASE(8, 1)
    ETP_NORM_CASE(16, 1)
    ETP_NORM_CASE(16, 2)
    ETP_NORM_CASE(16, 4)
    ETP_NORM_CASE(32, 2)
    ETP_NORM_CASE(32, 4)
    ETP_NORM_CASE(64, 2)
    ETP_NORM_CASE(64, 4)
    ETP_NORM_CASE(64, 8)
#undef ETP_NORM_CASE
    return hipErrorInvalidValue;
}

// Workgroups of `waves` waves over M rows, of which a wave takes rpw at a time.
static int64_t norm_blocks(int64_t M, int rpw, int waves)
{
    return (M + static_cast<int64_t>(waves) * rpw - 1) / (static_cast<int64_t>(waves) * rpw);
}

static unsigned norm_grid(int64_t M, int rpw, int most)
{
    const int64_t b = norm_blocks(M, rpw, 4);
    return static_cast<unsigned>(b < most ? b : most);
}

template <typename T>
static hipError_t norm_forward(const NormArgs &a, hipStream_t stream)
{
    if (a.C > kLongRow) {
        hipLaunchKernelGGL(layer_norm_long_kernel<T>, dim3(norm_grid(a.M, 1, 2048)), dim3(256), 0, stream, a);
        return hipGetLastError();
    }
    return by_shape<kVec<T>, false>(a.C, [&](auto l, auto n, auto rag) {
        hipLaunchKernelGGL((layer_norm_kernel<T, l(), n(), rag()>), dim3(norm_grid(a.M, 64 / l(), 1024)), dim3(256), 0,
                           stream, a);
        return hipGetLastError();
    });
}

hipError_t launch_layer_norm(const NormArgs &a, hipStream_t stream)
{
    if (a.M == 0)
        return hipSuccess;
    return a.bf16 ? norm_forward<bf16bits>(a, stream) : norm_forward<float>(a, stream);
}

// Partial column sums of the VJP: one set per workgroup, as many workgroups
// as the registers let run at once (two a compute unit up to eight columns a
// lane: 66 us against 70 with four, 75 with one, on 441172 x 64 floats; one
// beyond: 16 us against 22 with more, on 5184 x 777 bf16), all with the same
// number of turns.
static int norm_parts(int64_t M, int C, bool bf16)
{
    if (C > kLongRow) {
        const int64_t s = M / 16;
        return static_cast<int>(s < 1 ? 1 : s > 512 ? 512 : s);
    }
    const int V = bf16 ? 8 : 4;
    const NormShape s = norm_shape(C, V, true);
    const int64_t blocks = norm_blocks(M, 64 / s.lpr, kVjpWaves), most = s.ni * V <= 8 ? 512 : 256;
    const int64_t turns = (blocks + most - 1) / most;
    return static_cast<int>((blocks + turns - 1) / turns);
}

size_t layer_norm_vjp_workspace_bytes(int64_t M, int C, bool bf16)
{
    return M == 0 ? 0 : sizeof(float) * 2 * static_cast<size_t>(norm_parts(M, C, bf16)) * C;
}

template <typename T>
static hipError_t norm_vjp(const NormVjpArgs &a, int S, hipStream_t stream)
{
    if (a.C > kLongRow) {
        if (a.gx)
            hipLaunchKernelGGL(layer_norm_long_gx_kernel<T>, dim3(norm_grid(a.M, 1, 2048)), dim3(256), 0, stream, a);
        if (a.ws)
            hipLaunchKernelGGL(layer_norm_long_gw_kernel<T>, dim3(static_cast<unsigned>((a.C + 255) / 256), S),
                               dim3(256), 0, stream, a, S);
        return hipGetLastError();
    }
    return by_shape<kVec<T>, true>(a.C, [&](auto l, auto n, auto rag) {
        hipLaunchKernelGGL((layer_norm_vjp_kernel<T, l(), n(), rag()>), dim3(static_cast<unsigned>(S)),
                           dim3(64 * kVjpWaves), 0, stream, a);
        return hipGetLastError();
    });
}

hipError_t launch_layer_norm_vjp(const NormVjpArgs &args, hipStream_t stream)
{
    NormVjpArgs a = args;
    const bool sums = a.ggamma || a.gbeta;
    if (!sums)
        a.ws = nullptr;
    const int S = a.M == 0 ? 0 : norm_parts(a.M, a.C, a.bf16);
    hipError_t e = hipSuccess;
    if (S > 0 && (a.gx || sums))
        e = a.bf16 ? norm_vjp<bf16bits>(a, S, stream) : norm_vjp<float>(a, S, stream);
    const float *part = static_cast<const float *>(a.ws);
    if (e == hipSuccess && sums)
        e = launch_sum_parts(a.C, a.ggamma, a.C, a.gbeta, S, part, a.accumulate, stream);
    return e;
}

}  // namespace etp
