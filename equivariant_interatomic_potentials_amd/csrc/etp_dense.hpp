// etp_dense.hpp -- device code and launchers shared by the dense operators
// (linear layer, layer norm, grouped layer, orthogonalised update): typed loads
// and stores, activations, launch declarations.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace etp {

using bf16bits = uint16_t;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16bits v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v)
{
    return v;
}
// nearest even; a NaN stays one (the hardware conversion of gfx950)
template <>
__device__ __forceinline__ bf16bits from_f32<bf16bits>(float v)
{
    return __builtin_bit_cast(bf16bits, static_cast<__bf16>(v));
}

// The logistic function 1 / (1 + exp(-z)) from the hardware 2^t (1 ulp) and
// reciprocal (1 ulp): t = -z log2(e) is rounded, and its rounding error r is
// put back as the factor 2^r = 1 + r ln 2. z is clamped to +-128, where the
// result is 1 or (2^t having overflowed) 0 to float precision.
__device__ __forceinline__ float logistic(float z)
{
    const float zc = __builtin_amdgcn_fmed3f(z, -128.f, 128.f);
    constexpr float kL = 1.44269504f, kLlo = 1.92596299e-8f;  // log2(e) in two parts
    const float t = -zc * kL;
    const float r = __builtin_fmaf(-zc, kLlo, __builtin_fmaf(-zc, kL, -t));
    const float e = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(r, 0.693147181f, 1.f);
    return __builtin_amdgcn_rcpf(1.f + e);
}

constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2;

// The normal distribution function and density. With x = |z| / sqrt 2, the
// tail is Phi(-|z|) = exp(-x^2) u(t), t = 1 / (1 + 0.4 x), u the polynomial
// t (c0 + c1 t + ... + c7 t^7) fitted by least squares (reweighted towards the
// smallest largest error) to exp(x^2) erfc(x) / 2 on [0, 9]. With these
// coefficients it is within 4e-9 of Phi; evaluated in float within 2e-7, and
// within 8e-6 of the tail out to |z| = 6. A third of the cost of a
// library erf, which would bound the bf16 forward by its arithmetic.
__device__ __forceinline__ float normal_cdf(float z, float &density)
{
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.4f * 0.707106781f, fabsf(z), 1.f));
    const float e = __builtin_amdgcn_exp2f(-0.721347520f * z * z);
    float p = 0.0387523736f;
    p = __builtin_fmaf(p, t, -0.204188902f);
    p = __builtin_fmaf(p, t, 0.354209376f);
    p = __builtin_fmaf(p, t, -0.197550078f);
    p = __builtin_fmaf(p, t, 0.209061794f);
    p = __builtin_fmaf(p, t, 0.0691124589f);
    p = __builtin_fmaf(p, t, 0.118083984f);
    p = __builtin_fmaf(p, t, 0.112518994f);
    const float tail = p * t * e;
    density = 0.398942280f * e;
    return z > 0.f ? 1.f - tail : tail;
}

__device__ __forceinline__ float act_value(int act, float z)
{
    if (act == kActSilu)
        return z * logistic(z);
    if (act == kActGelu) {
        float density;
        return z * normal_cdf(z, density);
    }
    return z;
}

__device__ __forceinline__ float act_slope(int act, float z)
{
    if (act == kActSilu) {
        const float s = logistic(z);
        return s * __builtin_fmaf(z, 1.f - s, 1.f);
    }
    if (act == kActGelu) {
        float density;
        const float cdf = normal_cdf(z, density);
        return __builtin_fmaf(z, density, cdf);
    }
    return 1.f;
}

struct LinearArgs {
    int64_t M;  // rows
    int K, N;   // n_in, n_out
    bool bf16;
    const void *x;
    int64_t ldx;
    const void *W;
    const float *bias;
    int act;
    const void *res;
    int64_t ldr;
    void *y;
    int64_t ldy;
    void *z;
    int64_t ldz;
};
hipError_t launch_linear(const LinearArgs &a, hipStream_t stream);

struct LinearVjpArgs {
    int64_t M;
    int K, N;
    bool bf16, accumulate;
    const void *x;
    int64_t ldx;
    const void *W;
    const void *z;
    int64_t ldz;
    int act;
    const void *gy;
    int64_t ldgy;
    void *gx;
    int64_t ldgx;
    float *gW, *gb;
    void *ws;
};
size_t linear_vjp_workspace_bytes(int64_t M, int K, int N, bool bf16);
hipError_t launch_linear_vjp(const LinearVjpArgs &a, hipStream_t stream);

struct NormArgs {
    int64_t M;
    int C;
    bool bf16;
    const void *x;
    int64_t ldx;
    const float *gamma, *beta;
    float eps;
    void *y;
    int64_t ldy;
    float *mean, *rstd;
};
hipError_t launch_layer_norm(const NormArgs &a, hipStream_t stream);

struct NormVjpArgs {
    int64_t M;
    int C;
    bool bf16, accumulate;
    const void *x;
    int64_t ldx;
    const float *gamma, *mean, *rstd;
    const void *gy;
    int64_t ldgy;
    void *gx;
    int64_t ldgx;
    float *ggamma, *gbeta;
    void *ws;
};
size_t layer_norm_vjp_workspace_bytes(int64_t M, int C, bool bf16);
hipError_t launch_layer_norm_vjp(const NormVjpArgs &a, hipStream_t stream);

struct OrthArgs {
    int B, rows, cols;
    bool bf16;
    const void *G;
    int steps;
    float coef[3];
    float eps;
    void *X;
    void *ws;
};
size_t orthogonalize_workspace_bytes(int B, int rows, int cols);
hipError_t launch_orthogonalize(const OrthArgs &a, hipStream_t stream);

// The linear layer with a matrix for each group of rows: W, bias, gW and gb are
// those of group 0, the others follow.
struct GroupedLinearArgs {
    LinearArgs l;
    int n_groups;
    const int *group_ptr, *order;
};
hipError_t launch_grouped_linear(const GroupedLinearArgs &a, hipStream_t stream);

struct GroupedLinearVjpArgs {
    LinearVjpArgs v;
    int n_groups;
    const int *group_ptr, *order;
};
size_t grouped_linear_vjp_workspace_bytes(int64_t M, int G, int K, int N, bool bf16);
hipError_t launch_grouped_linear_vjp(const GroupedLinearVjpArgs &a, hipStream_t stream);

size_t group_rows_workspace_bytes(int64_t M, int G);
hipError_t launch_group_rows(int64_t M, int G, const int *ids, int *ptr, int *order, void *ws, hipStream_t stream);

// Sums of n sets of partial column sums: a set is n0 values that add up to
// out0 and n1 more for out1 (either output may be null: not written); n = 0
// writes zeros. Accumulating adds to what the outputs hold.
hipError_t launch_sum_parts(int64_t n0, float *out0, int64_t n1, float *out1, int n, const float *part,
                            bool accumulate, hipStream_t stream);

}  // namespace etp
