// etp_layer_norm.hip -- the layer norm over the columns of each row, and its
// VJP with the weights' gradients.
#include "etp_dense.hpp"

namespace etp {

__device__ __forceinline__ float wave_sum_xor(float v)
{
#pragma unroll
    for (int m = 32; m; m >>= 1)
        v += __shfl_xor(v, m);
    return v;
}

// a wave per row
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_kernel(const NormArgs a)
{
    const int lane = threadIdx.x & 63;
    for (int64_t r = blockIdx.x * 4ll + (threadIdx.x >> 6); r < a.M; r += gridDim.x * 4ll) {
        const T *x = static_cast<const T *>(a.x) + r * a.ldx;
        float s = 0.f;
        for (int c = lane; c < a.C; c += 64)
            s += to_f32(x[c]);
        const float mean = wave_sum_xor(s) / a.C;
        float q = 0.f;
        for (int c = lane; c < a.C; c += 64) {
            const float d = to_f32(x[c]) - mean;
            q = __builtin_fmaf(d, d, q);
        }
        const float rstd = 1.f / sqrtf(wave_sum_xor(q) / a.C + a.eps);
        T *y = static_cast<T *>(a.y) + r * a.ldy;
        for (int c = lane; c < a.C; c += 64) {
            const float h = (to_f32(x[c]) - mean) * rstd;
            y[c] = from_f32<T>(__builtin_fmaf(h, a.gamma ? a.gamma[c] : 1.f, a.beta ? a.beta[c] : 0.f));
        }
        if (lane == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) layer_norm_gx_kernel(const NormVjpArgs a)
{
    const int lane = threadIdx.x & 63;
    for (int64_t r = blockIdx.x * 4ll + (threadIdx.x >> 6); r < a.M; r += gridDim.x * 4ll) {
        const T *x = static_cast<const T *>(a.x) + r * a.ldx, *gy = static_cast<const T *>(a.gy) + r * a.ldgy;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s = 0.f, t = 0.f;
        for (int c = lane; c < a.C; c += 64) {
            const float h = (to_f32(x[c]) - mean) * rstd, d = to_f32(gy[c]) * (a.gamma ? a.gamma[c] : 1.f);
            s += d;
            t = __builtin_fmaf(d, h, t);
        }
        s = wave_sum_xor(s) / a.C;
        t = wave_sum_xor(t) / a.C;
        T *gx = static_cast<T *>(a.gx) + r * a.ldgx;
        for (int c = lane; c < a.C; c += 64) {
            const float h = (to_f32(x[c]) - mean) * rstd, d = to_f32(gy[c]) * (a.gamma ? a.gamma[c] : 1.f);
            const float g = rstd * (d - s - h * t);
            gx[c] = from_f32<T>(a.accumulate ? to_f32(gx[c]) + g : g);
        }
    }
}

// part[s][0][c] = sum over the rows of split s of gy h, part[s][1][c] of gy
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_gw_kernel(const NormVjpArgs a, const int nsplit)
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

static unsigned row_grid(int64_t M)
{
    const int64_t b = (M + 3) / 4;
    return static_cast<unsigned>(b < 8192 ? b : 8192);
}

hipError_t launch_layer_norm(const NormArgs &a, hipStream_t stream)
{
    if (a.M == 0)
        return hipSuccess;
    if (a.bf16)
        hipLaunchKernelGGL(layer_norm_kernel<bf16bits>, dim3(row_grid(a.M)), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(layer_norm_kernel<float>, dim3(row_grid(a.M)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

static int norm_splits(int64_t M)
{
    const int64_t s = M / 16;
    return static_cast<int>(s < 1 ? 1 : s > 512 ? 512 : s);
}

size_t layer_norm_vjp_workspace_bytes(int64_t M, int C, bool)
{
    return M == 0 ? 0 : sizeof(float) * 2 * static_cast<size_t>(norm_splits(M)) * C;
}

hipError_t launch_layer_norm_vjp(const NormVjpArgs &a, hipStream_t stream)
{
    if (a.M > 0 && a.gx) {
        if (a.bf16)
            hipLaunchKernelGGL(layer_norm_gx_kernel<bf16bits>, dim3(row_grid(a.M)), dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL(layer_norm_gx_kernel<float>, dim3(row_grid(a.M)), dim3(256), 0, stream, a);
    }
    if (!a.ggamma && !a.gbeta)
        return hipGetLastError();
    const int S = a.M == 0 ? 0 : norm_splits(a.M);
    if (S > 0) {
        const dim3 grid(static_cast<unsigned>((a.C + 255) / 256), S);
        if (a.bf16)
            hipLaunchKernelGGL(layer_norm_gw_kernel<bf16bits>, grid, dim3(256), 0, stream, a, S);
        else
            hipLaunchKernelGGL(layer_norm_gw_kernel<float>, grid, dim3(256), 0, stream, a, S);
    }
    const float *part = static_cast<const float *>(a.ws);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.ggamma)
        e = launch_sum_parts(a.C, S, 2 * a.C, part, a.ggamma, a.accumulate, stream);
    if (e == hipSuccess && a.gbeta)
        e = launch_sum_parts(a.C, S, 2 * a.C, part ? part + a.C : nullptr, a.gbeta, a.accumulate, stream);
    return e;
}

}  // namespace etp
