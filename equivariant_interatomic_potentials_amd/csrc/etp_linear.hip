// etp_linear.hip -- the linear layer with bias, activation and residual, and
// its VJP.
#include "etp_dense.hpp"

namespace etp {

// y = act(x W + bias) + res: a 16 x 16 output tile per workgroup, x and W
// through LDS in chunks of 16 of the inner dimension.
template <typename T>
__global__ void __launch_bounds__(256) linear_kernel(const LinearArgs a)
{
    __shared__ float xs[16][17], wsh[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 16 + ty;
    const int j = blockIdx.y * 16 + tx;
    const T *x = static_cast<const T *>(a.x), *W = static_cast<const T *>(a.W);
    float acc = 0.f;
    for (int k0 = 0; k0 < a.K; k0 += 16) {
        xs[ty][tx] = r < a.M && k0 + tx < a.K ? to_f32(x[r * a.ldx + k0 + tx]) : 0.f;
        wsh[ty][tx] = j < a.N && k0 + ty < a.K ? to_f32(W[static_cast<int64_t>(k0 + ty) * a.N + j]) : 0.f;
        __syncthreads();
        for (int k = 0; k < 16; ++k)
            acc = __builtin_fmaf(xs[ty][k], wsh[k][tx], acc);
        __syncthreads();
    }
    if (r >= a.M || j >= a.N)
        return;
    const float z = acc + (a.bias ? a.bias[j] : 0.f);
    float y = act_value(a.act, z);
    if (a.res)
        y += to_f32(static_cast<const T *>(a.res)[r * a.ldr + j]);
    static_cast<T *>(a.y)[r * a.ldy + j] = from_f32<T>(y);
    if (a.z)
        static_cast<T *>(a.z)[r * a.ldz + j] = from_f32<T>(z);
}

template <typename T>
__device__ __forceinline__ float slope_grad(const LinearVjpArgs &a, int64_t r, int j)
{
    const float g = to_f32(static_cast<const T *>(a.gy)[r * a.ldgy + j]);
    return a.act == kActNone ? g : g * act_slope(a.act, to_f32(static_cast<const T *>(a.z)[r * a.ldz + j]));
}

// gx = d W^T, d = gy act'(z)
template <typename T>
__global__ void __launch_bounds__(256) linear_gx_kernel(const LinearVjpArgs a)
{
    __shared__ float ds[16][17], wsh[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 16 + ty;
    const int k = blockIdx.y * 16 + tx;
    const T *W = static_cast<const T *>(a.W);
    float acc = 0.f;
    for (int j0 = 0; j0 < a.N; j0 += 16) {
        ds[ty][tx] = r < a.M && j0 + tx < a.N ? slope_grad<T>(a, r, j0 + tx) : 0.f;
        const int kw = blockIdx.y * 16 + ty;
        wsh[ty][tx] = kw < a.K && j0 + tx < a.N ? to_f32(W[static_cast<int64_t>(kw) * a.N + j0 + tx]) : 0.f;
        __syncthreads();
        for (int j = 0; j < 16; ++j)
            acc = __builtin_fmaf(ds[ty][j], wsh[tx][j], acc);
        __syncthreads();
    }
    if (r >= a.M || k >= a.K)
        return;
    T *o = static_cast<T *>(a.gx) + r * a.ldgx + k;
    *o = from_f32<T>(a.accumulate ? to_f32(*o) + acc : acc);
}

// part[s][k][j] = sum over the rows of split s of x[r][k] d[r][j]; the row
// k = K holds sum d (the bias gradient)
template <typename T>
__global__ void __launch_bounds__(256) linear_gw_kernel(const LinearVjpArgs a, const int nsplit)
{
    __shared__ float xs[16][17], ds[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int k = blockIdx.x * 16 + ty, j = blockIdx.y * 16 + tx, s = blockIdx.z;
    const int64_t r0 = a.M * s / nsplit, r1 = a.M * (s + 1) / nsplit;
    const T *x = static_cast<const T *>(a.x);
    float acc = 0.f;
    for (int64_t r = r0; r < r1; r += 16) {
        const int kk = blockIdx.x * 16 + tx;
        const bool ok = r + ty < r1;
        xs[ty][tx] = !ok || kk > a.K ? 0.f : kk == a.K ? 1.f : x ? to_f32(x[(r + ty) * a.ldx + kk]) : 0.f;
        ds[ty][tx] = ok && j < a.N ? slope_grad<T>(a, r + ty, j) : 0.f;
        __syncthreads();
        for (int i = 0; i < 16; ++i)
            acc = __builtin_fmaf(xs[i][ty], ds[i][tx], acc);
        __syncthreads();
    }
    if (k <= a.K && j < a.N)
        static_cast<float *>(a.ws)[(static_cast<int64_t>(s) * (a.K + 1) + k) * a.N + j] = acc;
}

__global__ void __launch_bounds__(256) sum_parts_kernel(const int64_t count, const int n, const int64_t stride,
                                                        const float *__restrict__ part, float *__restrict__ out,
                                                        const int accumulate)
{
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < count; i += gridDim.x * 256ll) {
        float v = 0.f;
        for (int s = 0; s < n; ++s)
            v += part[s * stride + i];
        out[i] = accumulate ? out[i] + v : v;
    }
}

hipError_t launch_sum_parts(int64_t count, int n, int64_t stride, const float *part, float *out, bool accumulate,
                            hipStream_t stream)
{
    const int64_t blocks = (count + 255) / 256;
    hipLaunchKernelGGL(sum_parts_kernel, dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)), dim3(256), 0,
                       stream, count, n, stride, part, out, accumulate ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_linear(const LinearArgs &a, hipStream_t stream)
{
    if (a.M == 0)
        return hipSuccess;
    const dim3 grid(static_cast<unsigned>((a.M + 15) / 16), static_cast<unsigned>((a.N + 15) / 16));
    if (a.bf16)
        hipLaunchKernelGGL(linear_kernel<bf16bits>, grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(linear_kernel<float>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

// Splits of the rows for the weight gradient: enough workgroups to fill the
// chip, at least 64 rows each.
static int gw_splits(int64_t M, int K, int N)
{
    const int64_t tiles = static_cast<int64_t>((K + 1 + 15) / 16) * ((N + 15) / 16);
    int64_t s = (2048 + tiles - 1) / tiles;
    s = s < M / 64 ? s : M / 64;
    return static_cast<int>(s < 1 ? 1 : s > 256 ? 256 : s);
}

size_t linear_vjp_workspace_bytes(int64_t M, int K, int N, bool)
{
    return M == 0 ? 0 : sizeof(float) * static_cast<size_t>(gw_splits(M, K, N)) * (K + 1) * static_cast<size_t>(N);
}

hipError_t launch_linear_vjp(const LinearVjpArgs &a, hipStream_t stream)
{
    const int64_t kn = static_cast<int64_t>(a.K) * a.N;
    if (a.M > 0 && a.gx) {
        const dim3 grid(static_cast<unsigned>((a.M + 15) / 16), static_cast<unsigned>((a.K + 15) / 16));
        if (a.bf16)
            hipLaunchKernelGGL(linear_gx_kernel<bf16bits>, grid, dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL(linear_gx_kernel<float>, grid, dim3(256), 0, stream, a);
    }
    if (!a.gW && !a.gb)
        return hipGetLastError();
    const int S = a.M == 0 ? 0 : gw_splits(a.M, a.K, a.N);
    if (S > 0) {
        const dim3 grid(static_cast<unsigned>((a.K + 1 + 15) / 16), static_cast<unsigned>((a.N + 15) / 16), S);
        if (a.bf16)
            hipLaunchKernelGGL(linear_gw_kernel<bf16bits>, grid, dim3(256), 0, stream, a, S);
        else
            hipLaunchKernelGGL(linear_gw_kernel<float>, grid, dim3(256), 0, stream, a, S);
    }
    const float *part = static_cast<const float *>(a.ws);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.gW)
        e = launch_sum_parts(kn, S, kn + a.N, part, a.gW, a.accumulate, stream);
    if (e == hipSuccess && a.gb)
        e = launch_sum_parts(a.N, S, kn + a.N, part ? part + kn : nullptr, a.gb, a.accumulate, stream);
    return e;
}

}  // namespace etp
