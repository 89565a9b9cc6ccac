// etp_orth.hip -- the orthogonalised update: Newton-Schulz steps
// X <- a X + (b A + c A^2) X, A = X X^T, on X / (|X|_F + eps).
#include "etp_dense.hpp"

namespace etp {

// norm[b] = 1 / (|G_b|_F + eps); one workgroup per matrix, sums in double
template <typename T>
__global__ void __launch_bounds__(1024) orth_norm_kernel(const T *__restrict__ G, const int64_t count,
                                                         const float eps, float *__restrict__ scale)
{
    __shared__ double part[1024];
    const T *g = G + blockIdx.x * count;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += 1024) {
        const double v = to_f32(g[i]);
        s += v * v;
    }
    part[threadIdx.x] = s;
    __syncthreads();
    for (int d = 512; d; d >>= 1) {
        if (threadIdx.x < d)
            part[threadIdx.x] += part[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0)
        scale[blockIdx.x] = static_cast<float>(1.0 / (sqrt(part[0]) + eps));
}

// X[b] = G[b] scale[b] as [n][m] (n <= m), transposed from G when tall
template <typename T>
__global__ void __launch_bounds__(256) orth_in_kernel(const T *__restrict__ G, const float *__restrict__ scale,
                                                      const int n, const int m, const int tall,
                                                      float *__restrict__ X)
{
    const int64_t nm = static_cast<int64_t>(n) * m, i = blockIdx.x * 256ll + threadIdx.x, b = blockIdx.y;
    if (i >= nm)
        return;
    const int64_t r = i / m, c = i - r * m;
    X[b * nm + i] = to_f32(G[b * nm + (tall ? c * n + r : i)]) * scale[b];
}

template <typename T>
__global__ void __launch_bounds__(256) orth_out_kernel(const float *__restrict__ X, const int n, const int m,
                                                       const int tall, T *__restrict__ out)
{
    const int64_t nm = static_cast<int64_t>(n) * m, i = blockIdx.x * 256ll + threadIdx.x, b = blockIdx.y;
    if (i >= nm)
        return;
    const int64_t r = i / m, c = i - r * m;
    out[b * nm + (tall ? c * n + r : i)] = from_f32<T>(X[b * nm + i]);
}

// C = alpha A op(B) + beta D, A [n][k], C and D [n][m], op(B) = B [k][m] or
// B^T with B [m][k]; batched over blockIdx.z
template <bool NT>
__global__ void __launch_bounds__(256) orth_product_kernel(const int n, const int m, const int k, const float alpha,
                                                           const float *__restrict__ A, const float *__restrict__ B,
                                                           const float beta, const float *__restrict__ D,
                                                           float *__restrict__ C)
{
    __shared__ float as[16][17], bs[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, b = blockIdx.z;
    const int i = blockIdx.x * 16 + ty, j0 = blockIdx.y * 16, j = j0 + tx;
    A += static_cast<int64_t>(b) * n * k;
    B += static_cast<int64_t>(b) * m * k;
    float acc = 0.f;
    for (int q = 0; q < k; q += 16) {
        as[ty][tx] = i < n && q + tx < k ? A[static_cast<int64_t>(i) * k + q + tx] : 0.f;
        if (NT)
            bs[tx][ty] = j0 + ty < m && q + tx < k ? B[static_cast<int64_t>(j0 + ty) * k + q + tx] : 0.f;
        else
            bs[ty][tx] = q + ty < k && j < m ? B[static_cast<int64_t>(q + ty) * m + j] : 0.f;
        __syncthreads();
        for (int t = 0; t < 16; ++t)
            acc = __builtin_fmaf(as[ty][t], bs[t][tx], acc);
        __syncthreads();
    }
    if (i < n && j < m) {
        const int64_t o = (static_cast<int64_t>(b) * n + i) * m + j;
        C[o] = D ? __builtin_fmaf(beta, D[o], alpha * acc) : alpha * acc;
    }
}

static int64_t pad4(int64_t n) { return (n + 3) / 4 * 4; }

size_t orthogonalize_workspace_bytes(int B, int rows, int cols, bool)
{
    const int64_t n = rows < cols ? rows : cols, m = rows < cols ? cols : rows;
    return sizeof(float) * static_cast<size_t>(pad4(B) + 2 * pad4(B * n * m) + 2 * pad4(B * n * n));
}

hipError_t launch_orthogonalize(const OrthArgs &a, hipStream_t stream)
{
    if (a.B == 0)
        return hipSuccess;
    const bool tall = a.rows > a.cols;
    const int n = tall ? a.cols : a.rows, m = tall ? a.rows : a.cols;
    const int64_t nm = static_cast<int64_t>(n) * m;
    float *scale = static_cast<float *>(a.ws);
    float *X = scale + pad4(a.B), *Y = X + pad4(a.B * nm), *A = Y + pad4(a.B * nm),
          *P = A + pad4(static_cast<int64_t>(a.B) * n * n);
    const dim3 ew(static_cast<unsigned>((nm + 255) / 256), a.B);
    if (a.bf16) {
        const auto G = static_cast<const bf16bits *>(a.G);
        hipLaunchKernelGGL(orth_norm_kernel<bf16bits>, dim3(a.B), dim3(1024), 0, stream, G, nm, a.eps, scale);
        hipLaunchKernelGGL(orth_in_kernel<bf16bits>, ew, dim3(256), 0, stream, G, scale, n, m, tall, X);
    } else {
        const auto G = static_cast<const float *>(a.G);
        hipLaunchKernelGGL(orth_norm_kernel<float>, dim3(a.B), dim3(1024), 0, stream, G, nm, a.eps, scale);
        hipLaunchKernelGGL(orth_in_kernel<float>, ew, dim3(256), 0, stream, G, scale, n, m, tall, X);
    }
    const dim3 gs(static_cast<unsigned>((n + 15) / 16), static_cast<unsigned>((n + 15) / 16), a.B);
    const dim3 gl(static_cast<unsigned>((n + 15) / 16), static_cast<unsigned>((m + 15) / 16), a.B);
    const float *none = nullptr;
    for (int s = 0; s < a.steps; ++s) {
        hipLaunchKernelGGL(orth_product_kernel<true>, gs, dim3(256), 0, stream, n, n, m, 1.f, X, X, 0.f, none, A);
        hipLaunchKernelGGL(orth_product_kernel<true>, gs, dim3(256), 0, stream, n, n, n, a.coef[2], A, A, a.coef[1],
                           A, P);
        hipLaunchKernelGGL(orth_product_kernel<false>, gl, dim3(256), 0, stream, n, m, n, 1.f, P, X, a.coef[0], X, Y);
        float *t = X;
        X = Y;
        Y = t;
    }
    if (a.bf16)
        hipLaunchKernelGGL(orth_out_kernel<bf16bits>, ew, dim3(256), 0, stream, X, n, m, tall,
                           static_cast<bf16bits *>(a.X));
    else
        hipLaunchKernelGGL(orth_out_kernel<float>, ew, dim3(256), 0, stream, X, n, m, tall,
                           static_cast<float *>(a.X));
    return hipGetLastError();
}

}  // namespace etp
