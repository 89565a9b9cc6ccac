// etp_grad_norm.hip -- the norm of many tensors taken as one vector, and their
// scaling to a largest norm.
//
// Squares are added in double: no square of a float overflows or vanishes, and
// what a sum of 2^30 terms loses is far below a float's rounding. A launch
// carries its tensors' addresses in its arguments (kTableTensors of them: 4 KiB),
// cut into chunks of kChunk entries; a workgroup owns a run of chunks and leaves
// one partial sum. Whoever needs the norm adds the partial sums in the same fixed
// order: the scaling launch does so in every workgroup, instead of a launch in
// between.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "etp_dense_mma.hpp"
#include "etp_grad_norm.hpp"

namespace etp {

constexpr int kChunk = 8192;
constexpr int kTableTensors = 140;
constexpr int kMostRuns = 2048;  // workgroups of a launch

struct TensorTable {
    const void *in[kTableTensors];
    void *out[kTableTensors];
    int64_t numel[kTableTensors];  // negative: bf16, of -numel entries
    int first[kTableTensors];      // chunk of the tensor's start
    int n, chunks, per;            // per: chunks of a workgroup
    int part0;                     // partial sums of the launches before
};
static_assert(sizeof(TensorTable) <= 4000);

// The last tensor that starts at or before a chunk.
__device__ __forceinline__ int tensor_of(const TensorTable &t, int chunk)
{
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The sum over a workgroup of 256 threads, in every thread.
__device__ __forceinline__ double block_sum(double v, double *lds)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d, 64);
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    __syncthreads();
    return v;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, int n)
{
    constexpr int V = kVec<T>;
    double s = 0.0;
    int i = threadIdx.x * V;
#pragma unroll 4
    for (; i + V <= n; i += 256 * V) {
        RawVec<T> v;
        v.load(p + i, V);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const double x = v.get(k);
            s = __builtin_fma(x, x, s);
        }
    }
    for (; i < n; ++i) {  // the piece that the end cuts
        const double x = to_f32(p[i]);
        s = __builtin_fma(x, x, s);
    }
    return s;
}

__global__ void __launch_bounds__(256) grad_squares_kernel(const TensorTable t, double *__restrict__ part)
{
    __shared__ double lds[4];
    const int from = blockIdx.x * t.per, stop = from + t.per < t.chunks ? from + t.per : t.chunks;
    int k = tensor_of(t, from);
    double s = 0.0;
    for (int c = from; c < stop; ++c) {
        while (k + 1 < t.n && t.first[k + 1] <= c)
            ++k;
        const int64_t at = static_cast<int64_t>(c - t.first[k]) * kChunk, size = t.numel[k];
        const int64_t rest = (size < 0 ? -size : size) - at;
        const int n = rest < kChunk ? static_cast<int>(rest) : kChunk;
        s += size < 0 ? chunk_squares(static_cast<const bf16bits *>(t.in[k]) + at, n)
                      : chunk_squares(static_cast<const float *>(t.in[k]) + at, n);
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0)
        part[t.part0 + blockIdx.x] = s;
}

__device__ __forceinline__ double norm_of_parts(const double *part, int parts, double *lds)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 256)
        s += part[i];
    return __builtin_sqrt(block_sum(s, lds));
}

__global__ void __launch_bounds__(256) grad_norm_kernel(const double *__restrict__ part, int parts, float *norm)
{
    __shared__ double lds[4];
    const double v = norm_of_parts(part, parts, lds);
    if (threadIdx.x == 0)
        *norm = static_cast<float>(v);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *p, T *o, int n, double scale)
{
    constexpr int V = kVec<T>;
    int i = threadIdx.x * V;
#pragma unroll 4
    for (; i + V <= n; i += 256 * V) {
        RawVec<T> v;
        v.load(p + i, V);
        float y[8];
#pragma unroll
        for (int k = 0; k < V; ++k)
            y[k] = static_cast<float>(v.get(k) * scale);
        store_n<V>(o + i, V, y);
    }
    for (; i < n; ++i)
        o[i] = from_f32<T>(static_cast<float>(to_f32(p[i]) * scale));
}

__global__ void __launch_bounds__(256) grad_scale_kernel(const TensorTable t, const double *__restrict__ part, int parts,
                                                         float max_norm, float *norm)
{
    __shared__ double lds[4];
    const double length = norm_of_parts(part, parts, lds);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0)
        *norm = static_cast<float>(length);
    // not a number: everything becomes one
    const double scale = length <= max_norm ? 1.0 : max_norm / length;
    // what was read last is read first: it may still be in the last level of cache
    const int from = blockIdx.x * t.per, stop = from + t.per < t.chunks ? from + t.per : t.chunks;
    int k = tensor_of(t, stop - 1);
    for (int c = stop - 1; c >= from; --c) {
        while (t.first[k] > c)
            --k;
        if (scale == 1.0 && t.in[k] == t.out[k])
            continue;
        const int64_t at = static_cast<int64_t>(c - t.first[k]) * kChunk, size = t.numel[k];
        const int64_t rest = (size < 0 ? -size : size) - at;
        const int n = rest < kChunk ? static_cast<int>(rest) : kChunk;
        if (size < 0)
            chunk_scale(static_cast<const bf16bits *>(t.in[k]) + at, static_cast<bf16bits *>(t.out[k]) + at, n, scale);
        else
            chunk_scale(static_cast<const float *>(t.in[k]) + at, static_cast<float *>(t.out[k]) + at, n, scale);
    }
}

// Fills the table with the tensors from i on that are not empty; returns the
// first one that does not fit.
static int fill_table(TensorTable &t, const GradList &g, int i)
{
    t.n = 0;
    int64_t chunks = 0;
    for (; i < g.n && t.n < kTableTensors; ++i) {
        const int64_t numel = g.tensors[i].numel, c = (numel + kChunk - 1) / kChunk;
        if (numel == 0)
            continue;
        if (chunks + c >= (int64_t{1} << 31))
            break;
        t.in[t.n] = g.tensors[i].data;
        t.out[t.n] = g.out ? g.out[i] : const_cast<void *>(g.tensors[i].data);
        t.numel[t.n] = g.tensors[i].dtype == ETP_BF16 ? -numel : numel;
        t.first[t.n] = static_cast<int>(chunks);
        ++t.n;
        chunks += c;
    }
    t.chunks = static_cast<int>(chunks);
    t.per = static_cast<int>((chunks + kMostRuns - 1) / kMostRuns);
    return i;
}

static int runs_of(const TensorTable &t) { return t.per ? (t.chunks + t.per - 1) / t.per : 0; }

size_t grad_norm_workspace_bytes(const GradList &g)
{
    size_t parts = 0;
    TensorTable t;
    for (int i = 0; i < g.n;) {
        i = fill_table(t, g, i);
        parts += runs_of(t);
    }
    return sizeof(double) * parts;
}

static hipError_t squares(const GradList &g, double *part, int *parts, hipStream_t stream)
{
    TensorTable t;
    *parts = 0;
    for (int i = 0; i < g.n;) {
        i = fill_table(t, g, i);
        if (t.chunks == 0)
            continue;
        t.part0 = *parts;
        hipLaunchKernelGGL(grad_squares_kernel, dim3(runs_of(t)), dim3(256), 0, stream, t, part);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        *parts += runs_of(t);
    }
    return hipSuccess;
}

hipError_t launch_grad_norm(const GradList &g, float *norm, void *ws, hipStream_t stream)
{
    int parts;
    const hipError_t e = squares(g, static_cast<double *>(ws), &parts, stream);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, stream, static_cast<const double *>(ws), parts, norm);
    return hipGetLastError();
}

hipError_t launch_clip_grads(const GradList &g, float max_norm, float *norm, void *ws, hipStream_t stream)
{
    int parts;
    hipError_t e = squares(g, static_cast<double *>(ws), &parts, stream);
    if (e != hipSuccess)
        return e;
    if (parts == 0) {
        if (!norm)
            return hipSuccess;
        hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, stream, static_cast<const double *>(ws), 0, norm);
        return hipGetLastError();
    }
    TensorTable t;
    for (int i = 0; i < g.n;) {
        i = fill_table(t, g, i);
        if (t.chunks == 0)
            continue;
        hipLaunchKernelGGL(grad_scale_kernel, dim3(runs_of(t)), dim3(256), 0, stream, t, static_cast<const double *>(ws),
                           parts, max_norm, norm);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        norm = nullptr;  // written once
    }
    return hipSuccess;
}

}  // namespace etp
