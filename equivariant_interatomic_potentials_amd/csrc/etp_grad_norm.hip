// etp_grad_norm.hip -- the norm of many tensors taken as one vector, and their
// scaling to a largest norm.
//
// Squares are added in double: no square of a float overflows or vanishes, and
// what a sum of 2^30 terms loses is far below a float's rounding. The tensors are
// cut into chunks of kChunk entries; a workgroup owns a run of chunks and leaves
// one partial sum. Whoever needs the norm adds the partial sums in the same fixed
// order: the scaling launch does so in every workgroup, while its first chunk is
// on its way, instead of a launch in between. Addresses and sizes travel in a
// launch's arguments (kTableTensors fill the 4 KiB); of more tensors they are
// written into the workspace first.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "etp_dense_mma.hpp"
#include "etp_grad_norm.hpp"

namespace etp {

constexpr int kChunk = 8192;
constexpr int kTableTensors = 120;
constexpr int kMostRuns = 2048;       // workgroups of a launch, and partial sums
constexpr int kSmallEntries = 32768;  // one workgroup reads and scales so many
constexpr int kPiece = 512;           // entries a wave of it takes at a time

struct TensorEntry {
    const void *in;
    void *out;
    int64_t numel;  // negative: bf16, of -numel entries
    int64_t first;  // chunk (piece) of the tensor's start
};
struct TensorTable {
    TensorEntry e[kTableTensors];
};
static_assert(sizeof(TensorTable) <= 3840);

struct Runs {
    int64_t chunks, per;  // in all, and of a workgroup
    int tensors;
};

// The last tensor that starts at or before a chunk.
__device__ __forceinline__ int tensor_of(const TensorEntry *e, int n, int64_t chunk)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (e[mid].first <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The sum over a workgroup of Waves waves, in every thread.
template <int Waves>
__device__ __forceinline__ double block_sum(double v, double *lds)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d, 64);
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < Waves; ++w)
        v += lds[w];
    __syncthreads();
    return v;
}

// A thread's share of Entries consecutive entries, Threads threads 16 bytes each in
// turn, as loaded.
template <typename T, int Threads, int Entries>
struct Share {
    static constexpr int V = kVec<T>, N = Entries / (Threads * V);
    static_assert(N >= 1 && N * Threads * V == Entries);
    RawVec<T> v[N];
    __device__ __forceinline__ void load(const TensorEntry &t, int64_t at, int n, int id)
    {
        const T *p = static_cast<const T *>(t.in) + at;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = (k * Threads + id) * V;
            v[k].load(p + (i < n ? i : 0), n - i);
        }
    }
    // (entries past the end were loaded as zeros)
    __device__ __forceinline__ double squares() const
    {
        double s = 0.0;
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const double x = v[k].get(j);
                s = __builtin_fma(x, x, s);
            }
        return s;
    }
    // the product with a double, rounded once to float (and once more to bf16)
    __device__ __forceinline__ void scale(const TensorEntry &t, int64_t at, int n, int id, double by) const
    {
        T *p = static_cast<T *>(t.out) + at;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = (k * Threads + id) * V;
            float y[8];
#pragma unroll
            for (int j = 0; j < V; ++j)
                y[j] = static_cast<float>(v[k].get(j) * by);
            if (i < n)
                store_n<V>(p + i, n - i, y);
        }
    }
};

// Where a chunk lies: its tensor, first entry and number of entries.
template <int Entries>
struct Place {
    int64_t at;
    int n;
    bool bf16;
    __device__ __forceinline__ Place(const TensorEntry &t, int64_t chunk)
    {
        const int64_t size = t.numel;
        bf16 = size < 0;
        at = (chunk - t.first) * Entries;
        const int64_t rest = (bf16 ? -size : size) - at;
        n = rest < Entries ? static_cast<int>(rest) : Entries;
    }
};

__global__ void __launch_bounds__(128) grad_table_kernel(const TensorTable t, int n, TensorEntry *__restrict__ to)
{
    if (static_cast<int>(threadIdx.x) < n)
        to[threadIdx.x] = t.e[threadIdx.x];
}

// In the place of a table that lies in memory.
struct NoTable {
    TensorEntry e[1];
};

template <typename Table>
__global__ void __launch_bounds__(256)
    grad_squares_kernel(const Table t, const TensorEntry *__restrict__ far, const Runs r, double *__restrict__ part)
{
    const TensorEntry *e = sizeof(Table) == sizeof(NoTable) ? far : t.e;
    __shared__ double lds[4];
    const int64_t from = blockIdx.x * r.per, stop = from + r.per < r.chunks ? from + r.per : r.chunks;
    int k = tensor_of(e, r.tensors, from);
    double s = 0.0;
    for (int64_t c = from; c < stop; ++c) {
        while (k + 1 < r.tensors && e[k + 1].first <= c)
            ++k;
        const Place<kChunk> p(e[k], c);
        if (p.bf16) {
            Share<bf16bits, 256, kChunk> v;
            v.load(e[k], p.at, p.n, threadIdx.x);
            s += v.squares();
        } else {
            Share<float, 256, kChunk> v;
            v.load(e[k], p.at, p.n, threadIdx.x);
            s += v.squares();
        }
    }
    s = block_sum<4>(s, lds);
    if (threadIdx.x == 0)
        part[blockIdx.x] = s;
}

__device__ __forceinline__ double norm_of_parts(const double *part, int parts, double *lds)
{
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < kMostRuns / 256; ++k) {
        const int i = k * 256 + threadIdx.x;
        s += i < parts ? part[i] : 0.0;
    }
    return __builtin_sqrt(block_sum<4>(s, lds));
}

// A norm that is not a number makes everything one.
__device__ __forceinline__ double scale_of(double norm, float max_norm) { return norm <= max_norm ? 1.0 : max_norm / norm; }

__global__ void __launch_bounds__(256) grad_norm_kernel(const double *__restrict__ part, int parts, float *norm)
{
    __shared__ double lds[4];
    const double v = norm_of_parts(part, parts, lds);
    if (threadIdx.x == 0)
        *norm = static_cast<float>(v);
}

template <typename Table>
__global__ void __launch_bounds__(256)
    grad_scale_kernel(const Table t, const TensorEntry *__restrict__ far, const Runs r, const double *__restrict__ part,
                      int parts, float max_norm, float *norm)
{
    const TensorEntry *e = sizeof(Table) == sizeof(NoTable) ? far : t.e;
    __shared__ double lds[4];
    // what was read last is read first: it may still be in the last level of cache
    const int64_t from = blockIdx.x * r.per, stop = from + r.per < r.chunks ? from + r.per : r.chunks;
    int k = tensor_of(e, r.tensors, stop - 1);
    double scale = -1.0;
    auto chunk = [&](auto share, const Place<kChunk> &p) __attribute__((always_inline)) {
        share.load(e[k], p.at, p.n, threadIdx.x);
        if (scale < 0.0) {  // once, with the first chunk on its way
            const double length = norm_of_parts(part, parts, lds);
            if (norm && blockIdx.x == 0 && threadIdx.x == 0)
                *norm = static_cast<float>(length);
            scale = scale_of(length, max_norm);
        }
        if (scale != 1.0 || e[k].in != e[k].out)
            share.scale(e[k], p.at, p.n, threadIdx.x, scale);
    };
    for (int64_t c = stop - 1; c >= from; --c) {
        while (e[k].first > c)
            --k;
        const Place<kChunk> p(e[k], c);
        if (p.bf16)
            chunk(Share<bf16bits, 256, kChunk>(), p);
        else
            chunk(Share<float, 256, kChunk>(), p);
    }
}

// Few entries: norm and scaling in one workgroup of 16 waves and one launch. out:
// whether to scale.
__global__ void __launch_bounds__(1024)
    grad_small_kernel(const TensorTable t, const Runs r, int scales, float max_norm, float *norm)
{
    __shared__ double lds[16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int pieces = static_cast<int>(r.chunks);
    double s = 0.0;
    for (int c = wave; c < pieces; c += 16) {
        const int k = tensor_of(t.e, r.tensors, c);
        const Place<kPiece> p(t.e[k], c);
        if (p.bf16) {
            Share<bf16bits, 64, kPiece> v;
            v.load(t.e[k], p.at, p.n, lane);
            s += v.squares();
        } else {
            Share<float, 64, kPiece> v;
            v.load(t.e[k], p.at, p.n, lane);
            s += v.squares();
        }
    }
    const double length = __builtin_sqrt(block_sum<16>(s, lds));
    if (norm && threadIdx.x == 0)
        *norm = static_cast<float>(length);
    if (!scales)
        return;
    const double scale = scale_of(length, max_norm);
    for (int c = wave; c < pieces; c += 16) {
        const int k = tensor_of(t.e, r.tensors, c);
        if (scale == 1.0 && t.e[k].in == t.e[k].out)
            continue;
        const Place<kPiece> p(t.e[k], c);
        if (p.bf16) {
            Share<bf16bits, 64, kPiece> v;
            v.load(t.e[k], p.at, p.n, lane);
            v.scale(t.e[k], p.at, p.n, lane, scale);
        } else {
            Share<float, 64, kPiece> v;
            v.load(t.e[k], p.at, p.n, lane);
            v.scale(t.e[k], p.at, p.n, lane, scale);
        }
    }
}

// The tensors that are not empty, in chunks of so many entries.
struct ListSize {
    int tensors = 0;
    int64_t entries = 0, chunks = 0;
};
static ListSize size_of(const GradList &g, int chunk)
{
    ListSize s;
    for (int i = 0; i < g.n; ++i) {
        const int64_t n = g.tensors[i].numel;
        s.tensors += n > 0;
        s.entries += n;
        s.chunks += (n + chunk - 1) / chunk;
    }
    return s;
}

// One table's entries from tensor i on; `first` runs on. Returns the tensor behind.
static int fill_table(TensorTable &t, int &n, const GradList &g, int i, int chunk, int64_t &first)
{
    for (n = 0; i < g.n && n < kTableTensors; ++i) {
        const etp_tensor &x = g.tensors[i];
        if (x.numel == 0)
            continue;
        t.e[n++] = {x.data, g.out ? g.out[i] : const_cast<void *>(x.data), x.dtype == ETP_BF16 ? -x.numel : x.numel, first};
        first += (x.numel + chunk - 1) / chunk;
    }
    return i;
}

static bool is_small(const ListSize &s) { return s.tensors <= kTableTensors && s.entries <= kSmallEntries; }

static Runs runs_of(const ListSize &s) { return {s.chunks, (s.chunks + kMostRuns - 1) / kMostRuns, s.tensors}; }

static int parts_of(const Runs &r) { return r.chunks ? static_cast<int>((r.chunks + r.per - 1) / r.per) : 0; }

size_t grad_norm_workspace_bytes(const GradList &g)
{
    const ListSize s = size_of(g, kChunk);
    if (is_small(s))
        return 0;
    return sizeof(double) * static_cast<size_t>((parts_of(runs_of(s)) + 1) / 2 * 2) +
           (s.tensors > kTableTensors ? sizeof(TensorEntry) * static_cast<size_t>(s.tensors) : 0);
}

// The norm, and with `scales` the scaling.
static hipError_t launch(const GradList &g, bool scales, float max_norm, float *norm, void *ws, hipStream_t stream)
{
    const ListSize s = size_of(g, kChunk);
    TensorTable t;
    int n;
    int64_t first = 0;
    if (is_small(s)) {
        fill_table(t, n, g, 0, kPiece, first);
        hipLaunchKernelGGL(grad_small_kernel, dim3(1), dim3(1024), 0, stream, t, Runs{first, 1, n}, scales ? 1 : 0, max_norm,
                           norm);
        return hipGetLastError();
    }
    const Runs r = runs_of(s);
    const int parts = parts_of(r);
    double *part = static_cast<double *>(ws);
    hipError_t e = hipSuccess;
    if (s.tensors <= kTableTensors) {
        fill_table(t, n, g, 0, kChunk, first);
        hipLaunchKernelGGL(grad_squares_kernel<TensorTable>, dim3(parts), dim3(256), 0, stream, t, nullptr, r, part);
        e = hipGetLastError();
        if (e == hipSuccess && scales) {
            hipLaunchKernelGGL(grad_scale_kernel<TensorTable>, dim3(parts), dim3(256), 0, stream, t, nullptr, r, part,
                               parts, max_norm, norm);
            e = hipGetLastError();
        }
    } else {
        TensorEntry *far = reinterpret_cast<TensorEntry *>(part + (parts + 1) / 2 * 2);
        for (int i = 0, at = 0; i < g.n; at += n) {
            i = fill_table(t, n, g, i, kChunk, first);
            hipLaunchKernelGGL(grad_table_kernel, dim3(1), dim3(128), 0, stream, t, n, far + at);
            if ((e = hipGetLastError()) != hipSuccess)
                return e;
        }
        const NoTable none{};
        hipLaunchKernelGGL(grad_squares_kernel<NoTable>, dim3(parts), dim3(256), 0, stream, none, far, r, part);
        e = hipGetLastError();
        if (e == hipSuccess && scales) {
            hipLaunchKernelGGL(grad_scale_kernel<NoTable>, dim3(parts), dim3(256), 0, stream, none, far, r, part, parts,
                               max_norm, norm);
            e = hipGetLastError();
        }
    }
    if (e != hipSuccess || scales)
        return e;
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, stream, part, parts, norm);
    return hipGetLastError();
}

hipError_t launch_grad_norm(const GradList &g, float *norm, void *ws, hipStream_t stream)
{
    return launch(g, false, 0.f, norm, ws, stream);
}

hipError_t launch_clip_grads(const GradList &g, float max_norm, float *norm, void *ws, hipStream_t stream)
{
    return launch(g, true, max_norm, norm, ws, stream);
}

}  // namespace etp
