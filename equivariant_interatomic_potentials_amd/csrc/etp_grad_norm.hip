// etp_grad_norm.hip -- the norm of many tensors taken as one vector, and their
// scaling to a largest norm.
//
// Squares are added in double: no square of a float overflows or vanishes, and
// what a sum of 2^30 terms loses is far below a float's rounding. The tensors are
// cut into chunks of kChunk bytes; a workgroup owns a run of chunks and leaves
// one partial sum. Whoever needs the norm adds the partial sums in the same fixed
// order: the scaling launch does so in every workgroup, while its first chunk is
// on its way, instead of a launch in between. Addresses and sizes travel in a
// launch's arguments (kTableTensors fill the 4 KiB); of more tensors they are
// written into the workspace first.
//
// HBM bounds both: the norm of 300 million entries of both types (772 MB) 137 us, 5.6
// TB/s; clipping 400 million bf16 entries reads them twice and writes them, 2.4 GB, 502
// us, 4.8 TB/s (what was read last comes from the last level of cache no faster;
// stores that pass it by move 45 us from the scaling to the next call's reading).
// Squares of bf16 added in pairs in float before the doubles: no faster.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "etp_dense_mma.hpp"
#include "etp_grad_norm.hpp"

namespace etp {

constexpr int kChunk = 16384;         // bytes
constexpr int kTableTensors = 120;
constexpr int kMostRuns = 2048;       // workgroups of a launch, and partial sums
constexpr int kSmallEntries = 32768;  // one workgroup reads and scales so many
constexpr int kPiece = 2048;          // bytes a wave of it takes at a time

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

// The last tensor that starts at or before a chunk: by halves in the arguments, by 64
// probes a step in memory, where a step costs a microsecond.
__device__ __forceinline__ int tensor_in_memory(const TensorEntry *e, int n, int64_t chunk)
{
    int first = 0, count = n;
    for (;;) {
        const int step = (count + 63) >> 6, i = (threadIdx.x & 63) * step;
        const bool starts = i < count && e[first + i].first <= chunk;
        const int k = __builtin_amdgcn_readfirstlane(__popcll(__ballot(starts))) - 1;
        first += k * step;
        if (step == 1)
            return first;
        count = count - k * step < step ? count - k * step : step;
    }
}

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

// Where a chunk of Bytes lies: its addresses, number of bytes and type. (Copied, not
// pointed to: of a table in the arguments a pointer would make a copy in memory.)
template <int Bytes>
struct Place {
    const unsigned char *in;
    unsigned char *out;
    int n;
    bool bf16;
    __device__ __forceinline__ Place(const TensorEntry &t, int64_t chunk)
    {
        const int64_t size = t.numel, at = (chunk - t.first) * Bytes;
        bf16 = size < 0;
        in = static_cast<const unsigned char *>(t.in) + at;
        out = static_cast<unsigned char *>(t.out) + at;
        const int64_t rest = (bf16 ? -2 * size : 4 * size) - at;
        n = rest < Bytes ? static_cast<int>(rest) : Bytes;
    }
};

// A thread's share of a chunk, 16 bytes of every 16 Threads, as loaded; zeros past
// the end.
template <int Threads, int Bytes>
struct Share {
    static constexpr int N = Bytes / (16 * Threads);
    static_assert(N >= 1 && N * 16 * Threads == Bytes);
    u32x4 v[N];
    __device__ __forceinline__ void load(const Place<Bytes> &p, int id)
    {
        const unsigned char *base = p.in;
        if (p.n == Bytes) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                v[k] = *reinterpret_cast<const u32x4_any *>(base + (k * Threads + id) * 16);
            return;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = (k * Threads + id) * 16;
            v[k] = load8(reinterpret_cast<const bf16bits *>(base + (i < p.n ? i : 0)), (p.n - i) / 2);
        }
    }
    __device__ __forceinline__ static float half(uint32_t u, int j) { return __uint_as_float(j ? u & 0xFFFF0000u : u << 16); }
    __device__ __forceinline__ double squares(bool bf16) const
    {
        double s = 0.0;
        if (bf16) {
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const double x = half(v[k][j >> 1], j & 1);
                    s = __builtin_fma(x, x, s);
                }
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const double x = __uint_as_float(v[k][j]);
                    s = __builtin_fma(x, x, s);
                }
        }
        return s;
    }
    // the product with a double, rounded once to float (and once more to bf16)
    __device__ __forceinline__ void scale(const Place<Bytes> &p, int id, double by) const
    {
        unsigned char *base = p.out;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = (k * Threads + id) * 16;
            if (i >= p.n)
                continue;
            float y[8];
            if (p.bf16) {
                // in float where the scale has a float's digits
                const float f = static_cast<float>(by);
                if (by >= 0x1p-100) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y[j] = half(v[k][j >> 1], j & 1) * f;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y[j] = static_cast<float>(half(v[k][j >> 1], j & 1) * by);
                }
                store8(reinterpret_cast<bf16bits *>(base + i), (p.n - i) / 2, y);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    y[j] = static_cast<float>(__uint_as_float(v[k][j]) * by);
                store_n<4>(reinterpret_cast<float *>(base + i), (p.n - i) / 4, y);
            }
        }
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
    constexpr bool kFar = sizeof(Table) == sizeof(NoTable);
    const TensorEntry *e = kFar ? far : t.e;
    __shared__ double lds[4];
    const int64_t from = blockIdx.x * r.per, stop = from + r.per < r.chunks ? from + r.per : r.chunks;
    int k = kFar ? tensor_in_memory(far, r.tensors, from) : tensor_of(e, r.tensors, from);
    Place<kChunk> p(e[k], from);
    Share<256, kChunk> v;
    v.load(p, threadIdx.x);
    double s = 0.0;
    for (int64_t c = from; c < stop; ++c) {
        // the next chunk is on its way while this one is squared
        const Share<256, kChunk> now = v;
        const bool bf16 = p.bf16;
        if (c + 1 < stop) {
            while (k + 1 < r.tensors && e[k + 1].first <= c + 1)
                ++k;
            p = Place<kChunk>(e[k], c + 1);
            v.load(p, threadIdx.x);
        }
        s += now.squares(bf16);
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
    constexpr bool kFar = sizeof(Table) == sizeof(NoTable);
    const TensorEntry *e = kFar ? far : t.e;
    __shared__ double lds[4];
    // what was read last is read first: it may still be in the last level of cache
    const int64_t from = blockIdx.x * r.per, stop = from + r.per < r.chunks ? from + r.per : r.chunks;
    int k = kFar ? tensor_in_memory(far, r.tensors, stop - 1) : tensor_of(e, r.tensors, stop - 1);
    Place<kChunk> p(e[k], stop - 1);
    Share<256, kChunk> v;
    v.load(p, threadIdx.x);
    const double length = norm_of_parts(part, parts, lds);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0)
        *norm = static_cast<float>(length);
    const double scale = scale_of(length, max_norm);
    for (int64_t c = stop - 1; c >= from; --c) {
        const Share<256, kChunk> now = v;
        const Place<kChunk> here = p;
        if (c > from) {
            while (e[k].first > c - 1)
                --k;
            p = Place<kChunk>(e[k], c - 1);
            v.load(p, threadIdx.x);
        }
        if (scale != 1.0 || here.in != here.out)
            now.scale(here, threadIdx.x, scale);
    }
}

// Few entries: norm and (where asked for) scaling in one workgroup of 16 waves and
// one launch.
__global__ void __launch_bounds__(1024)
    grad_small_kernel(const TensorTable t, const Runs r, int scales, float max_norm, float *norm)
{
    __shared__ double lds[16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int pieces = static_cast<int>(r.chunks);
    double s = 0.0;
    for (int c = wave; c < pieces; c += 16) {
        const Place<kPiece> p(t.e[tensor_of(t.e, r.tensors, c)], c);
        Share<64, kPiece> v;
        v.load(p, lane);
        s += v.squares(p.bf16);
    }
    const double length = __builtin_sqrt(block_sum<16>(s, lds));
    if (norm && threadIdx.x == 0)
        *norm = static_cast<float>(length);
    if (!scales)
        return;
    const double scale = scale_of(length, max_norm);
    for (int c = wave; c < pieces; c += 16) {
        const Place<kPiece> p(t.e[tensor_of(t.e, r.tensors, c)], c);
        if (scale == 1.0 && p.in == p.out)
            continue;
        Share<64, kPiece> v;
        v.load(p, lane);
        v.scale(p, lane, scale);
    }
}

static int64_t chunks_of(const etp_tensor &x, int bytes)
{
    const int64_t each = bytes / (x.dtype == ETP_BF16 ? 2 : 4);
    return (x.numel + each - 1) / each;
}

// The tensors that are not empty, in chunks.
struct ListSize {
    int tensors = 0;
    int64_t entries = 0, chunks = 0;
};
static ListSize size_of(const GradList &g)
{
    ListSize s;
    for (int i = 0; i < g.n; ++i) {
        s.tensors += g.tensors[i].numel > 0;
        s.entries += g.tensors[i].numel;
        s.chunks += chunks_of(g.tensors[i], kChunk);
    }
    return s;
}

// One table's entries from tensor i on, in chunks of so many bytes; `first` runs on.
// Returns the tensor behind.
static int fill_table(TensorTable &t, int &n, const GradList &g, int i, int chunk, int64_t &first)
{
    for (n = 0; i < g.n && n < kTableTensors; ++i) {
        const etp_tensor &x = g.tensors[i];
        if (x.numel == 0)
            continue;
        t.e[n++] = {x.data, g.out ? g.out[i] : const_cast<void *>(x.data), x.dtype == ETP_BF16 ? -x.numel : x.numel, first};
        first += chunks_of(x, chunk);
    }
    return i;
}

static bool is_small(const ListSize &s) { return s.tensors <= kTableTensors && s.entries <= kSmallEntries; }

static Runs runs_of(const ListSize &s) { return {s.chunks, (s.chunks + kMostRuns - 1) / kMostRuns, s.tensors}; }

static int parts_of(const Runs &r) { return r.chunks ? static_cast<int>((r.chunks + r.per - 1) / r.per) : 0; }

size_t grad_norm_workspace_bytes(const GradList &g)
{
    const ListSize s = size_of(g);
    if (is_small(s))
        return 0;
    return sizeof(double) * static_cast<size_t>((parts_of(runs_of(s)) + 1) / 2 * 2) +
           (s.tensors > kTableTensors ? sizeof(TensorEntry) * static_cast<size_t>(s.tensors) : 0);
}

// The norm, and with `scales` the scaling.
static hipError_t launch(const GradList &g, bool scales, float max_norm, float *norm, void *ws, hipStream_t stream)
{
    const ListSize s = size_of(g);
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
