// mx_grad.cu -- L2 norm over many gradient tensors, and their clipping by it
// (mx_grad_norm, mx_clip_grads).
//
//   norm = sqrt(sum over all tensors of g^2),  out = g * min(1, max_norm / (norm + eps))
//
// The tensors' addresses and sizes travel as kernel parameters, so a call
// needs no table in device memory and can be captured in a graph.  Sums run
// in fp32 per thread and in fp64 across threads and blocks, in an order that
// the sizes alone fix (no atomics): the same inputs give the same bits.
#include <cstdint>
#include <cuda_runtime.h>

#include "mx_internal.h"
#include "mx_ptx.cuh"
#include "mx_rows.cuh"

namespace mx {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kGrid = 608;          // four blocks for each of 152 SMs
constexpr int64_t kChunk = 8192;    // elements a block takes at a time
constexpr int kMostTensors = 1024;  // per launch (the table is a kernel parameter)

template <int N>
struct Table {
    const uint8_t *p[N];
    uint8_t *out[N];
    int64_t n[N];
    uint32_t first[N + 1];  // first chunk of each tensor
    uint8_t f32[N], out_f32[N];
    int count;
};

struct Piece {
    int tensor;
    int64_t begin, len;  // elements of the tensor
};

template <int N>
__device__ __forceinline__ Piece piece_of(const Table<N> &t, uint32_t chunk) {
    int lo = 0, hi = t.count;  // first[lo] <= chunk < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    Piece r;
    r.tensor = lo;
    r.begin = static_cast<int64_t>(chunk - t.first[lo]) * kChunk;
    const int64_t left = t.n[lo] - r.begin;
    r.len = left < kChunk ? left : kChunk;
    return r;
}

__device__ __forceinline__ float load1(const uint8_t *p, bool f32, int64_t i) {
    return f32 ? reinterpret_cast<const float *>(p)[i]
               : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << 16);
}

// Sum over the block in fp64, the same value in every thread.
__device__ __forceinline__ double sum_block(double v, double *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) v += part[i];
    return v;
}

template <typename T>
__device__ __forceinline__ float sum_squares(const uint8_t *p, int64_t len) {
    float s = 0.0f;
    const int64_t whole = len / 8;
    for (int64_t i = threadIdx.x; i < whole; i += kThreads) {
        Raw8<T> r;
        load8(r, p + i * 8 * T::kBytes);
        float v[8];
        to_f32(r, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fmaf(v[k], v[k], s);
    }
    for (int64_t i = whole * 8 + threadIdx.x; i < len; i += kThreads) {
        const float v = load1(p, T::kBytes == 4, i);
        s = fmaf(v, v, s);
    }
    return s;
}

template <int N>
__global__ void __launch_bounds__(kThreads) mx_grad_sums_kernel(const __grid_constant__ Table<N> t,
                                                                double *sums) {
    __shared__ double part[kThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    double s = 0.0;
    for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        const Piece q = piece_of(t, c);
        const bool f32 = t.f32[q.tensor] != 0;
        const uint8_t *p = t.p[q.tensor] + q.begin * (f32 ? 4 : 2);
        float v = 0.0f;
        if (reinterpret_cast<uintptr_t>(p) & 15u) {
            for (int64_t i = threadIdx.x; i < q.len; i += kThreads) {
                const float g = load1(p, f32, i);
                v = fmaf(g, g, v);
            }
        } else {
            v = f32 ? sum_squares<F32>(p, q.len) : sum_squares<BF16>(p, q.len);
        }
        s += static_cast<double>(v);
    }
    s = sum_block(s, part);
    if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// The norm from the blocks' sums (every block computes the same value).
__device__ __forceinline__ float norm_of(const double *sums, int64_t n, double *part) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) s += sums[i];
    return static_cast<float>(sqrt(sum_block(s, part)));
}

__global__ void __launch_bounds__(kThreads) mx_grad_norm_kernel(const double *sums, int64_t n,
                                                                float *norm) {
    __shared__ double part[kThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const float v = norm_of(sums, n, part);
    if (threadIdx.x == 0) *norm = v;
}

template <typename T, typename O>
__device__ __forceinline__ void scale_piece(const uint8_t *p, uint8_t *out, int64_t len, float coef) {
    const bool wide = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    const int64_t whole = wide ? len / 8 : 0;
    for (int64_t i = threadIdx.x; i < whole; i += kThreads) {
        Raw8<T> r;
        load8(r, p + i * 8 * T::kBytes);
        float v[8];
        to_f32(r, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= coef;
        Raw8<O> o;
        from_f32(o, v);
        uint4 *d = reinterpret_cast<uint4 *>(out + i * 8 * O::kBytes);
        d[0] = o.a;
        if constexpr (O::kBytes == 4) d[1] = o.b;
    }
    for (int64_t i = whole * 8 + threadIdx.x; i < len; i += kThreads) {
        const float v = load1(p, T::kBytes == 4, i) * coef;
        if constexpr (O::kBytes == 4) reinterpret_cast<float *>(out)[i] = v;
        else reinterpret_cast<uint16_t *>(out)[i] = static_cast<uint16_t>(bf16x2(v, 0.0f));
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads) mx_grad_scale_kernel(const __grid_constant__ Table<N> t,
                                                                 const double *sums, int64_t n_sums,
                                                                 float max_norm, float eps,
                                                                 float *norm) {
    __shared__ double part[kThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const float total = norm_of(sums, n_sums, part);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    float coef = max_norm / (total + eps);
    if (coef > 1.0f) coef = 1.0f;  // a NaN stays
    for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        const Piece q = piece_of(t, c);
        const bool f32 = t.f32[q.tensor] != 0, out_f32 = t.out_f32[q.tensor] != 0;
        const uint8_t *p = t.p[q.tensor] + q.begin * (f32 ? 4 : 2);
        uint8_t *out = t.out[q.tensor] + q.begin * (out_f32 ? 4 : 2);
        if (p == out && coef == 1.0f) continue;  // in place and nothing to change
        if (f32) {
            if (out_f32) scale_piece<F32, F32>(p, out, q.len, coef);
            else scale_piece<F32, BF16>(p, out, q.len, coef);
        } else {
            if (out_f32) scale_piece<BF16, F32>(p, out, q.len, coef);
            else scale_piece<BF16, BF16>(p, out, q.len, coef);
        }
    }
}

template <int N>
bool fill(Table<N> *t, const GradTensor *g, int count) {
    uint64_t chunks = 0;
    for (int i = 0; i < count; ++i) {
        t->p[i] = static_cast<const uint8_t *>(g[i].p);
        t->out[i] = static_cast<uint8_t *>(g[i].out);
        t->n[i] = g[i].n;
        t->f32[i] = g[i].f32;
        t->out_f32[i] = g[i].out_f32;
        t->first[i] = static_cast<uint32_t>(chunks);
        chunks += static_cast<uint64_t>((g[i].n + kChunk - 1) / kChunk);
        if (chunks > 0x7FFFFFFFull) return false;
    }
    t->first[count] = static_cast<uint32_t>(chunks);
    t->count = count;
    return true;
}

template <int N>
cudaError_t run_slice(const GradTensor *g, int count, bool sums, double *at, int64_t n_sums,
                      float max_norm, float eps, float *norm, cudaStream_t stream) {
    Table<N> t{};
    if (!fill(&t, g, count)) return cudaErrorInvalidValue;
    if (sums) return launch_dependent(mx_grad_sums_kernel<N>, kGrid, kThreads, stream, t, at);
    return launch_dependent(mx_grad_scale_kernel<N>, kGrid, kThreads, stream, t,
                            static_cast<const double *>(at), n_sums, max_norm, eps, norm);
}

}  // namespace

size_t grad_ws(int64_t count) {
    return static_cast<size_t>((count + kMostTensors - 1) / kMostTensors) * kGrid * sizeof(double);
}

cudaError_t launch_grad_clip(const GradTensor *g, int64_t count, bool scale, float max_norm,
                             float eps, float *norm, void *ws, const DeviceInfo &dev,
                             cudaStream_t stream) {
    double *sums = static_cast<double *>(ws);
    const int64_t slices = (count + kMostTensors - 1) / kMostTensors, n_sums = slices * kGrid;
    for (int pass = 0; pass < (scale ? 2 : 1); ++pass) {
        for (int64_t s = 0; s < slices; ++s) {
            const int64_t first = s * kMostTensors;
            const int n = static_cast<int>(count - first < kMostTensors ? count - first : kMostTensors);
            double *at = pass == 0 ? sums + s * kGrid : sums;
            const cudaError_t e =
                n <= 64 ? run_slice<64>(g + first, n, pass == 0, at, n_sums, max_norm, eps, norm, stream)
                        : run_slice<kMostTensors>(g + first, n, pass == 0, at, n_sums, max_norm, eps,
                                                  norm, stream);
            if (e != cudaSuccess) return e;
        }
    }
    if (scale) return cudaSuccess;
    return launch_dependent(mx_grad_norm_kernel, 1, kThreads, stream,
                            static_cast<const double *>(sums), n_sums, norm);
}

}  // namespace mx
