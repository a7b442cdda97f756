// mx_grad.cu -- L2 norm over many gradient tensors, and their clipping by it
// (mx_grad_norm, mx_clip_grads).
//
//   norm = sqrt(sum over all tensors of g^2),  out = g * min(1, max_norm / (norm + eps))
//
// The tensors' addresses and sizes travel as kernel parameters, so a call
// needs no table in device memory and can be captured in a graph.  Sums run
// in fp32 per thread and in pairs of fp32 across threads and blocks, in an order
// that the sizes, the types and the alignment (Parts below) fix, without atomics: the
// same inputs at the same alignment give the same bits.
//
// Bound by memory, and by the second read: the factor is known only after the
// whole norm.  218M fp32 gradients into bf16: 126 us for the norm (6.9 TB/s) and
// 195 us for the scaling (6.7 TB/s), 320 us in all, where one read and one write
// would take 192 us and two reads and one write 320 us at a plain copy's rate.  Going
// backwards finds some 40 MB in L2.  64 small tensors: 5 us, two launches.
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "mx_internal.h"
#include "mx_ptx.cuh"
#include "mx_rows.cuh"

namespace mx {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kGrid = 608;          // blocks at most: four for each of 152 SMs
constexpr int kFewTensors = 64;     // sizes of the table (a kernel parameter)
constexpr int kSomeTensors = 256;
constexpr int kMostTensors = 1024;  // per launch
constexpr int kUnroll = 4;          // 16-byte or element loads a thread has in flight
// Elements a block takes at a time: large ones cost fewer table searches, small
// ones spread a few small tensors over more SMs.
constexpr int64_t kChunk = 8192, kSmallChunk = 2048;

template <int N>
struct Table {
    const uint8_t *p[N];
    uint8_t *out[N];
    int64_t n[N];
    uint32_t first[N + 1];  // first chunk of each tensor
    uint8_t f32[N], out_f32[N];
    int count;
    int chunk;
};

// A block's chunks are a contiguous share of all; it walks them with the tensor
// it is in, which one search finds (the table lies in constant memory, a
// search costs as long as a chunk's loads).
template <int N>
struct Walk {
    uint32_t begin, end;  // chunks
    int tensor;

    __device__ __forceinline__ Walk(const Table<N> &t, bool backwards) {
        const uint64_t all = t.first[t.count];
        begin = static_cast<uint32_t>(all * blockIdx.x / gridDim.x);
        end = static_cast<uint32_t>(all * (blockIdx.x + 1) / gridDim.x);
        const uint32_t at = backwards ? end - 1 : begin;
        int lo = 0, hi = t.count;  // first[lo] <= at < first[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (t.first[mid] <= at) lo = mid;
            else hi = mid;
        }
        tensor = lo;
    }
    // Elements [first, first + len) of the tensor that chunk c lies in.
    __device__ __forceinline__ int piece(const Table<N> &t, uint32_t c, int64_t &first) {
        while (t.first[tensor + 1] <= c) ++tensor;
        while (t.first[tensor] > c) --tensor;
        first = static_cast<int64_t>(c - t.first[tensor]) * t.chunk;
        const int64_t left = t.n[tensor] - first;
        return static_cast<int>(left < t.chunk ? left : t.chunk);
    }
};

template <typename T>
__device__ __forceinline__ float load1(const uint8_t *p, int i) {
    if constexpr (T::kBytes == 4) return reinterpret_cast<const float *>(p)[i];
    else return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << 16);
}
template <typename T>
__device__ __forceinline__ void store1(const Out &o, uint8_t *p, int i, float v, int *status) {
    uint8_t *d = p + static_cast<size_t>(i) * T::kBytes;
    if (!MX_STORE_OK(d, T::kBytes, o.p, o.bytes, status)) return;
    if constexpr (T::kBytes == 4) *reinterpret_cast<float *>(d) = v;
    else *reinterpret_cast<uint16_t *>(d) = static_cast<uint16_t>(bf16x2(v, 0.0f));
}

// A piece of a tensor in three parts: elements up to the first boundary of a
// vector of 8 (16 bytes of bf16, 32 of fp32), such vectors, elements after them.
struct Parts {
    int head, whole;
};
template <typename T>
__device__ __forceinline__ Parts parts_of(const uint8_t *p, int len) {
    Parts r;
    constexpr uint32_t kLast = 8 * T::kBytes - 1;
    r.head = static_cast<int>((kLast + 1 - (reinterpret_cast<uintptr_t>(p) & kLast)) & kLast) / T::kBytes;
    if (r.head > len) r.head = len;
    r.whole = (len - r.head) / 8;
    return r;
}

// A sum as an fp32 value and what its roundings left out (Knuth's two-sum):
// about 48 bits.  fp64 would do, but a block's few fp64 additions take longer
// here than the rest of a small call (2 lanes a clock and SM).
struct Sum {
    float hi, lo;
};
__device__ __forceinline__ Sum add(const Sum &a, const Sum &b) {
    const float s = a.hi + b.hi, bb = s - a.hi;
    const float e = (a.hi - (s - bb)) + (b.hi - bb) + (a.lo + b.lo);
    const float t = s + e;
    if (!isfinite(t)) return {s, 0.0f};
    return {t, e - (t - s)};
}

// Sum over the block, the same value in every thread.
__device__ __forceinline__ Sum sum_block(Sum v, Sum *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = add(v, {__shfl_xor_sync(0xFFFFFFFFu, v.hi, o), __shfl_xor_sync(0xFFFFFFFFu, v.lo, o)});
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[threadIdx.x & 7];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        v = add(v, {__shfl_xor_sync(0xFFFFFFFFu, v.hi, o), __shfl_xor_sync(0xFFFFFFFFu, v.lo, o)});
    return v;
}

template <typename T>
__device__ __forceinline__ float sum_squares(const uint8_t *p, int len) {
    const Parts q = parts_of<T>(p, len);
    const int tail = q.head + 8 * q.whole, t = threadIdx.x;
    float ends = 0.0f;
    if (t < q.head) ends = load1<T>(p, t);
    ends *= ends;
    if (t < len - tail) {
        const float v = load1<T>(p, tail + t);
        ends = fmaf(v, v, ends);
    }
    const uint8_t *body = p + q.head * T::kBytes;
    uint64_t sums[kUnroll] = {};
    auto take = [&](const Raw8<T> &r, uint64_t &sum) {
        const V8 v = to_v8(r);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = fma2(v.v[j], v.v[j], sum);
    };
    auto at = [&](int i) { return body + static_cast<int64_t>(i) * 8 * T::kBytes; };
    int i = t;
    // Groups of loads without a condition between them, so that they are in flight
    // together (a condition each: one at a time, 136 us against 124 us for 218M fp32).
    for (; i + (kUnroll - 1) * kThreads < q.whole; i += kUnroll * kThreads) {
        Raw8<T> r[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) load8(r[k], at(i + k * kThreads));
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) take(r[k], sums[k]);
    }
    for (; i < q.whole; i += kThreads) {
        Raw8<T> r;
        load8(r, at(i));
        take(r, sums[0]);
    }
    return ends + sum2(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])));
}

template <int N>
__global__ void __launch_bounds__(kThreads) mx_grad_sums_kernel(const __grid_constant__ Table<N> t,
                                                                Sum *sums) {
    __shared__ Sum part[kThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    float s = 0.0f;
    Walk<N> walk(t, false);
    for (uint32_t c = walk.begin; c < walk.end; ++c) {
        int64_t first;
        const int len = walk.piece(t, c, first);
        const bool f32 = t.f32[walk.tensor] != 0;
        const uint8_t *p = t.p[walk.tensor] + first * (f32 ? 4 : 2);
        s += f32 ? sum_squares<F32>(p, len) : sum_squares<BF16>(p, len);
    }
    const Sum all = sum_block({s, 0.0f}, part);
    if (threadIdx.x == 0) sums[blockIdx.x] = all;
}

// The norm from the blocks' sums (every block computes the same value).
__device__ __forceinline__ float norm_of(const Sum *sums, int n, Sum *part) {
    Sum s{0.0f, 0.0f};
    for (int i = threadIdx.x; i < n; i += kThreads) s = add(s, sums[i]);
    return __fsqrt_rn(sum_block(s, part).hi);
}

__global__ void __launch_bounds__(kThreads) mx_grad_norm_kernel(const Sum *sums, int n,
                                                                float *norm) {
    __shared__ Sum part[kThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const float v = norm_of(sums, n, part);
    if (threadIdx.x == 0) *norm = v;
}

template <typename T, typename O>
__device__ __forceinline__ void scale_piece(const Out &whole, const uint8_t *p, uint8_t *out, int len,
                                            float coef, int *status) {
    Parts q = parts_of<T>(p, len);
    // The vectors' stores need the output's boundary at the same element.
    if ((reinterpret_cast<uintptr_t>(out) + q.head * O::kBytes) & 15u) q.head = q.whole = 0;
    const int tail = q.head + 8 * q.whole, t = threadIdx.x;
    if (t < q.head) store1<O>(whole, out, t, load1<T>(p, t) * coef, status);
    const uint8_t *body = p + q.head * T::kBytes;
    uint8_t *dst = out + q.head * O::kBytes;
    const bool aligned32 = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
    auto at = [&](int i) { return body + static_cast<int64_t>(i) * 8 * T::kBytes; };
    auto put = [&](const Raw8<T> &r, int i) {
        V8 v = to_v8(r);
#pragma unroll
        for (int j = 0; j < 4; ++j) v.v[j] = mul2(v.v[j], same2(coef));
        store8<O>(whole, dst + static_cast<int64_t>(i) * 8 * O::kBytes, v, aligned32, status);
    };
    int n = t;
    for (; n + (kUnroll - 1) * kThreads < q.whole; n += kUnroll * kThreads) {
        Raw8<T> r[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) load8(r[k], at(n + k * kThreads));
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) put(r[k], n + k * kThreads);
    }
    for (; n < q.whole; n += kThreads) {
        Raw8<T> r;
        load8(r, at(n));
        put(r, n);
    }
    for (int i = tail + t; i < len; i += 4 * kUnroll * kThreads) {
        float v[4 * kUnroll];
#pragma unroll
        for (int k = 0; k < 4 * kUnroll; ++k)
            v[k] = i + k * kThreads < len ? load1<T>(p, i + k * kThreads) : 0.0f;
#pragma unroll
        for (int k = 0; k < 4 * kUnroll; ++k)
            if (i + k * kThreads < len) store1<O>(whole, out, i + k * kThreads, v[k] * coef, status);
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads) mx_grad_scale_kernel(const __grid_constant__ Table<N> t,
                                                                 const Sum *sums, int n_sums,
                                                                 float max_norm, float eps,
                                                                 float *norm, int *status) {
    __shared__ Sum part[kThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const float total = norm_of(sums, n_sums, part);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    float coef = max_norm / (total + eps);
    if (coef > 1.0f) coef = 1.0f;  // a NaN stays
    // Backwards: what the sums read last is still in L2.
    Walk<N> walk(t, true);
    for (uint32_t c = walk.end; c-- > walk.begin;) {
        int64_t first;
        const int len = walk.piece(t, c, first), k = walk.tensor;
        const bool f32 = t.f32[k] != 0, out_f32 = t.out_f32[k] != 0;
        const uint8_t *p = t.p[k] + first * (f32 ? 4 : 2);
        uint8_t *out = t.out[k] + first * (out_f32 ? 4 : 2);
        const Out whole{t.out[k], static_cast<size_t>(t.n[k]) * (out_f32 ? 4 : 2)};
        if (p == out && coef == 1.0f) continue;  // in place and nothing to change
        if (f32) {
            if (out_f32) scale_piece<F32, F32>(whole, p, out, len, coef, status);
            else scale_piece<F32, BF16>(whole, p, out, len, coef, status);
        } else {
            if (out_f32) scale_piece<BF16, F32>(whole, p, out, len, coef, status);
            else scale_piece<BF16, BF16>(whole, p, out, len, coef, status);
        }
    }
}

uint64_t chunks_of(const GradTensor *g, int count, int64_t chunk) {
    uint64_t n = 0;
    for (int i = 0; i < count; ++i) n += static_cast<uint64_t>((g[i].n + chunk - 1) / chunk);
    return n;
}

// Up to N tensors of one launch.
struct Slice {
    const GradTensor *g;
    int count;
    int chunk, blocks;
};

template <int N>
cudaError_t run_slice(const Slice &s, bool scale, Sum *sums, int n_sums, float max_norm,
                      float eps, float *norm, int *status, cudaStream_t stream) {
    Table<N> t{};
    uint32_t at = 0;
    for (int i = 0; i < s.count; ++i) {
        const GradTensor &g = s.g[i];
        t.p[i] = static_cast<const uint8_t *>(g.p);
        t.out[i] = static_cast<uint8_t *>(g.out);
        t.n[i] = g.n;
        t.f32[i] = g.f32;
        t.out_f32[i] = g.out_f32;
        t.first[i] = at;
        at += static_cast<uint32_t>((g.n + s.chunk - 1) / s.chunk);
    }
    t.first[s.count] = at;
    t.count = s.count;
    t.chunk = s.chunk;
    if (!scale) return launch_dependent(mx_grad_sums_kernel<N>, s.blocks, kThreads, 0, stream, t, sums);
    return launch_dependent(mx_grad_scale_kernel<N>, s.blocks, kThreads, 0, stream, t,
                            static_cast<const Sum *>(sums), n_sums, max_norm, eps, norm, status);
}

}  // namespace

size_t grad_ws(int64_t count) {
    return static_cast<size_t>((count + kMostTensors - 1) / kMostTensors) * kGrid * sizeof(Sum);
}

cudaError_t launch_grad_clip(const GradTensor *g, int64_t count, bool scale, float max_norm,
                             float eps, float *norm, void *ws, const DeviceInfo &dev,
                             cudaStream_t stream) {
    Sum *sums = static_cast<Sum *>(ws);
    int n_sums = 0;
    for (int pass = 0; pass < (scale ? 2 : 1); ++pass) {
        // The last slice first in the second pass, like the chunks within one.
        const int64_t slices = (count + kMostTensors - 1) / kMostTensors;
        for (int64_t i = 0; i < slices; ++i) {
            const int64_t first = (pass == 0 ? i : slices - 1 - i) * kMostTensors;
            Slice s;
            s.g = g + first;
            s.count = static_cast<int>(count - first < kMostTensors ? count - first : kMostTensors);
            s.chunk = static_cast<int>(chunks_of(s.g, s.count, kChunk) >= kGrid ? kChunk : kSmallChunk);
            const uint64_t chunks = chunks_of(s.g, s.count, s.chunk);
            if (chunks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
            s.blocks = static_cast<int>(chunks < kGrid ? chunks : kGrid);
            Sum *at = pass == 0 ? sums + n_sums : sums;
            auto run = [&](auto size) {
                return run_slice<decltype(size)::value>(s, pass == 1, at, n_sums, max_norm, eps, norm,
                                                        dev.status, stream);
            };
            // The table is copied with every launch, 2, 7 or 29 KB.  At 65 / 200 / 256 small
            // tensors 7 KB instead of 29 takes a call from 15.3 / 22.0 / 24.8 us to 13.0 / 19.3 /
            // 22.9, and the two launches from 5.02 / 5.49 / 5.64 us to 4.81 / 5.40 / 5.43.
            const cudaError_t e =
                s.count <= kFewTensors    ? run(std::integral_constant<int, kFewTensors>{})
                : s.count <= kSomeTensors ? run(std::integral_constant<int, kSomeTensors>{})
                                          : run(std::integral_constant<int, kMostTensors>{});
            if (e != cudaSuccess) return e;
            if (pass == 0) n_sums += s.blocks;
        }
    }
    if (scale) return cudaSuccess;
    return launch_dependent(mx_grad_norm_kernel, 1, kThreads, 0, stream,
                            static_cast<const Sum *>(sums), n_sums, norm);
}

}  // namespace mx
