// mx_norm.cu -- RMS norm of the residual stream with an encoded output, and
// its gradient (mx_rmsnorm, mx_rmsnorm_backward).
//
//   h = x + r,  rstd = (mean(h^2) + eps)^(-1/2),  y = h * rstd * w
//   dx = rstd * (dy * w - h * rstd^2 * mean(dy * w * h)) + dres
//   dw = sum over rows of dy * h * rstd
//
// Sums and products are in fp32; y is rounded once, from fp32, to bf16 and
// (separately) to the codes.
#include <cstdint>
#include <cuda_runtime.h>

#include "mx_internal.h"
#include "mx_ptx.cuh"
#include "mx_rows.cuh"

namespace mx {
namespace {

using namespace rows;

struct NormArgs {
    const uint8_t *x, *res, *w;
    int64_t x_pitch, res_pitch, h_pitch;  // in elements
    Out h, y, rstd;
    Encoded enc;
    int64_t T, K;
    int64_t rows;  // T, or T padded to the scale layout's 128-line groups
    float eps;
    int w_f32;
    int tpr;  // threads per row, a multiple of 32
    int *status;
};

// Sum over the tpr threads of a row (the whole block takes part: rows of one
// block reduce in step).  `part` holds one float per warp.
__device__ __forceinline__ float sum_row(float v, int tpr, float *part) {
    v = sum_lanes(v, 32);
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, n = tpr >> 5, first = warp / n * n;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < n; ++i) v += part[first + i];
    return v;
}

// One row per tpr threads, C chunks of 8 columns per thread, the row in
// registers between its sum and its output.
template <typename X, typename S, bool RES, int C>
__global__ void __launch_bounds__(1024) mx_rmsnorm_kernel(const __grid_constant__ NormArgs p) {
    __shared__ float part[32];
    griddep_wait();
    griddep_launch_dependents();
    const int tr = threadIdx.x % p.tpr;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / p.tpr) + threadIdx.x / p.tpr;
    const bool live = row < p.T;
    float h[C][8];
    Raw8<X> xr[C];
    Raw8<S> rr[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int64_t col = 8 * (static_cast<int64_t>(j) * p.tpr + tr);
        const bool in = live && col < p.K;
        zero8(xr[j]);
        zero8(rr[j]);
        if (in) load8(xr[j], p.x + (row * p.x_pitch + col) * X::kBytes);
        if (RES && in) load8(rr[j], p.res + (row * p.res_pitch + col) * S::kBytes);
    }
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        to_f32(xr[j], h[j]);
        if (RES) {
            float r[8];
            to_f32(rr[j], r);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[j][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
    }
    ss = sum_row(ss, p.tpr, part);
    const float rstd = __frsqrt_rn(ss / static_cast<float>(p.K) + p.eps);
    if (live && tr == 0 && p.rstd.p != nullptr) {
        float *d = reinterpret_cast<float *>(p.rstd.p) + row;
        if (MX_STORE_OK(d, 4, p.rstd.p, p.rstd.bytes, p.status)) *d = rstd;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int64_t c = static_cast<int64_t>(j) * p.tpr + tr, col = 8 * c;
        const bool in = live && col < p.K;
        if (RES && in && p.h.p != nullptr) store8<S>(p.h, row * p.h_pitch + col, h[j], p.status);
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (in) {
            float w[8];
            load_weight8(p.w, p.w_f32 != 0, col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = h[j][i] * rstd * w[i];
            if (p.y.p != nullptr) store8<BF16>(p.y, row * p.K + col, y, p.status);
        }
        // Whole warps: a warp's chunks are all inside the padded width or all beyond it.
        if (p.enc.fmt != kEncNone && row < p.rows && c < p.enc.katoms * 16)
            encode8(p.enc, row, live ? p.K : 0, c, y, p.status);
    }
}

struct NormGradArgs {
    const uint8_t *dy, *h, *w, *dres;
    const float *rstd;
    int64_t dy_pitch, h_pitch, dres_pitch, dx_pitch;
    Out dx;
    float *parts;  // [gridDim.x * rows per block][K] partial weight gradients
    int64_t T, K;
    int w_f32;
    int tpr;
    int *status;
};

// Each group of tpr threads takes rows in turn and keeps its columns' sums of
// dy * h * rstd in registers; the groups' sums go to the workspace.
template <typename D, typename S, int C>
__global__ void __launch_bounds__(C > 4 ? 512 : 1024)
    mx_rmsnorm_backward_kernel(const __grid_constant__ NormGradArgs p) {
    __shared__ float part[2][32];
    griddep_wait();
    griddep_launch_dependents();
    const int tr = threadIdx.x % p.tpr, groups = blockDim.x / p.tpr;
    const int64_t group = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / p.tpr;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * groups;
    float dw[C][8];
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
    // Every group of a block makes the same number of turns (they share barriers).
    int turn = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < p.T; base += stride, turn ^= 1) {
        const int64_t row = base + threadIdx.x / p.tpr;
        const bool live = row < p.T;
        const float rstd = live ? p.rstd[row] : 0.0f;
        float a[C][8], x[C][8];  // dy * w, h * rstd
        float along = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int64_t col = 8 * (static_cast<int64_t>(j) * p.tpr + tr);
            const bool in = live && col < p.K;
            Raw8<D> dr;
            Raw8<S> hr;
            zero8(dr);
            zero8(hr);
            if (in) {
                load8(dr, p.dy + (row * p.dy_pitch + col) * D::kBytes);
                load8(hr, p.h + (row * p.h_pitch + col) * S::kBytes);
            }
            to_f32(dr, a[j]);
            to_f32(hr, x[j]);
            float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (col < p.K) load_weight8(p.w, p.w_f32 != 0, col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[j][i] *= rstd;
                dw[j][i] = fmaf(a[j][i], x[j][i], dw[j][i]);
                a[j][i] *= w[i];
                along = fmaf(a[j][i], x[j][i], along);
            }
        }
        along = sum_row(along, p.tpr, part[turn]) / static_cast<float>(p.K);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int64_t col = 8 * (static_cast<int64_t>(j) * p.tpr + tr);
            if (!live || col >= p.K) continue;
            float g[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (p.dres != nullptr) {
                Raw8<S> gr;
                load8(gr, p.dres + (row * p.dres_pitch + col) * S::kBytes);
                to_f32(gr, g);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = fmaf(rstd, a[j][i] - x[j][i] * along, g[i]);
            store8<S>(p.dx, row * p.dx_pitch + col, g, p.status);
        }
    }
    if (p.parts == nullptr) return;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int64_t col = 8 * (static_cast<int64_t>(j) * p.tpr + tr);
        if (col >= p.K) continue;
        float4 *d = reinterpret_cast<float4 *>(p.parts + group * p.K + col);
        d[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
        d[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
    }
}

// dw[col] = sum of the partial sums, in a fixed order: 32 columns a block,
// the partials split over its 8 warps.
__global__ void __launch_bounds__(256) mx_rmsnorm_dw_kernel(const float *parts, int64_t n, int64_t K,
                                                            Out dw, int *status) {
    __shared__ float sums[8][32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
    float s = 0.0f;
    if (col < K)
        for (int64_t i = threadIdx.x >> 5; i < n; i += 8) s += parts[i * K + col];
    sums[threadIdx.x >> 5][threadIdx.x & 31] = s;
    __syncthreads();
    if (threadIdx.x < 32 && col < K) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
        float *d = reinterpret_cast<float *>(dw.p) + col;
        if (MX_STORE_OK(d, 4, dw.p, dw.bytes, status)) *d = s;
    }
}

// Chunks of 8 columns a row's threads cover: the padded width of the scale layout.
int64_t padded_chunks(int64_t K) { return (K + 255) / 256 * 32; }

struct RowShape {
    int chunks_per_thread, tpr, groups;
};
// Few chunks a thread keep the registers few and the loads of a row in flight
// at once; a block has at least 256 threads.
RowShape row_shape(int64_t K, int most) {
    const int64_t n = padded_chunks(K);
    const int c = n <= 32 ? 1 : n <= 2 * most ? 2 : n <= 4 * most ? 4 : 8;
    const int tpr = static_cast<int>(((n + c - 1) / c + 31) / 32 * 32);
    return {c, tpr, tpr >= 256 ? 1 : 256 / tpr};
}

template <typename X, typename S, bool RES>
cudaError_t launch_norm(const NormArgs &p, const RowShape &s, cudaStream_t stream) {
    const int64_t grid = (p.rows + s.groups - 1) / s.groups;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const int threads = s.tpr * s.groups;
    switch (s.chunks_per_thread) {
        case 1: return launch_dependent(mx_rmsnorm_kernel<X, S, RES, 1>, grid, threads, stream, p);
        case 2: return launch_dependent(mx_rmsnorm_kernel<X, S, RES, 2>, grid, threads, stream, p);
        case 4: return launch_dependent(mx_rmsnorm_kernel<X, S, RES, 4>, grid, threads, stream, p);
        default: return launch_dependent(mx_rmsnorm_kernel<X, S, RES, 8>, grid, threads, stream, p);
    }
}

template <typename D, typename S>
cudaError_t launch_norm_grad(const NormGradArgs &p, const RowShape &s, int grid, cudaStream_t stream) {
    const int threads = s.tpr * s.groups;
    switch (s.chunks_per_thread) {
        case 1: return launch_dependent(mx_rmsnorm_backward_kernel<D, S, 1>, grid, threads, stream, p);
        case 2: return launch_dependent(mx_rmsnorm_backward_kernel<D, S, 2>, grid, threads, stream, p);
        case 4: return launch_dependent(mx_rmsnorm_backward_kernel<D, S, 4>, grid, threads, stream, p);
        default: return launch_dependent(mx_rmsnorm_backward_kernel<D, S, 8>, grid, threads, stream, p);
    }
}

constexpr int kGradGrid = 304;  // blocks of the gradient at most: two for each of 152 SMs

int grad_grid(int64_t T, const RowShape &s) {
    const int64_t want = (T + s.groups - 1) / s.groups;
    return static_cast<int>(want < kGradGrid ? want : kGradGrid);
}

}  // namespace

cudaError_t launch_rmsnorm(const RowIn &x, const RowIn &res, const void *w, int w_f32, float eps,
                           int64_t T, int64_t K, void *h, int64_t h_pitch, void *y,
                           const RowEncode &e, float *rstd, const DeviceInfo &dev,
                           cudaStream_t stream) {
    NormArgs p{};
    p.x = static_cast<const uint8_t *>(x.p);
    p.res = static_cast<const uint8_t *>(res.p);
    p.w = static_cast<const uint8_t *>(w);
    p.x_pitch = x.pitch;
    p.res_pitch = res.pitch;
    p.h_pitch = h_pitch;
    const size_t sb = res.f32 ? 4 : 2;
    p.h = {static_cast<uint8_t *>(h), (static_cast<size_t>(T - 1) * h_pitch + K) * sb};
    p.y = {static_cast<uint8_t *>(y), static_cast<size_t>(T) * K * 2};
    p.rstd = {reinterpret_cast<uint8_t *>(rstd), static_cast<size_t>(T) * 4};
    p.enc = row_encoded(e, T, K);
    p.T = T;
    p.K = K;
    p.rows = e.fmt != kEncNone ? 128 * scale_groups(T) : T;
    p.eps = eps;
    p.w_f32 = w_f32;
    p.status = dev.status;
    const RowShape s = row_shape(K, 1024);
    p.tpr = s.tpr;
    if (res.p == nullptr) return x.f32 ? launch_norm<F32, F32, false>(p, s, stream)
                                       : launch_norm<BF16, BF16, false>(p, s, stream);
    if (x.f32) return res.f32 ? launch_norm<F32, F32, true>(p, s, stream)
                              : launch_norm<F32, BF16, true>(p, s, stream);
    return res.f32 ? launch_norm<BF16, F32, true>(p, s, stream)
                   : launch_norm<BF16, BF16, true>(p, s, stream);
}

size_t rmsnorm_backward_ws(int64_t T, int64_t K) {
    const RowShape s = row_shape(K, 512);
    return static_cast<size_t>(grad_grid(T, s)) * s.groups * static_cast<size_t>(K) * 4;
}

cudaError_t launch_rmsnorm_backward(const RowIn &dy, const RowIn &h, const void *w, int w_f32,
                                    const float *rstd, const RowIn &dres, int64_t T, int64_t K,
                                    void *dx, int64_t dx_pitch, float *dw, void *ws,
                                    const DeviceInfo &dev, cudaStream_t stream) {
    NormGradArgs p{};
    p.dy = static_cast<const uint8_t *>(dy.p);
    p.h = static_cast<const uint8_t *>(h.p);
    p.w = static_cast<const uint8_t *>(w);
    p.dres = static_cast<const uint8_t *>(dres.p);
    p.rstd = rstd;
    p.dy_pitch = dy.pitch;
    p.h_pitch = h.pitch;
    p.dres_pitch = dres.pitch;
    p.dx_pitch = dx_pitch;
    p.dx = {static_cast<uint8_t *>(dx),
            (static_cast<size_t>(T - 1) * dx_pitch + K) * static_cast<size_t>(h.f32 ? 4 : 2)};
    p.parts = dw != nullptr ? static_cast<float *>(ws) : nullptr;
    p.T = T;
    p.K = K;
    p.w_f32 = w_f32;
    p.status = dev.status;
    const RowShape s = row_shape(K, 512);
    p.tpr = s.tpr;
    const int grid = grad_grid(T, s);
    cudaError_t e = dy.f32 ? (h.f32 ? launch_norm_grad<F32, F32>(p, s, grid, stream)
                                    : launch_norm_grad<F32, BF16>(p, s, grid, stream))
                           : (h.f32 ? launch_norm_grad<BF16, F32>(p, s, grid, stream)
                                    : launch_norm_grad<BF16, BF16>(p, s, grid, stream));
    if (e != cudaSuccess || dw == nullptr) return e;
    return launch_dependent(mx_rmsnorm_dw_kernel, (K + 31) / 32, 256, stream,
                            static_cast<const float *>(ws), static_cast<int64_t>(grid) * s.groups, K,
                            Out{reinterpret_cast<uint8_t *>(dw), static_cast<size_t>(K) * 4},
                            dev.status);
}

}  // namespace mx
