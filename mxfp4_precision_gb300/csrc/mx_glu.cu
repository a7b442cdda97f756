// mx_glu.cu -- SwiGLU of a gate/up product with an encoded output, and its
// gradient (mx_swiglu, mx_swiglu_backward).
//
//   y = g * s * u,  s = 1 / (1 + exp(-g));  g = gu[:, :F], u = gu[:, F:]
//   dg = dy * u * s * (1 + g * (1 - s)),  du = dy * g * s
#include <cstdint>
#include <cuda_runtime.h>

#include "mx_internal.h"
#include "mx_ptx.cuh"
#include "mx_rows.cuh"

namespace mx {
namespace {

using namespace rows;

struct GluArgs {
    const uint8_t *gu, *dy;
    int64_t gu_pitch, dy_pitch;
    Out y;  // y [T][F], or dgu [T][2F]
    Encoded enc;
    int64_t T, F;
    int64_t chunks;  // chunks of 8 columns per row, padded to a multiple of 32
    int64_t total;   // chunks over all rows (padded rows included when encoding)
    int *status;
};

template <typename G>
__global__ void __launch_bounds__(256) mx_swiglu_kernel(const __grid_constant__ GluArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    // total is a multiple of 32: whole warps take part.
    const int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (at >= p.total) return;
    const int64_t row = at / p.chunks, c = at % p.chunks, col = 8 * c;
    const bool in = row < p.T && col < p.F;
    float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in) {
        Raw8<G> gr, ur;
        const uint8_t *src = p.gu + (row * p.gu_pitch + col) * G::kBytes;
        load8(gr, src);
        load8(ur, src + p.F * G::kBytes);
        float g[8], u[8];
        to_f32(gr, g);
        to_f32(ur, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = g[i] / (1.0f + expf(-g[i])) * u[i];
        if (p.y.p != nullptr) store8<BF16>(p.y, row * p.F + col, y, p.status);
    }
    if (p.enc.fmt != kEncNone) encode8(p.enc, row, row < p.T ? p.F : 0, c, y, p.status);
}

template <typename D, typename G>
__global__ void __launch_bounds__(256) mx_swiglu_backward_kernel(const __grid_constant__ GluArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (at >= p.total) return;
    const int64_t row = at / p.chunks, col = 8 * (at % p.chunks);
    Raw8<G> gr, ur;
    Raw8<D> dr;
    const uint8_t *src = p.gu + (row * p.gu_pitch + col) * G::kBytes;
    load8(dr, p.dy + (row * p.dy_pitch + col) * D::kBytes);
    load8(gr, src);
    load8(ur, src + p.F * G::kBytes);
    float g[8], u[8], d[8];
    to_f32(dr, d);
    to_f32(gr, g);
    to_f32(ur, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float s = 1.0f / (1.0f + expf(-g[i])), ds = d[i] * s;
        u[i] = ds * u[i] * (1.0f + g[i] * (1.0f - s));
        d[i] = ds * g[i];
    }
    store8<BF16>(p.y, row * 2 * p.F + col, u, p.status);
    store8<BF16>(p.y, row * 2 * p.F + p.F + col, d, p.status);
}

}  // namespace

cudaError_t launch_swiglu(const RowIn &gu, int64_t T, int64_t F, void *y, const RowEncode &e,
                          const DeviceInfo &dev, cudaStream_t stream) {
    GluArgs p{};
    p.gu = static_cast<const uint8_t *>(gu.p);
    p.gu_pitch = gu.pitch;
    p.y = {static_cast<uint8_t *>(y), static_cast<size_t>(T) * F * 2};
    p.enc = row_encoded(e, T, F);
    p.T = T;
    p.F = F;
    p.chunks = (F + 255) / 256 * 32;
    p.total = (e.fmt != kEncNone ? 128 * scale_groups(T) : T) * p.chunks;
    p.status = dev.status;
    const int64_t grid = (p.total + 255) / 256;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return gu.f32 ? launch_dependent(mx_swiglu_kernel<F32>, grid, 256, stream, p)
                  : launch_dependent(mx_swiglu_kernel<BF16>, grid, 256, stream, p);
}

cudaError_t launch_swiglu_backward(const RowIn &dy, const RowIn &gu, int64_t T, int64_t F,
                                   void *dgu, const DeviceInfo &dev, cudaStream_t stream) {
    GluArgs p{};
    p.dy = static_cast<const uint8_t *>(dy.p);
    p.dy_pitch = dy.pitch;
    p.gu = static_cast<const uint8_t *>(gu.p);
    p.gu_pitch = gu.pitch;
    p.y = {static_cast<uint8_t *>(dgu), static_cast<size_t>(T) * F * 4};
    p.T = T;
    p.F = F;
    p.chunks = F / 8;
    p.total = T * p.chunks;
    p.status = dev.status;
    const int64_t grid = (p.total + 255) / 256;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (dy.f32)
        return gu.f32 ? launch_dependent(mx_swiglu_backward_kernel<F32, F32>, grid, 256, stream, p)
                      : launch_dependent(mx_swiglu_backward_kernel<F32, BF16>, grid, 256, stream, p);
    return gu.f32 ? launch_dependent(mx_swiglu_backward_kernel<BF16, F32>, grid, 256, stream, p)
                  : launch_dependent(mx_swiglu_backward_kernel<BF16, BF16>, grid, 256, stream, p);
}

}  // namespace mx
