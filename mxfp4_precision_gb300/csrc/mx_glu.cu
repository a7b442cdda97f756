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

// Three forms of the sigmoid s = 1 / (1 + exp(-g)) and of silu(g) = g s, u = 2^-24.
//
// kFast, |g| <= 80: the hardware's 2^x and reciprocal.  Their errors (2 and 1
// units in the last place, 6 u), the rounded sum (u), the rounded product g log2 e
// and the rounding of log2 e itself (|g| u and 0.23 |g| u of the exponential) leave
// it within (7 + 1.23 |g|) u, 106 u at most: inside the outputs' roundings of 2^16 u
// (bf16) and more.  With bf16 input, where instructions bound the kernel, the form
// below takes 125 us against 99 us (8192 x 14336, codes alone; the memory 87 us).
//
// kFine, |g| <= 80: silu(g) = g / (1 + expf(-g)), each step rounded as fp32 rounds
// it, where the kernel has the time for it (fp32 in, bound by memory).  y, its codes
// and its scales then have the bits of the formula in fp32; a sigmoid that was
// multiplied by g put 6 in a million bf16 y on a rounding boundary's other side, at
// the same time.
//
// kFar, any g: beyond 80, where the exponential of the forms above leaves fp32's
// range, s is exp(g) down to the smallest subnormal below, within 116 u (the product
// is rounded at up to 2^8, 89 u) and a step of 2^-149, and 1 above; NaN for NaN.
enum : int { kFast, kFine, kFar };
template <int FORM>
__device__ __forceinline__ float sigmoid(float g) {
    float e, r;
    if (FORM == kFar && g < -80.0f) {
        asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(g * 0x1.715476p+0f));
        return e;
    }
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -0x1.715476p+0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// g / d to nearest for |g| <= 80 and d = 1 + exp(-g): a reciprocal with one Newton
// step, and a quotient with one correction from its remainder (Markstein, IBM J. Res.
// Dev. 34(1), 1990).  On the host it is the division's value for 4 10^8 such pairs, with
// the reciprocal one unit off either way.  The division itself takes the kernel from
// 178 to 182 us (fp32 in, 8192 x 14336).
__device__ __forceinline__ float quotient(float g, float d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    r = fmaf(r, fmaf(-d, r, 1.0f), r);
    const float q = g * r;
    return fmaf(-fmaf(d, q, -g), r, q);  // the remainder's sign so that -0 stays -0
}

// silu(g) in form NEAR up to 80; beyond, where FAR allows for such gates, in kFar: an
// element's form does not depend on its neighbours.
template <int NEAR, bool FAR>
__device__ __forceinline__ float silu(float g) {
    if (FAR && !(fabsf(g) <= 80.0f)) return g * sigmoid<kFar>(g);
    if constexpr (NEAR == kFine) return quotient(g, __fadd_rn(1.0f, expf(-g)));
    else return g * sigmoid<kFast>(g);
}

// Whether one of eight values lies beyond 80 or is NaN.
__device__ __forceinline__ bool any_far(const float (&g)[8]) {
    float top = enc::absmax2_nan(enc::absmax3_nan(g[0], g[1], g[2]), enc::absmax3_nan(g[3], g[4], g[5]));
    top = enc::absmax3_nan(top, g[6], g[7]);
    return !(top <= 80.0f);
}

// y = g * s * u of eight columns.
template <int NEAR, bool FAR>
__device__ __forceinline__ V8 gated(const float (&g)[8], const float (&u)[8]) {
    V8 y;
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        y.v[i / 2] = pack2(silu<NEAR, FAR>(g[i]) * u[i], silu<NEAR, FAR>(g[i + 1]) * u[i + 1]);
    return y;
}

// dg into u, du into d (which hold u and dy).
template <int FORM>
__device__ __forceinline__ void ungated(const float (&g)[8], float (&u)[8], float (&d)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float s = sigmoid<FORM>(g[i]), ds = d[i] * s;
        u[i] = ds * u[i] * fmaf(g[i], 1.0f - s, 1.0f);
        d[i] = ds * g[i];
    }
}

// One read, one write, bound by memory with fp32 input: 8192 x 14336 with bf16 y
// and MXFP8 codes 178 us, 1.30 GB = 7.3 TB/s (107% of a plain copy's rate: it
// writes less than it reads); the gradient 254 us, 1.88 GB = 7.4 TB/s (109%).  With
// bf16 input and codes alone the instructions bound it: 98.8 us, 591 MB = 6.0 TB/s
// (88%).
// Both kernels: a block is `deep` rows by `wide` chunks of 8 columns (a
// multiple of 32 threads), `segments` blocks side by side make a row; each
// thread keeps its columns and takes `turns` rows, two at a time.
// Small blocks: a finished one makes room for the next sooner (128 threads against
// 256: bf16 8192 x 4096 to codes alone 87% of a plain copy's rate, 81%).
constexpr int kBlock = 128;
struct GluArgs {
    const uint8_t *gu, *dy;
    int64_t gu_pitch, dy_pitch;  // bytes
    Out y;                       // y [T][F], or dgu [T][2F]
    Encoded enc;
    int64_t T;
    uint32_t F;
    int wide, segments, turns;
    uint32_t tiles;  // blocks that hold rows; those after them zero the scales' padding lines
    bool aligned32;
    int *status;
};

struct Place {
    int64_t row, end;  // rows row, row + deep, ... below end
    int deep;
    uint32_t c;
};
__device__ __forceinline__ Place place(const GluArgs &p) {
    const uint32_t band = blockIdx.x / p.segments, r = threadIdx.x / p.wide;
    Place at;
    at.deep = blockDim.x / p.wide;
    at.row = static_cast<int64_t>(band) * at.deep * p.turns + r;
    at.end = min(p.T, (static_cast<int64_t>(band) + 1) * at.deep * p.turns);
    at.c = (blockIdx.x - band * p.segments) * p.wide + (threadIdx.x - r * p.wide);
    return at;
}

template <typename G>
__global__ void __launch_bounds__(kBlock, G::kBytes == 4 ? 8 : 10) mx_swiglu_kernel(const __grid_constant__ GluArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x >= p.tiles) {
        zero_padding(p.enc, p.T, static_cast<int64_t>(blockIdx.x - p.tiles) * blockDim.x + threadIdx.x,
                     static_cast<int64_t>(gridDim.x - p.tiles) * blockDim.x, p.status);
        return;
    }
    const Place at = place(p);
    const uint32_t col = 8 * at.c;
    const bool in = col < p.F;
    // Only a warp that the row ends in has lanes to clear.
    const bool full = col - 8 * (at.c & 31) + 256 <= p.F;
    const uint8_t *src = p.gu + static_cast<size_t>(col) * G::kBytes;
    const size_t up = static_cast<size_t>(p.F) * G::kBytes;
    // Whole warps share a row, so that its blocks are encoded together.
    for (int64_t row = at.row; row < at.end; row += 2 * at.deep) {
        Raw8<G> gr[2], ur[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t r = row + k * at.deep;
            if (!full) {
                zero8(gr[k]);
                zero8(ur[k]);
            }
            if (in && r < at.end) {
                load8(gr[k], src + r * p.gu_pitch, p.aligned32);
                load8(ur[k], src + r * p.gu_pitch + up, p.aligned32);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t r = row + k * at.deep;
            if (r >= at.end) break;
            float g[8], u[8];
            floats_of(to_v8(gr[k]), g);
            floats_of(to_v8(ur[k]), u);
            constexpr int kNear = G::kBytes == 4 ? kFine : kFast;
            const V8 y = any_far(g) ? gated<kNear, true>(g, u) : gated<kNear, false>(g, u);
            if (in && p.y.p != nullptr)
                store8<BF16>(p.y, p.y.p + (r * p.F + col) * 2, y, p.aligned32, p.status);
            if (p.enc.fmt != kEncNone && at.c < p.enc.katoms * 16)
                encode8(p.enc, encoded_row(p.enc, r), at.c, in, y, p.status);
        }
    }
}

template <typename D, typename G>
__global__ void __launch_bounds__(kBlock) mx_swiglu_backward_kernel(const __grid_constant__ GluArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const Place at = place(p);
    const uint32_t col = 8 * at.c;
    if (col >= p.F) return;
    const uint8_t *src = p.gu + static_cast<size_t>(col) * G::kBytes;
    const uint8_t *dsrc = p.dy + static_cast<size_t>(col) * D::kBytes;
    const size_t up = static_cast<size_t>(p.F) * G::kBytes;
    for (int64_t row = at.row; row < at.end; row += at.deep) {
        Raw8<G> gr, ur;
        Raw8<D> dr;
        load8(dr, dsrc + row * p.dy_pitch, p.aligned32);
        load8(gr, src + row * p.gu_pitch, p.aligned32);
        load8(ur, src + row * p.gu_pitch + up, p.aligned32);
        float g[8], u[8], d[8];
        floats_of(to_v8(gr), g);
        floats_of(to_v8(ur), u);
        floats_of(to_v8(dr), d);
        if (any_far(g)) ungated<kFar>(g, u, d);
        else ungated<kFast>(g, u, d);
        V8 dg, du;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dg.v[i] = pack2(u[2 * i], u[2 * i + 1]);
            du.v[i] = pack2(d[2 * i], d[2 * i + 1]);
        }
        uint8_t *dst = p.y.p + (row * 2 * p.F + col) * 2;
        store8<BF16>(p.y, dst, dg, p.aligned32, p.status);
        store8<BF16>(p.y, dst + 2 * static_cast<size_t>(p.F), du, p.aligned32, p.status);
    }
}

// Tiles of rows whose `chunks` are cut into equal segments of at most a block;
// several rows a thread once there are blocks enough for every SM to be filled
// kWaves times.
constexpr int64_t kWaves = 2;
bool shape(GluArgs &p, int64_t chunks, int64_t pad_words, int most, const DeviceInfo &dev,
           int64_t *grid, int *threads) {
    p.segments = static_cast<int>((chunks + kBlock - 1) / kBlock);
    p.wide = static_cast<int>(((chunks + p.segments - 1) / p.segments + 31) / 32 * 32);
    const int deep = kBlock / p.wide;
    *threads = p.wide * deep;
    p.turns = most;
    auto tiles = [&] { return (p.T + deep * p.turns - 1) / (deep * p.turns) * p.segments; };
    while (p.turns > 1 && tiles() < kWaves * (2048 / kBlock) * dev.sm_count) p.turns /= 2;
    *grid = tiles() + (pad_words + *threads - 1) / *threads;
    p.tiles = static_cast<uint32_t>(tiles());
    return *grid <= 0x7FFFFFFF;
}

}  // namespace

cudaError_t launch_swiglu(const RowIn &gu, int64_t T, int64_t F, void *y, const RowEncode &e,
                          const DeviceInfo &dev, cudaStream_t stream) {
    GluArgs p{};
    p.gu = static_cast<const uint8_t *>(gu.p);
    p.gu_pitch = gu.pitch * (gu.f32 ? 4 : 2);
    p.y = {static_cast<uint8_t *>(y), static_cast<size_t>(T) * F * 2};
    p.enc = row_encoded(e, T, F);
    p.T = T;
    p.F = static_cast<uint32_t>(F);
    p.aligned32 = aligned32(gu.p);
    p.status = dev.status;
    int64_t grid = 0;
    int threads = 0;
    if (!shape(p, (F + 255) / 256 * 32, padding_words(p.enc, T), 4, dev, &grid, &threads))
        return cudaErrorInvalidValue;
    return gu.f32 ? launch_dependent(mx_swiglu_kernel<F32>, grid, threads, 0, stream, p)
                  : launch_dependent(mx_swiglu_kernel<BF16>, grid, threads, 0, stream, p);
}

cudaError_t launch_swiglu_backward(const RowIn &dy, const RowIn &gu, int64_t T, int64_t F,
                                   void *dgu, const DeviceInfo &dev, cudaStream_t stream) {
    GluArgs p{};
    p.dy = static_cast<const uint8_t *>(dy.p);
    p.dy_pitch = dy.pitch * (dy.f32 ? 4 : 2);
    p.gu = static_cast<const uint8_t *>(gu.p);
    p.gu_pitch = gu.pitch * (gu.f32 ? 4 : 2);
    p.y = {static_cast<uint8_t *>(dgu), static_cast<size_t>(T) * F * 4};
    p.T = T;
    p.F = static_cast<uint32_t>(F);
    p.aligned32 = aligned32(dy.p) && aligned32(gu.p);
    p.status = dev.status;
    int64_t grid = 0;
    int threads = 0;
    if (!shape(p, F / 8, 0, 1, dev, &grid, &threads)) return cudaErrorInvalidValue;
    if (dy.f32)
        return gu.f32 ? launch_dependent(mx_swiglu_backward_kernel<F32, F32>, grid, threads, 0, stream, p)
                      : launch_dependent(mx_swiglu_backward_kernel<F32, BF16>, grid, threads, 0, stream, p);
    return gu.f32 ? launch_dependent(mx_swiglu_backward_kernel<BF16, F32>, grid, threads, 0, stream, p)
                  : launch_dependent(mx_swiglu_backward_kernel<BF16, BF16>, grid, threads, 0, stream, p);
}

}  // namespace mx
