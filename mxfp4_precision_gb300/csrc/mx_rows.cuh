// mx_rows.cuh -- device building blocks of the row operators between the
// GEMMs (RMS norm, SwiGLU and their gradients): typed 8-column loads and
// stores, sums over the threads of a row, and the MXFP8 / MXFP4 encode of
// rows whose columns lie across lanes.
//
// Every kernel here gives each thread chunks of 8 consecutive columns: 16
// bytes of bf16, 32 of fp32.  Four lanes hold one 32-column block, 16 lanes
// the four blocks whose scale bytes are one word of the tiled layout.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mx_encode.cuh"
#include "mx_internal.h"
#include "mx_ptx.cuh"

namespace mx {
namespace rows {

// Element types of the row operators' tensors (mx_type in mx.h).
struct BF16 {
    static constexpr int kBytes = 2;
};
struct F32 {
    static constexpr int kBytes = 4;
};

// Eight columns as loaded (kept packed until they are used, so that several
// loads can be in flight without their converted values taking registers).
template <typename T>
struct Raw8;
template <>
struct Raw8<BF16> {
    uint4 a;
};
template <>
struct Raw8<F32> {
    uint4 a, b;
};

__device__ __forceinline__ void load8(Raw8<BF16> &r, const uint8_t *p) {
    r.a = __ldcs(reinterpret_cast<const uint4 *>(p));
}
__device__ __forceinline__ void load8(Raw8<F32> &r, const uint8_t *p) {
    r.a = __ldcs(reinterpret_cast<const uint4 *>(p));
    r.b = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
}
__device__ __forceinline__ void zero8(Raw8<BF16> &r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero8(Raw8<F32> &r) { r.a = r.b = make_uint4(0, 0, 0, 0); }

__device__ __forceinline__ void to_f32(const Raw8<BF16> &r, float (&v)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void to_f32(const Raw8<F32> &r, float (&v)[8]) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}

// Two bf16 in a word, lo in the low half (round to nearest even).
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void from_f32(Raw8<BF16> &r, const float (&v)[8]) {
    r.a = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                     bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void from_f32(Raw8<F32> &r, const float (&v)[8]) {
    r.a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3]));
    r.b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                     __float_as_uint(v[7]));
}

// A written buffer: its base and extent (the bounds-checked build tests every
// store against them).
struct Out {
    uint8_t *p;
    size_t bytes;
};

template <typename T>
__device__ __forceinline__ void store8(const Out &o, int64_t at, const float (&v)[8], int *status) {
    Raw8<T> r;
    from_f32(r, v);
    uint8_t *d = o.p + at * T::kBytes;
    if (!MX_STORE_OK(d, 8 * T::kBytes, o.p, o.bytes, status)) return;
    reinterpret_cast<uint4 *>(d)[0] = r.a;
    if constexpr (T::kBytes == 4) reinterpret_cast<uint4 *>(d)[1] = r.b;
}

// A weight vector's 8 columns, of either type (uniform branch).
__device__ __forceinline__ void load_weight8(const uint8_t *w, bool w_f32, int64_t col,
                                             float (&v)[8]) {
    if (w_f32) {
        Raw8<F32> r;
        r.a = __ldg(reinterpret_cast<const uint4 *>(w + col * 4));
        r.b = __ldg(reinterpret_cast<const uint4 *>(w + col * 4) + 1);
        to_f32(r, v);
    } else {
        Raw8<BF16> r;
        r.a = __ldg(reinterpret_cast<const uint4 *>(w + col * 2));
        to_f32(r, v);
    }
}

// ---------------------------------------------------------------- encode
struct Encoded {
    Out codes, scales;
    int64_t katoms;  // scale atoms (4 blocks) per 128-line group
    int fmt;
};

// Encodes columns 8c .. 8c+7 of a row (c: the lane's chunk, lanes holding
// consecutive chunks with c % 16 == lane % 16; v = 0 past the row's end) and
// stores codes and scales.  Called by whole groups of 16 lanes.  The rules are those
// of mx_quantize and mx_quantize_mxfp8: the exponent of the block's largest
// magnitude less the format's largest exponent, codes to nearest even and
// saturating, a block with Inf or NaN: scale 0xFF and zero codes.  Chunks
// past the row's end give the zero bytes of the scales' padding.
__device__ __forceinline__ void encode8(const Encoded &e, int64_t row, int64_t cols, int64_t c,
                                        const float (&v)[8], int *status) {
    const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
    float m = enc::absmax2_nan(enc::absmax3_nan(v[0], v[1], v[2]), enc::absmax3_nan(v[3], v[4], v[5]));
    m = enc::absmax3_nan(m, v[6], v[7]);
    m = enc::absmax2_nan(m, __shfl_xor_sync(mask, m, 1));
    m = enc::absmax2_nan(m, __shfl_xor_sync(mask, m, 2));
    float inv;
    const uint32_t s = e.fmt == kEncMX8 ? enc::scale_of_e4m3(m, inv) : enc::scale_of(m, inv);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(v[i], inv);
    if (8 * c < cols) {
        if (e.fmt == kEncMX8) {
            uint2 w = make_uint2(enc::cvt_e4m3x4(q[0], q[1], q[2], q[3]),
                                 enc::cvt_e4m3x4(q[4], q[5], q[6], q[7]));
            if (s == 0xFFu) w = make_uint2(0, 0);
            uint8_t *d = e.codes.p + row * cols + 8 * c;
            if (MX_STORE_OK(d, 8, e.codes.p, e.codes.bytes, status))
                *reinterpret_cast<uint2 *>(d) = w;
        } else {
            uint32_t w = enc::cvt_e2m1x8(q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]);
            if (s == 0xFFu) w = 0;
            uint8_t *d = e.codes.p + row * (cols / 2) + 4 * c;
            if (MX_STORE_OK(d, 4, e.codes.p, e.codes.bytes, status))
                *reinterpret_cast<uint32_t *>(d) = w;
        }
    }
    // The bytes of four blocks to the lane of the first: one word.
    uint32_t w = s << (2 * (threadIdx.x & 12));
    w |= __shfl_xor_sync(mask, w, 4);
    w |= __shfl_xor_sync(mask, w, 8);
    if ((threadIdx.x & 15) == 0) {
        uint8_t *d = e.scales.p + enc::scale_offset(row, c / 4, e.katoms);
        if (MX_STORE_OK(d, 4, e.scales.p, e.scales.bytes, status))
            *reinterpret_cast<uint32_t *>(d) = w;
    }
}

// ---------------------------------------------------------------- sums
// Sum over the `width` lanes (a power of two) that share a row.
__device__ __forceinline__ float sum_lanes(float v, int width) {
    for (int o = width / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// ---------------------------------------------------------------- host
inline Encoded row_encoded(const RowEncode &e, int64_t T, int64_t K) {
    Encoded r{};
    r.fmt = e.fmt;
    r.katoms = scale_katoms(K);
    r.codes = {static_cast<uint8_t *>(e.codes),
               static_cast<size_t>(T) * static_cast<size_t>(e.fmt == kEncMX8 ? K : K / 2)};
    r.scales = {static_cast<uint8_t *>(e.scales),
                static_cast<size_t>(scale_groups(T)) * static_cast<size_t>(r.katoms) * 512};
    return r;
}

// Launch under the library's programmatic-dependent-launch rule (the kernel
// waits in griddep_wait before it touches global memory).
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int64_t grid, int threads,
                             cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rows
}  // namespace mx
