// mx_rows.cuh -- device building blocks of the row operators between the
// GEMMs (RMS norm, SwiGLU and their gradients): typed 8-column loads and
// stores, sums over the threads of a row, and the MXFP8 / MXFP4 encode of
// rows whose columns lie across lanes.
//
// Every kernel here gives each thread chunks of 8 consecutive columns: 16
// bytes of bf16, 32 of fp32.  Four lanes hold one 32-column block.
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

// ---------------------------------------------------------------- pairs
// Eight columns as four packed fp32 pairs {even column (low), odd (high)}: the
// f32x2 instructions round each half like the scalar ones, at half the issue
// slots, which is what these kernels run short of first.
struct V8 {
    uint64_t v[4];
};
using enc::add2;
using enc::mul2;
using enc::pack2;
using enc::sub2;
using enc::unpack2;
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t same2(float v) { return pack2(v, v); }
__device__ __forceinline__ float sum2(uint64_t a) {
    float lo, hi;
    unpack2(a, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ V8 zero_v8() { return V8{{0, 0, 0, 0}}; }
__device__ __forceinline__ void floats_of(const V8 &a, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(a.v[i], f[2 * i], f[2 * i + 1]);
}

// ---------------------------------------------------------------- loads and stores
// Eight columns as loaded: kept packed until they are used, so that several
// loads can be in flight without their converted values taking registers.
template <typename T>
struct Raw8 {
    uint32_t w[2 * T::kBytes];
};

__device__ __forceinline__ void load16(uint32_t *w, const uint8_t *p) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
}
template <typename T>
__device__ __forceinline__ void zero8(Raw8<T> &r) {
#pragma unroll
    for (int i = 0; i < 2 * T::kBytes; ++i) r.w[i] = 0;
}
// From shared memory, or from global memory that is read again shortly.
template <typename T>
__device__ __forceinline__ void load8_again(Raw8<T> &r, const uint8_t *p) {
    load16(r.w, p);
    if constexpr (T::kBytes == 4) load16(r.w + 4, p + 16);
}
// From global memory, without a copy in L1.  A lane's 32 bytes of fp32 are one
// instruction where they are 32-byte aligned: two of 16 bytes touch every sector
// twice, and once its first touch has left L1 the second goes to L2 again
// (SwiGLU's gradient, fp32 8192 x 14336: 403 us against 254 us, decided by how
// the compiler spaced the two).  Volatile, because the compiler otherwise spaces
// a group of loads out to save registers and fewer are in flight.  L2 keeps its
// default policy: marking these lines to leave first costs 3 to 5% of the
// bandwidth (SwiGLU, the same matrix: 187 us against 178 us).
__device__ __forceinline__ void load8(Raw8<BF16> &r, const uint8_t *p, bool = true) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p));
}
__device__ __forceinline__ void load8(Raw8<F32> &r, const uint8_t *p, bool aligned32 = true) {
    if (aligned32)
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                       "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                     : "l"(p));
    else
        load8_again(r, p);
}

__device__ __forceinline__ V8 to_v8(const Raw8<BF16> &r) {
    V8 a;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a.v[i] = pack2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u));
    return a;
}
__device__ __forceinline__ V8 to_v8(const Raw8<F32> &r) {
    V8 a;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a.v[i] = pack2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    return a;
}

// Two bf16 in a word, lo in the low half (round to nearest even).
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void from_v8(Raw8<BF16> &r, const V8 &a) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(a.v[i], lo, hi);
        r.w[i] = bf16x2(lo, hi);
    }
}
__device__ __forceinline__ void from_v8(Raw8<F32> &r, const V8 &a) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(a.v[i], lo, hi);
        r.w[2 * i] = __float_as_uint(lo), r.w[2 * i + 1] = __float_as_uint(hi);
    }
}

// A written buffer: its base and extent (the bounds-checked build tests every
// store against them).
struct Out {
    uint8_t *p;
    size_t bytes;
};

// Eight columns at d, inside o.
template <typename T>
__device__ __forceinline__ void store8(const Out &o, uint8_t *d, const V8 &a, bool aligned32,
                                       int *status) {
    Raw8<T> r;
    from_v8(r, a);
    if (!MX_STORE_OK(d, 8 * T::kBytes, o.p, o.bytes, status)) return;
    if constexpr (T::kBytes == 4) {
        if (aligned32) {
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(d), "r"(r.w[0]),
                         "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]),
                         "r"(r.w[6]), "r"(r.w[7])
                         : "memory");
            return;
        }
        reinterpret_cast<uint4 *>(d)[1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
    }
    reinterpret_cast<uint4 *>(d)[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
}

// Eight columns of a weight vector of either type (uniform branch).
__device__ __forceinline__ V8 load_weight8(const uint8_t *w, bool w_f32, uint32_t col) {
    if (w_f32) {
        Raw8<F32> r;
        load8_again(r, w + 4 * static_cast<size_t>(col));
        return to_v8(r);
    }
    Raw8<BF16> r;
    load8_again(r, w + 2 * static_cast<size_t>(col));
    return to_v8(r);
}

// ---------------------------------------------------------------- encode
struct Encoded {
    Out codes, scales;
    int64_t katoms;  // scale atoms (4 blocks) per 128-line group
    int64_t pitch;   // bytes of a row of codes
    int fmt;
};

// A row's codes and scales: where its chunk 0 and its block 0 go.
struct EncodedRow {
    uint8_t *codes, *scales;
};
__device__ __forceinline__ EncodedRow encoded_row(const Encoded &e, int64_t row) {
    const uint32_t r = static_cast<uint32_t>(row) & 127u;
    return {e.codes.p + row * e.pitch,
            e.scales.p + (static_cast<uint64_t>(row) >> 7) * static_cast<uint64_t>(e.katoms) * 512u +
                (r & 31u) * 16u + (r >> 5) * 4u};
}

// Encodes columns 8c .. 8c+7 of a row (c: the lane's chunk, lanes holding
// consecutive chunks with c % 32 == lane; `in`: the chunk lies in the row)
// and stores codes and scales.  Called by whole
// warps.  The rules are those of mx_quantize and
// mx_quantize_mxfp8: the exponent of the block's largest magnitude less the
// format's largest exponent, codes to nearest even and saturating, a block
// with Inf or NaN: scale 0xFF and zero codes.  Chunks past the row's end give
// the zero bytes of the scales' padding whatever a holds (0 times a row's Inf or
// NaN rstd is NaN).
__device__ __forceinline__ void encode8(const Encoded &e, const EncodedRow &at, uint32_t c, bool in,
                                        const V8 &a, int *status) {
    float f[8];
    floats_of(a, f);
    float m = enc::absmax2_nan(enc::absmax3_nan(f[0], f[1], f[2]), enc::absmax3_nan(f[3], f[4], f[5]));
    m = enc::absmax3_nan(m, f[6], f[7]);
    m = enc::absmax2_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = enc::absmax2_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    float inv;
    const bool fp8 = e.fmt == kEncMX8;
    const uint32_t s = fp8 ? enc::scale_of_e4m3(m, inv) : enc::scale_of(m, inv);
    V8 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q.v[i] = mul2(a.v[i], same2(inv));
    floats_of(q, f);
    if (in) {
        if (fp8) {
            uint2 w = make_uint2(enc::cvt_e4m3x4(f[0], f[1], f[2], f[3]),
                                 enc::cvt_e4m3x4(f[4], f[5], f[6], f[7]));
            if (s == 0xFFu) w = make_uint2(0, 0);
            uint8_t *d = at.codes + 8u * c;
            if (MX_STORE_OK(d, 8, e.codes.p, e.codes.bytes, status)) *reinterpret_cast<uint2 *>(d) = w;
        } else {
            uint32_t w = enc::cvt_e2m1x8(f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]);
            if (s == 0xFFu) w = 0;
            uint8_t *d = at.codes + 4u * c;
            if (MX_STORE_OK(d, 4, e.codes.p, e.codes.bytes, status)) *reinterpret_cast<uint32_t *>(d) = w;
        }
    }
    // One byte a block: the eight of a warp lie in two sectors, as two gathered words would.
    if ((threadIdx.x & 3) == 0) {
        uint8_t *d = at.scales + (c >> 4) * 512u + ((c >> 2) & 3u);
        if (MX_STORE_OK(d, 1, e.scales.p, e.scales.bytes, status)) *d = static_cast<uint8_t>(in ? s : 0u);
    }
}

// Words (4 blocks of a line) of the scales' padding lines T .. 128 * ceil(T / 128) - 1.
__host__ __device__ __forceinline__ int64_t padding_words(const Encoded &e, int64_t T) {
    return e.fmt == kEncNone ? 0 : (128 - T % 128) % 128 * e.katoms;
}
// Zeroes them: the n-th of `threads` threads.
__device__ __forceinline__ void zero_padding(const Encoded &e, int64_t T, int64_t n, int64_t threads,
                                             int *status) {
    const int64_t words = padding_words(e, T);
    const uint32_t katoms = static_cast<uint32_t>(e.katoms);  // words fit 32 bits: columns are below 2^30
    for (int64_t i = n; i < words; i += threads) {
        const uint32_t line = static_cast<uint32_t>(i) / katoms;
        const uint32_t atom = static_cast<uint32_t>(i) - line * katoms;
        uint8_t *d = encoded_row(e, T + line).scales + static_cast<size_t>(atom) * 512;
        if (MX_STORE_OK(d, 4, e.scales.p, e.scales.bytes, status)) *reinterpret_cast<uint32_t *>(d) = 0;
    }
}

// ---------------------------------------------------------------- sums
// Sum over the warp.
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// ---------------------------------------------------------------- host
inline Encoded row_encoded(const RowEncode &e, int64_t T, int64_t K) {
    Encoded r{};
    r.fmt = e.fmt;
    r.katoms = scale_katoms(K);
    r.pitch = e.fmt == kEncMX8 ? K : K / 2;
    r.codes = {static_cast<uint8_t *>(e.codes),
               static_cast<size_t>(T) * static_cast<size_t>(r.pitch)};
    r.scales = {static_cast<uint8_t *>(e.scales),
                static_cast<size_t>(scale_groups(T)) * static_cast<size_t>(r.katoms) * 512};
    return r;
}

inline bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// Launch under the library's programmatic-dependent-launch rule (the kernel
// waits in griddep_wait before it touches global memory).
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int64_t grid, int threads, size_t smem,
                             cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.dynamicSmemBytes = smem;
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
