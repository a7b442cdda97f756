// mx_few.cu -- the products of mx_product.cu for few rows of A (tokens of a
// decoding step), dense and by expert (many experts: the second half of this file).
//
// With a handful of rows the product is a read of B: 2 M N K operations over
// N K / 2 bytes.  Tiles of 256 columns leave most SMs without one (4096 columns:
// 16 pairs) and walk their whole contraction one stage after the other.  Here a
// block takes 32 columns and splits the contraction over its warps, four blocks of 32
// elements at a time, so that all of B is on its way at once; the warps' sums
// are joined in shared memory in their order.
//
// A warp multiplies 32 lines of B by 8 rows of A per mma.sync.m16n8k16 (f16 in, fp32
// out): E2M1 and E4M3 values are f16 values, so the products are exact, and the
// instruction's rate does not matter where the read bounds the kernel.  Which element of
// the contraction takes which of its places is free as long as both operands
// agree, so lane c of four takes elements 8 c .. 8 c + 7 of a block: one load, and
// two instructions to a block, after which the sums get the block's scales.
//
// Measured: 8 x 4096 x 4096 6.0 us, of which an empty launch is 2.5 (the tiles: 9.5), 5 x 4128 x 2080 in MXFP8
// 5.0 us; 1 x 4096 x 14336 11.3 us = 2.8 TB/s.  (A plain sum over 67 MB, not written for this, runs at 3.4 TB/s.)  A
// ring of asynchronous copies a warp instead of the register loads: 13.4 us where these took 11.2 to 13.2.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>

#include "../../include/mx.h"
#include "mx_act.cuh"
#include "mx_encode.cuh"
#include "mx_internal.h"
#include "mx_ptx.cuh"
#include "mx_rows.cuh"

namespace mx {
namespace {

constexpr int kColumns = 32;  // of a block: one block of an encoded row
// Dense: one block an SM and all of B at once.  By expert: several smaller ones, since each first looks up
// its expert.
constexpr int kDenseWarps = 16, kExpertWarps = 8;

struct FewArgs {
    const uint8_t *Aq, *As, *Bq, *Bs;
    int64_t M, N;         // rows of A (by expert: the capacity of all segments)
    int64_t line_bytes;   // codes of a line
    int64_t katoms, b_groups;
    int blocks;           // blocks of 32 elements of a line
    int experts;          // 0: dense
    int columns;          // by lines: the items' columns, kLines at a time
    const int32_t *offsets, *counts;
    const uint8_t *bias, *res;
    int64_t res_pitch;    // bytes
    uint8_t *y, *z, *codes, *scales;
    size_t y_bytes, z_bytes, codes_bytes, scales_bytes;
    int64_t out_katoms;
    int act, bias_f32, res_f32, y_f32, fmt;
    int *status;
};

// Eight elements of a line as four f16 pairs.
template <bool FP8>
struct Codes;
template <>
struct Codes<false> {
    static constexpr int kBytes = 4;
    uint32_t w;
    __device__ __forceinline__ void load(const uint8_t *p) { w = *reinterpret_cast<const uint32_t *>(p); }
    __device__ __forceinline__ void clear() { w = 0; }
    __device__ __forceinline__ void values(uint32_t (&h)[4]) const {
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "mov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w));
    }
};
template <>
struct Codes<true> {
    static constexpr int kBytes = 8;
    uint2 w;
    __device__ __forceinline__ void load(const uint8_t *p) { w = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void clear() { w = make_uint2(0, 0); }
    __device__ __forceinline__ void values(uint32_t (&h)[4]) const {
        asm("{\n\t.reg .b16 a, b, c, d;\n\t"
            "mov.b32 {a, b}, %4;\n\t"
            "mov.b32 {c, d}, %5;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t"
            "cvt.rn.f16x2.e4m3x2 %2, c;\n\t"
            "cvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w.x), "r"(w.y));
    }
};

// D += A B: A 16 x 16 (a[0], a[2]: row r, a[1], a[3]: row r + 8), B 16 x 8.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// v 2^(a - 127) 2^(b - 127) for scale bytes a, b (255: NaN), in two steps of half the
// exponent each, so that nothing overflows that the result does not.
__device__ __forceinline__ float scaled(float v, uint32_t a, uint32_t b) {
    const uint32_t e = a + b, half = e >> 1;
    v = (v * __uint_as_float(half << 23)) * __uint_as_float((e - half) << 23);
    return a == 255u || b == 255u ? __uint_as_float(0x7FC00000u) : v;
}

// Where the scale bytes of a line's blocks 0 .. 3 lie; those of 4 n .. 4 n + 3 are 512 n further.
__device__ __forceinline__ const uint8_t *scales_of(const uint8_t *s, int64_t katoms, int64_t line) {
    return s + (line >> 7) * katoms * 512 + (line & 31) * 16 + ((line & 127) >> 5) * 4;
}
// Whether four scale bytes are all in 63 .. 190: two such powers of two have a product, -128 ..
// 126, that fp32 holds.  (b + 1 has one of its upper two bits then, and not both.)
__device__ __forceinline__ bool moderate(uint32_t s) {
    const uint32_t x = s + 0x01010101u;
    return ((x ^ (x << 1)) & 0x80808080u) == 0x80808080u;
}
__device__ __forceinline__ float power(uint32_t s, int j) { return __uint_as_float(((s >> (8 * j)) & 0xFFu) << 23); }
constexpr uint32_t kOnes = 0x7F7F7F7Fu;  // four scales of 1

__device__ __forceinline__ float activated(float x, int which) {
    const uint64_t v = act::same2(x);
    uint64_t r = v;
    switch (which) {
        case act::kRelu: r = act::value2<act::kRelu>(v); break;
        case act::kRelu2: r = act::value2<act::kRelu2>(v); break;
        case act::kGelu: r = act::value2<act::kGelu>(v); break;
        case act::kGeluTanh: r = act::value2<act::kGeluTanh>(v); break;
        case act::kSilu: r = act::value2<act::kSilu>(v); break;
        default: break;
    }
    float a, b;
    act::unpack2(r, a, b);
    return a;
}
__device__ __forceinline__ float element(const uint8_t *p, int64_t i, bool f32) {
    if (f32) return reinterpret_cast<const float *>(p)[i];
    return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << 16);
}
__device__ __forceinline__ void put_bf16(uint8_t *base, int64_t i, float v, size_t bytes, int *status) {
    uint8_t *p = base + 2 * i;
    if (MX_STORE_OK(p, 2, base, bytes, status)) *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(rows::bf16x2(v, 0.0f));
}

// One row's 32 columns, a lane each: v is the product (0 in padding).  Whole warps.
__device__ __forceinline__ void finish(const FewArgs &g, int64_t row, int expert, int col, bool real, float v) {
    const bool in = col < g.N;
    const int64_t e = row * g.N + col;
    if (real && in && g.bias != nullptr) v += element(g.bias, expert * g.N + col, g.bias_f32);
    if (g.z != nullptr && in) put_bf16(g.z, e, v, g.z_bytes, g.status);
    v = activated(v, g.act);
    if (g.res != nullptr && in) v += element(g.res + row * g.res_pitch, col, g.res_f32);
    if (g.y != nullptr && in) {
        if (g.y_f32) {
            uint8_t *p = g.y + 4 * e;
            if (MX_STORE_OK(p, 4, g.y, g.y_bytes, g.status)) *reinterpret_cast<float *>(p) = v;
        } else {
            put_bf16(g.y, e, v, g.y_bytes, g.status);
        }
    }
    if (g.fmt == kEncNone) return;
    const int lane = threadIdx.x & 31;
    float top = fabsf(v);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = enc::absmax2_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    float inv;
    const bool fp8 = g.fmt == kEncMX8;
    const uint32_t s = fp8 ? enc::scale_of_e4m3(top, inv) : enc::scale_of(top, inv);
    const float q = v * inv;
    if (fp8) {
        const uint32_t c = s == 0xFFu ? 0u : enc::cvt_e4m3x4(q, 0.0f, 0.0f, 0.0f) & 0xFFu;
        if (in && MX_STORE_OK(g.codes + e, 1, g.codes, g.codes_bytes, g.status)) g.codes[e] = static_cast<uint8_t>(c);
    } else {
        const float next = __shfl_down_sync(0xFFFFFFFFu, q, 1);
        const uint32_t c = s == 0xFFu ? 0u : enc::cvt_e2m1x8(q, next, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f) & 0xFFu;
        if (in && (lane & 1) == 0 && MX_STORE_OK(g.codes + e / 2, 1, g.codes, g.codes_bytes, g.status))
            g.codes[e / 2] = static_cast<uint8_t>(c);
    }
    if (lane == 0) {
        uint8_t *p = g.scales + enc::scale_offset(row, col / 32, g.out_katoms);
        if (MX_STORE_OK(p, 1, g.scales, g.scales_bytes, g.status)) *p = static_cast<uint8_t>(in ? s : 0u);
    }
}

// Zeroes the block's columns of rows first .. end - 1 (scales alone: the padding of a dense
// output's scales).  A thread per (row, 8 columns).
__device__ __forceinline__ void zero_rows(const FewArgs &g, int col0, int64_t first, int64_t end, bool scales_alone) {
    for (int64_t i = threadIdx.x; i < (end - first) * 4; i += blockDim.x) {
        const int64_t row = first + i / 4;
        const int part = static_cast<int>(i & 3), col = col0 + 8 * part;
        if (col < g.N && !scales_alone) {
            const int64_t e = row * g.N + col;
            const uint4 none = make_uint4(0, 0, 0, 0);
            if (g.z != nullptr && MX_STORE_OK(g.z + 2 * e, 16, g.z, g.z_bytes, g.status)) *reinterpret_cast<uint4 *>(g.z + 2 * e) = none;
            if (g.y != nullptr)
                for (int k = 0; k < (g.y_f32 ? 2 : 1); ++k) {
                    uint8_t *p = g.y + (g.y_f32 ? 4 : 2) * e + 16 * k;
                    if (MX_STORE_OK(p, 16, g.y, g.y_bytes, g.status)) *reinterpret_cast<uint4 *>(p) = none;
                }
            if (g.fmt == kEncMX8 && MX_STORE_OK(g.codes + e, 8, g.codes, g.codes_bytes, g.status))
                *reinterpret_cast<uint2 *>(g.codes + e) = make_uint2(0, 0);
            if (g.fmt == kEncMX4 && MX_STORE_OK(g.codes + e / 2, 4, g.codes, g.codes_bytes, g.status))
                *reinterpret_cast<uint32_t *>(g.codes + e / 2) = 0;
        }
        if (part == 0 && g.fmt != kEncNone) {
            uint8_t *p = g.scales + enc::scale_offset(row, col0 / 32, g.out_katoms);
            if (MX_STORE_OK(p, 1, g.scales, g.scales_bytes, g.status)) *p = 0;
        }
    }
}

// 32 columns (blockIdx.x; those behind the last are padding of the scales) of all rows, or by
// expert of 128 rows (blockIdx.y), which are one expert's or lie behind the last segment.
template <bool FP8, int NT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == kExpertWarps ? 3 : 1) mx_few_kernel(const __grid_constant__ FewArgs g) {
    griddep_wait();
    griddep_launch_dependents();
    const int col0 = static_cast<int>(blockIdx.x) * kColumns;
    int64_t first = 0, real = g.M;  // rows: taken by tokens up to `real`
    int expert = 0;
    __shared__ float part[WARPS][8 * NT][kColumns + 1];
    if (WARPS == kExpertWarps) {
        // Offsets are held to the rows that exist; any that go backwards: no rows (of segments that overlap
        // none would be the one).
        __shared__ int found, taken, backwards;
        first = static_cast<int64_t>(blockIdx.y) * 128;
        if (threadIdx.x == 0) found = taken = backwards = 0;
        __syncthreads();
        for (int e = threadIdx.x; e < g.experts; e += 32 * WARPS) {
            const int group = static_cast<int>(blockIdx.y), limit = static_cast<int>(g.M >> 7);
            const int begin = max(0, min(limit, g.offsets[e] >> 7)), end = max(0, min(limit, g.offsets[e + 1] >> 7));
            if (end < begin) backwards = 1;
            if (begin <= group && group < end) found = e, taken = max(0, min(128, max(0, g.counts[e]) - 128 * (group - begin)));
        }
        __syncthreads();
        expert = found;
        real = first + (backwards != 0 ? 0 : taken);
        zero_rows(g, col0, real, first + 128, false);
    } else if (g.fmt != kEncNone) {
        zero_rows(g, col0, g.M, (g.M + 127) / 128 * 128, true);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    using E = Codes<FP8>;
    const bool any = col0 < g.N;
    const int64_t line0 = expert * g.N + col0;
    const uint8_t *bs = g.Bs + expert * g.b_groups * g.katoms * 512;
    // Lines r, r + 8, r + 16, r + 24 of B; those beyond the last column stand on line 0 and are
    // not stored.
    const uint8_t *bq[4], *sb_at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int line = col0 + 8 * i + r < g.N ? 8 * i + r : 0;
        bq[i] = g.Bq + (line0 + line) * g.line_bytes + c * E::kBytes;
        sb_at[i] = scales_of(bs, g.katoms, col0 + line);
    }
    for (int64_t row0 = first; row0 < real; row0 += 8 * NT) {
        // Rows r of A (scales: rows 2 c, 2 c + 1); those beyond the last likewise.
        const uint8_t *aq[NT], *sa_at[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t row = row0 + 8 * t;
            aq[t] = g.Aq + min(row + r, real - 1) * g.line_bytes + c * E::kBytes;
#pragma unroll
            for (int k = 0; k < 2; ++k) sa_at[t][k] = scales_of(g.As, g.katoms, min(row + 2 * c + k, real - 1));
        }
        float sum[2][NT][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) sum[i][t][0] = sum[i][t][1] = sum[i][t][2] = sum[i][t][3] = 0.0f;
        for (int n = warp; any && 4 * n < g.blocks; n += WARPS) {
            // Four blocks of 32 elements; the last may be fewer (zeros with scales of 1).
            const int left = g.blocks - 4 * n;
            const int64_t at = static_cast<int64_t>(n) * 16 * E::kBytes, at_s = static_cast<int64_t>(n) * 512;
            const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : (1u << (8 * left)) - 1u;
            E b[4][4], a[NT][4];
            uint32_t sb[4], sa[NT][2];
            bool plain = true;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sb[i] = *reinterpret_cast<const uint32_t *>(sb_at[i] + at_s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    b[i][j].clear();
                    if (j < left) b[i][j].load(bq[i] + at + j * 4 * E::kBytes);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[t][j].clear();
                    if (j < left) a[t][j].load(aq[t] + at + j * 4 * E::kBytes);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    sa[t][k] = *reinterpret_cast<const uint32_t *>(sa_at[t][k] + at_s) & keep | kOnes & ~keep;
                    plain = plain && moderate(sa[t][k]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sb[i] = sb[i] & keep | kOnes & ~keep;
                plain = plain && moderate(sb[i]);
            }
            plain = __all_sync(0xFFFFFFFFu, plain);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t h[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i][j].values(h[i]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    uint32_t x[4];
                    a[t][j].values(x);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma(d, h[2 * i][0], h[2 * i + 1][0], h[2 * i][1], h[2 * i + 1][1], x[0], x[1]);
                        mma(d, h[2 * i][2], h[2 * i + 1][2], h[2 * i][3], h[2 * i + 1][3], x[2], x[3]);
                        if (plain) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                sum[i][t][k] = fmaf(d[k], power(sb[2 * i + (k >> 1)], j) * power(sa[t][k & 1], j), sum[i][t][k]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                sum[i][t][k] += scaled(d[k], (sb[2 * i + (k >> 1)] >> (8 * j)) & 0xFFu, (sa[t][k & 1] >> (8 * j)) & 0xFFu);
                        }
                    }
                }
            }
        }
        // d[k]: line r (k < 2) or r + 8 of the sixteen, row 2 c + (k & 1) of the eight.
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) part[warp][8 * t + 2 * c + (k & 1)][16 * i + 8 * (k >> 1) + r] = sum[i][t][k];
        __syncthreads();
        for (int m = warp; m < 8 * NT && row0 + m < real; m += WARPS) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) v += part[w][m][lane];
            finish(g, row0 + m, expert, col0 + lane, true, v);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- by expert, many of them
// The weights are the instruction's 128 rows and an expert's tokens its columns, as
// few as there are (a multiple of 16): nothing is decoded, and the tensor cores have a fraction
// of a tile's work.  A block stays on its SM and takes items in turn, kLines lines of an expert for up to
// 128 of its rows: one warp copies, one multiplies, four bring the scales to tensor memory, four have a
// lane quarter (32 lines, which are 32 columns of the output) each at the end, and two zero the rows without a
// token meanwhile.
//
// Measured: 24 rows to 64 experts of 2048 x 2048 (20 of them used, 42 MB, and 13 MB of zeros) 14.4 us; the tiles 17.8, the
// blocks above 21.5, of which their decoding is 7.  Without the zeros 1.5 less; a plain read of 42 MB takes 13, 2.5 of
// them the launch.  Items of 64 lines 20.4: a step's copies and scales cost the same for half the bytes.  Scales copied
// from shared to tensor memory by the products' own thread (tcgen05.cp) 23.3, two sets of warps for them 15.4.
constexpr int kLines = 128;       // of an item: the instruction's
constexpr int kTokens = 16;       // rows of a copy of A
constexpr int kRing = 6;
constexpr int kLineThreads = 384;
constexpr int kZeroWarp0 = 2, kZeroThreads = 64, kScaleWarp0 = 4, kEndWarp0 = 8;
constexpr uint32_t kLineBytes = 128;             // of a step
constexpr uint32_t kWeightBytes = kLines * kLineBytes, kTokenBytes = 128 * kLineBytes;
constexpr uint32_t kAtomBytes = 1024;            // room for a step's scales of 128 lines
constexpr uint32_t kAccColumns = 128, kScaleColumn = 2 * kAccColumns, kScaleColumns = 16, kAllColumns = 512;
static_assert(kScaleColumn + kRing * kScaleColumns <= kAllColumns, "scales fit in tensor memory");

template <bool FP8>
struct Step {
    static constexpr int kUnits = FP8 ? 1 : 2;  // of 128 elements, an atom of scales each
};
struct LineCtl {
    uint64_t full[kRing], scaled[kRing], empty[kRing], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort_flag;
    int backwards;
    uint32_t warp_groups[kLineThreads / 32];
    int start[MX_EXPERTS_MAX + 1];   // segments' first rows in units of 128
    int taken[MX_EXPERTS_MAX];       // rows of a segment with a token
    int before[MX_EXPERTS_MAX + 1];  // groups of 128 rows with a token of the experts before
};
constexpr size_t kLineSmem = 1024 + kRing * (kWeightBytes + kTokenBytes + 2 * kAtomBytes);
static_assert(kLineSmem + sizeof(LineCtl) + 1024 <= 232448, "shared memory of an SM");

// The last entry of at[0 .. n - 1] that is at most x (the first, if none is).
__device__ __forceinline__ int last_of(const int *at, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// An item: the expert, its first row and the end of its rows, the first column.  Items run
// over the columns, then an expert's rows, then the experts.
struct Item {
    int expert, row, end, col;
};
__device__ __forceinline__ Item item_of(const FewArgs &g, const LineCtl &ctl, int i) {
    const int group = i / g.columns, e = last_of(ctl.before, g.experts, group);
    const int first = ctl.start[e] * 128;
    return {e, first + 128 * (group - ctl.before[e]), first + ctl.taken[e], (i - group * g.columns) * kLines};
}
// The next one; there is one.
__device__ __forceinline__ void advance(const FewArgs &g, const LineCtl &ctl, Item &it) {
    it.col += kLines;
    if (it.col < g.columns * kLines) return;
    it.col = 0;
    it.row += 128;
    if (it.row < it.end) return;
    do ++it.expert;
    while (ctl.taken[it.expert] == 0);
    it.row = ctl.start[it.expert] * 128;
    it.end = it.row + ctl.taken[it.expert];
}
// Its rows in whole copies.
__device__ __forceinline__ int tokens_of(const Item &it) { return (min(128, it.end - it.row) + kTokens - 1) / kTokens * kTokens; }

// Zeroes part `n` of `parts` of bytes [from, to) of an output (whole 16 bytes).
__device__ __forceinline__ void zero_bytes(const FewArgs &g, uint8_t *base, int64_t from, int64_t to, size_t bytes, int n, int parts) {
    const int t = threadIdx.x - 32 * kZeroWarp0;
    if (base == nullptr) return;
    for (int64_t i = from + (static_cast<int64_t>(n) * kZeroThreads + t) * 16; i < to; i += static_cast<int64_t>(parts) * kZeroThreads * 16)
        if (MX_STORE_OK(base + i, 16, base, bytes, g.status)) *reinterpret_cast<uint4 *>(base + i) = make_uint4(0, 0, 0, 0);
}
// Rows without a token: of every 128 rows those behind their expert's, all before the first segment and behind
// the last.
// Each 128 rows are several blocks' (or a block has several).
__device__ __forceinline__ void zero_padding(const FewArgs &g, const LineCtl &ctl) {
    const int t = threadIdx.x - 32 * kZeroWarp0;
    const int groups = static_cast<int>(g.M >> 7), parts = max(1, static_cast<int>(gridDim.x) / groups);
    for (int u = blockIdx.x; u < groups * parts; u += gridDim.x) {
        const int n = u / groups, b = u - n * groups;
        int real = 0;
        if (b >= ctl.start[0] && b < ctl.start[g.experts]) {
            const int e = last_of(ctl.start, g.experts, b);
            real = max(0, min(128, ctl.taken[e] - 128 * (b - ctl.start[e])));
        }
        const int64_t from = static_cast<int64_t>(b) * 128 + real, to = static_cast<int64_t>(b) * 128 + 128;
        zero_bytes(g, g.y, from * g.N * (g.y_f32 ? 4 : 2), to * g.N * (g.y_f32 ? 4 : 2), g.y_bytes, n, parts);
        zero_bytes(g, g.z, from * g.N * 2, to * g.N * 2, g.z_bytes, n, parts);
        if (g.fmt == kEncNone) continue;
        zero_bytes(g, g.codes, g.fmt == kEncMX8 ? from * g.N : from * g.N / 2, g.fmt == kEncMX8 ? to * g.N : to * g.N / 2, g.codes_bytes, n, parts);
        // A row's four scale bytes of each atom.
        for (int64_t i = static_cast<int64_t>(n) * kZeroThreads + t; i < g.out_katoms * 128; i += static_cast<int64_t>(parts) * kZeroThreads) {
            const int row = static_cast<int>(i & 127);
            if (row < real) continue;
            uint8_t *p = g.scales + (b * g.out_katoms + (i >> 7)) * 512 + (row & 31) * 16 + (row >> 5) * 4;
            if (MX_STORE_OK(p, 4, g.scales, g.scales_bytes, g.status)) *reinterpret_cast<uint32_t *>(p) = 0;
        }
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kLineThreads, 1)
    mx_few_lines_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const __grid_constant__ FewArgs g) {
    constexpr int kUnits = Step<FP8>::kUnits;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ LineCtl ctl;
    uint8_t *weights = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *tokens = weights + kRing * kWeightBytes, *atoms = tokens + kRing * kTokenBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&ctl.full[i], 1), mbar_init(&ctl.scaled[i], 4), mbar_init(&ctl.empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&ctl.acc_full[i], 1), mbar_init(&ctl.acc_empty[i], kLineThreads / 32 - kEndWarp0);
        mbar_init(&ctl.drain, 1);
        ctl.abort_flag = ctl.backwards = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&ctl.tmem, kAllColumns);
        tmem_relinquish();
    }
    griddep_wait();
    griddep_launch_dependents();
    // The segments, held to the rows that exist whatever the plan says; ends before their starts: no rows.
    const int limit = static_cast<int>(g.M >> 7);
    for (int e = threadIdx.x; e <= g.experts; e += kLineThreads) {
        const int s = g.offsets[e] >> 7;
        ctl.start[e] = s < 0 ? 0 : s > limit ? limit : s;
        if (e < g.experts) ctl.taken[e] = g.counts[e];
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    static_assert(kLineThreads / 32 - kEndWarp0 == 4 && kEndWarp0 - kScaleWarp0 == 4, "a warp for each lane quarter");
    static_assert(MX_EXPERTS_MAX <= 2 * kLineThreads, "two experts a thread");
    int n[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e = 2 * threadIdx.x + k;
        if (e >= g.experts) continue;
        const int length = ctl.start[e + 1] - ctl.start[e];
        if (length < 0) ctl.backwards = 1;
        const int taken = max(0, min(ctl.taken[e], 128 * max(0, length)));
        ctl.taken[e] = taken;
        n[k] = (taken + 127) / 128;
    }
    uint32_t sum = n[0] + n[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) ctl.warp_groups[warp] = sum;
    __syncthreads();
    const bool none = ctl.backwards != 0;
    int before = sum - n[0] - n[1], all = 0;
    for (int i = 0; i < kLineThreads / 32; ++i) {
        const int v = ctl.warp_groups[i];
        if (i < warp) before += v;
        all += v;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e = 2 * threadIdx.x + k;
        if (e < g.experts) ctl.before[e] = before + (k ? n[0] : 0);
    }
    if (none)
        for (int e = threadIdx.x; e <= g.experts; e += kLineThreads) ctl.start[e] = 0;
    __syncthreads();
    // A block's items follow one another.  Every role walks over the same ones.
    const int64_t items = none ? 0 : static_cast<int64_t>(all) * g.columns;
    const int first = static_cast<int>(items * blockIdx.x / gridDim.x), end = static_cast<int>(items * (blockIdx.x + 1) / gridDim.x);
    const int units = (g.blocks + 3) / 4, steps = (units + kUnits - 1) / kUnits;
    volatile int *abort = &ctl.abort_flag;
    Item it{};
    if (first < end) it = item_of(g, ctl, first);
    // Columns that exist, and something to add up.
    const auto product = [&]() { return steps > 0 && it.col < g.N; };

    if (warp == 0 && lane == 0) {
        // ---------------------------------------------------------------- copies
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = first; ok && i < end; ++i) {
            if (i > first) advance(g, ctl, it);
            if (!product()) continue;
            const int rows = tokens_of(it);
            const uint8_t *bs = g.Bs + (it.expert * g.b_groups + (it.col >> 7)) * g.katoms * 512, *as = g.As + (it.row >> 7) * g.katoms * 512;
            for (int s = 0; s < steps; ++s) {
                if (!mbar_wait_inl(&ctl.empty[stage], phase ^ 1u, g.status, abort)) {
                    ok = false;
                    break;
                }
                uint64_t *bar = &ctl.full[stage];
                constexpr uint32_t scales = kUnits * 512;  // of 128 lines; the layout's width is a multiple of it
                mbar_arrive_expect_tx(bar, kWeightBytes + rows * kLineBytes + 2 * scales);
                const int x = s * static_cast<int>(kLineBytes);
                tma_load_2d(weights + stage * kWeightBytes, &map_b, bar, x, it.expert * static_cast<int>(g.N) + it.col);
                bulk_load(atoms + stage * 2 * kAtomBytes, bs + static_cast<int64_t>(s) * scales, scales, bar);
                bulk_load(atoms + stage * 2 * kAtomBytes + kAtomBytes, as + static_cast<int64_t>(s) * scales, scales, bar);
                for (int m = 0; m < rows; m += kTokens)
                    tma_load_2d(tokens + stage * kTokenBytes + m * kLineBytes, &map_a, bar, x, it.row + m);
                if (++stage == kRing) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1 && lane == 0) {
        // ---------------------------------------------------------------- products
        const uint32_t tmem = ctl.tmem;
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int i = first; ok && i < end; ++i) {
            if (i > first) advance(g, ctl, it);
            if (!product()) continue;
            const int rows = tokens_of(it);
            if (!mbar_wait_inl(&ctl.acc_empty[acc], acc_phase ^ 1u, g.status, abort)) break;
            tc_fence_after();
            for (int s = 0; s < steps; ++s) {
                if (!mbar_wait_inl(&ctl.scaled[stage], phase, g.status, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sf = tmem + kScaleColumn + kScaleColumns * stage;
                const uint32_t sw = smem_u32(weights + stage * kWeightBytes), st = smem_u32(tokens + stage * kTokenBytes);
                const int left = min(kUnits, units - s * kUnits);
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // 32 bytes of a line each
                    if (j >= 4 * left / kUnits) break;
                    const uint32_t more = s > 0 || j > 0 ? 1u : 0u;
                    if constexpr (FP8) {
                        mma_mxf8(tmem + kAccColumns * acc, sdesc_sw128(sw + 32u * j), sdesc_sw128(st + 32u * j), idesc_mxf8(128, rows, j, j), sf, sf + 8u, more);
                    } else {
                        mma_mxf4(tmem + kAccColumns * acc, sdesc_sw128(sw + 32u * j), sdesc_sw128(st + 32u * j),
                                 idesc_mxf4(128, rows, 2 * (j & 1), 2 * (j & 1)), sf + 4u * (j / 2), sf + 8u + 4u * (j / 2), more);
                    }
                }
                tc_commit(&ctl.empty[stage]);
                if (++stage == kRing) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            tc_commit(&ctl.acc_full[acc]);
            if ((acc ^= 1) == 0) acc_phase ^= 1u;
        }
        // Every tensor-core operation has finished before the tensor memory is released.
        tc_commit(&ctl.drain);
        mbar_wait_inl(&ctl.drain, 0, g.status, nullptr, 100ull * 1000ull * 1000ull);
    } else if (warp >= kZeroWarp0 && warp < kScaleWarp0) {
        zero_padding(g, ctl);
    } else if (warp >= kScaleWarp0 && warp < kEndWarp0) {
        // ---------------------------------------------------------------- scales
        // Lane l of every quarter gets lines l, l + 32, l + 64 and l + 96 of an atom in four columns, which is how
        // an atom lies in memory.  A step's columns are written again once its products are done (`empty`).
        const uint32_t lanes = ctl.tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kScaleColumn;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = first; ok && i < end; ++i) {
            if (i > first) advance(g, ctl, it);
            if (!product()) continue;
            for (int s = 0; s < steps; ++s) {
                ok = mbar_wait_inl(&ctl.full[stage], phase, g.status, abort);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint8_t *from = atoms + stage * 2 * kAtomBytes + lane * 16;
                uint32_t v[16] = {};
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(from + k * kAtomBytes + u * 512);
                        v[8 * k + 4 * u] = w.x, v[8 * k + 4 * u + 1] = w.y, v[8 * k + 4 * u + 2] = w.z, v[8 * k + 4 * u + 3] = w.w;
                    }
                tmem_st_32x32b_x16(lanes + kScaleColumns * stage, v);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.scaled[stage]);
                if (++stage == kRing) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp >= kEndWarp0) {
        // ---------------------------------------------------------------- ends
        const int q = warp & 3;  // tensor-memory lane quarter
        const uint32_t lanes = ctl.tmem + (static_cast<uint32_t>(32 * q) << 16);
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int i = first; i < end; ++i) {
            if (i > first) advance(g, ctl, it);
            const bool filled = product();
            const int real = min(128, it.end - it.row), col = it.col + 32 * q + lane;
            if (filled) {
                int ok = 1;
                if (lane == 0) ok = mbar_wait_inl(&ctl.acc_full[acc], acc_phase, g.status, abort) ? 1 : 0;
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                if (!ok) break;
                tc_fence_after();
            }
            for (int m0 = 0; m0 < real; m0 += 8) {
                uint32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (filled) {
                    tmem_ld_32x32b_x8(lanes + kAccColumns * acc + m0, v);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int m = 0; m < 8; ++m)
                    if (m0 + m < real) finish(g, it.row + m0 + m, it.expert, col, true, __uint_as_float(v[m]));
            }
            if (filled) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.acc_empty[acc]);
                if ((acc ^= 1) == 0) acc_phase ^= 1u;
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(ctl.tmem, kAllColumns);
    }
}

template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}
template <bool FP8>
cudaError_t launch_as(const FewArgs &g, dim3 grid, cudaStream_t stream) {
    if (g.experts > 0) return launch(mx_few_kernel<FP8, 1, kExpertWarps>, grid, 32 * kExpertWarps, 0, stream, g);
    return g.M > 8 ? launch(mx_few_kernel<FP8, 2, kDenseWarps>, grid, 32 * kDenseWarps, 0, stream, g)
                   : launch(mx_few_kernel<FP8, 1, kDenseWarps>, grid, 32 * kDenseWarps, 0, stream, g);
}
template <bool FP8>
cudaError_t launch_lines(const CUtensorMap &map_a, const CUtensorMap &map_b, const FewArgs &g, const DeviceInfo &dev, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};  // devices that know the kernel's shared memory
    const uint64_t bit = uint64_t{1} << (dev.ordinal & 63);
    if ((ready.load(std::memory_order_relaxed) & bit) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(mx_few_lines_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kLineSmem));
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch(mx_few_lines_kernel<FP8>, dim3(dev.sm_count, 1, 1), kLineThreads, kLineSmem, stream, map_a, map_b, g);
}

}  // namespace

// Where the tiles of mx_product.cu (256 columns, at most 76 pairs of SMs at a time) would leave most
// SMs idle.  Measured, us, the blocks of 32 columns and the tiles (MXFP4): 8 x 4096 x 4096 5.8 and 9.5,
// 8 x 4096 x 14336 13.2 and 20.8, 16 x 4096 x 14336 17.2 and 20.8; but 8 x 14336 x 4096 (56 tiles)
// 15.1 and 12.3.  By expert the host knows the capacity alone.  Below 128 rows an expert it is 128 times
// the number of rows, n < experts, each of which may be of another expert; at 128 rows an expert, n
// is anything from `experts` to experts + 127, and all may be of one.
namespace {
int64_t expert_tiles(const Product &p) { return p.M / 128 * ((p.N + 255) / 256); }
// Few tiles: the blocks of 32 columns fill more SMs than the blocks of 128 (2048 x 2048, 2 rows, 16 tiles: 5.4 us and 7.8;
// 512 x 1024, 16 rows, 32 tiles: 6.0 and 6.7; but 64 tiles of 2048 x 2048: 10.7 and 8.0).  They read an expert's weights once
// for every 8 of its rows, so few experts whose capacity is full go to the tiles (blocks and tiles, MXFP4): one of 4096 x 4096,
// 1, 16 and 128 rows: 8.3, 13.7, 82.5 and 11.9; two of 2048 x 2048, 2, 17 and 129 rows in equal shares: 5.8, 8.5, 28.7 and 9.5;
// four of 512 x 1024, 4, 67 and 131 rows: 3.9, 7.4, 10.8 and 7.9, all 131 in one: 29.4.  With eight, of 17 rows at most in the
// mean, 8, 71 and 135 rows: 4.3, 6.0, 7.7 and 8.3 (256 x 4096: 8.5, 13.2, 18.2 and 11.9; 135 in one expert 80).
bool few_blocks(const Product &p) {
    return p.mode == kProductRows && (p.M < 128 * p.experts || (p.M == 128 * p.experts && p.experts >= 8)) && expert_tiles(p) <= 32;
}
// More tiles, MXFP4, blocks of 128 columns and tiles: 64 experts of 2048 x 2048, 16 to 128 rows: 11.3 and 13.3 us to 31.2 and
// 33.6; 256 of 512 x 1024, 128 rows: 10.6 and 16.1; 128 of 1536 x 4096, 128 rows, 768 tiles: 63.0 and 63.1; but 16 of
// 14336 x 4096, 16 rows, 896 tiles: 63.7 and 62.3.  Few experts whose capacity is full may have many rows each: 8 of
// 4096 x 4096, 64 rows: 21.2 and 20.1, 128 rows: 22.6 and 20.1.  MXFP8 goes by the same bounds: 64 of 2048 x 2048 18.3 and
// 20.1 to 50.9 and 51.0; 896 tiles 128 and 133; 8 of 4096 x 4096 33.3 and 33.7, 35.1 and 33.5.
bool few_lines(const Product &p) {
    return p.mode == kProductRows && (p.M < 128 * p.experts || (p.M == 128 * p.experts && p.experts >= 32)) && expert_tiles(p) <= 768;
}
}  // namespace

bool few_rows(const Product &p) {
    const int64_t n_tiles = (p.N + 255) / 256;
    if (p.mode == kProductDense) return p.M <= 8 ? n_tiles <= 32 : p.M <= 16 && n_tiles <= 16;
    return few_blocks(p) || few_lines(p);
}

cudaError_t launch_few(const Product &p, const DeviceInfo &dev, cudaStream_t stream) {
    FewArgs g{};
    g.Aq = static_cast<const uint8_t *>(p.Aq), g.As = static_cast<const uint8_t *>(p.As);
    g.Bq = static_cast<const uint8_t *>(p.Bq), g.Bs = static_cast<const uint8_t *>(p.Bs);
    g.M = p.M;
    g.N = p.N;
    g.line_bytes = p.fp8 ? p.K : p.K / 2;
    g.katoms = scale_katoms(p.K);
    g.b_groups = scale_groups(p.N);
    g.blocks = static_cast<int>(p.K / 32);
    g.experts = p.mode == kProductRows ? static_cast<int>(p.experts) : 0;
    g.offsets = p.offsets;
    g.counts = p.counts;
    g.bias = static_cast<const uint8_t *>(p.bias);
    g.bias_f32 = p.bias_f32;
    g.res = static_cast<const uint8_t *>(p.res.p);
    g.res_f32 = p.res.f32;
    g.res_pitch = p.res.pitch * (p.res.f32 ? 4 : 2);
    const size_t out = static_cast<size_t>(p.M) * static_cast<size_t>(p.N);
    g.y = static_cast<uint8_t *>(p.y);
    g.y_f32 = p.y_f32;
    g.y_bytes = out * (p.y_f32 ? 4 : 2);
    g.z = static_cast<uint8_t *>(p.z);
    g.z_bytes = out * 2;
    g.fmt = p.enc.fmt;
    g.codes = static_cast<uint8_t *>(p.enc.codes);
    g.codes_bytes = p.enc.fmt == kEncMX8 ? out : out / 2;
    g.scales = static_cast<uint8_t *>(p.enc.scales);
    g.out_katoms = scale_katoms(p.N);
    g.scales_bytes = static_cast<size_t>(scale_groups(p.M)) * static_cast<size_t>(g.out_katoms) * 512;
    g.act = p.act;
    g.status = dev.status;
    // Columns up to the end of the scales' padding where there are scales.
    const int64_t end = p.enc.fmt == kEncNone ? p.N : g.out_katoms * 128;
    if (few_lines(p) && !few_blocks(p)) {
        g.columns = static_cast<int>((end + kLines - 1) / kLines);
        CUtensorMap map_a, map_b;
        std::memset(&map_a, 0, sizeof(map_a));
        std::memset(&map_b, 0, sizeof(map_b));
        if (p.K > 0) {  // without a contraction nothing is loaded
            const auto map = [&](CUtensorMap *m, const void *codes, int64_t lines, uint32_t box) {
                return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, g.line_bytes, lines, g.line_bytes, kLineBytes, box, CU_TENSOR_MAP_SWIZZLE_128B);
            };
            if (!map(&map_a, p.Aq, p.M, kTokens) || !map(&map_b, p.Bq, p.N * p.experts, kLines)) return cudaErrorInvalidValue;
        }
        return p.fp8 ? launch_lines<true>(map_a, map_b, g, dev, stream) : launch_lines<false>(map_a, map_b, g, dev, stream);
    }
    const int64_t columns = (end + kColumns - 1) / kColumns;
    const dim3 grid(static_cast<unsigned>(columns), static_cast<unsigned>(g.experts > 0 ? p.M / 128 : 1), 1);
    return p.fp8 ? launch_as<true>(g, grid, stream) : launch_as<false>(g, grid, stream);
}

}  // namespace mx
