// mx_product.cu -- block-scaled products with an epilogue, and products grouped
// by expert, on the sm_103a tensor cores (mx_gemm_bias_act, mx_gemm_experts,
// mx_gemm_experts_wgrad).
//
//   dense    z = A . B^T + bias,   y = act(z) + residual
//   rows     the same for the rows of each expert e with B_e and bias_e; A's rows lie
//            in the experts' order, each expert's segment at a multiple of 128 rows
//   depth    C_e = A_e . B_e^T over expert e's slice of the contraction (Wgrad:
//            both operands are encoded along the same rows)
//
// The main loop is the one of mx_gemm.cu (there: why it is built so, and what it measured): one 2-CTA
// cluster per SM pair and 256 x 256 output tiles by tcgen05.mma.cta_group::2, operands through a
// 3-stage TMA ring, block scales through a 5-slot ring of their own into tensor memory by four writer
// warps, epilogue warps that take the accumulator into registers at once, so that the next tile
// multiplies while they work.  What differs is where a tile lies: every role walks the same list of
// tiles, and a tile names its rows of A and B, its scale atoms and its length.
//
// Segments at multiples of 128 rows are what makes the groups cheap: 128 lines are one scale group
// (rows) and 128 elements one scale atom (depth), so no scale has to be moved, a tile's half (one CTA's
// 128 rows) belongs to one expert, and only the last K sub-tile of a slice can be half a sub-tile (two
// of its four MMAs are issued).  The experts' offsets are read on the device, so a plan made there
// needs no copy to the host.
//
// Epilogue.  Bias, activation, residual, both outputs and the codes take some 30 instructions a column
// where all are asked for (GELU 13 of them, two columns at a time), against which the tensor cores' time for
// a tile of K = 4096 is 5.3 us.  Sixteen warps of 64 columns and not eight of 128: 8192 x 14336 x 4096
// with bias, GELU, z, bf16 y and MXFP8 rows takes 210 us, 244 with eight, whose instructions wait for one another
// (96 registers hold 64 columns and what they need, so the 768 threads' 80 at launch are split
// 48 / 96).  With bf16 y alone it is 148 us, where the operations at the tensor cores' measured rate take 100.
// Stores leave as they come: spreading them over the next tile's stages, which mx_gemm.cu gains by, cost 5 to 25% in
// every form here.  An L2 prefetch of the next B panel made no difference.  z and y are rounded from fp32
// once each, codes from y in fp32.
// Measured (calls replayed one after another), as shares of the tensor cores' 9,650 TFLOP/s for FP4 and half of it for
// FP8: MXFP4 operands, bf16 y alone 67%, everything 47%; 8 experts of 14336 x 4096 over 16384 rows with bias and SiLU 54%
// (366 us); their Wgrad writes 1.88 GB of fp32 in 453 us.  MXFP8 operands: bf16 y alone 262 us (76%), everything 314 to 323.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mx.h"
#include "mx_act.cuh"
#include "mx_encode.cuh"
#include "mx_internal.h"
#include "mx_ptx.cuh"

namespace mx {
namespace {

constexpr int kTile = 256;                        // output tile (rows and columns) per pair
constexpr int kHalf = 128;                        // rows of A / of B per CTA
constexpr int kBKBytes = 128;                     // bytes per row of a K sub-tile
constexpr int kKSub = 2;                          // sub-tiles per stage
constexpr int kStages = 3;
constexpr int kSFRing = kStages + 2;
constexpr int kWriterWarp0 = 4;                   // warps 4..7: scale writers
constexpr int kEpiWarp0 = 8;                      // warps 8..23: epilogue
constexpr int kEpiWarps = 16;
constexpr int kEpiCols = 64;                      // columns of an epilogue warp
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kLaunchRegs = 80;
constexpr int kRegsLow = 48, kRegsHigh = 96;
static_assert(32 * (kEpiWarp0 * kRegsLow + kEpiWarps * kRegsHigh) <= kThreads * kLaunchRegs, "register split fits the launch");
static_assert(kThreads * kLaunchRegs <= 65536, "launch registers fit the SM");
constexpr uint32_t kSubBytes = kHalf * kBKBytes;  // 16 KB: 128 rows x one K sub-tile
constexpr uint32_t kStageBytes = 2 * kKSub * kSubBytes;
constexpr uint32_t kOffB = kKSub * kSubBytes;
constexpr uint32_t kSFSub = 1024;                 // scale room per sub-tile and 128 rows
constexpr uint32_t kOffSFB = kKSub * kSFSub;
constexpr uint32_t kSFSlotBytes = 3 * kKSub * kSFSub;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kAccCol = 0, kSFCol = 256;
constexpr uint32_t kSFCols = 24;                  // tensor-memory columns per sub-tile: A 8, B 16
constexpr uint32_t kSFSlot = kSFCols * kKSub;
static_assert(kSFCol + kStages * kSFSlot <= kTmemCols, "scale slots fit in tensor memory");
constexpr int kBand = 16;                         // tile rows of a band (L2 reuse, see mx_gemm.cu)

constexpr int kFmtMX4 = 0, kFmtMX8 = 1;
template <int FMT>
struct Elem {
    static constexpr int kUnits = FMT == kFmtMX8 ? 1 : 2;       // 128-element units per sub-tile
    static constexpr int kAtoms = kUnits;                       // scale atoms per sub-tile
    static constexpr uint32_t kUnitBytes = FMT == kFmtMX8 ? 128 : 64;
};

enum : int { kDense = 0, kRows = 1, kDepth = 2 };

// n / d for 0 <= n < 2^31 as a multiplication: with 2^(l-1) < d <= 2^l, m = floor(2^(31+l) / d) + 1
// fits 32 bits, and n m / 2^(31+l) is above n / d by less than n / 2^(31+l) <= 1 / d.
struct Divisor {
    uint32_t m, shift, d;
};
inline Divisor divisor(int64_t d) {
    uint32_t l = 0;
    while ((int64_t{1} << l) < d) ++l;
    return {static_cast<uint32_t>((uint64_t{1} << (31 + l)) / static_cast<uint64_t>(d) + 1), 31 + l, static_cast<uint32_t>(d)};
}
__device__ __forceinline__ int divide(int n, const Divisor &d) {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * d.m) >> d.shift);
}

struct ProductArgs {
    const uint8_t *As, *Bs;
    int64_t M, N;            // rows: M is the capacity of all segments; depth: per expert
    int64_t katoms;          // scale atoms along the contraction per 128-line group
    int64_t a_groups, b_groups;  // 128-line scale groups of A, and of B (per expert in `rows`)
    int k_units;             // contraction in units of 128 elements (depth: of all experts)
    int m_tiles, n_tiles;    // per expert in `depth`
    Divisor by_n, by_band, by_last, by_expert;  // n_tiles, a band's tiles, the last band's rows, an expert's tiles (depth)
    int num_items;           // dense, depth
    int experts;
    const int32_t *offsets;  // [experts + 1] rows
    const int32_t *counts;   // [experts] rows that are real (rows)
    // Epilogue.
    const uint8_t *bias;     // [N] or [experts][N]
    const uint8_t *res;      // [M][N], pitch in bytes
    int64_t res_pitch;
    uint8_t *y, *z, *codes, *scales;
    size_t y_bytes, z_bytes, codes_bytes, scales_bytes;
    int64_t out_katoms;
    int act, bias_f32, res_f32, y_f32, fmt;
    int wide, wide_codes;    // y's and z's rows, and codes, allow 32-byte stores
    int *status;
};

struct SharedCtl {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t sf_full[kSFRing];
    uint64_t sf_free[kSFRing];
    uint64_t acc_full;
    uint64_t acc_empty;
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    uint32_t warp_tiles[kThreads / 32];
    int start[MX_EXPERTS_MAX + 1];              // segments' first rows in units of 128
    uint16_t tiles_before[MX_EXPERTS_MAX + 1];  // tile rows of the experts before (rows)
};
static_assert(MX_EXPERTS_MAX < kThreads, "one thread per expert in the set-up");

constexpr size_t kSmem = kStages * kStageBytes + kSFRing * kSFSlotBytes + sizeof(SharedCtl) + 1024;
static_assert(kSmem <= 232448, "shared memory of an SM");

// Where a tile lies.  Every role of a CTA computes the same tiles in the same order.
struct Tile {
    int a_row, b_row;          // first rows of A and of B (before this CTA's half)
    int64_t a_group, b_group;  // their 128-line scale groups
    int a_left, b_left;        // groups that exist from there (0: none)
    int units;                 // length in units of 128 elements
    int unit0;                 // first unit of the contraction
    int expert;
    int row, col;              // first row and column of the output
    int m_left;                // rows of the expert's segment from `row` on (padding included)
};

// Tile t of m_tiles x n_tiles: bands of kBand tile rows, column by column within a band.
// by_last: the last band's rows (0: not known, an ordinary division).
__device__ __forceinline__ void band_coords(const ProductArgs &g, int t, int m_tiles, const Divisor *by_last, int &mb, int &nb) {
    const int band = divide(t, g.by_band), r = t - band * kBand * g.n_tiles;
    const int first = band * kBand, rows = m_tiles - first;
    nb = rows >= kBand ? r / kBand : by_last != nullptr ? divide(r, *by_last) : r / rows;
    mb = first + r - nb * (rows >= kBand ? kBand : rows);
}

template <int MODE>
__device__ __forceinline__ Tile tile_of(const ProductArgs &g, const SharedCtl *ctl, int t) {
    Tile w;
    int mb, nb;
    w.unit0 = 0;
    w.units = g.k_units;
    w.expert = 0;
    if constexpr (MODE == kDense) {
        band_coords(g, t, g.m_tiles, &g.by_last, mb, nb);
        w.row = mb * kTile;
        w.b_row = nb * kTile;
        w.b_group = 2 * static_cast<int64_t>(nb);
        w.m_left = static_cast<int>(g.M - w.row);
    } else if constexpr (MODE == kRows) {
        // The last expert whose tiles begin at or before t (experts without rows have none).
        const int tm = divide(t, g.by_n);
        int lo = 0, hi = g.experts - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (ctl->tiles_before[mid] <= tm) lo = mid;
            else hi = mid - 1;
        }
        const int before = ctl->tiles_before[lo];
        band_coords(g, t - before * g.n_tiles, ctl->tiles_before[lo + 1] - before, nullptr, mb, nb);
        w.expert = lo;
        w.row = ctl->start[lo] * 128 + mb * kTile;
        w.m_left = ctl->start[lo + 1] * 128 - w.row;
        w.b_row = lo * static_cast<int>(g.N) + nb * kTile;
        w.b_group = static_cast<int64_t>(lo) * g.b_groups + 2 * nb;
    } else {
        w.expert = divide(t, g.by_expert);
        band_coords(g, t - w.expert * static_cast<int>(g.by_expert.d), g.m_tiles, &g.by_last, mb, nb);
        w.unit0 = ctl->start[w.expert];
        w.units = max(0, ctl->start[w.expert + 1] - w.unit0);
        w.row = mb * kTile;
        w.b_row = nb * kTile;
        w.b_group = 2 * static_cast<int64_t>(nb);
        w.m_left = static_cast<int>(g.M - w.row);
    }
    w.a_row = w.row;
    w.a_group = w.row >> 7;
    w.a_left = static_cast<int>(g.a_groups - w.a_group);
    w.b_left = static_cast<int>(g.b_groups) - 2 * nb;
    w.col = nb * kTile;
    return w;
}
template <int FMT>
__device__ __forceinline__ int stages_of(const Tile &w) {
    return (w.units + kKSub * Elem<FMT>::kUnits - 1) / (kKSub * Elem<FMT>::kUnits);
}

// Reads the segments' bounds, held to the rows that exist whatever the plan says, and counts
// the tile rows before each expert.  An end before its start: no rows of that expert (depth), or
// of any (rows: segments that overlap could hold more tiles than the counts do).  All threads.
template <int MODE>
__device__ __forceinline__ int read_segments(const ProductArgs &g, SharedCtl *ctl, int64_t rows) {
    const int e = threadIdx.x;
    const int limit = static_cast<int>(rows >> 7);
    if (e <= g.experts) {
        const int s = g.offsets[e] >> 7;
        ctl->start[e] = s < 0 ? 0 : s > limit ? limit : s;
    }
    __syncthreads();
    if constexpr (MODE == kDepth) return g.num_items;
    const int lane = e & 31, warp = e >> 5;
    const int length = e < g.experts ? ctl->start[e + 1] - ctl->start[e] : 0;
    const uint32_t n = length > 0 ? (length + 1) / 2 : 0;
    uint32_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
    }
    constexpr uint32_t kBackwards = 1u << 31;  // beside a warp's tiles, which are below 2^28
    const bool backwards = __any_sync(0xFFFFFFFFu, length < 0);
    if (lane == 31) ctl->warp_tiles[warp] = backwards ? kBackwards : sum;
    __syncthreads();
    uint32_t before = 0, all = 0, any = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        const uint32_t v = ctl->warp_tiles[i];
        if (i < warp) before += v;
        all += v;
        any |= v;
    }
    if (any & kBackwards) {
        if (e <= g.experts) ctl->start[e] = 0;
        __syncthreads();
        return 0;
    }
    if (e < g.experts) ctl->tiles_before[e] = static_cast<uint16_t>(before + sum - n);
    if (e == 0) ctl->tiles_before[g.experts] = static_cast<uint16_t>(all);
    __syncthreads();
    return static_cast<int>(all) * g.n_tiles;
}

__device__ __forceinline__ void arrive_even(uint64_t *bar) {
    mbar_arrive_remote(mapa_shared(smem_u32(bar), 0u));
}

// Outputs are written once and not read here: past L1, first to leave L2.
__device__ __forceinline__ void st_out32(void *p, const uint32_t *v) {
    asm volatile("st.global.L1::no_allocate.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void st_out16(void *p, const uint32_t *v) {
    asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(uint64_t v) {
    float lo, hi;
    enc::unpack2(v, lo, hi);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 32 columns of a row, as 16 packed fp32 pairs.
struct Row32 {
    uint64_t v[16];
};

// To p (columns c .. c + 31 of a row of N, the first `cols` of them inside it; nothing where the
// lane's row is not stored) in bf16 or fp32.  N is a multiple of 8; cols is the warp's.
__device__ __forceinline__ void store_bf16(uint8_t *p, const uint8_t *base, size_t bytes, const Row32 &a, int cols,
                                           bool stored, bool wide, int *status) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = bf16_pair(a.v[i]);
    if (wide && cols >= 32) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (stored && MX_STORE_OK(p + 32 * i, 32, base, bytes, status)) st_out32(p + 32 * i, &w[8 * i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (stored && 8 * i < cols && MX_STORE_OK(p + 16 * i, 16, base, bytes, status)) st_out16(p + 16 * i, &w[4 * i]);
}
__device__ __forceinline__ void store_f32(uint8_t *p, const uint8_t *base, size_t bytes, const Row32 &a, int cols,
                                          bool stored, bool wide, int *status) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (!stored || 8 * i >= cols || !MX_STORE_OK(p + 32 * i, 32, base, bytes, status)) continue;
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float lo, hi;
            enc::unpack2(a.v[4 * i + k], lo, hi);
            w[2 * k] = __float_as_uint(lo), w[2 * k + 1] = __float_as_uint(hi);
        }
        if (wide) {
            st_out32(p + 32 * i, w);
        } else {
            st_out16(p + 32 * i, w);
            st_out16(p + 32 * i + 16, w + 4);
        }
    }
}

// Adds 32 columns of a bf16 or fp32 row (16-byte aligned).
__device__ __forceinline__ void add_row(Row32 &a, const uint8_t *p, bool f32, int cols) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (8 * i >= cols) break;
        if (f32) {
            const ulonglong2 s = *reinterpret_cast<const ulonglong2 *>(p + 32 * i);
            const ulonglong2 t = *reinterpret_cast<const ulonglong2 *>(p + 32 * i + 16);
            a.v[4 * i] = enc::add2(a.v[4 * i], s.x), a.v[4 * i + 1] = enc::add2(a.v[4 * i + 1], s.y);
            a.v[4 * i + 2] = enc::add2(a.v[4 * i + 2], t.x), a.v[4 * i + 3] = enc::add2(a.v[4 * i + 3], t.y);
        } else {
            const uint4 s = *reinterpret_cast<const uint4 *>(p + 16 * i);
            const uint32_t w[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                a.v[4 * i + k] = enc::add2(a.v[4 * i + k], enc::pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)));
        }
    }
}

template <int ACT, int P>
__device__ __forceinline__ void activate(uint64_t (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = act::value2<ACT>(v[i]);
}

// Codes of one 32-column block; its scale byte is returned.
__device__ __forceinline__ uint32_t encode32(const ProductArgs &g, uint8_t *p, const Row32 &a, bool stored) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 16; ++i) enc::unpack2(a.v[i], v[2 * i], v[2 * i + 1]);
    const float top = enc::block_amax32(v);
    float inv;
    const bool fp8 = g.fmt == kEncMX8;
    const uint32_t s = fp8 ? enc::scale_of_e4m3(top, inv) : enc::scale_of(top, inv);
    const uint64_t inv2 = act::same2(inv);
#pragma unroll
    for (int i = 0; i < 16; ++i) enc::unpack2(enc::mul2(a.v[i], inv2), v[2 * i], v[2 * i + 1]);
    uint32_t w[8];
    if (fp8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = s == 0xFFu ? 0u : enc::cvt_e4m3x4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        if (stored && MX_STORE_OK(p, 32, g.codes, g.codes_bytes, g.status)) {
            if (g.wide_codes) {
                st_out32(p, w);
            } else {
                st_out16(p, w);
                st_out16(p + 16, w + 4);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = s == 0xFFu ? 0u
                              : enc::cvt_e2m1x8(v[8 * i], v[8 * i + 1], v[8 * i + 2], v[8 * i + 3], v[8 * i + 4], v[8 * i + 5],
                                                v[8 * i + 6], v[8 * i + 7]);
        if (stored && MX_STORE_OK(p, 16, g.codes, g.codes_bytes, g.status)) st_out16(p, w);
    }
    return s;
}

// A warp's place in the epilogue: 32 rows and 64 columns of a tile.
struct EpiTile {
    int row;     // the lane's row of the output (depth: of its expert's)
    int expert;
    int col;     // first column
    int left;    // rows from the lane's on that are inside the output (none: 0 or less)
    int real;    // ... that are not padding
    int scaled;  // ... whose scales exist
};

// Two blocks' scale bytes of a row (blocks of columns col, col + 32): half a word of the tiled
// layout.  Rows and columns of its padding get zeros.
__device__ __forceinline__ void put_scales(const ProductArgs &g, const EpiTile &at, int more, uint32_t two) {
    if (g.fmt == kEncNone || more >= at.scaled) return;
    const int row = at.row + more;
    uint8_t *p = g.scales + ((row >> 7) * g.out_katoms + (at.col >> 7)) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 + ((at.col >> 5) & 3);
    if (MX_STORE_OK(p, 2, g.scales, g.scales_bytes, g.status)) *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(two);
}

template <int P>
__device__ __forceinline__ void activate(const ProductArgs &g, uint64_t (&v)[P]) {
    switch (g.act) {  // all of them keep 0 (padding rows)
        case act::kRelu: activate<act::kRelu, P>(v); break;
        case act::kRelu2: activate<act::kRelu2, P>(v); break;
        case act::kGelu: activate<act::kGelu, P>(v); break;
        case act::kGeluTanh: activate<act::kGeluTanh, P>(v); break;
        case act::kSilu: activate<act::kSilu, P>(v); break;
        default: break;
    }
}

// Columns at.col + part .. + 31 of the lane's row from its accumulator.  Returns the scale byte.
template <int MODE>
__device__ __forceinline__ uint32_t finish32(const ProductArgs &g, const EpiTile &at, int part, const uint32_t (&acc)[32]) {
    const int col = at.col + part;
    const int cols = static_cast<int>(g.N) - col;
    if (cols <= 0) return 0;
    const bool stored = at.left > 0;
    Row32 a;
#pragma unroll
    for (int i = 0; i < 16; ++i) a.v[i] = enc::pack2(__uint_as_float(acc[2 * i]), __uint_as_float(acc[2 * i + 1]));
    if constexpr (MODE == kDepth) {
        const int64_t e = (at.expert * g.M + at.row) * g.N + col;
        if (g.y_f32) store_f32(g.y + 4 * e, g.y, g.y_bytes, a, cols, stored, g.wide, g.status);
        else store_bf16(g.y + 2 * e, g.y, g.y_bytes, a, cols, stored, g.wide, g.status);
        return 0;
    }
    if (g.bias != nullptr)
        add_row(a, g.bias + ((MODE == kRows ? at.expert * g.N : 0) + col) * (g.bias_f32 ? 4 : 2), g.bias_f32, cols);
    if constexpr (MODE == kRows) {
        if (at.real <= 0) {  // padding: zero, which every activation keeps
#pragma unroll
            for (int i = 0; i < 16; ++i) a.v[i] = 0;
        }
    }
    const int64_t e = at.row * g.N + col;
    if (g.z != nullptr) store_bf16(g.z + 2 * e, g.z, g.z_bytes, a, cols, stored, g.wide, g.status);
    activate(g, a.v);
    if (MODE == kDense && g.res != nullptr && stored)
        add_row(a, g.res + at.row * g.res_pitch + static_cast<int64_t>(col) * (g.res_f32 ? 4 : 2), g.res_f32, cols);
    if (g.y != nullptr) {
        if (g.y_f32) store_f32(g.y + 4 * e, g.y, g.y_bytes, a, cols, stored, g.wide, g.status);
        else store_bf16(g.y + 2 * e, g.y, g.y_bytes, a, cols, stored, g.wide, g.status);
    }
    if (g.fmt == kEncNone) return 0;
    const uint32_t scale = encode32(g, g.codes + (g.fmt == kEncMX8 ? e : e / 2), a, stored);
    return stored ? scale : 0u;
}
template <int MODE>
__device__ __forceinline__ void finish_row(const ProductArgs &g, const EpiTile &at, uint32_t (&v0)[32], const uint32_t (&v1)[32]) {
    uint32_t scales = 0;
    // A loop and not two copies: half the code, which a tile runs through once.
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        scales |= finish32<MODE>(g, at, 32 * h, v0) << (8 * h);
#pragma unroll
        for (int i = 0; i < 32; ++i) v0[i] = v1[i];
    }
    if (MODE != kDepth) put_scales(g, at, 0, scales);
}

// ---- N a multiple of 64: four lanes have 16 columns each of a row
// A store of 32 lanes on 32 rows touches 32 lines, one a clock and SM, which is what an
// epilogue of fp32 spends its time on.  So the B lines of a 64-line group are loaded in
// another order, such that the tensor memory's 16 x 256-bit load, which gives lane 4 r + c of a
// warp columns 8 i + 2 c + {0, 1} of rows r and r + 8, gives it 16 columns that follow one
// another: column 8 i + 2 c + b holds line line_of(8 i + 2 c + b) = 16 c + 2 i + b, and the
// scale writers gather the lines' scales in that order.  Four lanes then write a line together.
__device__ __forceinline__ uint32_t line_of(uint32_t p) { return 16u * ((p >> 1) & 3u) + 2u * (p >> 3) + (p & 1u); }

// Brings the bias of a warp's 64 columns into L1 while it waits for the tile (dense).
template <int MODE>
__device__ __forceinline__ void warm_bias(const ProductArgs &g, const EpiTile &at) {
    const int lane = threadIdx.x & 31, per = g.bias_f32 ? 4 : 8;  // columns of 16 bytes
    if (MODE == kDepth || g.bias == nullptr || per * lane >= kEpiCols || at.col >= g.N) return;
    asm volatile("{\n\t.reg .b32 a, b, c, d;\n\tld.global.v4.b32 {a, b, c, d}, [%0];\n\t}" ::"l"(
        g.bias + static_cast<int64_t>(at.col + per * lane) * (g.bias_f32 ? 4 : 2)));
}

// Adds 16 columns of a bf16 or fp32 row (16-byte aligned).
__device__ __forceinline__ void add16(uint64_t *v, const uint8_t *p, bool f32) {
    if (f32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const ulonglong2 s = *reinterpret_cast<const ulonglong2 *>(p + 16 * i);
            v[2 * i] = enc::add2(v[2 * i], s.x), v[2 * i + 1] = enc::add2(v[2 * i + 1], s.y);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 s = *reinterpret_cast<const uint4 *>(p + 16 * i);
        const uint32_t w[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[4 * i + k] = enc::add2(v[4 * i + k], enc::pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)));
    }
}
__device__ __forceinline__ void put16_bf16(uint8_t *p, const uint8_t *base, size_t bytes, const uint64_t *v, bool wide, int *status) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = bf16_pair(v[i]);
    if (!MX_STORE_OK(p, 32, base, bytes, status)) return;
    if (wide) {
        st_out32(p, w);
    } else {
        st_out16(p, w);
        st_out16(p + 16, w + 4);
    }
}
__device__ __forceinline__ void put16_f32(uint8_t *p, const uint8_t *base, size_t bytes, const uint64_t *v, bool wide, int *status) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float lo, hi;
            enc::unpack2(v[4 * i + k], lo, hi);
            w[2 * k] = __float_as_uint(lo), w[2 * k + 1] = __float_as_uint(hi);
        }
        if (!MX_STORE_OK(p + 32 * i, 32, base, bytes, status)) continue;
        if (wide) {
            st_out32(p + 32 * i, w);
        } else {
            st_out16(p + 32 * i, w);
            st_out16(p + 32 * i + 16, w + 4);
        }
    }
}
__device__ __forceinline__ void put16(uint8_t *y, int64_t e, size_t bytes, const uint64_t *v, bool f32, bool wide, int *status) {
    if (f32) put16_f32(y + 4 * e, y, bytes, v, wide, status);
    else put16_bf16(y + 2 * e, y, bytes, v, wide, status);
}

// Codes of the lane's 16 columns of a row, of which two lanes hold a block (whole warps); the
// block's scale byte is returned.
__device__ __forceinline__ uint32_t encode16(const ProductArgs &g, int64_t e, const uint64_t *v, bool stored) {
    float f[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) enc::unpack2(v[i], f[2 * i], f[2 * i + 1]);
    float top = enc::absmax2_nan(f[0], f[1]);
#pragma unroll
    for (int i = 1; i < 8; ++i) top = enc::absmax3_nan(top, f[2 * i], f[2 * i + 1]);
    top = enc::absmax2_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    float inv;
    const bool fp8 = g.fmt == kEncMX8;
    const uint32_t s = fp8 ? enc::scale_of_e4m3(top, inv) : enc::scale_of(top, inv);
    const uint64_t inv2 = act::same2(inv);
#pragma unroll
    for (int i = 0; i < 8; ++i) enc::unpack2(enc::mul2(v[i], inv2), f[2 * i], f[2 * i + 1]);
    const bool none = s == 0xFFu;
    if (fp8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = none ? 0u : enc::cvt_e4m3x4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        uint8_t *p = g.codes + e;
        if (stored && MX_STORE_OK(p, 16, g.codes, g.codes_bytes, g.status)) st_out16(p, w);
    } else {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = none ? 0u
                        : enc::cvt_e2m1x8(f[8 * i], f[8 * i + 1], f[8 * i + 2], f[8 * i + 3], f[8 * i + 4], f[8 * i + 5], f[8 * i + 6],
                                          f[8 * i + 7]);
        uint8_t *p = g.codes + e / 2;
        if (stored && MX_STORE_OK(p, 8, g.codes, g.codes_bytes, g.status)) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
    return stored ? s : 0u;
}

// The lane's 16 columns of rows `more` and `more + 8` below its own (dense and depth).
// Returns both rows' two scale bytes (in lane 0 of four), the first row's in the low half.
template <int MODE>
__device__ __forceinline__ uint32_t finish_two(const ProductArgs &g, const EpiTile &at, int more, const uint32_t (&acc)[32]) {
    static_assert(MODE == kDense || MODE == kDepth, "an expert's rows and their padding are finish_row's");
    const int col = at.col + 16 * static_cast<int>(threadIdx.x & 3);
    uint64_t v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = enc::pack2(__uint_as_float(acc[4 * i]), __uint_as_float(acc[4 * i + 1]));
        v[8 + i] = enc::pack2(__uint_as_float(acc[4 * i + 2]), __uint_as_float(acc[4 * i + 3]));
    }
    const bool first = more < at.left, second = more + 8 < at.left;
    const int64_t e0 = ((MODE == kDepth ? at.expert * g.M : 0) + at.row + more) * g.N + col, e1 = e0 + 8 * g.N;
    if constexpr (MODE == kDepth) {
        if (first) put16(g.y, e0, g.y_bytes, v, g.y_f32, g.wide, g.status);
        if (second) put16(g.y, e1, g.y_bytes, v + 8, g.y_f32, g.wide, g.status);
        return 0;
    }
    if (g.bias != nullptr) {
        const uint8_t *p = g.bias + static_cast<int64_t>(col) * (g.bias_f32 ? 4 : 2);
        add16(v, p, g.bias_f32);
        add16(v + 8, p, g.bias_f32);
    }
    if (g.z != nullptr) {
        if (first) put16_bf16(g.z + 2 * e0, g.z, g.z_bytes, v, g.wide, g.status);
        if (second) put16_bf16(g.z + 2 * e1, g.z, g.z_bytes, v + 8, g.wide, g.status);
    }
    activate(g, v);
    if (g.res != nullptr) {
        const uint8_t *p = g.res + (at.row + more) * g.res_pitch + static_cast<int64_t>(col) * (g.res_f32 ? 4 : 2);
        if (first) add16(v, p, g.res_f32);
        if (second) add16(v + 8, p + 8 * g.res_pitch, g.res_f32);
    }
    if (g.y != nullptr) {
        if (first) put16(g.y, e0, g.y_bytes, v, g.y_f32, g.wide, g.status);
        if (second) put16(g.y, e1, g.y_bytes, v + 8, g.y_f32, g.wide, g.status);
    }
    if (g.fmt == kEncNone) return 0;
    const uint32_t s = encode16(g, e0, v, first) | encode16(g, e1, v + 8, second) << 16;
    return s | __shfl_down_sync(0xFFFFFFFFu, s, 2) << 8;
}
template <int MODE>
__device__ __forceinline__ void finish_rows(const ProductArgs &g, const EpiTile &at, uint32_t (&v0)[32], const uint32_t (&v1)[32]) {
    const bool inside = at.col < g.N;  // else only padding of the scales
    uint32_t low = 0, high = 0;        // scales of rows 0 and 8, 16 and 24 from the lane's own
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        low = high;
        high = inside ? finish_two<MODE>(g, at, 16 * h, v0) : 0u;
#pragma unroll
        for (int i = 0; i < 32; ++i) v0[i] = v1[i];
    }
    if (MODE == kDepth || g.fmt == kEncNone) return;
    // Each of four lanes stores one of their four rows' halves of a word.
    const int lane = threadIdx.x & 31, c = lane & 3;
    low = __shfl_sync(0xFFFFFFFFu, low, lane & ~3);
    high = __shfl_sync(0xFFFFFFFFu, high, lane & ~3);
    put_scales(g, at, 8 * c, (c < 2 ? low : high) >> (16 * (c & 1)));
}

// Zeroes an output's bytes [0, until) and [from, bytes), 16 at a time: the n-th of `threads` threads.
__device__ __forceinline__ void zero_around(uint8_t *base, size_t until, size_t from, size_t bytes, size_t n, size_t threads, int *status) {
    if (base == nullptr) return;
    const uint32_t none[4] = {0, 0, 0, 0};
    for (size_t i = 16 * n; i < until; i += 16 * threads)
        if (MX_STORE_OK(base + i, 16, base, bytes, status)) st_out16(base + i, none);
    for (size_t i = from + 16 * n; i < bytes; i += 16 * threads)
        if (MX_STORE_OK(base + i, 16, base, bytes, status)) st_out16(base + i, none);
}

template <int FMT, int MODE, bool GATHER>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx_product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ ProductArgs g) {
    using E = Elem<FMT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sf_ring = smem + kStages * kStageBytes;
    SharedCtl *ctl = reinterpret_cast<SharedCtl *>(sf_ring + kSFRing * kSFSlotBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            // The even CTA's producer (arming the operand bytes) and the four
            // scale writers of each CTA.
            mbar_init(&ctl->full[s], 1 + 2 * 4);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int j = 0; j < kSFRing; ++j) {
            mbar_init(&ctl->sf_full[j], 1);
            mbar_init(&ctl->sf_free[j], 4);
        }
        mbar_init(&ctl->acc_full, 1);
        mbar_init(&ctl->acc_empty, 2 * kEpiWarps);
        mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int *abort = &ctl->abort_flag;
    griddep_wait();
    griddep_launch_dependents();
    int num_items = g.num_items;
    if constexpr (MODE == kRows) num_items = read_segments<MODE>(g, ctl, g.M);
    if constexpr (MODE == kDepth) num_items = read_segments<MODE>(g, ctl, static_cast<int64_t>(g.k_units) * 128);

    if (warp < kWriterWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow) : "memory");
        if ((warp == 0 || warp == 2) && lane == 0) {
            // ------------------------------------------------------------ producers
            // Warp 0 fills the operand ring, warp 2 the scale ring.
            const bool scales = warp == 2;
            const int ring = scales ? kSFRing : kStages;
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = pair; ok && t < num_items; t += npairs) {
                const Tile w = tile_of<MODE>(g, ctl, t);
                const int ns = stages_of<FMT>(w);
                for (int ks = 0; ks < ns; ++ks) {
                    if (!mbar_wait_inl(scales ? &ctl->sf_free[stage] : &ctl->empty[stage], phase ^ 1u, g.status, abort)) {
                        ok = false;
                        break;
                    }
                    const int u0 = ks * kKSub * E::kUnits;  // units of this stage: u0 ..
                    const int nu = w.units - u0 < kKSub * E::kUnits ? w.units - u0 : kKSub * E::kUnits;
                    if (scales) {
                        uint8_t *sfs = sf_ring + stage * kSFSlotBytes;
                        const uint32_t bytes = static_cast<uint32_t>(nu) * 512u;
                        const int64_t atom = w.unit0 + u0;
                        uint32_t all = 0;
                        const bool a = static_cast<int>(rank) < w.a_left;
                        if (a) all += bytes;
                        for (int rb = 0; rb < 2; ++rb)
                            if (rb < w.b_left) all += bytes;
                        mbar_arrive_expect_tx(&ctl->sf_full[stage], all);
                        if (a)
                            bulk_load(sfs, g.As + ((w.a_group + rank) * g.katoms + atom) * 512, bytes, &ctl->sf_full[stage]);
                        for (int rb = 0; rb < 2; ++rb)
                            if (rb < w.b_left)
                                bulk_load(sfs + kOffSFB + rb * kKSub * kSFSub, g.Bs + ((w.b_group + rb) * g.katoms + atom) * 512,
                                          bytes, &ctl->sf_full[stage]);
                    } else {
                        // Both CTAs' loads complete on the even CTA's barrier (boxes partly or
                        // wholly outside an operand count in full; the TMA fills zeros).
                        uint8_t *st = smem + stage * kStageBytes;
                        const int nsub = (nu + E::kUnits - 1) / E::kUnits;
                        if (rank == 0)
                            mbar_arrive_expect_tx(&ctl->full[stage], static_cast<uint32_t>(nsub) * 4u * kSubBytes);
                        const uint32_t full_even = mapa_shared(smem_u32(&ctl->full[stage]), 0u);
                        const int byte0 = (w.unit0 + u0) * static_cast<int>(E::kUnitBytes);
                        for (int u = 0; u < nsub; ++u) {
                            tma_load_2d_pair(st + u * kSubBytes, &map_a, full_even, byte0 + u * kBKBytes,
                                             w.a_row + kHalf * static_cast<int>(rank));
                            const int b_row = w.b_row + kHalf * static_cast<int>(rank);
                            if constexpr (GATHER)
                                tma_load_5d_pair(st + kOffB + u * kSubBytes, &map_b, full_even, byte0 + u * kBKBytes, 0, 0, 0, b_row >> 6);
                            else
                                tma_load_2d_pair(st + kOffB + u * kSubBytes, &map_b, full_even, byte0 + u * kBKBytes, b_row);
                        }
                    }
                    if (++stage == ring) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            // ------------------------------------------------------------ MMA issuer
            int stage = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            const uint32_t idesc0 = idesc_mxf4(2 * kHalf, kTile, 0, 0);
            const uint32_t idesc2 = idesc_mxf4(2 * kHalf, kTile, 2, 2);
            uint32_t idesc8[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) idesc8[j] = idesc_mxf8(2 * kHalf, kTile, j, j);
            for (int t = pair; ok && t < num_items; t += npairs) {
                const Tile w = tile_of<MODE>(g, ctl, t);
                const int ns = stages_of<FMT>(w);
                if (ns == 0) continue;
                if (!mbar_wait_inl(&ctl->acc_empty, acc_phase ^ 1u, g.status, abort)) break;
                tc_fence_after();
                for (int ks = 0; ks < ns; ++ks) {
                    if (!mbar_wait_inl(&ctl->full[stage], phase, g.status, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int left = w.units - ks * kKSub * E::kUnits;
                    const uint32_t sbase = smem_u32(smem + stage * kStageBytes);
                    const uint32_t slot = tmem + kSFCol + kSFSlot * static_cast<uint32_t>(stage);
                    // The issue of these leaves no slack: a full stage's eight go without a test in between.
                    const auto multiply = [&](int u, int j) {
                        const uint32_t sa = sbase + u * kSubBytes + 32u * j;
                        const uint32_t sb = sbase + kOffB + u * kSubBytes + 32u * j;
                        const uint32_t sf = slot + kSFCols * static_cast<uint32_t>(u);
                        const uint32_t acc = (ks > 0 || u > 0 || j > 0) ? 1u : 0u;
                        if constexpr (FMT == kFmtMX8) {
                            mma_mxf8_pair(tmem + kAccCol, sdesc_sw128(sa), sdesc_sw128(sb), idesc8[j], sf, sf + 8u, acc);
                        } else {
                            const uint32_t ka = static_cast<uint32_t>(j / 2);
                            mma_mxf4_pair(tmem + kAccCol, sdesc_sw128(sa), sdesc_sw128(sb), (j & 1) ? idesc2 : idesc0,
                                          sf + 4u * ka, sf + 8u + 8u * ka, acc);
                        }
                    };
                    if (left >= kKSub * E::kUnits) {
#pragma unroll
                        for (int u = 0; u < kKSub; ++u)
#pragma unroll
                            for (int j = 0; j < 4; ++j) multiply(u, j);
                    } else {
                        // An odd length ends in half an FP4 sub-tile: what follows in shared memory is
                        // zeros, or (depth) the next expert's.
#pragma unroll
                        for (int u = 0; u < kKSub; ++u)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (4 * u + j < 4 * left / E::kUnits) multiply(u, j);
                    }
                    tc_commit_pair(&ctl->empty[stage], 0x3);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                tc_commit_pair(&ctl->acc_full, 0x3);
                acc_phase ^= 1u;
            }
            // Every tensor-core operation issued here has finished before
            // either CTA releases its tensor memory.
            tc_commit_pair(&ctl->drain, 0x1);
            mbar_wait_inl(&ctl->drain, 0, g.status, nullptr, 100ull * 1000ull * 1000ull);
        }
    } else if (warp < kEpiWarp0) {
        // ------------------------------------------------------------ scale writers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow) : "memory");
        // The tensor-memory layout of a sub-tile's scales is described in mx_gemm.cu.
        const int q = warp & 3;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
        // GATHER: where the four B lines of this lane lie in an atom (line_of's order).
        uint32_t b_at[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t n = 64u * (k >> 1) + line_of(32u * (k & 1) + lane);
            b_at[k] = (n & 31u) * 16u + (n >> 5) * 4u;
        }
        int stage = 0, sj = 0;
        uint32_t phase = 0, sphase = 0;
        for (int t = pair; t < num_items; t += npairs) {
            const Tile w = tile_of<MODE>(g, ctl, t);
            const int ns = stages_of<FMT>(w);
            bool ok = true;
            for (int ks = 0; ks < ns; ++ks) {
                int okw = 1;
                if (lane == 0) {
                    okw = mbar_wait_inl(&ctl->sf_full[sj], sphase, g.status, abort) ? 1 : 0;
                    if (okw) okw = mbar_wait_inl(&ctl->empty[stage], phase ^ 1u, g.status, abort) ? 1 : 0;
                }
                okw = __shfl_sync(0xFFFFFFFFu, okw, 0);
                if (!okw) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int left = w.units - ks * kKSub * E::kUnits;
                const uint8_t *sfs = sf_ring + sj * kSFSlotBytes;
                const uint32_t slot = lane_base + kSFCol + kSFSlot * static_cast<uint32_t>(stage);
                for (int u = 0; u < kKSub && u * E::kUnits < left; ++u) {
                    const uint8_t *sfa = sfs + u * E::kAtoms * 512;
                    const uint8_t *sfb = sfs + kOffSFB + u * E::kAtoms * 512;
                    const uint32_t col = slot + kSFCols * static_cast<uint32_t>(u);
                    uint32_t a[4 * E::kAtoms], b[8 * E::kAtoms];
#pragma unroll
                    for (int ka = 0; ka < E::kAtoms; ++ka) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(sfa + ka * 512 + lane * 16);
                        a[4 * ka + 0] = v.x, a[4 * ka + 1] = v.y, a[4 * ka + 2] = v.z, a[4 * ka + 3] = v.w;
#pragma unroll
                        for (int rb = 0; rb < 2; ++rb) {
                            const uint8_t *from = sfb + rb * kKSub * kSFSub + ka * 512;
                            if constexpr (GATHER) {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    b[8 * ka + 4 * rb + k] = *reinterpret_cast<const uint32_t *>(from + b_at[k]);
                            } else {
                                const uint4 s = *reinterpret_cast<const uint4 *>(from + lane * 16);
                                b[8 * ka + 4 * rb + 0] = s.x, b[8 * ka + 4 * rb + 1] = s.y;
                                b[8 * ka + 4 * rb + 2] = s.z, b[8 * ka + 4 * rb + 3] = s.w;
                            }
                        }
                    }
                    if constexpr (FMT == kFmtMX8) {
                        tmem_st_32x32b_x4(col, a);
                        tmem_st_32x32b_x8(col + 8u, b);
                    } else {
                        tmem_st_32x32b_x8(col, a);
                        tmem_st_32x32b_x16(col + 8u, b);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ctl->sf_free[sj]);
                    arrive_even(&ctl->full[stage]);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++sj == kSFRing) {
                    sj = 0;
                    sphase ^= 1u;
                }
            }
            if (!ok) break;
        }
    } else {
        // ------------------------------------------------------------ epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh) : "memory");
        const int q = warp & 3;                   // tensor-memory lane quarter this warp may access
        const int part = (warp - kEpiWarp0) / 4;  // column quarter of the 256-wide tile
        const uint32_t tbase = tmem + (static_cast<uint32_t>(32 * q) << 16) + kAccCol + kEpiCols * static_cast<uint32_t>(part);
        uint32_t acc_phase = 0;
        for (int t = pair; t < num_items; t += npairs) {
            const Tile w = tile_of<MODE>(g, ctl, t);
            const bool empty = stages_of<FMT>(w) == 0;
            EpiTile at;
            const int r = kHalf * static_cast<int>(rank) + 32 * q + (GATHER ? lane >> 2 : lane);
            at.row = w.row + r;
            at.expert = w.expert;
            at.col = w.col + kEpiCols * part;
            at.left = w.m_left - r;
            at.scaled = ((w.m_left + 127) & ~127) - r;
            at.real = at.left;
            if constexpr (MODE == kRows) at.real = min(at.left, g.counts[w.expert] - (at.row - ctl->start[w.expert] * 128));
            if constexpr (GATHER) warm_bias<MODE>(g, at);
            uint32_t v0[32], v1[32];
            if (!empty) {
                // One lane waits; its result is broadcast so the warp stays
                // converged for the .sync.aligned tensor-memory loads.
                int ok = 1;
                if (lane == 0) ok = mbar_wait_inl(&ctl->acc_full, acc_phase, g.status, abort) ? 1 : 0;
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                if (!ok) break;
                tc_fence_after();
                acc_phase ^= 1u;
                if constexpr (GATHER) {
                    tmem_ld_16x256b_x8(tbase, v0);
                    tmem_ld_16x256b_x8(tbase + (16u << 16), v1);
                } else {
                    tmem_ld_32x32b_x32(tbase, v0);
                    tmem_ld_32x32b_x32(tbase + 32u, v1);
                }
                tmem_ld_wait();
                // The accumulator is in registers: the next tile may start.
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_even(&ctl->acc_empty);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v0[i] = v1[i] = 0;
            }
            if constexpr (GATHER) finish_rows<MODE>(g, at, v0, v1);
            else finish_row<MODE>(g, at, v0, v1);
        }
        if constexpr (MODE == kRows) {
            // Rows before the first segment and behind the last are zero.
            const size_t first = static_cast<size_t>(ctl->start[0]), last = static_cast<size_t>(ctl->start[g.experts]);
            const size_t n = static_cast<size_t>(blockIdx.x) * 32 * kEpiWarps + threadIdx.x - 32 * kEpiWarp0,
                         all = static_cast<size_t>(gridDim.x) * 32 * kEpiWarps;
            const size_t N = static_cast<size_t>(g.N);
            const auto zero = [&](uint8_t *base, size_t group_bytes, size_t bytes) {  // of 128 rows
                zero_around(base, first * group_bytes, last * group_bytes, bytes, n, all, g.status);
            };
            zero(g.y, 128 * N * (g.y_f32 ? 4 : 2), g.y_bytes);
            zero(g.z, 128 * N * 2, g.z_bytes);
            zero(g.codes, g.fmt == kEncMX8 ? 128 * N : 64 * N, g.codes_bytes);
            zero(g.scales, static_cast<size_t>(g.out_katoms) * 512, g.scales_bytes);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // Neither CTA of the pair releases tensor memory (or leaves) while the
    // other's operations may still touch it.
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// Co-resident 2-CTA clusters of a kernel variant on a device, measured once.
template <int FMT, int MODE, bool GATHER>
int product_clusters(const DeviceInfo &dev) {
    static std::atomic<int> cache[64];
    const int idx = dev.ordinal >= 0 && dev.ordinal < 64 ? dev.ordinal : 0;
    int n = cache[idx].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaFuncSetAttribute(mx_product_kernel<FMT, MODE, GATHER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmem)) != cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    if (cudaOccupancyMaxActiveClusters(&n, mx_product_kernel<FMT, MODE, GATHER>, &cfg) != cudaSuccess || n < 1) return 0;
    cache[idx].store(n, std::memory_order_relaxed);
    return n;
}

template <int FMT, int MODE, bool GATHER>
cudaError_t launch_variant(const CUtensorMap &map_a, const CUtensorMap &map_b, const ProductArgs &g, int64_t most_items,
                           const DeviceInfo &dev, cudaStream_t stream) {
    const int pairs_max = product_clusters<FMT, MODE, GATHER>(dev);
    if (pairs_max < 1) return cudaErrorLaunchOutOfResources;
    int64_t pairs = std::min<int64_t>(most_items, pairs_max);
    // As many rounds of tiles as all pairs need, spread evenly over fewer pairs (where the
    // tiles are of one length and their number is known here).
    if (MODE == kDense) {
        const int64_t rounds = (most_items + pairs - 1) / pairs;
        pairs = (most_items + rounds - 1) / rounds;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, mx_product_kernel<FMT, MODE, GATHER>, map_a, map_b, g);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int MODE, bool GATHER>
cudaError_t launch_mode(bool fp8, const CUtensorMap &map_a, const CUtensorMap &map_b, const ProductArgs &g, int64_t most_items,
                        const DeviceInfo &dev, cudaStream_t stream) {
    return fp8 ? launch_variant<kFmtMX8, MODE, GATHER>(map_a, map_b, g, most_items, dev, stream)
               : launch_variant<kFmtMX4, MODE, GATHER>(map_a, map_b, g, most_items, dev, stream);
}
}  // namespace

cudaError_t launch_product(const Product &p, const DeviceInfo &dev, cudaStream_t stream) {
    const bool rows = p.mode == kProductRows, depth = p.mode == kProductDepth;
    const int64_t row_bytes = p.fp8 ? p.K : p.K / 2;
    // Four lanes a row (GATHER) where lines are what the epilogue waits for: a residual is read
    // (8192 x 14336 x 4096: 167 us, 230 without), and the experts' Wgrad, whose outputs are many
    // for the length of its products (8 experts of 14336 x 4096 over 16384 rows, fp32: 453 us, 543
    // without).  Elsewhere a lane's own row is no slower (bf16 148 us, 151 to 156) or faster
    // (z, y and codes with gelu 210 us, 242).  Whole groups of 64 lines alone can be loaded in
    // that order: a partial one could not be kept inside its buffer.
    const bool gather = p.N % 64 == 0 && (depth || p.res.p != nullptr);
    CUtensorMap map_a, map_b;
    std::memset(&map_a, 0, sizeof(map_a));
    std::memset(&map_b, 0, sizeof(map_b));
    if (p.K > 0) {  // without a contraction nothing is loaded
        const int64_t b_lines = rows ? p.N * p.experts : p.N;
        if (!encode_tmap_2d(&map_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.Aq, row_bytes, p.M, row_bytes, kBKBytes, kHalf,
                            CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
        if (gather ? !encode_tmap_lines64(&map_b, p.Bq, row_bytes, b_lines, kBKBytes, kHalf, CU_TENSOR_MAP_SWIZZLE_128B)
                   : !encode_tmap_2d(&map_b, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.Bq, row_bytes, b_lines, row_bytes, kBKBytes, kHalf,
                                     CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    ProductArgs g{};
    g.As = static_cast<const uint8_t *>(p.As);
    g.Bs = static_cast<const uint8_t *>(p.Bs);
    g.M = p.M;
    g.N = p.N;
    g.katoms = scale_katoms(p.K);
    g.a_groups = scale_groups(p.M);
    g.b_groups = scale_groups(p.N);
    g.k_units = static_cast<int>((p.K + 127) / 128);
    const int64_t m_tiles = (p.M + kTile - 1) / kTile, n_tiles = (p.N + kTile - 1) / kTile;
    const int64_t experts = std::max<int64_t>(1, p.experts);
    // Tile rows of all segments: each may end in half a tile.
    const int64_t tiles = rows ? (m_tiles + experts) * n_tiles : depth ? experts * m_tiles * n_tiles : m_tiles * n_tiles;
    if (tiles > 0x3FFFFFFF || (rows && m_tiles + experts > 0xFFFF)) return cudaErrorNotSupported;
    g.m_tiles = static_cast<int>(m_tiles);
    g.n_tiles = static_cast<int>(n_tiles);
    g.num_items = static_cast<int>(tiles);
    g.by_n = divisor(n_tiles);
    g.by_band = divisor(kBand * n_tiles);
    g.by_last = divisor((m_tiles - 1) % kBand + 1);
    g.by_expert = divisor(m_tiles * n_tiles);
    g.experts = static_cast<int>(p.experts);
    g.offsets = p.offsets;
    g.counts = p.counts;
    const size_t out = static_cast<size_t>(p.M) * static_cast<size_t>(p.N) * (depth ? static_cast<size_t>(experts) : 1u);
    g.bias = static_cast<const uint8_t *>(p.bias);
    g.bias_f32 = p.bias_f32;
    g.res = static_cast<const uint8_t *>(p.res.p);
    g.res_f32 = p.res.f32;
    g.res_pitch = p.res.pitch * (p.res.f32 ? 4 : 2);
    g.y = static_cast<uint8_t *>(p.y);
    g.y_f32 = p.y_f32;
    g.y_bytes = out * (p.y_f32 ? 4 : 2);
    g.z = static_cast<uint8_t *>(p.z);
    g.z_bytes = out * 2;
    g.fmt = p.enc.fmt;
    g.codes = static_cast<uint8_t *>(p.enc.codes);
    g.scales = static_cast<uint8_t *>(p.enc.scales);
    g.codes_bytes = p.enc.fmt == kEncMX8 ? out : out / 2;
    g.out_katoms = scale_katoms(p.N);
    g.scales_bytes = static_cast<size_t>(scale_groups(p.M)) * static_cast<size_t>(g.out_katoms) * 512;
    g.act = p.act;
    const uintptr_t ends = reinterpret_cast<uintptr_t>(p.y) | reinterpret_cast<uintptr_t>(p.z);
    g.wide = (ends & 31) == 0 && p.N % 16 == 0;
    g.wide_codes = (reinterpret_cast<uintptr_t>(p.enc.codes) & 31) == 0;
    g.status = dev.status;
    if (depth)
        return gather ? launch_mode<kDepth, true>(p.fp8, map_a, map_b, g, tiles, dev, stream)
                      : launch_mode<kDepth, false>(p.fp8, map_a, map_b, g, tiles, dev, stream);
    if (rows) return launch_mode<kRows, false>(p.fp8, map_a, map_b, g, tiles, dev, stream);
    return gather ? launch_mode<kDense, true>(p.fp8, map_a, map_b, g, tiles, dev, stream)
                  : launch_mode<kDense, false>(p.fp8, map_a, map_b, g, tiles, dev, stream);
}

}  // namespace mx
