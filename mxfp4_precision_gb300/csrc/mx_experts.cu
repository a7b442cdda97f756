// mx_experts.cu -- the rows' way to their experts and back (mx_expert_plan,
// mx_expert_dispatch, mx_expert_combine, mx_expert_combine_backward).
//
//   plan       entry i = token * picks + choice names an expert; the entries of each
//              expert, in their order, take the rows of its segment, and every
//              segment begins at a multiple of 128 rows
//   dispatch   rows[slot] = x[token], in bf16 and / or encoded; other rows zero
//   combine    y[token] = residual[token] + sum over choices of weight * rows[slot]
//   its gradient: drows[slot] = weight * dy[token],  dweight = <dy[token], rows[slot]>
//
// Slots that lie outside the rows stand for dropped choices.
//
// Measured, 8192 tokens of 4096 columns to 4 of 64 experts (32768 rows and 8064 without a token, bf16): plan
// 9 us (two launches), rows in with bf16 and MXFP8 90 us = 6.4 TB/s, rows out 64 us = 6.3 TB/s, their gradient with
// the weights' 120 us = 5.6 TB/s (128 registers leave two blocks an SM; two rows at a time with three blocks 122,
// and 135 with four).
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mx.h"
#include "mx_internal.h"
#include "mx_ptx.cuh"
#include "mx_rows.cuh"

namespace mx {
namespace {

using namespace rows;

// ---------------------------------------------------------------- plan
// A stable counting sort.  A block takes one chunk of entries, its 16 warps
// equal parts of it in order; a warp ranks 32 entries at a time among those of the
// same expert (match_any).  A first launch counts each chunk's entries by expert (not
// needed for one chunk); in the second every block adds the chunks before its
// own, and the segments' starts follow from the totals in the block itself.
constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kChunk = 2048;     // entries of a block, at least
constexpr int kMaxChunks = 128;  // more entries: larger chunks
static_assert(MX_EXPERTS_MAX <= kPlanThreads, "one thread per expert");

struct PlanArgs {
    const void *index;
    int64_t n, rows;
    int experts, chunks;
    int64_t chunk;           // a multiple of kChunk
    int32_t *offsets, *counts, *slot, *source;
    uint32_t *chunk_counts;  // [chunks][experts]
    int *status;
};

// Expert of entry i; -1 for none (past the end, or no expert).
template <typename I>
__device__ __forceinline__ int expert_of(const PlanArgs &p, int64_t i) {
    if (i >= p.n) return -1;
    const I e = static_cast<const I *>(p.index)[i];
    return e >= 0 && e < static_cast<I>(p.experts) ? static_cast<int>(e) : -1;
}

template <typename I>
__global__ void __launch_bounds__(kPlanThreads) mx_expert_count_kernel(const __grid_constant__ PlanArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ uint32_t count[MX_EXPERTS_MAX];
    for (int e = threadIdx.x; e < p.experts; e += kPlanThreads) count[e] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * p.chunk;
    for (int64_t i = threadIdx.x; i < p.chunk; i += kPlanThreads) {
        const int e = expert_of<I>(p, first + i);
        if (e >= 0) atomicAdd(&count[e], 1u);  // whole numbers: any order gives the same
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kPlanThreads)
        p.chunk_counts[static_cast<int64_t>(blockIdx.x) * p.experts + e] = count[e];
}

// A warp's entries, kGroups times 32 at a time so that their loads are in flight together.
constexpr int kGroups = 4;
template <typename I>
struct Entries {
    int x[kGroups];
    __device__ __forceinline__ Entries(const PlanArgs &p, int64_t first) {
#pragma unroll
        for (int k = 0; k < kGroups; ++k) x[k] = expert_of<I>(p, first + 32 * k + (threadIdx.x & 31));
    }
};

template <typename I>
__global__ void __launch_bounds__(kPlanThreads) mx_expert_plan_kernel(const __grid_constant__ PlanArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ uint32_t at[kPlanWarps][MX_EXPERTS_MAX];  // counts, then next rows
    __shared__ uint32_t part[kPlanWarps];
    __shared__ uint32_t begin[MX_EXPERTS_MAX], full[MX_EXPERTS_MAX];  // first row of the padding, first row behind it
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = threadIdx.x;
    const int64_t each = p.chunk / kPlanWarps;  // a multiple of 32 * kGroups
    const int64_t first = blockIdx.x * p.chunk + warp * each;
    const Entries<I> head(p, first);
    for (int i = lane; i < p.experts; i += 32) at[warp][i] = 0;
    __syncwarp();
    for (int64_t i = 0; i < each; i += 32 * kGroups) {
        const Entries<I> now = i == 0 ? head : Entries<I>(p, first + i);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int x = now.x[k];
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, x);
            if (x >= 0 && lane == __ffs(same) - 1) at[warp][x] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // Entries of expert e in the chunks before this one, and in all.
    uint32_t before = 0, total = 0;
    if (e < p.experts) {
        if (p.chunks == 1) {
#pragma unroll
            for (int w = 0; w < kPlanWarps; ++w) total += at[w][e];
        } else {
#pragma unroll 8
            for (int c = 0; c < p.chunks; ++c) {
                const uint32_t v = p.chunk_counts[static_cast<int64_t>(c) * p.experts + e];
                total += v;
                if (c < static_cast<int>(blockIdx.x)) before += v;
            }
        }
    }
    // Segments' starts: a running sum of the totals, each rounded up to 128.
    const uint32_t size = (total + 127u) & ~127u;
    uint32_t sum = size;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) part[warp] = sum;
    __syncthreads();
    uint32_t start = sum - size, used = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) start += part[w];
        used += part[w];
    }
    if (e < p.experts) {
        if (blockIdx.x == 0) {
            p.offsets[e] = static_cast<int32_t>(start);
            p.counts[e] = static_cast<int32_t>(total);
        }
        begin[e] = start + total;
        full[e] = start + size;
        uint32_t next = start + before;
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            const uint32_t v = at[w][e];
            at[w][e] = next;
            next += v;
        }
    }
    if (threadIdx.x == 0 && blockIdx.x == 0) p.offsets[p.experts] = static_cast<int32_t>(used);
    __syncthreads();
    for (int64_t i = 0; i < each; i += 32 * kGroups) {
        const Entries<I> now = i == 0 ? head : Entries<I>(p, first + i);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int x = now.x[k];
            const int64_t entry = first + i + 32 * k + lane;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, x);
            int32_t row = -1;
            if (x >= 0) row = static_cast<int32_t>(at[warp][x] + __popc(same & ((1u << lane) - 1u)));
            __syncwarp();
            if (x >= 0 && lane == __ffs(same) - 1) at[warp][x] += __popc(same);
            __syncwarp();
            if (entry < p.n) {
                p.slot[entry] = row;
                if (row >= 0 && row < p.rows) p.source[row] = static_cast<int32_t>(entry);
            }
        }
    }
    // Padding rows (a warp takes an expert's), and the rows behind the last segment.
    for (int i = blockIdx.x * kPlanWarps + warp; i < p.experts; i += gridDim.x * kPlanWarps)
        for (uint32_t r = begin[i] + lane; r < full[i] && r < p.rows; r += 32) p.source[r] = -1;
    for (int64_t r = used + static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x; r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * kPlanThreads)
        p.source[r] = -1;
}

// ---------------------------------------------------------------- rows in
// A warp takes one token's strip of 512 columns, a lane 16 of them (two lanes a block), reads it
// once, encodes it once and stores it to each of the token's rows; bound by memory.
// Blocks before those of the tokens zero the rows without a token.
constexpr int kWarps = 8;
constexpr int kZeroRows = 8;  // rows a warp looks through for padding
constexpr int kStrip = 512;

struct RowsArgs {
    const uint8_t *x, *rows, *res;
    int64_t x_pitch, rows_pitch, res_pitch;  // bytes
    const int32_t *slot, *source;
    const float *weights;
    Out y, dweights;
    Encoded enc;
    int64_t T, P;
    uint32_t K;
    int picks, strips;
    uint32_t zeros;  // blocks that look for rows without a token
    bool aligned32, aligned_out;
    int *status;
};

__device__ __forceinline__ bool there(const RowsArgs &p, int32_t slot) {
    return static_cast<uint32_t>(slot) < static_cast<uint64_t>(p.P);
}

// The lane's 16 columns: those from 8 col on, and whether each eight are inside the row.
struct Lane16 {
    uint32_t col;
    bool in0, in1;
};
__device__ __forceinline__ Lane16 lane16(const RowsArgs &p, uint32_t strip) {
    const uint32_t col = strip * kStrip + 16 * (threadIdx.x & 31);
    return {col, col < p.K, col + 8 < p.K};
}
template <typename X>
__device__ __forceinline__ void load(Raw8<X> (&r)[2], const uint8_t *row, const Lane16 &at, bool aligned32) {
    zero8(r[0]);
    zero8(r[1]);
    if (at.in0) load8(r[0], row + static_cast<size_t>(at.col) * X::kBytes, aligned32);
    if (at.in1) load8(r[1], row + static_cast<size_t>(at.col + 8) * X::kBytes, aligned32);
}

// The lane's 16 columns of an output row, kept to be stored to several rows: bf16, codes, scale byte.
struct Packed16 {
    uint32_t y[8], w[4], scale;
};
__device__ __forceinline__ void pack(Packed16 &q, const RowsArgs &p, const V8 &a, const V8 &b) {
    Raw8<BF16> r;
    from_v8(r, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) q.y[i] = r.w[i];
    from_v8(r, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) q.y[4 + i] = r.w[i];
    if (p.enc.fmt == kEncNone) return;
    float f[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(a.v[i], f[2 * i], f[2 * i + 1]), unpack2(b.v[i], f[8 + 2 * i], f[9 + 2 * i]);
    float m = enc::absmax2_nan(f[0], f[1]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = enc::absmax3_nan(m, f[2 * i], f[2 * i + 1]);
    m = enc::absmax2_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    float inv;
    q.scale = p.enc.fmt == kEncMX8 ? enc::scale_of_e4m3(m, inv) : enc::scale_of(m, inv);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] *= inv;
    if (p.enc.fmt == kEncMX8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q.w[i] = enc::cvt_e4m3x4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            q.w[i] = enc::cvt_e2m1x8(f[8 * i], f[8 * i + 1], f[8 * i + 2], f[8 * i + 3], f[8 * i + 4], f[8 * i + 5], f[8 * i + 6], f[8 * i + 7]);
    }
    if (q.scale == 0xFFu) q.w[0] = q.w[1] = q.w[2] = q.w[3] = 0;
}
__device__ __forceinline__ void put(const RowsArgs &p, int64_t row, const Lane16 &at, const Packed16 &q) {
    if (p.y.p != nullptr) {
        uint8_t *d = p.y.p + (row * p.K + at.col) * 2;
        if (at.in1 && p.aligned_out) {
            if (MX_STORE_OK(d, 32, p.y.p, p.y.bytes, p.status))
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(d), "r"(q.y[0]), "r"(q.y[1]), "r"(q.y[2]),
                             "r"(q.y[3]), "r"(q.y[4]), "r"(q.y[5]), "r"(q.y[6]), "r"(q.y[7])
                             : "memory");
        } else {
            if (at.in0 && MX_STORE_OK(d, 16, p.y.p, p.y.bytes, p.status))
                reinterpret_cast<uint4 *>(d)[0] = make_uint4(q.y[0], q.y[1], q.y[2], q.y[3]);
            if (at.in1 && MX_STORE_OK(d + 16, 16, p.y.p, p.y.bytes, p.status))
                reinterpret_cast<uint4 *>(d)[1] = make_uint4(q.y[4], q.y[5], q.y[6], q.y[7]);
        }
    }
    if (p.enc.fmt == kEncNone) return;
    // Encoded rows are whole blocks: both eights are inside or neither.
    const EncodedRow to = encoded_row(p.enc, row);
    if (at.in1) {
        if (p.enc.fmt == kEncMX8) {
            uint8_t *d = to.codes + at.col;
            if (MX_STORE_OK(d, 16, p.enc.codes.p, p.enc.codes.bytes, p.status))
                *reinterpret_cast<uint4 *>(d) = make_uint4(q.w[0], q.w[1], q.w[2], q.w[3]);
        } else {
            uint8_t *d = to.codes + at.col / 2;
            if (MX_STORE_OK(d, 8, p.enc.codes.p, p.enc.codes.bytes, p.status)) *reinterpret_cast<uint2 *>(d) = make_uint2(q.w[0], q.w[1]);
        }
    }
    const uint32_t block = at.col >> 5;
    if ((threadIdx.x & 1) == 0 && block < 4 * static_cast<uint32_t>(p.enc.katoms)) {
        uint8_t *d = to.scales + (block >> 2) * 512u + (block & 3u);
        if (MX_STORE_OK(d, 1, p.enc.scales.p, p.enc.scales.bytes, p.status)) *d = static_cast<uint8_t>(at.in0 ? q.scale : 0u);
    }
}

// Zeroes the rows without a token: the n-th warp looks through kZeroRows of them.
__device__ __forceinline__ void zero_rows(const RowsArgs &p, int64_t n) {
    const int lane = threadIdx.x & 31;
    const int64_t first = n * kZeroRows;
    const bool free_row = lane < kZeroRows && first + lane < p.P && p.source[first + lane] < 0;
    const Packed16 none{};
    for (uint32_t mask = __ballot_sync(0xFFFFFFFFu, free_row); mask != 0; mask &= mask - 1) {
        const int64_t row = first + __ffs(mask) - 1;
        for (int s = 0; s < p.strips; ++s) put(p, row, lane16(p, s), none);
    }
}

template <typename X>
__global__ void __launch_bounds__(32 * kWarps) mx_expert_dispatch_kernel(const __grid_constant__ RowsArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5;
    if (blockIdx.x < p.zeros) {
        zero_rows(p, static_cast<int64_t>(blockIdx.x) * kWarps + warp);
        return;
    }
    const int64_t unit = static_cast<int64_t>(blockIdx.x - p.zeros) * kWarps + warp;
    const int64_t t = unit / p.strips;
    if (t >= p.T) return;
    const Lane16 at = lane16(p, static_cast<uint32_t>(unit - t * p.strips));
    Raw8<X> r[2];
    load(r, p.x + t * p.x_pitch, at, p.aligned32);
    // The first four rows' numbers are on their way beside the columns.
    int32_t s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = j < p.picks ? p.slot[t * p.picks + j] : -1;
    Packed16 q;
    pack(q, p, to_v8(r[0]), to_v8(r[1]));
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (there(p, s[j])) put(p, s[j], at, q);
    for (int j = 4; j < p.picks; ++j) {
        const int32_t row = p.slot[t * p.picks + j];
        if (there(p, row)) put(p, row, at, q);
    }
}

// ---------------------------------------------------------------- rows out
// A warp takes one token's strip of 256 columns and adds up to four of its rows at
// a time, all in flight; bound by memory.
constexpr int kOutStrip = 256;
template <typename R, typename S, typename Y>
__global__ void __launch_bounds__(32 * kWarps) mx_expert_combine_kernel(const __grid_constant__ RowsArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int64_t t = unit / p.strips;
    if (t >= p.T) return;
    const uint32_t col = 8 * (static_cast<uint32_t>(unit - t * p.strips) * 32 + lane);
    if (col >= p.K) return;
    V8 sum = zero_v8();
    if (p.res != nullptr) {
        Raw8<S> r;
        load8(r, p.res + t * p.res_pitch + static_cast<size_t>(col) * S::kBytes, p.aligned32);
        sum = to_v8(r);
    }
    constexpr int kAhead = 4;
    for (int j0 = 0; j0 < p.picks; j0 += kAhead) {
        Raw8<R> r[kAhead];
        float w[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            zero8(r[k]);
            w[k] = 0.0f;
            if (j0 + k >= p.picks) continue;
            const int64_t i = t * p.picks + j0 + k;
            const int32_t s = p.slot[i];
            if (!there(p, s)) continue;
            w[k] = p.weights != nullptr ? p.weights[i] : 1.0f;
            load8(r[k], p.rows + s * p.rows_pitch + static_cast<size_t>(col) * R::kBytes, p.aligned32);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const V8 a = to_v8(r[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum.v[i] = fma2(a.v[i], same2(w[k]), sum.v[i]);
        }
    }
    store8<Y>(p.y, p.y.p + (t * p.K + col) * Y::kBytes, sum, p.aligned_out, p.status);
}

// ---------------------------------------------------------------- gradient of rows out
// A block takes one token, a warp a strip of 512 columns at a time: dy and up to four of the
// token's rows (two of fp32, which fill the registers) are read together, the rows' gradients leave as they are made, and the products with
// the rows are added up over the block in a fixed order.  Blocks before those of the tokens
// zero the rows without a token.
template <typename D, typename R>
__global__ void __launch_bounds__(32 * kWarps, 2) mx_expert_combine_backward_kernel(const __grid_constant__ RowsArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (blockIdx.x < p.zeros) {
        zero_rows(p, static_cast<int64_t>(blockIdx.x) * warps + warp);
        return;
    }
    constexpr int kAtOnce = R::kBytes == 4 ? 2 : 4;
    __shared__ float part[kWarps][kAtOnce];
    const int64_t t = blockIdx.x - p.zeros;
    const uint8_t *dy = p.x + t * p.x_pitch;
    const bool writes = p.y.p != nullptr || p.enc.fmt != kEncNone, dots = p.dweights.p != nullptr;
    for (int j0 = 0; j0 < p.picks; j0 += kAtOnce) {
        int32_t s[kAtOnce];
        float w[kAtOnce];
        uint64_t dot[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int64_t i = t * p.picks + j0 + k;
            const bool has = j0 + k < p.picks;
            s[k] = has ? p.slot[i] : -1;
            w[k] = has ? p.weights[i] : 0.0f;
            if (!there(p, s[k])) s[k] = -1;
            dot[k] = 0;
        }
        for (int strip = warp; strip < p.strips; strip += warps) {
            const Lane16 at = lane16(p, strip);
            Raw8<D> dr[2];
            load(dr, dy, at, p.aligned32);
            Raw8<R> r[kAtOnce][2];
            if (dots) {
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    zero8(r[k][0]);
                    zero8(r[k][1]);
                    if (s[k] >= 0) load(r[k], p.rows + s[k] * p.rows_pitch, at, p.aligned32);
                }
            }
            const V8 d0 = to_v8(dr[0]), d1 = to_v8(dr[1]);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (s[k] < 0) continue;
                if (dots) {
                    const V8 a = to_v8(r[k][0]), b = to_v8(r[k][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dot[k] = fma2(b.v[i], d1.v[i], fma2(a.v[i], d0.v[i], dot[k]));
                }
                if (!writes) continue;
                V8 a, b;
#pragma unroll
                for (int i = 0; i < 4; ++i) a.v[i] = mul2(d0.v[i], same2(w[k])), b.v[i] = mul2(d1.v[i], same2(w[k]));
                Packed16 q;
                pack(q, p, a, b);
                put(p, s[k], at, q);
            }
        }
        if (!dots) continue;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const float v = sum_lanes(sum2(dot[k]));
            if (lane == 0) part[warp][k] = v;
        }
        __syncthreads();
        if (threadIdx.x < kAtOnce && j0 + static_cast<int>(threadIdx.x) < p.picks) {
            float v = 0.0f;
            for (int i = 0; i < warps; ++i) v += part[i][threadIdx.x];
            uint8_t *o = p.dweights.p + (t * p.picks + j0 + threadIdx.x) * 4;
            if (MX_STORE_OK(o, 4, p.dweights.p, p.dweights.bytes, p.status)) *reinterpret_cast<float *>(o) = v;
        }
        __syncthreads();
    }
}

RowsArgs rows_args(const ExpertRows &r, const DeviceInfo &dev) {
    RowsArgs p{};
    p.slot = r.slot;
    p.source = r.source;
    p.T = r.T;
    p.P = r.rows;
    p.K = static_cast<uint32_t>(r.K);
    p.picks = static_cast<int>(r.picks);
    p.strips = static_cast<int>((r.K + kStrip - 1) / kStrip);
    p.status = dev.status;
    return p;
}
int64_t zero_blocks(const RowsArgs &p, int warps) {
    return (p.P + kZeroRows * warps - 1) / (kZeroRows * warps);
}

template <typename I>
cudaError_t launch_plan(const PlanArgs &p, cudaStream_t stream) {
    if (p.chunks > 1) {
        const cudaError_t e = launch_dependent(mx_expert_count_kernel<I>, p.chunks, kPlanThreads, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(mx_expert_plan_kernel<I>, p.chunks, kPlanThreads, 0, stream, p);
}

int64_t chunk_entries(int64_t n) {
    const int64_t most = (n + kMaxChunks - 1) / kMaxChunks;
    return (std::max<int64_t>(1, most) + kChunk - 1) / kChunk * kChunk;
}

template <typename R, typename S>
cudaError_t launch_combine(const RowsArgs &p, bool y_f32, int64_t grid, cudaStream_t stream) {
    return y_f32 ? launch_dependent(mx_expert_combine_kernel<R, S, F32>, grid, 32 * kWarps, 0, stream, p)
                 : launch_dependent(mx_expert_combine_kernel<R, S, BF16>, grid, 32 * kWarps, 0, stream, p);
}

}  // namespace

size_t expert_plan_ws(int64_t n, int64_t experts) {
    const int64_t chunk = chunk_entries(n), chunks = (n + chunk - 1) / chunk;
    return chunks <= 1 ? 0 : static_cast<size_t>(chunks) * static_cast<size_t>(experts) * sizeof(uint32_t);
}

cudaError_t launch_expert_plan(const void *index, bool wide, int64_t n, int64_t experts, int64_t rows,
                               int32_t *offsets, int32_t *counts, int32_t *slot, int32_t *source, void *ws,
                               const DeviceInfo &dev, cudaStream_t stream) {
    PlanArgs p{};
    p.index = index;
    p.n = n;
    p.rows = rows;
    p.experts = static_cast<int>(experts);
    p.chunk = chunk_entries(n);
    p.chunks = static_cast<int>(std::max<int64_t>(1, (n + p.chunk - 1) / p.chunk));
    p.offsets = offsets;
    p.counts = counts;
    p.slot = slot;
    p.source = source;
    p.chunk_counts = static_cast<uint32_t *>(ws);
    p.status = dev.status;
    return wide ? launch_plan<int64_t>(p, stream) : launch_plan<int32_t>(p, stream);
}

cudaError_t launch_expert_dispatch(const RowIn &x, const ExpertRows &r, void *y, const RowEncode &e,
                                   const DeviceInfo &dev, cudaStream_t stream) {
    RowsArgs p = rows_args(r, dev);
    p.x = static_cast<const uint8_t *>(x.p);
    p.x_pitch = x.pitch * (x.f32 ? 4 : 2);
    p.y = {static_cast<uint8_t *>(y), static_cast<size_t>(r.rows) * r.K * 2};
    p.enc = row_encoded(e, r.rows, r.K);
    p.aligned32 = aligned32(x.p);
    p.aligned_out = y == nullptr || (aligned32(y) && r.K % 16 == 0);
    if (r.picks == 0) p.T = 0;  // x is not read (and may be null)
    const int64_t zeros = zero_blocks(p, kWarps), grid = zeros + (p.T * p.strips + kWarps - 1) / kWarps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.zeros = static_cast<uint32_t>(zeros);
    return x.f32 ? launch_dependent(mx_expert_dispatch_kernel<F32>, grid, 32 * kWarps, 0, stream, p)
                 : launch_dependent(mx_expert_dispatch_kernel<BF16>, grid, 32 * kWarps, 0, stream, p);
}

cudaError_t launch_expert_combine(const RowIn &rows, const ExpertRows &r, const float *weights, const RowIn &res,
                                  void *y, int y_f32, const DeviceInfo &dev, cudaStream_t stream) {
    RowsArgs p = rows_args(r, dev);
    p.rows = static_cast<const uint8_t *>(rows.p);
    p.rows_pitch = rows.pitch * (rows.f32 ? 4 : 2);
    p.res = static_cast<const uint8_t *>(res.p);
    p.res_pitch = res.pitch * (res.f32 ? 4 : 2);
    p.weights = weights;
    p.y = {static_cast<uint8_t *>(y), static_cast<size_t>(r.T) * r.K * (y_f32 ? 4 : 2)};
    p.aligned32 = aligned32(rows.p) && aligned32(res.p);
    p.aligned_out = aligned32(y);
    p.strips = static_cast<int>((r.K + kOutStrip - 1) / kOutStrip);
    const int64_t grid = (r.T * p.strips + kWarps - 1) / kWarps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (rows.f32)
        return res.f32 ? launch_combine<F32, F32>(p, y_f32, grid, stream) : launch_combine<F32, BF16>(p, y_f32, grid, stream);
    return res.f32 ? launch_combine<BF16, F32>(p, y_f32, grid, stream) : launch_combine<BF16, BF16>(p, y_f32, grid, stream);
}

cudaError_t launch_expert_combine_backward(const RowIn &dy, const RowIn &rows, const ExpertRows &r,
                                           const float *weights, void *drows, const RowEncode &e, float *dweights,
                                           const DeviceInfo &dev, cudaStream_t stream) {
    RowsArgs p = rows_args(r, dev);
    p.x = static_cast<const uint8_t *>(dy.p);
    p.x_pitch = dy.pitch * (dy.f32 ? 4 : 2);
    p.rows = static_cast<const uint8_t *>(rows.p);
    p.rows_pitch = rows.pitch * (rows.f32 ? 4 : 2);
    p.weights = weights;
    p.y = {static_cast<uint8_t *>(drows), static_cast<size_t>(r.rows) * r.K * 2};
    p.dweights = {reinterpret_cast<uint8_t *>(dweights), static_cast<size_t>(r.T) * r.picks * 4};
    p.enc = row_encoded(e, r.rows, r.K);
    p.aligned32 = aligned32(dy.p) && aligned32(rows.p);
    p.aligned_out = drows == nullptr || (aligned32(drows) && r.K % 16 == 0);
    // As many warps as a row has strips, at most a block.
    const int warps = std::min(kWarps, p.strips), threads = 32 * warps;
    const bool writes = drows != nullptr || e.fmt != kEncNone;
    const int64_t zeros = writes ? zero_blocks(p, warps) : 0, grid = zeros + r.T;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.zeros = static_cast<uint32_t>(zeros);
    if (dy.f32)
        return rows.f32 ? launch_dependent(mx_expert_combine_backward_kernel<F32, F32>, grid, threads, 0, stream, p)
                        : launch_dependent(mx_expert_combine_backward_kernel<F32, BF16>, grid, threads, 0, stream, p);
    return rows.f32 ? launch_dependent(mx_expert_combine_backward_kernel<BF16, F32>, grid, threads, 0, stream, p)
                    : launch_dependent(mx_expert_combine_backward_kernel<BF16, BF16>, grid, threads, 0, stream, p);
}

}  // namespace mx
