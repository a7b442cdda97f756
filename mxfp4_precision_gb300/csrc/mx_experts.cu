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
    int64_t chunk;           // a multiple of 512
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

template <typename I>
__global__ void __launch_bounds__(kPlanThreads) mx_expert_plan_kernel(const __grid_constant__ PlanArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ uint32_t at[kPlanWarps][MX_EXPERTS_MAX];  // counts, then next rows
    __shared__ uint32_t part[kPlanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = threadIdx.x;
    for (int i = threadIdx.x; i < kPlanWarps * MX_EXPERTS_MAX; i += kPlanThreads) (&at[0][0])[i] = 0;
    __syncthreads();
    const int64_t each = p.chunk / kPlanWarps;  // a multiple of 32
    const int64_t first = blockIdx.x * p.chunk + warp * each;
    for (int64_t i = lane; i < each; i += 32) {
        const int x = expert_of<I>(p, first + i);
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, x);
        if (x >= 0 && lane == __ffs(same) - 1) at[warp][x] += __popc(same);
        __syncwarp();
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
        uint32_t next = start + before;
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            const uint32_t v = at[w][e];
            at[w][e] = next;
            next += v;
        }
        // This expert's padding rows.
        if (e % gridDim.x == blockIdx.x)
            for (uint32_t r = start + total; r < start + size && r < p.rows; ++r) p.source[r] = -1;
    }
    if (threadIdx.x == 0 && blockIdx.x == 0) p.offsets[p.experts] = static_cast<int32_t>(used);
    __syncthreads();
    for (int64_t i = lane; i < each; i += 32) {
        const int x = expert_of<I>(p, first + i);
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, x);
        int32_t row = -1;
        if (x >= 0) row = static_cast<int32_t>(at[warp][x] + __popc(same & ((1u << lane) - 1u)));
        __syncwarp();
        if (x >= 0 && lane == __ffs(same) - 1) at[warp][x] += __popc(same);
        __syncwarp();
        if (first + i < p.n) {
            p.slot[first + i] = row;
            if (row >= 0 && row < p.rows) p.source[row] = static_cast<int32_t>(first + i);
        }
    }
    // Rows behind the last segment.
    for (int64_t r = used + static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x; r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * kPlanThreads)
        p.source[r] = -1;
}

// ---------------------------------------------------------------- rows in
// A warp takes one token's strip of 256 columns (a 32-column block is four
// lanes), reads it once, encodes it once and stores it to each of the token's rows;
// bound by memory.  Blocks behind those of the tokens zero the rows without a token.
constexpr int kWarps = 8;
constexpr int kZeroRows = 8;  // rows a warp looks through for padding

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
    uint32_t tiles;  // blocks that hold tokens
    bool aligned32, aligned_out;
    int *status;
};

__device__ __forceinline__ bool there(const RowsArgs &p, int32_t slot) {
    return static_cast<uint32_t>(slot) < static_cast<uint64_t>(p.P);
}

// Codes and scale byte of the lane's eight columns, kept to be stored to several rows.
struct Codes8 {
    uint32_t w[2];
    uint32_t scale;
};
__device__ __forceinline__ Codes8 codes8(int fmt, const V8 &a) {
    float f[8];
    floats_of(a, f);
    float m = enc::absmax2_nan(enc::absmax3_nan(f[0], f[1], f[2]), enc::absmax3_nan(f[3], f[4], f[5]));
    m = enc::absmax3_nan(m, f[6], f[7]);
    m = enc::absmax2_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = enc::absmax2_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    float inv;
    Codes8 r;
    r.scale = fmt == kEncMX8 ? enc::scale_of_e4m3(m, inv) : enc::scale_of(m, inv);
    V8 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q.v[i] = mul2(a.v[i], same2(inv));
    floats_of(q, f);
    if (fmt == kEncMX8) {
        r.w[0] = enc::cvt_e4m3x4(f[0], f[1], f[2], f[3]);
        r.w[1] = enc::cvt_e4m3x4(f[4], f[5], f[6], f[7]);
    } else {
        r.w[0] = enc::cvt_e2m1x8(f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]);
        r.w[1] = 0;
    }
    if (r.scale == 0xFFu) r.w[0] = r.w[1] = 0;
    return r;
}

// The lane's eight columns (chunk c) of a row of the output: bf16, codes and scale byte; all
// lanes of a warp on one row.
__device__ __forceinline__ void put8(const RowsArgs &p, int64_t row, uint32_t c, bool in, const V8 &a, const Codes8 &q) {
    if (in && p.y.p != nullptr) store8<BF16>(p.y, p.y.p + (row * p.K + 8 * c) * 2, a, true, p.status);
    if (p.enc.fmt == kEncNone) return;
    const EncodedRow at = encoded_row(p.enc, row);
    if (in) {
        if (p.enc.fmt == kEncMX8) {
            uint8_t *d = at.codes + 8u * c;
            if (MX_STORE_OK(d, 8, p.enc.codes.p, p.enc.codes.bytes, p.status))
                *reinterpret_cast<uint2 *>(d) = make_uint2(q.w[0], q.w[1]);
        } else {
            uint8_t *d = at.codes + 4u * c;
            if (MX_STORE_OK(d, 4, p.enc.codes.p, p.enc.codes.bytes, p.status)) *reinterpret_cast<uint32_t *>(d) = q.w[0];
        }
    }
    if ((threadIdx.x & 3) == 0) {
        uint8_t *d = at.scales + (c >> 4) * 512u + ((c >> 2) & 3u);
        if (MX_STORE_OK(d, 1, p.enc.scales.p, p.enc.scales.bytes, p.status)) *d = static_cast<uint8_t>(in ? q.scale : 0u);
    }
}

// Zeroes the rows without a token: the n-th warp looks through kZeroRows of them.
__device__ __forceinline__ void zero_rows(const RowsArgs &p, int64_t n) {
    const int lane = threadIdx.x & 31;
    const int64_t first = n * kZeroRows;
    const bool free_row = lane < kZeroRows && first + lane < p.P && p.source[first + lane] < 0;
    for (uint32_t mask = __ballot_sync(0xFFFFFFFFu, free_row); mask != 0; mask &= mask - 1) {
        const int64_t row = first + __ffs(mask) - 1;
        const Codes8 none{{0, 0}, 0};
        for (int s = 0; s < p.strips; ++s) {
            const uint32_t c = static_cast<uint32_t>(s) * 32 + lane;
            put8(p, row, c, 8 * c < p.K, zero_v8(), none);
        }
    }
}

template <typename X>
__global__ void __launch_bounds__(32 * kWarps) mx_expert_dispatch_kernel(const __grid_constant__ RowsArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x >= p.tiles) {
        zero_rows(p, static_cast<int64_t>(blockIdx.x - p.tiles) * kWarps + warp);
        return;
    }
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int64_t t = unit / p.strips;
    if (t >= p.T) return;
    const uint32_t c = static_cast<uint32_t>(unit - t * p.strips) * 32 + lane;
    const bool in = 8 * c < p.K;
    Raw8<X> r;
    zero8(r);
    if (in) load8(r, p.x + t * p.x_pitch + static_cast<size_t>(8 * c) * X::kBytes, p.aligned32);
    const V8 a = to_v8(r);
    Codes8 q{{0, 0}, 0};
    if (p.enc.fmt != kEncNone) q = codes8(p.enc.fmt, a);
    for (int j = 0; j < p.picks; ++j) {
        const int32_t s = p.slot[t * p.picks + j];
        if (there(p, s)) put8(p, s, c, in, a, q);
    }
}

// ---------------------------------------------------------------- rows out
// A warp takes one token's strip of 256 columns and adds up to four of its rows at
// a time, all in flight; bound by memory.
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
// A block takes one token: dy is read once for up to four of its choices, whose rows'
// gradients leave as they are made; the products with the rows are added up over the
// block in a fixed order.  Blocks behind those of the tokens zero the rows without a token.
constexpr int kAtOnce = 4;
constexpr int kGradThreads = 256;

template <typename D, typename R>
__global__ void __launch_bounds__(kGradThreads) mx_expert_combine_backward_kernel(const __grid_constant__ RowsArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (blockIdx.x >= p.tiles) {
        zero_rows(p, static_cast<int64_t>(blockIdx.x - p.tiles) * warps + warp);
        return;
    }
    __shared__ float part[kGradThreads / 32][kAtOnce];
    const int64_t t = blockIdx.x;
    const uint8_t *dy = p.x + t * p.x_pitch;
    const uint32_t chunks = static_cast<uint32_t>(p.strips) * 32;
    for (int j0 = 0; j0 < p.picks; j0 += kAtOnce) {
        int32_t s[kAtOnce];
        float w[kAtOnce];
        uint64_t dot[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int64_t i = t * p.picks + j0 + k;
            s[k] = j0 + k < p.picks ? p.slot[i] : -1;
            if (!there(p, s[k])) s[k] = -1;
            w[k] = s[k] >= 0 ? p.weights[i] : 0.0f;
            dot[k] = 0;
        }
        for (uint32_t c = threadIdx.x; c < chunks; c += blockDim.x) {
            const bool in = 8 * c < p.K;
            Raw8<D> dr;
            Raw8<R> r[kAtOnce];
            zero8(dr);
            if (in) load8(dr, dy + static_cast<size_t>(8 * c) * D::kBytes, p.aligned32);
            if (p.dweights.p != nullptr) {
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    zero8(r[k]);
                    if (in && s[k] >= 0) load8(r[k], p.rows + s[k] * p.rows_pitch + static_cast<size_t>(8 * c) * R::kBytes, p.aligned32);
                }
            }
            const V8 d = to_v8(dr);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (s[k] < 0) continue;
                if (p.dweights.p != nullptr) {
                    const V8 a = to_v8(r[k]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dot[k] = fma2(a.v[i], d.v[i], dot[k]);
                }
                if (p.y.p == nullptr && p.enc.fmt == kEncNone) continue;
                V8 g;
#pragma unroll
                for (int i = 0; i < 4; ++i) g.v[i] = mul2(d.v[i], same2(w[k]));
                Codes8 q{{0, 0}, 0};
                if (p.enc.fmt != kEncNone) q = codes8(p.enc.fmt, g);
                put8(p, s[k], c, in, g, q);
            }
        }
        if (p.dweights.p == nullptr) continue;
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
    p.strips = static_cast<int>((r.K + 255) / 256);
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
    return most <= kChunk ? kChunk : (most + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
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
    const int64_t tiles = (r.T * p.strips + kWarps - 1) / kWarps, grid = tiles + zero_blocks(p, kWarps);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.tiles = static_cast<uint32_t>(tiles);
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
    // As many threads as a row has chunks of 8 columns, at most a block.
    const int threads = std::min(kGradThreads, p.strips * 32);
    const bool writes = drows != nullptr || e.fmt != kEncNone;
    const int64_t grid = r.T + (writes ? zero_blocks(p, threads / 32) : 0);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.tiles = static_cast<uint32_t>(r.T);
    if (dy.f32)
        return rows.f32 ? launch_dependent(mx_expert_combine_backward_kernel<F32, F32>, grid, threads, 0, stream, p)
                        : launch_dependent(mx_expert_combine_backward_kernel<F32, BF16>, grid, threads, 0, stream, p);
    return rows.f32 ? launch_dependent(mx_expert_combine_backward_kernel<BF16, F32>, grid, threads, 0, stream, p)
                    : launch_dependent(mx_expert_combine_backward_kernel<BF16, BF16>, grid, threads, 0, stream, p);
}

}  // namespace mx
