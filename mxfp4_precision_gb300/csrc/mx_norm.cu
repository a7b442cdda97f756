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
    int64_t x_pitch, res_pitch, h_pitch;  // bytes
    Out h, y, rstd;
    Encoded enc;
    int64_t T;
    uint32_t K;
    float eps;
    bool aligned32;
    int w_f32;
    int tpr, groups;  // threads per row (a multiple of 32), rows per block
    uint32_t tiles;  // blocks that hold rows; those after them zero the scales' padding lines
    int *status;
};

// Sum over the tpr threads of a row (the whole block takes part: rows of one
// block reduce in step).  `part` holds one float per warp.
__device__ __forceinline__ float sum_row(float v, int g, int tpr, float *part) {
    v = sum_lanes(v);
    if (tpr == 32) return v;
    const int n = tpr >> 5;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < n; ++i) v += part[g * n + i];
    return v;
}

__device__ __forceinline__ float rstd_of(float sum, uint32_t K, float eps) {
    return __frsqrt_rn(sum / static_cast<float>(K) + eps);
}

// Where a row's outputs go.
struct NormRow {
    uint8_t *h, *y;
    EncodedRow enc;
};
__device__ __forceinline__ NormRow norm_row(const NormArgs &p, int64_t row) {
    return {p.h.p + row * p.h_pitch, p.y.p + row * 2 * p.K, encoded_row(p.enc, row)};
}
// The outputs of one chunk (8 columns) of a row: h, y and y's codes.
template <typename S, bool RES>
__device__ __forceinline__ void norm_out(const NormArgs &p, const NormRow &at, uint32_t c, const V8 &h,
                                         const V8 &w, float rstd) {
    const bool in = 8 * c < p.K;
    if (RES && in && p.h.p != nullptr) store8<S>(p.h, at.h + 8 * S::kBytes * c, h, p.aligned32, p.status);
    V8 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y.v[i] = mul2(mul2(h.v[i], same2(rstd)), w.v[i]);
    if (in && p.y.p != nullptr) store8<BF16>(p.y, at.y + 16 * c, y, true, p.status);
    // Whole warps: a warp's chunks are all inside the padded width or all beyond it.
    if (p.enc.fmt != kEncNone && c < p.enc.katoms * 16) encode8(p.enc, at.enc, c, in, y, p.status);
}

// h = x + r of a chunk, and its squares added to a pair of sums.
template <typename X, typename S, bool RES>
__device__ __forceinline__ V8 join(const Raw8<X> &x, const Raw8<S> &r, uint64_t &ss) {
    V8 h = to_v8(x);
    if (RES) {
        const V8 b = to_v8(r);
#pragma unroll
        for (int i = 0; i < 4; ++i) h.v[i] = add2(h.v[i], b.v[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) ss = fma2(h.v[i], h.v[i], ss);
    return h;
}

__device__ __forceinline__ void rstd_out(const NormArgs &p, int64_t row, float rstd) {
    if (p.rstd.p == nullptr) return;
    float *d = reinterpret_cast<float *>(p.rstd.p) + row;
    if (MX_STORE_OK(d, 4, p.rstd.p, p.rstd.bytes, p.status)) *d = rstd;
}

// One row per tpr threads and no turn after it, C chunks of 8 columns per
// thread, the row in registers between its sum and its output: one read, one
// write.  Bound by memory; what it needs is loads in flight, and several short
// blocks per SM have more of them than one long-lived block that feeds itself
// through a ring of shared-memory slots (8192 x 4096: 62 to 66 us so).  fp32 x,
// bf16 stream and bf16 y, MXFP8 codes, 8192 x 4096: 56.8 us, 370 MB = 6.5 TB/s (96%
// of a plain copy's rate); 16384 x 4096 without y: 89.5 us, 6.8 TB/s (99.6%).
// norm_blocks: blocks per SM that the registers must allow; the compiler left
// alone takes C = 4 to one block of 512 threads (bf16, 2048 x 16384: 67 us against
// 51 us).
template <typename X, typename S, int C, int THREADS>
constexpr int norm_blocks() {
    if (THREADS > 256) return THREADS > 512 ? 1 : 2;
    return C == 1 ? 6 : C == 2 ? 5 : C <= 4 ? 4 : X::kBytes + S::kBytes == 8 ? 2 : 3;
}
template <typename X, typename S, bool RES, int C, int THREADS>
__global__ void __launch_bounds__(THREADS, norm_blocks<X, S, C, THREADS>()) mx_rmsnorm_kernel(const __grid_constant__ NormArgs p) {
    __shared__ float part[32];
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x >= p.tiles) {
        zero_padding(p.enc, p.T, static_cast<int64_t>(blockIdx.x - p.tiles) * blockDim.x + threadIdx.x,
                     static_cast<int64_t>(gridDim.x - p.tiles) * blockDim.x, p.status);
        return;
    }
    int g = 0, tr = threadIdx.x;
    if (p.groups > 1) {
        g = p.tpr == 32 ? tr >> 5 : tr / p.tpr;
        tr -= g * p.tpr;
    }
    const int64_t row = static_cast<int64_t>(blockIdx.x) * p.groups + g;
    const bool live = row < p.T;
    const uint8_t *x = p.x + row * p.x_pitch, *res = p.res + row * p.res_pitch;
    Raw8<X> xr[C];
    Raw8<S> rr[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint32_t col = 8 * (j * p.tpr + tr);
        // Only a warp that the row ends in has lanes to clear.
        if (!live || col - 8 * (tr & 31) + 256 > p.K) {
            zero8(xr[j]);
            zero8(rr[j]);
            if (!live || col >= p.K) continue;
        }
        load8(xr[j], x + col * X::kBytes, p.aligned32);
        if (RES) load8(rr[j], res + col * S::kBytes, p.aligned32);
    }
    V8 h[C];
    uint64_t ss = 0;
#pragma unroll
    for (int j = 0; j < C; ++j) h[j] = join<X, S, RES>(xr[j], rr[j], ss);
    const float rstd = rstd_of(sum_row(sum2(ss), g, p.tpr, part), p.K, p.eps);
    if (!live) return;
    if (tr == 0) rstd_out(p, row, rstd);
    const NormRow at = norm_row(p, row);
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint32_t c = j * p.tpr + tr;
        const V8 w = 8 * c < p.K ? load_weight8(p.w, p.w_f32 != 0, 8 * c) : zero_v8();
        norm_out<S, RES>(p, at, c, h[j], w, rstd);
    }
}

// ---------------------------------------------------------------- rows through a ring
// For the gradient over many rows: one block per SM, its threads in groups of
// tpr that each take rows in turn.  A group's next rows are on their way
// (cp.async.bulk, one per input and row) into its ring of shared-memory slots
// while it works on the present one, so that the loads never wait for a row's
// sum.  A group meets once a row, in the barrier of its sum; by then every
// thread has the row in registers, and the slot is filled again.
struct Ring {
    uint8_t *slots;  // of this group
    uint64_t *full;
    float *part;     // [2][32]
    int id, tpr, stages, slot_bytes;
    int s = 0;
    uint32_t parity = 0;

    __device__ __forceinline__ uint8_t *slot() const { return slots + s * slot_bytes; }
    __device__ __forceinline__ void next() {
        if (++s == stages) s = 0, parity ^= 1;
    }
    // Sum over the group, and whether every thread's wait ended well.
    __device__ __forceinline__ bool sum(float &v, bool ok, int turn) {
        v = sum_lanes(v);
        if (tpr == 32) return __all_sync(0xFFFFFFFFu, ok);
        float *at = part + (turn & 1) * 32;
        const int tr = threadIdx.x % tpr;
        if ((tr & 31) == 0) at[tr >> 5] = v;
        ok = bar_and(id, tpr, ok);
        v = 0.0f;
        for (int i = 0; i < tpr >> 5; ++i) v += at[i];
        return ok;
    }
    // Every thread of the group is done with the slot.
    __device__ __forceinline__ void done() {
        if (tpr == 32) __syncwarp();
        else bar_and(id, tpr, true);
    }
    // After a wait that ran out: the slots still being filled, before the block ends.
    __device__ __forceinline__ void drain(int64_t left) {
        for (int64_t i = 0; i < left && i < stages; ++i, next())
            mbar_wait_inl(&full[s], parity, nullptr, nullptr);
    }
};

// Carves the block's dynamic shared memory: groups x stages slots, then the
// barriers, then the groups' partial sums; sets up this thread's group.
__device__ __forceinline__ Ring ring_of(uint8_t *smem, int tpr, int stages, int slot_bytes) {
    const int groups = blockDim.x / tpr, g = threadIdx.x / tpr;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + static_cast<size_t>(groups) * stages * slot_bytes);
    float *parts = reinterpret_cast<float *>(bars + groups * stages);
    Ring r;
    r.slots = smem + static_cast<size_t>(g) * stages * slot_bytes;
    r.full = bars + g * stages;
    r.part = parts + g * 64;
    r.id = g + 1;
    r.tpr = tpr;
    r.stages = stages;
    r.slot_bytes = slot_bytes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < groups * stages; ++i) mbar_init(&bars[i], 1);
        fence_barrier_init();
    }
    __syncthreads();
    return r;
}

// ---------------------------------------------------------------- gradient
struct NormGradArgs {
    const uint8_t *dy, *h, *w, *dres;
    const float *rstd;
    int64_t dy_pitch, h_pitch, dres_pitch, dx_pitch;  // bytes
    Out dx, parts;  // parts [n][K] fp32: partial weight gradients (null: not wanted)
    int64_t T;
    uint32_t K;
    int w_f32;
    int tpr, stages;
    bool aligned32;
    int *status;
};

// Columns col .. col+7 of partial gradient n.
__device__ __forceinline__ void part_out(const NormGradArgs &p, int64_t n, uint32_t col, const V8 &v) {
    store8<F32>(p.parts, p.parts.p + (n * p.K + col) * 4, v, false, p.status);
}

// The block's partial gradient from its groups', through sums [groups][K].
template <int C>
__device__ __forceinline__ void sum_groups(const NormGradArgs &p, float *sums, const V8 (&dw)[C]) {
    const int tr = threadIdx.x % p.tpr, groups = blockDim.x / p.tpr, g = threadIdx.x / p.tpr;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint32_t col = 8 * (j * p.tpr + tr);
        if (col >= p.K) continue;
        float v[8];
        floats_of(dw[j], v);
        float4 *d = reinterpret_cast<float4 *>(sums + g * p.K + col);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __syncthreads();
    for (uint32_t col = 8 * threadIdx.x; col < p.K; col += 8 * blockDim.x) {
        V8 v = zero_v8();
        for (int k = 0; k < groups; ++k) {
            Raw8<F32> r;
            load8_again(r, reinterpret_cast<const uint8_t *>(sums + k * p.K + col));
            const V8 b = to_v8(r);
#pragma unroll
            for (int i = 0; i < 4; ++i) v.v[i] = add2(v.v[i], b.v[i]);
        }
        part_out(p, blockIdx.x, col, v);
    }
}

// First look at a chunk: dw += dy * xhat and along += dy * w * xhat, with
// xhat = h * rstd; leaves dy * w in a.
__device__ __forceinline__ void look(V8 &a, const V8 &h, const V8 &w, float rstd, V8 &dw,
                                     uint64_t &along) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t x = mul2(h.v[i], same2(rstd));
        dw.v[i] = fma2(a.v[i], x, dw.v[i]);
        a.v[i] = mul2(a.v[i], w.v[i]);
        along = fma2(a.v[i], x, along);
    }
}
// dx = rstd * (a - xhat * along) + dres, into g (which holds dres).
__device__ __forceinline__ void finish(const V8 &a, const V8 &h, float rstd, float along, V8 &g) {
    const uint64_t r = same2(rstd), m = same2(-along);
#pragma unroll
    for (int i = 0; i < 4; ++i) g.v[i] = fma2(r, fma2(mul2(h.v[i], r), m, a.v[i]), g.v[i]);
}

// Few rows, or rows too wide for two in the ring below (fp32 beyond 9000 columns or
// so: 10240 to 16384 columns 61 to 74% of a plain copy's rate, beyond that 45 to 67%): each group of tpr threads takes rows in turn and keeps its columns' sums of
// dy * h * rstd in registers; they are added up over the block's groups at the
// end: one partial per block.  AGAIN: rows too wide for the registers are
// loaded twice (the second time from L1 or L2), once for mean(dy * w * h), once
// for dx.
template <typename D, typename S, int C, int THREADS, bool AGAIN>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 2 : 1)
    mx_rmsnorm_backward_kernel(const __grid_constant__ NormGradArgs p) {
    __shared__ float part[2][32];
    extern __shared__ __align__(128) uint8_t smem[];  // [groups][K] fp32 where groups > 1
    griddep_wait();
    griddep_launch_dependents();
    const int tr = threadIdx.x % p.tpr, groups = blockDim.x / p.tpr, g = threadIdx.x / p.tpr;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * groups;
    V8 dw[C];
#pragma unroll
    for (int j = 0; j < C; ++j) dw[j] = zero_v8();
    // Every group of a block makes the same number of turns (they share barriers).
    int turn = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < p.T; base += stride, turn ^= 1) {
        const int64_t row = base + g;
        const bool live = row < p.T;
        const uint8_t *dy = p.dy + row * p.dy_pitch, *hp = p.h + row * p.h_pitch;
        const uint8_t *gp = p.dres + row * p.dres_pitch;
        Raw8<D> dr[C];
        Raw8<S> hr[C], gr[C];
        const float rstd = live ? p.rstd[row] : 0.0f;
        uint64_t sums = 0;
        if (!AGAIN) {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const uint32_t col = 8 * (j * p.tpr + tr);
                zero8(dr[j]);
                zero8(hr[j]);
                zero8(gr[j]);
                if (live && col < p.K) {
                    load8(dr[j], dy + col * D::kBytes, p.aligned32);
                    load8(hr[j], hp + col * S::kBytes, p.aligned32);
                    if (p.dres != nullptr) load8(gr[j], gp + col * S::kBytes, p.aligned32);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const uint32_t col = 8 * (j * p.tpr + tr);
            if (!live || col >= p.K) continue;
            if (AGAIN) {
                load8_again(dr[j], dy + col * D::kBytes);
                load8_again(hr[j], hp + col * S::kBytes);
            }
            V8 a = to_v8(dr[j]);
            look(a, to_v8(hr[j]), load_weight8(p.w, p.w_f32 != 0, col), rstd, dw[j], sums);
        }
        const float along = sum_row(sum2(sums), g, p.tpr, part[turn]) / static_cast<float>(p.K);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const uint32_t col = 8 * (j * p.tpr + tr);
            if (!live || col >= p.K) continue;
            if (AGAIN) {
                load8_again(dr[j], dy + col * D::kBytes);
                load8_again(hr[j], hp + col * S::kBytes);
                zero8(gr[j]);
                if (p.dres != nullptr) load8(gr[j], gp + col * S::kBytes, p.aligned32);
            }
            V8 a = to_v8(dr[j]), v = to_v8(gr[j]);
            const V8 w = load_weight8(p.w, p.w_f32 != 0, col);
#pragma unroll
            for (int i = 0; i < 4; ++i) a.v[i] = mul2(a.v[i], w.v[i]);
            finish(a, to_v8(hr[j]), rstd, along, v);
            store8<S>(p.dx, p.dx.p + row * p.dx_pitch + col * S::kBytes, v, p.aligned32, p.status);
        }
    }
    if (p.parts.p == nullptr) return;
    if (groups == 1) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const uint32_t col = 8 * (j * p.tpr + tr);
            if (col < p.K) part_out(p, blockIdx.x, col, dw[j]);
        }
        return;
    }
    sum_groups<C>(p, reinterpret_cast<float *>(smem), dw);
}

// Many rows, through the ring (bf16 stream 8192 x 4096: 54 us, 81 us directly).
// Bound by memory: with fp32 dy 336 MB = 6.2 TB/s (91% of a plain copy's rate)
// there; the sum of the partial weight gradients takes 2 us and the ring's filling
// and emptying 4 us.  LOOK2 (one warp a row, or four chunks a thread): a row is read from its slot twice, once
// for mean(dy * w * h) and once for dx, instead of staying in registers between
// them; the slot is then free only after the second.  The groups' weight
// gradients are summed in shared memory at the end: one partial per block.
template <typename D, typename S, int C, int THREADS, bool LOOK2>
__global__ void __launch_bounds__(THREADS)
    mx_rmsnorm_backward_ring_kernel(const __grid_constant__ NormGradArgs p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t db = p.K * D::kBytes, sb = p.K * S::kBytes;
    const bool res = p.dres != nullptr;
    const uint32_t bytes = db + sb + (res ? sb : 0);
    Ring ring = ring_of(smem, p.tpr, p.stages, bytes);
    griddep_wait();
    griddep_launch_dependents();
    const int tr = threadIdx.x % p.tpr, groups = blockDim.x / p.tpr, g = threadIdx.x / p.tpr;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * groups;
    // Neighbouring blocks take neighbouring rows.
    int64_t row = static_cast<int64_t>(g) * gridDim.x + blockIdx.x;
    auto fill = [&](int64_t r, int s) {
        uint8_t *d = ring.slots + s * ring.slot_bytes;
        mbar_arrive_expect_tx(&ring.full[s], bytes);
        bulk_load(d, p.dy + r * p.dy_pitch, db, &ring.full[s]);
        bulk_load(d + db, p.h + r * p.h_pitch, sb, &ring.full[s]);
        if (res) bulk_load(d + db + sb, p.dres + r * p.dres_pitch, sb, &ring.full[s]);
    };
    if (tr == 0)
        for (int s = 0; s < p.stages; ++s)
            if (row + s * stride < p.T) fill(row + s * stride, s);
    V8 w[C], dw[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint32_t col = 8 * (j * p.tpr + tr);
        w[j] = col < p.K ? load_weight8(p.w, p.w_f32 != 0, col) : zero_v8();
        dw[j] = zero_v8();
    }
    for (int turn = 0; row < p.T; row += stride, ++turn) {
        const float rstd = p.rstd[row];
        bool ok = mbar_wait_inl(&ring.full[ring.s], ring.parity, p.status, nullptr);
        const uint8_t *slot = ring.slot();
        V8 a[C];
        Raw8<S> hr[C], gr[C];
        uint64_t sums = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const uint32_t col = 8 * (j * p.tpr + tr);
            Raw8<D> dr;
            zero8(dr);
            zero8(hr[j]);
            zero8(gr[j]);
            if (col < p.K) {
                load8_again(dr, slot + col * D::kBytes);
                load8_again(hr[j], slot + db + col * S::kBytes);
                if (!LOOK2 && res) load8_again(gr[j], slot + db + sb + col * S::kBytes);
            }
            a[j] = to_v8(dr);
            look(a[j], to_v8(hr[j]), w[j], rstd, dw[j], sums);
        }
        float along = sum2(sums);
        ok = ring.sum(along, ok, turn);
        if (!ok) {
            if (tr == 0) ring.drain((p.T - row + stride - 1) / stride);
            break;
        }
        const int64_t next = row + p.stages * stride;
        if (!LOOK2 && tr == 0 && next < p.T) fill(next, ring.s);
        along /= static_cast<float>(p.K);
        uint8_t *dx = p.dx.p + row * p.dx_pitch;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const uint32_t col = 8 * (j * p.tpr + tr);
            if (col >= p.K) continue;
            if (LOOK2) {
                Raw8<D> dr;
                load8_again(dr, slot + col * D::kBytes);
                load8_again(hr[j], slot + db + col * S::kBytes);
                if (res) load8_again(gr[j], slot + db + sb + col * S::kBytes);
                a[j] = to_v8(dr);
#pragma unroll
                for (int i = 0; i < 4; ++i) a[j].v[i] = mul2(a[j].v[i], w[j].v[i]);
            }
            V8 v = to_v8(gr[j]);
            finish(a[j], to_v8(hr[j]), rstd, along, v);
            store8<S>(p.dx, dx + col * S::kBytes, v, p.aligned32, p.status);
        }
        if (LOOK2) {
            ring.done();
            if (tr == 0 && next < p.T) fill(next, ring.s);
        }
        ring.next();
    }
    if (p.parts.p == nullptr) return;
    // All slots are consumed (or drained): the ring's memory holds the groups' sums.
    __syncthreads();
    sum_groups<C>(p, reinterpret_cast<float *>(smem), dw);
}

// dw[col] = sum of the n partial sums, in a fixed order: 32 columns a block, four
// a lane, the partials split over the block's other threads, four of them in
// flight (the last again, unused, beyond the end): one round of loads from L2
// up to 512 partials, which with the launch is what bounds it.
__global__ void __launch_bounds__(1024) mx_rmsnorm_dw_kernel(const float *parts, int n, uint32_t K, Out dw,
                                                             int *status) {
    __shared__ float sums[32][32];
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t col = blockIdx.x * 32 + 4 * (threadIdx.x & 7);
    float s[4] = {0, 0, 0, 0};
    if (col < K) {
        for (int i = threadIdx.x >> 3; i < n; i += 4 * 128) {
            float4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = *reinterpret_cast<const float4 *>(parts + static_cast<int64_t>(min(i + 128 * k, n - 1)) * K + col);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + 128 * k < n) s[0] += v[k].x, s[1] += v[k].y, s[2] += v[k].z, s[3] += v[k].w;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], 8);
        s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], 16);
    }
    if ((threadIdx.x & 31) < 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) sums[threadIdx.x >> 5][4 * (threadIdx.x & 7) + k] = s[k];
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < K) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += sums[i][threadIdx.x];
        float *d = reinterpret_cast<float *>(dw.p) + blockIdx.x * 32 + threadIdx.x;
        if (MX_STORE_OK(d, 4, dw.p, dw.bytes, status)) *d = t;
    }
}

// ---------------------------------------------------------------- shapes
// Threads of a row and its chunks of 8 columns per thread, and the rows of a block
// of `block` threads or one row; `n` chunks is the padded width of the scale
// layout (a multiple of 32).
struct RowShape {
    int c, tpr, groups, stages;
    size_t smem;
};
int64_t padded_chunks(int64_t K) { return (K + 255) / 256 * 32; }
RowShape row_shape(int64_t n, int c, int block) {
    const int tpr = static_cast<int>((n + 32 * c - 1) / (32 * c)) * 32;
    return {c, tpr, tpr >= block ? 1 : block / tpr, 0, 0};
}

// How a row is cut, by what keeps the most loads in flight (rates of a plain
// copy's, at 2^25 elements unless said):
//   blocks of 128 threads where a row needs no more, since a finished one makes room
//     sooner (bf16 2048 columns, codes alone: 86%, 78% in blocks of 256);
//   up to 32 chunks (K <= 256): one warp a row;
//   up to 160, once the rows fill the SMs with warps: one warp a row, no barrier
//     (bf16 16383 x 1056: 29.7 us, 34.4 us at two chunks a thread);
//   two chunks a thread, or three where that leaves fewer threads without one
//     (bf16 16383 x 2080: 52 us, 63 us at two);
//   three or four beyond 128 threads at two, for rows of up to 4 bytes a column, whose
//     threads hold little (bf16 4096 columns, codes alone: 90%, 82% at two), and
//     beyond 256 for rows of 6 (fp32 x and bf16 stream, 4096 x 8192: 57.9 us, 60.5 us;
//     at 4096 columns 96%, 97% at two), but not for rows of 8 (fp32 both, 4096 x 8192:
//     82 us, 76 us at two);
//   above 1024 chunks: four.
RowShape norm_shape(int64_t T, int64_t K, int bytes, const DeviceInfo &dev) {
    const int64_t n = padded_chunks(K);
    const bool many = T >= 16ll * dev.sm_count;
    if (n <= 32 || (n <= 160 && many)) return row_shape(n, static_cast<int>(n / 32), 128);
    if (n > 1024) return row_shape(n, 4, 128);
    const RowShape two = row_shape(n, 2, 128), three = row_shape(n, 3, 128), four = row_shape(n, 4, 128);
    const int most = bytes <= 4 ? 128 : bytes <= 6 ? 256 : 1024;
    if (many && two.tpr > most) return three.tpr <= most && three.tpr * 3 <= four.tpr * 4 ? three : four;
    return three.tpr * 3 < two.tpr * 2 ? three : two;
}

template <typename X, typename S, bool RES>
cudaError_t launch_norm(NormArgs &p, const DeviceInfo &dev, cudaStream_t stream) {
    const RowShape s = norm_shape(p.T, p.K, X::kBytes + (RES ? S::kBytes : 0), dev);
    p.tpr = s.tpr;
    p.groups = s.groups;
    const int threads = s.tpr * s.groups;
    const int64_t tiles = (p.T + s.groups - 1) / s.groups;
    const int64_t grid = tiles + (padding_words(p.enc, p.T) + threads - 1) / threads;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.tiles = static_cast<uint32_t>(tiles);
#define MX_NORM_CASE(C, THREADS) \
    launch_dependent(mx_rmsnorm_kernel<X, S, RES, C, THREADS>, grid, threads, 0, stream, p)
    switch (s.c) {
        case 1: return MX_NORM_CASE(1, 256);
        case 2: return threads <= 256 ? MX_NORM_CASE(2, 256) : MX_NORM_CASE(2, 512);
        case 3: return threads <= 256 ? MX_NORM_CASE(3, 256) : MX_NORM_CASE(3, 512);
        case 5: return MX_NORM_CASE(5, 256);
        default:
            return threads <= 256   ? MX_NORM_CASE(4, 256)
                   : threads <= 512 ? MX_NORM_CASE(4, 512)
                                    : MX_NORM_CASE(4, 1024);
    }
#undef MX_NORM_CASE
}

constexpr int kGradBlocks = 304;  // of the direct gradient kernel, at most
constexpr int kRingBlocks = 160;  // one per SM; devices with more SMs take the direct kernel
constexpr int kRingThreads = 512;
constexpr size_t kRingSmem = 220 * 1024;

RowShape grad_shape(int64_t T, int64_t K) {
    const int64_t n = padded_chunks(K);
    RowShape s = n <= 160 ? row_shape(n, static_cast<int>(n / 32), 256) : row_shape(n, n <= 512 ? 2 : 4, 256);
    if (T < s.groups) s.groups = static_cast<int>(T);
    s.smem = s.groups > 1 ? s.groups * static_cast<size_t>(K) * 4 : 0;
    return s;
}
int64_t grad_grid(int64_t T, const RowShape &s) {
    const int64_t want = (T + s.groups - 1) / s.groups;
    return want < kGradBlocks ? want : kGradBlocks;
}

// The ring's shape for rows of `bytes`, or stages = 0 where it does not apply: one
// warp a row up to 160 chunks; then two chunks a thread, or three or four where
// that gives an SM two rows at a time (bf16 8192 columns: 85% of a plain copy's
// rate, 76% with one row at a time; fp32 dy 5120 columns: 90%, 75%).
RowShape ring_shape(int64_t T, int64_t K, size_t bytes, const DeviceInfo &dev) {
    const int64_t n = padded_chunks(K);
    const int slots = static_cast<int>((kRingSmem - 4096) / (bytes + 8));
    RowShape s{};
    if (dev.sm_count > kRingBlocks) return s;
    for (int c = n <= 160 ? static_cast<int>(n / 32) : n <= 1024 ? 2 : 4; c <= 5; ++c) {
        RowShape t = row_shape(n, c, 256);
        t.groups = kRingThreads / t.tpr < slots / 2 ? kRingThreads / t.tpr : slots / 2;
        if (t.groups < 1) continue;
        if (s.groups == 0) s = t;
        if (t.groups >= 2) s = t;
        if (n <= 160 || s.groups >= 2 || c == 4) break;
    }
    // It pays from one row a group on (1024 rows of 2048 columns, bf16 stream: 7.4 us,
    // 7.9 us directly), two for one-warp rows (4096 of 512: 6.9 us directly, 7.4 us).
    if (s.groups < 1 || T < (s.tpr == 32 ? 2ll : 1ll) * s.groups * dev.sm_count) return s;
    s.stages = slots / s.groups < 8 ? slots / s.groups : 8;
    s.smem = s.groups * (s.stages * (bytes + 8) + 256);
    return s;
}

template <typename D, typename S>
cudaError_t launch_norm_grad(NormGradArgs &p, int64_t *n_parts, const DeviceInfo &dev,
                             cudaStream_t stream) {
    RowShape s = ring_shape(
        p.T, p.K, static_cast<size_t>(p.K) * (D::kBytes + (p.dres != nullptr ? 2 : 1) * S::kBytes), dev);
    const bool ring = s.stages > 0;
    if (!ring) s = grad_shape(p.T, p.K);
    p.tpr = s.tpr;
    p.stages = s.stages;
    const int64_t grid = ring ? dev.sm_count : grad_grid(p.T, s);
    *n_parts = grid;
    p.parts.bytes = static_cast<size_t>(grid) * p.K * 4;
    const int threads = s.tpr * s.groups;
    auto go = [&](auto kernel) { return launch_dependent(kernel, grid, threads, s.smem, stream, p); };
    if (ring) {
        // The limit is the kernel's, not the call's: always the same one.
        auto large = [&](auto kernel) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(kRingSmem));
            return e != cudaSuccess ? e : go(kernel);
        };
        if (s.tpr > 32 && s.c == 2) return large(mx_rmsnorm_backward_ring_kernel<D, S, 2, kRingThreads, false>);
        switch (s.c) {
            case 1: return large(mx_rmsnorm_backward_ring_kernel<D, S, 1, kRingThreads, true>);
            case 2: return large(mx_rmsnorm_backward_ring_kernel<D, S, 2, kRingThreads, true>);
            case 3: return large(mx_rmsnorm_backward_ring_kernel<D, S, 3, kRingThreads, true>);
            case 4: return large(mx_rmsnorm_backward_ring_kernel<D, S, 4, kRingThreads, true>);
            default: return large(mx_rmsnorm_backward_ring_kernel<D, S, 5, kRingThreads, true>);
        }
    }
    switch (s.c) {
        case 1: return go(mx_rmsnorm_backward_kernel<D, S, 1, 256, false>);
        case 2: return go(mx_rmsnorm_backward_kernel<D, S, 2, 256, false>);
        case 3: return go(mx_rmsnorm_backward_kernel<D, S, 3, 256, false>);
        case 5: return go(mx_rmsnorm_backward_kernel<D, S, 5, 256, false>);
        default:
            return threads <= 256   ? go(mx_rmsnorm_backward_kernel<D, S, 4, 256, false>)
                   : threads <= 512 ? go(mx_rmsnorm_backward_kernel<D, S, 4, 512, true>)
                                    : go(mx_rmsnorm_backward_kernel<D, S, 4, 1024, true>);
    }
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
    p.x_pitch = x.pitch * (x.f32 ? 4 : 2);
    p.res_pitch = res.pitch * (res.f32 ? 4 : 2);
    p.h_pitch = h_pitch * (res.f32 ? 4 : 2);
    p.aligned32 = aligned32(x.p) && aligned32(res.p) && aligned32(h);
    const size_t sb = res.f32 ? 4 : 2;
    p.h = {static_cast<uint8_t *>(h), (static_cast<size_t>(T - 1) * h_pitch + K) * sb};
    p.y = {static_cast<uint8_t *>(y), static_cast<size_t>(T) * K * 2};
    p.rstd = {reinterpret_cast<uint8_t *>(rstd), static_cast<size_t>(T) * 4};
    p.enc = row_encoded(e, T, K);
    p.T = T;
    p.K = static_cast<uint32_t>(K);
    p.eps = eps;
    p.w_f32 = w_f32;
    p.status = dev.status;
    if (res.p == nullptr) return x.f32 ? launch_norm<F32, F32, false>(p, dev, stream)
                                       : launch_norm<BF16, BF16, false>(p, dev, stream);
    if (x.f32) return res.f32 ? launch_norm<F32, F32, true>(p, dev, stream)
                              : launch_norm<F32, BF16, true>(p, dev, stream);
    return res.f32 ? launch_norm<BF16, F32, true>(p, dev, stream)
                   : launch_norm<BF16, BF16, true>(p, dev, stream);
}

size_t rmsnorm_backward_ws(int64_t T, int64_t K) {
    // One partial for each block of either kernel.
    const int64_t direct = grad_grid(T, grad_shape(T, K)), ring = T < kRingBlocks ? T : kRingBlocks;
    return static_cast<size_t>(direct > ring ? direct : ring) * static_cast<size_t>(K) * 4;
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
    p.dy_pitch = dy.pitch * (dy.f32 ? 4 : 2);
    p.h_pitch = h.pitch * (h.f32 ? 4 : 2);
    p.dres_pitch = dres.pitch * (h.f32 ? 4 : 2);
    p.dx_pitch = dx_pitch * (h.f32 ? 4 : 2);
    p.aligned32 = aligned32(dy.p) && aligned32(h.p) && aligned32(dres.p) && aligned32(dx);
    p.dx = {static_cast<uint8_t *>(dx),
            (static_cast<size_t>(T - 1) * dx_pitch + K) * static_cast<size_t>(h.f32 ? 4 : 2)};
    p.parts.p = dw != nullptr ? static_cast<uint8_t *>(ws) : nullptr;
    p.T = T;
    p.K = static_cast<uint32_t>(K);
    p.w_f32 = w_f32;
    p.status = dev.status;
    int64_t n = 0;
    const cudaError_t e = dy.f32 ? (h.f32 ? launch_norm_grad<F32, F32>(p, &n, dev, stream)
                                          : launch_norm_grad<F32, BF16>(p, &n, dev, stream))
                                 : (h.f32 ? launch_norm_grad<BF16, F32>(p, &n, dev, stream)
                                          : launch_norm_grad<BF16, BF16>(p, &n, dev, stream));
    if (e != cudaSuccess || dw == nullptr) return e;
    return launch_dependent(mx_rmsnorm_dw_kernel, (K + 31) / 32, 1024, 0, stream,
                            static_cast<const float *>(ws), static_cast<int>(n), static_cast<uint32_t>(K),
                            Out{reinterpret_cast<uint8_t *>(dw), static_cast<size_t>(K) * 4},
                            dev.status);
}

}  // namespace mx
