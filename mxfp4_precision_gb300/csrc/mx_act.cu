// mx_act.cu -- gradient of a product's bias and activation
// (mx_bias_act_backward):
//
//   dz = dy * act'(z),   dbias = sum over rows of dz
//
// One read of dy and z, one write of dz; the columns' sums ride along.  A block is a
// strip of 256 columns (a warp: 32 lanes of 8 columns, so a 32-column block
// is four lanes) and a share of the rows; its warps take rows in turn, each
// lane adds its columns up in fp32, the block's warps are joined in shared
// memory and leave one partial row per share.  A second launch adds the
// shares in their order, so the same inputs give the same bits.  A call of few rows is one
// share of 16 warps, which writes dbias itself.  Bound by memory: 8192 x 14336 with fp32 dy and
// gelu 143 us, 940 MB = 6.6 TB/s (97% of a plain copy's rate); bf16 dy 130 us, where gelu's
// instructions show (relu 112 us).
#include <cstdint>
#include <cuda_runtime.h>

#include "mx_act.cuh"
#include "mx_internal.h"
#include "mx_ptx.cuh"
#include "mx_rows.cuh"

namespace mx {
namespace {

using namespace rows;

constexpr int kStrip = 256;      // columns of a block
constexpr int kMaxShares = 128;  // partial rows of dbias

struct ActGradArgs {
    const uint8_t *dy, *z;
    int64_t dy_pitch, z_pitch;  // bytes
    Out dz, sums;               // sums: dbias, or the shares' partial rows
    Encoded enc;
    int64_t T;
    uint32_t N;
    int act;
    int strips;
    int64_t share;              // rows of a block
    uint32_t tiles;             // blocks that hold rows; those after them zero the scales' padding lines
    bool aligned32;
    int *status;
};

template <int ACT>
__device__ __forceinline__ void slopes(const V8 &z, V8 &d) {
#pragma unroll
    for (int i = 0; i < 4; ++i) d.v[i] = mul2(d.v[i], act::slope2<ACT>(z.v[i]));
}

// Two rows in flight a warp and four blocks an SM: with four rows, whose registers leave two
// blocks, gelu's slope waits for its own instructions (fp32 dy, 8192 x 14336: 160 us, 143 us).
// The few rows of a small call are all read at once.
template <typename D, typename Z, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 8 ? 4 : 1) mx_bias_act_backward_kernel(const __grid_constant__ ActGradArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x >= p.tiles) {
        zero_padding(p.enc, p.T, static_cast<int64_t>(blockIdx.x - p.tiles) * blockDim.x + threadIdx.x,
                     static_cast<int64_t>(gridDim.x - p.tiles) * blockDim.x, p.status);
        return;
    }
    const uint32_t share = blockIdx.x / p.strips, strip = blockIdx.x - share * p.strips;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t c = strip * (kStrip / 8) + lane, col = 8 * c;
    const bool in = col < p.N;
    const int64_t first = static_cast<int64_t>(share) * p.share;
    const int64_t end = min(p.T, first + p.share);
    const uint8_t *dy = p.dy + static_cast<size_t>(col) * D::kBytes;
    const uint8_t *z = p.z + static_cast<size_t>(col) * Z::kBytes;
    constexpr int kAhead = WARPS == 8 ? 2 : 4;  // rows in flight
    V8 sum = zero_v8();
    for (int64_t row = first + warp; row < end; row += kAhead * WARPS) {
        Raw8<D> dr[kAhead];
        Raw8<Z> zr[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t r = row + k * WARPS;
            zero8(dr[k]);
            zero8(zr[k]);
            if (in && r < end) {
                load8(dr[k], dy + r * p.dy_pitch, p.aligned32);
                if (p.act != act::kNone) load8(zr[k], z + r * p.z_pitch, p.aligned32);
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t r = row + k * WARPS;
            if (r >= end) break;
            V8 g = to_v8(dr[k]);
            const V8 x = to_v8(zr[k]);
            switch (p.act) {
                case act::kRelu: slopes<act::kRelu>(x, g); break;
                case act::kRelu2: slopes<act::kRelu2>(x, g); break;
                case act::kGelu: slopes<act::kGelu>(x, g); break;
                case act::kGeluTanh: slopes<act::kGeluTanh>(x, g); break;
                case act::kSilu: slopes<act::kSilu>(x, g); break;
                default: break;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sum.v[i] = add2(sum.v[i], g.v[i]);
            if (in && p.dz.p != nullptr) store8<BF16>(p.dz, p.dz.p + (r * p.N + col) * 2, g, true, p.status);
            if (p.enc.fmt != kEncNone && c < p.enc.katoms * 16)
                encode8(p.enc, encoded_row(p.enc, r), c, in, g, p.status);
        }
    }
    if (p.sums.p == nullptr) return;
    // The warps' sums of a column, in the warps' order.
    __shared__ float part[WARPS][kStrip + 4];
    float s[8];
    floats_of(sum, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) part[warp][8 * lane + i] = s[i];
    __syncthreads();
    for (int i = threadIdx.x; i < kStrip; i += 32 * WARPS) {
        const uint32_t at = strip * kStrip + i;
        if (at >= p.N) break;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += part[w][i];
        uint8_t *d = p.sums.p + (static_cast<size_t>(share) * p.N + at) * 4;
        if (MX_STORE_OK(d, 4, p.sums.p, p.sums.bytes, p.status)) *reinterpret_cast<float *>(d) = v;
    }
}

// dbias = the shares' partial rows, added in their order: eight groups of shares at a
// time, then the groups.
__global__ void __launch_bounds__(256) mx_bias_sum_kernel(const float *part, int shares, uint32_t N, Out dbias,
                                                          int *status) {
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t col = blockIdx.x * 32 + (threadIdx.x & 31);
    const int group = threadIdx.x >> 5;
    __shared__ float joined[8][32];
    float v = 0.0f;
    if (col < N) {
        const int each = (shares + 7) / 8, end = min(shares, (group + 1) * each);
#pragma unroll 8
        for (int i = group * each; i < end; ++i) v += part[static_cast<size_t>(i) * N + col];
    }
    joined[group][threadIdx.x & 31] = v;
    __syncthreads();
    if (group != 0 || col >= N) return;
    v = 0.0f;
#pragma unroll
    for (int g = 0; g < 8; ++g) v += joined[g][threadIdx.x];
    uint8_t *d = dbias.p + 4 * static_cast<size_t>(col);
    if (MX_STORE_OK(d, 4, dbias.p, dbias.bytes, status)) *reinterpret_cast<float *>(d) = v;
}

// Rows of a share: a few rows are one share; more are cut so that every SM has blocks
// enough, into at most kMaxShares.
constexpr int64_t kFewRows = 128;
int64_t share_rows(int64_t T, int64_t N) {
    if (T <= kFewRows) return kFewRows;
    const int64_t strips = (N + kStrip - 1) / kStrip;
    int64_t rows = 256;
    while (rows > 32 && (T + rows - 1) / rows * strips < 152 * 8) rows /= 2;
    while ((T + rows - 1) / rows > kMaxShares) rows *= 2;
    return rows;
}

template <typename D, typename Z>
cudaError_t launch(const ActGradArgs &p, int64_t pad_words, bool few, cudaStream_t stream) {
    const int threads = few ? 512 : 256;
    const int64_t grid = p.tiles + (pad_words + threads - 1) / threads;
    return few ? launch_dependent(mx_bias_act_backward_kernel<D, Z, 16>, grid, threads, 0, stream, p)
               : launch_dependent(mx_bias_act_backward_kernel<D, Z, 8>, grid, threads, 0, stream, p);
}

}  // namespace

size_t bias_act_backward_ws(int64_t T, int64_t N) {
    const int64_t rows = share_rows(T, N), shares = (T + rows - 1) / rows;
    return shares <= 1 ? 0 : static_cast<size_t>(shares) * static_cast<size_t>(N) * sizeof(float);
}

cudaError_t launch_bias_act_backward(const RowIn &dy, const RowIn &z, int act, int64_t T, int64_t N, void *dz,
                                     const RowEncode &e, float *dbias, void *ws, const DeviceInfo &dev,
                                     cudaStream_t stream) {
    ActGradArgs p{};
    p.dy = static_cast<const uint8_t *>(dy.p);
    p.dy_pitch = dy.pitch * (dy.f32 ? 4 : 2);
    p.z = static_cast<const uint8_t *>(z.p);
    p.z_pitch = z.pitch * (z.f32 ? 4 : 2);
    p.dz = {static_cast<uint8_t *>(dz), static_cast<size_t>(T) * N * 2};
    p.enc = row_encoded(e, T, N);
    p.T = T;
    p.N = static_cast<uint32_t>(N);
    p.act = act;
    p.strips = static_cast<int>((N + kStrip - 1) / kStrip);
    p.share = share_rows(T, N);
    const int64_t shares = (T + p.share - 1) / p.share;
    if (dbias != nullptr)
        p.sums = shares == 1 ? Out{reinterpret_cast<uint8_t *>(dbias), static_cast<size_t>(N) * 4}
                             : Out{static_cast<uint8_t *>(ws), bias_act_backward_ws(T, N)};
    if (shares * p.strips > 0x3FFFFFFF) return cudaErrorInvalidValue;
    p.tiles = static_cast<uint32_t>(shares * p.strips);
    p.aligned32 = aligned32(dy.p) && aligned32(z.p);
    p.status = dev.status;
    const int64_t pad = padding_words(p.enc, T);
    const bool few = T <= kFewRows;
    cudaError_t err = dy.f32 ? (z.f32 ? launch<F32, F32>(p, pad, few, stream) : launch<F32, BF16>(p, pad, few, stream))
                             : (z.f32 ? launch<BF16, F32>(p, pad, few, stream) : launch<BF16, BF16>(p, pad, few, stream));
    if (err != cudaSuccess || dbias == nullptr || shares == 1) return err;
    return launch_dependent(mx_bias_sum_kernel, (N + 31) / 32, 256, 0, stream, static_cast<const float *>(ws),
                            static_cast<int>(shares), p.N, Out{reinterpret_cast<uint8_t *>(dbias), static_cast<size_t>(N) * 4},
                            dev.status);
}

}  // namespace mx
