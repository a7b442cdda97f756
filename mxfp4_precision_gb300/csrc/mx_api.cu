// mx_api.cu -- the library's C ABI (include/mx.h): argument checks, workspace
// carving, tensor-map encoding, per-device status word, and the launches.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "../../include/mx.h"
#include <nvtx3/nvToolsExt.h>
#include "mx_internal.h"
#include "mx_ptx.cuh"

// One status word per device (lives as long as the module is loaded).
static __device__ int g_mx_status;

namespace mx {
namespace {

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
DeviceInfo g_devices[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

bool load_encode_fn() {
    if (g_encode != nullptr) return true;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
        return false;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    return true;
}

__global__ void timeout_probe_kernel(int *status, uint64_t limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
    }
    __syncthreads();
    // Nothing ever arrives on `bar`: the bounded wait must give up.
    if (threadIdx.x == 0) mbar_wait(&bar, 0, status, nullptr, limit_ns);
    __syncthreads();
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool valid_rot(int rot, int rot_block) {
    if (rot == MX_ROT_NONE) return true;
    if (rot != MX_ROT_HADAMARD_DET && rot != MX_ROT_HADAMARD_RAND) return false;
    return rot_block == 16 || rot_block == 32 || rot_block == 64 || rot_block == 128 ||
           rot_block == 256;
}
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

mx_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MX_OK : MX_ERR_CUDA; }

// Checks shared by every encode: enums, shape (contraction length multiple of
// 32 and of rot_block), pointer alignment.
mx_status check_encode(const void *src, int64_t rows, int64_t cols, int contract, int rot,
                       int rot_block, int rnd, const void *codes, const void *scales) {
    if (contract != MX_CONTRACT_ROWS && contract != MX_CONTRACT_COLS) return MX_ERR_INVALID_ARG;
    if (!valid_rot(rot, rot_block)) return MX_ERR_INVALID_ARG;
    if (rnd != MX_ROUND_RNE && rnd != MX_ROUND_SR) return MX_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0) return MX_ERR_SHAPE;
    if (rows > 0x7FFFFFFF || cols > 0x7FFFFFFF) return MX_ERR_SHAPE;
    if (rows == 0 || cols == 0) return MX_OK;
    if (src == nullptr || codes == nullptr || scales == nullptr) return MX_ERR_INVALID_ARG;
    const int64_t L = contract == MX_CONTRACT_ROWS ? rows : cols;
    if (L % 32 != 0) return MX_ERR_SHAPE;
    if (rot != MX_ROT_NONE && L % rot_block != 0) return MX_ERR_SHAPE;
    if (!aligned16(src) || !aligned16(codes) || !aligned16(scales)) return MX_ERR_ALIGN;
    if (cols % 8 != 0) return MX_ERR_ALIGN;  // 16-byte rows for the TMA
    return MX_OK;
}

mx_status check_gemm(const void *Aq, const void *As, const void *Bq, const void *Bs,
                     const float *C, int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0) return MX_ERR_SHAPE;
    if (M > 0x7FFFFFFF || N > 0x7FFFFFFF || K > 0x7FFFFFFF) return MX_ERR_SHAPE;
    if (M == 0 || N == 0) return MX_OK;
    if (C == nullptr) return MX_ERR_INVALID_ARG;
    if (K % 32 != 0) return MX_ERR_SHAPE;
    if (N % 4 != 0 || !aligned16(C)) return MX_ERR_ALIGN;
    if (K == 0) return MX_OK;
    if (!Aq || !As || !Bq || !Bs) return MX_ERR_INVALID_ARG;
    if (!aligned16(Aq) || !aligned16(As) || !aligned16(Bq) || !aligned16(Bs)) return MX_ERR_ALIGN;
    return MX_OK;
}

// Lines and contraction length of both operands of a linear op.
struct OpShape {
    int64_t a_lines, b_lines, k;
};
bool op_shape(int op, int64_t T, int64_t N, int64_t K, OpShape *s) {
    switch (op) {
        case MX_OP_FPROP: *s = {T, N, K}; return true;
        case MX_OP_DGRAD: *s = {T, K, N}; return true;
        case MX_OP_WGRAD: *s = {N, K, T}; return true;
        default: return false;
    }
}

}  // namespace

const DeviceInfo *current_device(cudaError_t *err) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        *err = e != cudaSuccess ? e : cudaErrorInvalidDevice;
        return nullptr;
    }
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceInfo &d = g_devices[dev];
    if (d.ordinal == dev) return &d;
    cudaDeviceProp prop;
    if ((e = cudaGetDeviceProperties(&prop, dev)) != cudaSuccess) {
        *err = e;
        return nullptr;
    }
    void *status = nullptr;
    if ((e = cudaGetSymbolAddress(&status, g_mx_status)) != cudaSuccess) {
        *err = e;
        return nullptr;
    }
    if (!load_encode_fn()) {
        *err = cudaErrorSymbolNotFound;
        return nullptr;
    }
    d.sm_count = prop.multiProcessorCount;
    d.cc_major = prop.major;
    d.cc_minor = prop.minor;
    d.status = static_cast<int *>(status);
    d.ordinal = dev;
    return &d;
}

bool encode_tmap_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base,
                    uint64_t inner_elems, uint64_t outer_elems, uint64_t row_bytes,
                    uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle) {
    if (g_encode == nullptr) return false;
    cuuint64_t dims[2] = {inner_elems, outer_elems};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = g_encode(map, dtype, 2, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool encode_tmap_lines64(CUtensorMap *map, const void *base, uint64_t row_bytes, uint64_t lines,
                         uint32_t box_inner, uint32_t box_lines, CUtensorMapSwizzle swizzle) {
    if (g_encode == nullptr) return false;
    cuuint64_t dims[5] = {row_bytes, 2, 4, 8, lines / 64};
    cuuint64_t strides[4] = {row_bytes, 16 * row_bytes, 2 * row_bytes, 64 * row_bytes};
    cuuint32_t box[5] = {box_inner, 2, 4, 8, box_lines / 64};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

}  // namespace mx

using namespace mx;

namespace {
mx_status device_or_error(const DeviceInfo **out) {
    cudaError_t e = cudaSuccess;
    const DeviceInfo *d = current_device(&e);
    if (d == nullptr) return MX_ERR_CUDA;
    if (!(d->cc_major == 10 && d->cc_minor == 3)) return MX_ERR_UNSUPPORTED;
    *out = d;
    return MX_OK;
}

mx_status quantize_impl(const void *src, int64_t rows, int64_t cols, int contract, int rot,
                        int rot_block, int rnd, uint64_t seed, uint64_t sr_tag, void *codes,
                        void *scales, cudaStream_t stream) {
    mx_status st = check_encode(src, rows, cols, contract, rot, rot_block, rnd, codes, scales);
    if (st != MX_OK || rows == 0 || cols == 0) return st;
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_quantize(src, rows, cols, contract, rot, rot_block, rnd, seed, sr_tag,
                                     codes, scales, *dev, stream));
}

mx_status quantize_pair_impl(const void *src0, int64_t rows0, int64_t cols0, const void *src1,
                             int64_t rows1, int64_t cols1, int rot, int rot_block, int rnd,
                             uint64_t seed, void *codes0, void *scales0, void *codes1,
                             void *scales1, cudaStream_t stream) {
    if (rows0 != rows1) return MX_ERR_SHAPE;
    mx_status st = check_encode(src0, rows0, cols0, MX_CONTRACT_ROWS, rot, rot_block, rnd, codes0,
                                scales0);
    if (st != MX_OK) return st;
    st = check_encode(src1, rows1, cols1, MX_CONTRACT_ROWS, rot, rot_block, rnd, codes1, scales1);
    if (st != MX_OK) return st;
    const bool e0 = rows0 == 0 || cols0 == 0, e1 = rows1 == 0 || cols1 == 0;
    if (e0 && e1) return MX_OK;
    if (e0 || e1)  // one side empty: plain single-operand encode of the other
        return e0 ? quantize_impl(src1, rows1, cols1, MX_CONTRACT_ROWS, rot, rot_block, rnd, seed,
                                  2, codes1, scales1, stream)
                  : quantize_impl(src0, rows0, cols0, MX_CONTRACT_ROWS, rot, rot_block, rnd, seed,
                                  1, codes0, scales0, stream);
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_quantize_pair_colwise(src0, rows0, cols0, src1, rows1, cols1, rot,
                                                  rot_block, rnd, seed, codes0, scales0, codes1,
                                                  scales1, *dev, stream));
}

mx_status quantize_dual_impl(const void *src, int64_t T, int64_t N, int rot, int rot_block,
                             int rnd, uint64_t seed, void *codes_t, void *scales_t, void *codes_n,
                             void *scales_n, cudaStream_t stream) {
    mx_status st = check_encode(src, T, N, MX_CONTRACT_ROWS, rot, rot_block, rnd, codes_t,
                                scales_t);
    if (st != MX_OK) return st;
    st = check_encode(src, T, N, MX_CONTRACT_COLS, MX_ROT_NONE, 32, rnd, codes_n, scales_n);
    if (st != MX_OK || T == 0 || N == 0) return st;
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_quantize_dual(src, T, N, rot, rot_block, rnd, seed, codes_t, scales_t,
                                          codes_n, scales_n, *dev, stream));
}

mx_status gemm_impl(const void *Aq, const void *As, const void *Bq, const void *Bs, float *C,
                    int64_t M, int64_t N, int64_t K, cudaStream_t stream) {
    mx_status st = check_gemm(Aq, As, Bq, Bs, C, M, N, K);
    if (st != MX_OK || M == 0 || N == 0) return st;
    if (K == 0)
        return from_cuda(cudaMemsetAsync(C, 0, static_cast<size_t>(M) * N * sizeof(float), stream));
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_gemm(Aq, As, Bq, Bs, C, M, N, K, *dev, stream));
}

// MXFP8 comparator: encode down the rows of one or two operands, contract.
mx_status quantize_mxfp8_impl(const void *src0, int64_t rows0, int64_t cols0, const void *src1,
                              int64_t rows1, int64_t cols1, void *codes0, void *scales0,
                              void *codes1, void *scales1, cudaStream_t stream) {
    mx_status st = check_encode(src0, rows0, cols0, MX_CONTRACT_ROWS, MX_ROT_NONE, 32,
                                MX_ROUND_RNE, codes0, scales0);
    if (st != MX_OK) return st;
    if (src1 != nullptr) {
        st = check_encode(src1, rows1, cols1, MX_CONTRACT_ROWS, MX_ROT_NONE, 32, MX_ROUND_RNE,
                          codes1, scales1);
        if (st != MX_OK) return st;
        if (rows1 == 0 || cols1 == 0) src1 = nullptr;
    }
    if (rows0 == 0 || cols0 == 0) {
        if (src1 == nullptr) return MX_OK;
        src0 = src1, rows0 = rows1, cols0 = cols1, codes0 = codes1, scales0 = scales1;
        src1 = nullptr;
    }
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_quantize_mxfp8_colwise(src0, rows0, cols0, src1, rows1, cols1, codes0,
                                                   scales0, codes1, scales1, *dev, stream));
}

mx_status gemm_mxfp8_impl(const void *Aq, const void *As, const void *Bq, const void *Bs,
                          float *C, int64_t M, int64_t N, int64_t K, cudaStream_t stream) {
    mx_status st = check_gemm(Aq, As, Bq, Bs, C, M, N, K);
    if (st != MX_OK || M == 0 || N == 0) return st;
    if (K == 0)
        return from_cuda(cudaMemsetAsync(C, 0, static_cast<size_t>(M) * N * sizeof(float), stream));
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_gemm_fmt(kGemmMXFP8, Aq, As, Bq, Bs, C, M, N, K, nullptr, nullptr,
                                     *dev, stream));
}

// NVFP4 variant: encode down the rows of one or two operands (two launches:
// tensor amax, then the encode), contract with the tensor scales.
mx_status quantize_nvfp4_impl(const void *src0, int64_t rows0, int64_t cols0, const void *src1,
                              int64_t rows1, int64_t cols1, int rot, int rot_block, uint64_t seed,
                              void *codes0, void *scales0, void *codes1, void *scales1,
                              float *amax, cudaStream_t stream) {
    mx_status st = check_encode(src0, rows0, cols0, MX_CONTRACT_ROWS, rot, rot_block,
                                MX_ROUND_RNE, codes0, scales0);
    if (st != MX_OK) return st;
    if (rot != MX_ROT_NONE && rot_block != 16 && rot_block != 32) return MX_ERR_UNSUPPORTED;
    if (src1 != nullptr) {
        st = check_encode(src1, rows1, cols1, MX_CONTRACT_ROWS, rot, rot_block, MX_ROUND_RNE,
                          codes1, scales1);
        if (st != MX_OK) return st;
        if (rows1 == 0 || cols1 == 0) return MX_ERR_SHAPE;
    }
    if (rows0 == 0 || cols0 == 0) return src1 == nullptr ? MX_OK : MX_ERR_SHAPE;
    if (amax == nullptr) return MX_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(amax) & 7u) != 0) return MX_ERR_ALIGN;
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_quantize_nvfp4_colwise(src0, rows0, cols0, src1, rows1, cols1, rot,
                                                   rot_block, seed, codes0, scales0, codes1,
                                                   scales1, amax, *dev, stream));
}

mx_status gemm_nvfp4_impl(const void *Aq, const void *As, const float *amax_a, const void *Bq,
                          const void *Bs, const float *amax_b, float *C, int64_t M, int64_t N,
                          int64_t K, cudaStream_t stream) {
    mx_status st = check_gemm(Aq, As, Bq, Bs, C, M, N, K);
    if (st != MX_OK || M == 0 || N == 0) return st;
    if (K == 0)
        return from_cuda(cudaMemsetAsync(C, 0, static_cast<size_t>(M) * N * sizeof(float), stream));
    if (amax_a == nullptr || amax_b == nullptr) return MX_ERR_INVALID_ARG;
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_gemm_fmt(kGemmNVFP4, Aq, As, Bq, Bs, C, M, N, K, amax_a, amax_b,
                                     *dev, stream));
}

// Quantise both operands of a linear op into the workspace, then contract.
mx_status linear_impl(int op, const void *a_src, int64_t a_rows, int64_t a_cols, int a_contract,
                      const void *b_src, int64_t b_rows, int64_t b_cols, int b_contract, float *out,
                      int64_t T, int64_t N, int64_t K, int rot, int rot_block, int rnd,
                      uint64_t seed, void *ws, size_t ws_bytes, cudaStream_t stream,
                      bool fused = false) {
    OpShape s;
    if (!op_shape(op, T, N, K, &s)) return MX_ERR_INVALID_ARG;
    if (T < 0 || N < 0 || K < 0) return MX_ERR_SHAPE;
    if (s.a_lines == 0 || s.b_lines == 0) return MX_OK;
    if (out == nullptr) return MX_ERR_INVALID_ARG;
    if (s.k == 0) return gemm_impl(nullptr, nullptr, nullptr, nullptr, out, s.a_lines, s.b_lines, 0, stream);
    // Operand checks (the workspace is checked separately below).
    mx_status st = check_encode(a_src, a_rows, a_cols, a_contract, rot, rot_block, rnd, a_src,
                                a_src);
    if (st != MX_OK) return st;
    st = check_encode(b_src, b_rows, b_cols, b_contract, rot, rot_block, rnd, b_src, b_src);
    if (st != MX_OK) return st;
    if (s.b_lines % 4 != 0 || !aligned16(out)) return MX_ERR_ALIGN;
    const size_t need = mx_linear_workspace_bytes(op, T, N, K);
    if (ws == nullptr || ws_bytes < need) return MX_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MX_ERR_ALIGN;
    uint8_t *p = static_cast<uint8_t *>(ws);
    uint8_t *aq = p;
    p += align256(mx_codes_bytes(s.a_lines, s.k));
    uint8_t *as = p;
    p += align256(mx_scales_bytes(s.a_lines, s.k));
    uint8_t *bq = p;
    p += align256(mx_codes_bytes(s.b_lines, s.k));
    uint8_t *bs = p;
    if (fused) {
        // One launch: the GEMM's own encoder warps encode both operands while
        // it runs (its chunk counters, after the operands in the workspace,
        // are zeroed first).
        if (op != MX_OP_WGRAD || !wgrad_fusable(T, N, K, rot, rot_block, rnd))
            return MX_ERR_UNSUPPORTED;
        const DeviceInfo *dev = nullptr;
        if ((st = device_or_error(&dev)) != MX_OK) return st;
        uint8_t *counters = bs + align256(mx_scales_bytes(s.b_lines, s.k));
        return from_cuda(launch_wgrad_fused(a_src, b_src, out, T, N, K, rot, rot_block, aq, as, bq,
                                            bs, counters, *dev, stream));
    }
    if (a_contract == MX_CONTRACT_ROWS && b_contract == MX_CONTRACT_ROWS) {
        // Wgrad: both operands encoded down their rows in a single launch.
        st = quantize_pair_impl(a_src, a_rows, a_cols, b_src, b_rows, b_cols, rot, rot_block, rnd,
                                seed, aq, as, bq, bs, stream);
    } else {
        st = quantize_impl(a_src, a_rows, a_cols, a_contract, rot, rot_block, rnd, seed, 1, aq, as,
                           stream);
        if (st == MX_OK)
            st = quantize_impl(b_src, b_rows, b_cols, b_contract, rot, rot_block, rnd, seed, 2,
                               bq, bs, stream);
    }
    if (st != MX_OK) return st;
    return gemm_impl(aq, as, bq, bs, out, s.a_lines, s.b_lines, s.k, stream);
}
}  // namespace

namespace {
// ---- operators between the GEMMs
bool valid_type(int t) { return t == MX_TYPE_BF16 || t == MX_TYPE_F32; }

mx_status check_row_sizes(int64_t T, int64_t cols) {
    if (T < 0 || cols < 0 || T > 0x7FFFFFFF || cols > 0x3FFFFFFF) return MX_ERR_SHAPE;
    return MX_OK;
}

// A row-major matrix: 16-byte rows at a pitch that holds them.
mx_status check_rows(const void *p, int64_t pitch, int64_t cols) {
    if (p == nullptr) return MX_ERR_INVALID_ARG;
    if (pitch < cols || pitch > 0x7FFFFFFF) return MX_ERR_SHAPE;
    if (cols % 8 != 0 || pitch % 8 != 0 || !aligned16(p)) return MX_ERR_ALIGN;
    return MX_OK;
}

mx_status check_row_encode(const RowEncode &e, int64_t T, int64_t cols) {
    if (e.fmt == MX_FORMAT_NONE)
        return e.codes == nullptr && e.scales == nullptr ? MX_OK : MX_ERR_INVALID_ARG;
    if (e.fmt != MX_FORMAT_MXFP4 && e.fmt != MX_FORMAT_MXFP8) return MX_ERR_INVALID_ARG;
    if (cols % 32 != 0) return MX_ERR_SHAPE;
    if (T == 0 || cols == 0) return MX_OK;
    if (e.codes == nullptr || e.scales == nullptr) return MX_ERR_INVALID_ARG;
    return aligned16(e.codes) && aligned16(e.scales) ? MX_OK : MX_ERR_ALIGN;
}

// ---- products with an epilogue, and by expert
bool valid_act(int act) { return act >= MX_ACT_NONE && act <= MX_ACT_SILU; }

// Outputs and bias of a product of p.M x p.N; set in p.
mx_status check_epilogue(Product &p, const void *bias, int bias_type, int act, void *y, int y_type, void *z,
                         int format, void *codes, void *scales) {
    if (!valid_act(act) || (bias != nullptr && !valid_type(bias_type)) || (y != nullptr && !valid_type(y_type)))
        return MX_ERR_INVALID_ARG;
    if (p.M > 0 && p.N > 0 && y == nullptr && z == nullptr && format == MX_FORMAT_NONE) return MX_ERR_INVALID_ARG;
    p.enc = {format, codes, scales};
    mx_status st = check_row_sizes(p.M, p.N);
    if (st != MX_OK || (st = check_row_encode(p.enc, p.M, p.N)) != MX_OK) return st;
    if (!aligned16(bias) || !aligned16(y) || !aligned16(z)) return MX_ERR_ALIGN;
    p.bias = bias;
    p.bias_f32 = bias_type == MX_TYPE_F32;
    p.act = act;
    p.y = y;
    p.y_f32 = y_type == MX_TYPE_F32;
    p.z = z;
    return MX_OK;
}

// Operands and sizes.
mx_status check_product(Product &p, int operands) {
    if (operands != MX_FORMAT_MXFP4 && operands != MX_FORMAT_MXFP8) return MX_ERR_INVALID_ARG;
    p.fp8 = operands == MX_FORMAT_MXFP8;
    if (p.M < 0 || p.N < 0 || p.K < 0 || p.M > 0x7FFFFF00 || p.N > 0x3FFFFFFF || p.K > 0x7FFFFFFF) return MX_ERR_SHAPE;
    if (p.M == 0 || p.N == 0) return MX_OK;
    if (p.K % 32 != 0) return MX_ERR_SHAPE;
    if (p.N % 8 != 0) return MX_ERR_ALIGN;
    if (p.K == 0) return MX_OK;
    if (!p.Aq || !p.As || !p.Bq || !p.Bs) return MX_ERR_INVALID_ARG;
    if (!aligned16(p.Aq) || !aligned16(p.As) || !aligned16(p.Bq) || !aligned16(p.Bs)) return MX_ERR_ALIGN;
    return MX_OK;
}

mx_status check_experts(int64_t experts, const int32_t *offsets) {
    if (experts < 1) return MX_ERR_SHAPE;
    if (experts > MX_EXPERTS_MAX) return MX_ERR_UNSUPPORTED;
    if (offsets == nullptr) return MX_ERR_INVALID_ARG;
    return aligned16(offsets) ? MX_OK : MX_ERR_ALIGN;
}

// A plan's sizes: entries and rows are counted in 32 bits.
mx_status check_expert_rows(const ExpertRows &r) {
    if (r.T < 0 || r.picks < 0 || r.rows < 0 || r.T > 0x7FFFFFFF || r.picks > 0x7FFFFFFF) return MX_ERR_SHAPE;
    if (r.T * r.picks > 0x7FFFFFFF || r.rows > 0x7FFFFFFF || r.rows % 128 != 0) return MX_ERR_SHAPE;
    return aligned16(r.slot) && aligned16(r.source) ? MX_OK : MX_ERR_ALIGN;
}

mx_status run_product(const Product &p, void *stream) {
    const DeviceInfo *dev = nullptr;
    const mx_status st = device_or_error(&dev);
    if (st != MX_OK) return st;
    const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    const cudaError_t e = few_rows(p) ? launch_few(p, *dev, st_) : launch_product(p, *dev, st_);
    return e == cudaErrorNotSupported ? MX_ERR_UNSUPPORTED : from_cuda(e);
}

mx_status experts_wgrad_impl(const void *Aq, const void *As, const void *Bq, const void *Bs, int operands,
                             const int32_t *offsets, int64_t experts, int64_t rows, int64_t M, int64_t N, void *C,
                             int c_type, void *stream) {
    Product p{};
    p.mode = kProductDepth;
    p.M = M, p.N = N, p.K = rows, p.experts = experts;
    p.Aq = Aq, p.As = As, p.Bq = Bq, p.Bs = Bs;
    p.offsets = offsets;
    if (!valid_type(c_type)) return MX_ERR_INVALID_ARG;
    mx_status st = check_product(p, operands);
    if (st != MX_OK) return st;
    if (rows % 128 != 0) return MX_ERR_SHAPE;
    if ((st = check_experts(experts, offsets)) != MX_OK || M == 0 || N == 0) return st;
    if (C == nullptr) return MX_ERR_INVALID_ARG;
    if (!aligned16(C)) return MX_ERR_ALIGN;
    p.y = C;
    p.y_f32 = c_type == MX_TYPE_F32;
    return run_product(p, stream);
}

mx_status grad_impl(const void *const *h_grads, const int64_t *h_sizes, const int *h_types,
                    void *const *h_outs, const int *h_out_types, int64_t count, bool scale,
                    float max_norm, float eps, float *d_norm, void *ws, size_t ws_bytes,
                    cudaStream_t stream) {
    if (count < 0 || count > (1 << 20)) return MX_ERR_SHAPE;
    if (d_norm == nullptr) return MX_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(d_norm) & 3u) != 0) return MX_ERR_ALIGN;
    if (count > 0 && (h_grads == nullptr || h_sizes == nullptr || h_types == nullptr))
        return MX_ERR_INVALID_ARG;
    if (h_outs != nullptr && h_out_types == nullptr) return MX_ERR_INVALID_ARG;
    std::vector<GradTensor> g;
    try {
        g.reserve(static_cast<size_t>(count));
    } catch (const std::bad_alloc &) {
        return MX_ERR_WORKSPACE;
    }
    for (int64_t i = 0; i < count; ++i) {
        if (!valid_type(h_types[i])) return MX_ERR_INVALID_ARG;
        if (h_sizes[i] < 0) return MX_ERR_SHAPE;
        if (h_sizes[i] == 0) continue;
        GradTensor t{h_grads[i], nullptr, h_sizes[i], h_types[i] == MX_TYPE_F32, false};
        if (t.p == nullptr) return MX_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(t.p) & (t.f32 ? 3u : 1u)) != 0) return MX_ERR_ALIGN;
        if (scale) {
            t.out = h_outs != nullptr ? h_outs[i] : const_cast<void *>(t.p);
            if (h_outs != nullptr && !valid_type(h_out_types[i])) return MX_ERR_INVALID_ARG;
            t.out_f32 = h_outs != nullptr ? h_out_types[i] == MX_TYPE_F32 : t.f32;
            if (t.out == nullptr || (t.out == t.p && t.out_f32 != t.f32)) return MX_ERR_INVALID_ARG;
            if ((reinterpret_cast<uintptr_t>(t.out) & (t.out_f32 ? 3u : 1u)) != 0)
                return MX_ERR_ALIGN;
        }
        g.push_back(t);
    }
    const int64_t n = static_cast<int64_t>(g.size());
    if (n == 0) return from_cuda(cudaMemsetAsync(d_norm, 0, sizeof(float), stream));
    if (ws == nullptr || ws_bytes < mx_grad_workspace_bytes(n)) return MX_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MX_ERR_ALIGN;
    const DeviceInfo *dev = nullptr;
    const mx_status st = device_or_error(&dev);
    if (st != MX_OK) return st;
    return from_cuda(launch_grad_clip(g.data(), n, scale, max_norm, eps, d_norm, ws, *dev, stream));
}
}  // namespace

namespace {
// Names each exported call in profiler timelines (NVTX; free without a tool attached).
struct TraceRange {
    explicit TraceRange(const char *name) { nvtxRangePushA(name); }
    ~TraceRange() { nvtxRangePop(); }
    TraceRange(const TraceRange &) = delete;
    TraceRange &operator=(const TraceRange &) = delete;
};
}  // namespace

extern "C" {

size_t mx_codes_bytes(int64_t mn, int64_t k) {
    if (mn <= 0 || k <= 0) return 0;
    return static_cast<size_t>(mn) * static_cast<size_t>(k / 2);
}

size_t mx_scales_bytes(int64_t mn, int64_t k) {
    if (mn <= 0 || k <= 0) return 0;
    return static_cast<size_t>(scale_groups(mn)) * 128u * static_cast<size_t>(8 * ((k + 255) / 256));
}

mx_status mx_quantize(const void *d_src, int64_t rows, int64_t cols, int contract, int rot,
                      int rot_block, int rnd, uint64_t seed, void *d_codes, void *d_scales,
                      void *stream) {
    TraceRange trace("mx_quantize");
    return quantize_impl(d_src, rows, cols, contract, rot, rot_block, rnd, seed, 1, d_codes,
                         d_scales, static_cast<cudaStream_t>(stream));
}

mx_status mx_quantize_pair(const void *d_src0, int64_t rows0, int64_t cols0, const void *d_src1,
                           int64_t rows1, int64_t cols1, int rot, int rot_block, int rnd,
                           uint64_t seed, void *d_codes0, void *d_scales0, void *d_codes1,
                           void *d_scales1, void *stream) {
    TraceRange trace("mx_quantize_pair");
    return quantize_pair_impl(d_src0, rows0, cols0, d_src1, rows1, cols1, rot, rot_block, rnd, seed,
                              d_codes0, d_scales0, d_codes1, d_scales1,
                              static_cast<cudaStream_t>(stream));
}

mx_status mx_quantize_dual(const void *d_src, int64_t T, int64_t N, int rot, int rot_block,
                           int rnd, uint64_t seed, void *d_codes_t, void *d_scales_t,
                           void *d_codes_n, void *d_scales_n, void *stream) {
    TraceRange trace("mx_quantize_dual");
    return quantize_dual_impl(d_src, T, N, rot, rot_block, rnd, seed, d_codes_t, d_scales_t,
                              d_codes_n, d_scales_n, static_cast<cudaStream_t>(stream));
}

mx_status mx_scales_to_canonical(const void *d_scales, int64_t lines, int64_t k, void *d_canon,
                                 void *stream) {
    TraceRange trace("mx_scales_to_canonical");
    if (lines < 0 || k < 0) return MX_ERR_SHAPE;
    if (k % 32 != 0) return MX_ERR_SHAPE;
    if (lines == 0 || k == 0) return MX_OK;
    if (d_scales == nullptr || d_canon == nullptr) return MX_ERR_INVALID_ARG;
    const DeviceInfo *dev = nullptr;
    mx_status st = device_or_error(&dev);
    if (st != MX_OK) return st;
    return from_cuda(launch_scales_to_canonical(d_scales, lines, k, d_canon, *dev,
                                                static_cast<cudaStream_t>(stream)));
}

mx_status mx_gemm(const void *d_Aq, const void *d_As, const void *d_Bq, const void *d_Bs,
                  float *d_C, int64_t M, int64_t N, int64_t K, void *stream) {
    TraceRange trace("mx_gemm");
    return gemm_impl(d_Aq, d_As, d_Bq, d_Bs, d_C, M, N, K, static_cast<cudaStream_t>(stream));
}

size_t mx_linear_workspace_bytes(int op, int64_t T, int64_t N, int64_t K) {
    OpShape s;
    if (!op_shape(op, T, N, K, &s)) return 0;
    size_t bytes = align256(mx_codes_bytes(s.a_lines, s.k)) + align256(mx_scales_bytes(s.a_lines, s.k)) +
                   align256(mx_codes_bytes(s.b_lines, s.k)) + align256(mx_scales_bytes(s.b_lines, s.k));
    // Wgrad: room for the fused launch's (panel, chunk) counters.
    if (op == MX_OP_WGRAD && T > 0 && N > 0 && K > 0) bytes += align256(wgrad_fused_counter_bytes(T, N, K));
    return bytes;
}

mx_status mx_linear_wgrad(const void *d_dY, const void *d_X, float *d_dW, int64_t T, int64_t N,
                          int64_t K, int rot, int rot_block, int rnd, uint64_t seed, void *d_ws,
                          size_t ws_bytes, void *stream) {
    TraceRange trace("mx_linear_wgrad");
    // dW[N][K] = dY^T X: both operands encoded down their rows (contraction T).
    return linear_impl(MX_OP_WGRAD, d_dY, T, N, MX_CONTRACT_ROWS, d_X, T, K, MX_CONTRACT_ROWS,
                       d_dW, T, N, K, rot, rot_block, rnd, seed, d_ws, ws_bytes,
                       static_cast<cudaStream_t>(stream));
}

mx_status mx_linear_fprop(const void *d_X, const void *d_W, float *d_Y, int64_t T, int64_t N,
                          int64_t K, int rot, int rot_block, int rnd, uint64_t seed, void *d_ws,
                          size_t ws_bytes, void *stream) {
    TraceRange trace("mx_linear_fprop");
    // Y[T][N] = X W^T: X[T][K] and W[N][K] encoded along their rows (contraction K).
    return linear_impl(MX_OP_FPROP, d_X, T, K, MX_CONTRACT_COLS, d_W, N, K, MX_CONTRACT_COLS, d_Y,
                       T, N, K, rot, rot_block, rnd, seed, d_ws, ws_bytes,
                       static_cast<cudaStream_t>(stream));
}

mx_status mx_linear_dgrad(const void *d_dY, const void *d_W, float *d_dX, int64_t T, int64_t N,
                          int64_t K, int rot, int rot_block, int rnd, uint64_t seed, void *d_ws,
                          size_t ws_bytes, void *stream) {
    TraceRange trace("mx_linear_dgrad");
    // dX[T][K] = dY W: dY[T][N] along its rows, W[N][K] down its rows (contraction N).
    return linear_impl(MX_OP_DGRAD, d_dY, T, N, MX_CONTRACT_COLS, d_W, N, K, MX_CONTRACT_ROWS,
                       d_dX, T, N, K, rot, rot_block, rnd, seed, d_ws, ws_bytes,
                       static_cast<cudaStream_t>(stream));
}

size_t mx_mxfp8_codes_bytes(int64_t mn, int64_t k) {
    if (mn <= 0 || k <= 0) return 0;
    return static_cast<size_t>(mn) * static_cast<size_t>(k);
}

mx_status mx_quantize_mxfp8(const void *d_src, int64_t rows, int64_t cols, void *d_codes,
                            void *d_scales, void *stream) {
    TraceRange trace("mx_quantize_mxfp8");
    return quantize_mxfp8_impl(d_src, rows, cols, nullptr, 0, 0, d_codes, d_scales, nullptr,
                               nullptr, static_cast<cudaStream_t>(stream));
}

mx_status mx_gemm_mxfp8(const void *d_Aq, const void *d_As, const void *d_Bq, const void *d_Bs,
                        float *d_C, int64_t M, int64_t N, int64_t K, void *stream) {
    TraceRange trace("mx_gemm_mxfp8");
    return gemm_mxfp8_impl(d_Aq, d_As, d_Bq, d_Bs, d_C, M, N, K,
                           static_cast<cudaStream_t>(stream));
}

size_t mx_linear_wgrad_mxfp8_workspace_bytes(int64_t T, int64_t N, int64_t K) {
    if (T <= 0 || N <= 0 || K <= 0) return 0;
    return align256(mx_mxfp8_codes_bytes(N, T)) + align256(mx_scales_bytes(N, T)) +
           align256(mx_mxfp8_codes_bytes(K, T)) + align256(mx_scales_bytes(K, T));
}

mx_status mx_linear_wgrad_mxfp8(const void *d_dY, const void *d_X, float *d_dW, int64_t T,
                                int64_t N, int64_t K, void *d_ws, size_t ws_bytes, void *stream) {
    TraceRange trace("mx_linear_wgrad_mxfp8");
    const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    if (T < 0 || N < 0 || K < 0) return MX_ERR_SHAPE;
    if (N == 0 || K == 0) return MX_OK;
    if (d_dW == nullptr) return MX_ERR_INVALID_ARG;
    if (T == 0) return gemm_mxfp8_impl(nullptr, nullptr, nullptr, nullptr, d_dW, N, K, 0, st_);
    mx_status st = check_encode(d_dY, T, N, MX_CONTRACT_ROWS, MX_ROT_NONE, 32, MX_ROUND_RNE,
                                d_dY, d_dY);
    if (st != MX_OK) return st;
    st = check_encode(d_X, T, K, MX_CONTRACT_ROWS, MX_ROT_NONE, 32, MX_ROUND_RNE, d_X, d_X);
    if (st != MX_OK) return st;
    if (K % 4 != 0 || !aligned16(d_dW)) return MX_ERR_ALIGN;
    if (d_ws == nullptr || ws_bytes < mx_linear_wgrad_mxfp8_workspace_bytes(T, N, K))
        return MX_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return MX_ERR_ALIGN;
    uint8_t *aq = static_cast<uint8_t *>(d_ws);
    uint8_t *as = aq + align256(mx_mxfp8_codes_bytes(N, T));
    uint8_t *bq = as + align256(mx_scales_bytes(N, T));
    uint8_t *bs = bq + align256(mx_mxfp8_codes_bytes(K, T));
    st = quantize_mxfp8_impl(d_dY, T, N, d_X, T, K, aq, as, bq, bs, st_);
    if (st != MX_OK) return st;
    return gemm_mxfp8_impl(aq, as, bq, bs, d_dW, N, K, T, st_);
}

size_t mx_nvfp4_scales_bytes(int64_t mn, int64_t k) {
    if (mn <= 0 || k <= 0) return 0;
    return static_cast<size_t>(scale_groups(mn)) * 128u * static_cast<size_t>(16 * ((k + 255) / 256));
}

mx_status mx_quantize_nvfp4(const void *d_src, int64_t rows, int64_t cols, int rot, int rot_block,
                            uint64_t seed, void *d_codes, void *d_scales, float *d_amax,
                            void *stream) {
    TraceRange trace("mx_quantize_nvfp4");
    return quantize_nvfp4_impl(d_src, rows, cols, nullptr, 0, 0, rot, rot_block, seed, d_codes,
                               d_scales, nullptr, nullptr, d_amax,
                               static_cast<cudaStream_t>(stream));
}

mx_status mx_gemm_nvfp4(const void *d_Aq, const void *d_As, const float *d_amax_a,
                        const void *d_Bq, const void *d_Bs, const float *d_amax_b, float *d_C,
                        int64_t M, int64_t N, int64_t K, void *stream) {
    TraceRange trace("mx_gemm_nvfp4");
    return gemm_nvfp4_impl(d_Aq, d_As, d_amax_a, d_Bq, d_Bs, d_amax_b, d_C, M, N, K,
                           static_cast<cudaStream_t>(stream));
}

size_t mx_linear_wgrad_nvfp4_workspace_bytes(int64_t T, int64_t N, int64_t K) {
    if (T <= 0 || N <= 0 || K <= 0) return 0;
    return align256(mx_codes_bytes(N, T)) + align256(mx_nvfp4_scales_bytes(N, T)) +
           align256(mx_codes_bytes(K, T)) + align256(mx_nvfp4_scales_bytes(K, T)) + 256;
}

mx_status mx_linear_wgrad_nvfp4(const void *d_dY, const void *d_X, float *d_dW, int64_t T,
                                int64_t N, int64_t K, int rot, int rot_block, uint64_t seed,
                                void *d_ws, size_t ws_bytes, void *stream) {
    TraceRange trace("mx_linear_wgrad_nvfp4");
    const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    if (T < 0 || N < 0 || K < 0) return MX_ERR_SHAPE;
    if (N == 0 || K == 0) return MX_OK;
    if (d_dW == nullptr) return MX_ERR_INVALID_ARG;
    if (T == 0) {
        mx_status st = check_gemm(nullptr, nullptr, nullptr, nullptr, d_dW, N, K, 0);
        if (st != MX_OK) return st;
        return from_cuda(cudaMemsetAsync(d_dW, 0, static_cast<size_t>(N) * K * sizeof(float), st_));
    }
    mx_status st = check_encode(d_dY, T, N, MX_CONTRACT_ROWS, rot, rot_block, MX_ROUND_RNE, d_dY,
                                d_dY);
    if (st != MX_OK) return st;
    st = check_encode(d_X, T, K, MX_CONTRACT_ROWS, rot, rot_block, MX_ROUND_RNE, d_X, d_X);
    if (st != MX_OK) return st;
    if (rot != MX_ROT_NONE && rot_block != 16 && rot_block != 32) return MX_ERR_UNSUPPORTED;
    if (K % 4 != 0 || !aligned16(d_dW)) return MX_ERR_ALIGN;
    if (d_ws == nullptr || ws_bytes < mx_linear_wgrad_nvfp4_workspace_bytes(T, N, K))
        return MX_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return MX_ERR_ALIGN;
    uint8_t *aq = static_cast<uint8_t *>(d_ws);
    uint8_t *as = aq + align256(mx_codes_bytes(N, T));
    uint8_t *bq = as + align256(mx_nvfp4_scales_bytes(N, T));
    uint8_t *bs = bq + align256(mx_codes_bytes(K, T));
    float *amax = reinterpret_cast<float *>(bs + align256(mx_nvfp4_scales_bytes(K, T)));
    st = quantize_nvfp4_impl(d_dY, T, N, d_X, T, K, rot, rot_block, seed, aq, as, bq, bs, amax,
                             st_);
    if (st != MX_OK) return st;
    return gemm_nvfp4_impl(aq, as, amax, bq, bs, amax + 1, d_dW, N, K, T, st_);
}

int mx_linear_wgrad_fused_supported(int64_t T, int64_t N, int64_t K, int rot, int rot_block,
                                    int rnd) {
    return wgrad_fusable(T, N, K, rot, rot_block, rnd) ? 1 : 0;
}

mx_status mx_linear_wgrad_fused(const void *d_dY, const void *d_X, float *d_dW, int64_t T,
                                int64_t N, int64_t K, int rot, int rot_block, int rnd,
                                uint64_t seed, void *d_ws, size_t ws_bytes, void *stream) {
    TraceRange trace("mx_linear_wgrad_fused");
    return linear_impl(MX_OP_WGRAD, d_dY, T, N, MX_CONTRACT_ROWS, d_X, T, K, MX_CONTRACT_ROWS,
                       d_dW, T, N, K, rot, rot_block, rnd, seed, d_ws, ws_bytes,
                       static_cast<cudaStream_t>(stream), true);
}

mx_status mx_rmsnorm(const void *d_x, int x_type, int64_t x_pitch, const void *d_res, int res_type,
                     int64_t res_pitch, const void *d_w, int w_type, float eps, int64_t T,
                     int64_t K, void *d_h, int64_t h_pitch, void *d_y, int format, void *d_codes,
                     void *d_scales, float *d_rstd, void *stream) {
    TraceRange trace("mx_rmsnorm");
    if (!valid_type(x_type) || !valid_type(w_type) || !(eps >= 0.0f)) return MX_ERR_INVALID_ARG;
    if (d_res != nullptr && !valid_type(res_type)) return MX_ERR_INVALID_ARG;
    if (d_res == nullptr && d_h != nullptr) return MX_ERR_INVALID_ARG;
    mx_status st = check_row_sizes(T, K);
    if (st != MX_OK) return st;
    const RowEncode e{format, d_codes, d_scales};
    if ((st = check_row_encode(e, T, K)) != MX_OK || T == 0 || K == 0) return st;
    if (d_w == nullptr) return MX_ERR_INVALID_ARG;
    if ((st = check_rows(d_x, x_pitch, K)) != MX_OK) return st;
    if (d_res != nullptr && (st = check_rows(d_res, res_pitch, K)) != MX_OK) return st;
    if (d_h != nullptr && (st = check_rows(d_h, h_pitch, K)) != MX_OK) return st;
    if (!aligned16(d_w) || !aligned16(d_y) || !aligned16(d_rstd)) return MX_ERR_ALIGN;
    if (K > MX_ROW_COLUMNS_MAX) return MX_ERR_UNSUPPORTED;
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_rmsnorm({d_x, x_pitch, x_type == MX_TYPE_F32},
                                    {d_res, res_pitch, res_type == MX_TYPE_F32}, d_w,
                                    w_type == MX_TYPE_F32, eps, T, K, d_h, h_pitch, d_y, e, d_rstd,
                                    *dev, static_cast<cudaStream_t>(stream)));
}

size_t mx_rmsnorm_backward_workspace_bytes(int64_t T, int64_t K) {
    if (T <= 0 || K <= 0 || K > MX_ROW_COLUMNS_MAX) return 0;
    return align256(rmsnorm_backward_ws(T, K));
}

mx_status mx_rmsnorm_backward(const void *d_dy, int dy_type, int64_t dy_pitch, const void *d_h,
                              int h_type, int64_t h_pitch, const void *d_w, int w_type,
                              const float *d_rstd, const void *d_dres, int64_t dres_pitch,
                              int64_t T, int64_t K, void *d_dx, int64_t dx_pitch, float *d_dw,
                              void *d_ws, size_t ws_bytes, void *stream) {
    TraceRange trace("mx_rmsnorm_backward");
    if (!valid_type(dy_type) || !valid_type(h_type) || !valid_type(w_type))
        return MX_ERR_INVALID_ARG;
    mx_status st = check_row_sizes(T, K);
    if (st != MX_OK || K == 0) return st;
    if (!aligned16(d_dw)) return MX_ERR_ALIGN;
    if (T == 0)
        return d_dw == nullptr ? MX_OK
                               : from_cuda(cudaMemsetAsync(d_dw, 0, static_cast<size_t>(K) * sizeof(float),
                                                           static_cast<cudaStream_t>(stream)));
    if (d_w == nullptr || d_rstd == nullptr) return MX_ERR_INVALID_ARG;
    if ((st = check_rows(d_dy, dy_pitch, K)) != MX_OK) return st;
    if ((st = check_rows(d_h, h_pitch, K)) != MX_OK) return st;
    if ((st = check_rows(d_dx, dx_pitch, K)) != MX_OK) return st;
    if (d_dres != nullptr && (st = check_rows(d_dres, dres_pitch, K)) != MX_OK) return st;
    if (!aligned16(d_w) || !aligned16(d_rstd)) return MX_ERR_ALIGN;
    if (K > MX_ROW_COLUMNS_MAX) return MX_ERR_UNSUPPORTED;
    if (d_dw != nullptr) {
        if (d_ws == nullptr || ws_bytes < mx_rmsnorm_backward_workspace_bytes(T, K))
            return MX_ERR_WORKSPACE;
        if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return MX_ERR_ALIGN;
    }
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_rmsnorm_backward(
        {d_dy, dy_pitch, dy_type == MX_TYPE_F32}, {d_h, h_pitch, h_type == MX_TYPE_F32}, d_w,
        w_type == MX_TYPE_F32, d_rstd, {d_dres, dres_pitch, h_type == MX_TYPE_F32}, T, K, d_dx,
        dx_pitch, d_dw, d_ws, *dev, static_cast<cudaStream_t>(stream)));
}

mx_status mx_swiglu(const void *d_gu, int gu_type, int64_t gu_pitch, int64_t T, int64_t F,
                    void *d_y, int format, void *d_codes, void *d_scales, void *stream) {
    TraceRange trace("mx_swiglu");
    if (!valid_type(gu_type)) return MX_ERR_INVALID_ARG;
    mx_status st = check_row_sizes(T, F);
    if (st != MX_OK) return st;
    const RowEncode e{format, d_codes, d_scales};
    if ((st = check_row_encode(e, T, F)) != MX_OK || T == 0 || F == 0) return st;
    if ((st = check_rows(d_gu, gu_pitch, 2 * F)) != MX_OK) return st;
    if (F % 8 != 0 || !aligned16(d_y)) return MX_ERR_ALIGN;
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_swiglu({d_gu, gu_pitch, gu_type == MX_TYPE_F32}, T, F, d_y, e, *dev,
                                   static_cast<cudaStream_t>(stream)));
}

mx_status mx_swiglu_backward(const void *d_dy, int dy_type, int64_t dy_pitch, const void *d_gu,
                             int gu_type, int64_t gu_pitch, int64_t T, int64_t F, void *d_dgu,
                             void *stream) {
    TraceRange trace("mx_swiglu_backward");
    if (!valid_type(dy_type) || !valid_type(gu_type)) return MX_ERR_INVALID_ARG;
    mx_status st = check_row_sizes(T, F);
    if (st != MX_OK || T == 0 || F == 0) return st;
    if ((st = check_rows(d_dy, dy_pitch, F)) != MX_OK) return st;
    if ((st = check_rows(d_gu, gu_pitch, 2 * F)) != MX_OK) return st;
    if (d_dgu == nullptr) return MX_ERR_INVALID_ARG;
    if (F % 8 != 0 || !aligned16(d_dgu)) return MX_ERR_ALIGN;
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_swiglu_backward({d_dy, dy_pitch, dy_type == MX_TYPE_F32},
                                            {d_gu, gu_pitch, gu_type == MX_TYPE_F32}, T, F, d_dgu,
                                            *dev, static_cast<cudaStream_t>(stream)));
}

size_t mx_grad_workspace_bytes(int64_t count) {
    return count <= 0 ? 0 : align256(grad_ws(count));
}

mx_status mx_grad_norm(const void *const *h_grads, const int64_t *h_sizes, const int *h_types,
                       int64_t count, float *d_norm, void *d_ws, size_t ws_bytes, void *stream) {
    TraceRange trace("mx_grad_norm");
    return grad_impl(h_grads, h_sizes, h_types, nullptr, nullptr, count, false, 0.0f, 0.0f, d_norm,
                     d_ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

mx_status mx_clip_grads(const void *const *h_grads, const int64_t *h_sizes, const int *h_types,
                        void *const *h_outs, const int *h_out_types, int64_t count, float max_norm,
                        float eps, float *d_norm, void *d_ws, size_t ws_bytes, void *stream) {
    TraceRange trace("mx_clip_grads");
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f)) return MX_ERR_INVALID_ARG;
    return grad_impl(h_grads, h_sizes, h_types, h_outs, h_out_types, count, true, max_norm, eps,
                     d_norm, d_ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

mx_status mx_gemm_bias_act(const void *d_Aq, const void *d_As, const void *d_Bq, const void *d_Bs,
                           int operands, int64_t M, int64_t N, int64_t K, const void *d_bias,
                           int bias_type, int act, const void *d_res, int res_type,
                           int64_t res_pitch, void *d_y, int y_type, void *d_z, int format,
                           void *d_codes, void *d_scales, void *stream) {
    TraceRange trace("mx_gemm_bias_act");
    Product p{};
    p.mode = kProductDense;
    p.M = M, p.N = N, p.K = K;
    p.Aq = d_Aq, p.As = d_As, p.Bq = d_Bq, p.Bs = d_Bs;
    mx_status st = check_epilogue(p, d_bias, bias_type, act, d_y, y_type, d_z, format, d_codes, d_scales);
    if (st != MX_OK) return st;
    if (d_res != nullptr && !valid_type(res_type)) return MX_ERR_INVALID_ARG;
    if ((st = check_product(p, operands)) != MX_OK || M == 0 || N == 0) return st;
    if (d_res != nullptr && (st = check_rows(d_res, res_pitch, N)) != MX_OK) return st;
    p.res = {d_res, res_pitch, res_type == MX_TYPE_F32};
    return run_product(p, stream);
}

size_t mx_bias_act_backward_workspace_bytes(int64_t T, int64_t N) {
    return T <= 0 || N <= 0 ? 0 : align256(bias_act_backward_ws(T, N));
}

mx_status mx_bias_act_backward(const void *d_dy, int dy_type, int64_t dy_pitch, const void *d_z,
                               int z_type, int64_t z_pitch, int act, int64_t T, int64_t N,
                               void *d_dz, int format, void *d_codes, void *d_scales,
                               float *d_dbias, void *d_ws, size_t ws_bytes, void *stream) {
    TraceRange trace("mx_bias_act_backward");
    if (!valid_type(dy_type) || !valid_act(act)) return MX_ERR_INVALID_ARG;
    if (act != MX_ACT_NONE && !valid_type(z_type)) return MX_ERR_INVALID_ARG;
    if (T > 0 && N > 0 && d_dz == nullptr && format == MX_FORMAT_NONE && d_dbias == nullptr) return MX_ERR_INVALID_ARG;
    mx_status st = check_row_sizes(T, N);
    if (st != MX_OK) return st;
    const RowEncode e{format, d_codes, d_scales};
    if ((st = check_row_encode(e, T, N)) != MX_OK || N == 0) return st;
    if (!aligned16(d_dbias)) return MX_ERR_ALIGN;
    if (T == 0)
        return d_dbias == nullptr ? MX_OK
                                  : from_cuda(cudaMemsetAsync(d_dbias, 0, static_cast<size_t>(N) * sizeof(float),
                                                              static_cast<cudaStream_t>(stream)));
    if ((st = check_rows(d_dy, dy_pitch, N)) != MX_OK) return st;
    if (act != MX_ACT_NONE && (st = check_rows(d_z, z_pitch, N)) != MX_OK) return st;
    if (!aligned16(d_dz)) return MX_ERR_ALIGN;
    if (d_dbias != nullptr && bias_act_backward_ws(T, N) > 0) {
        if (d_ws == nullptr || ws_bytes < mx_bias_act_backward_workspace_bytes(T, N)) return MX_ERR_WORKSPACE;
        if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return MX_ERR_ALIGN;
    }
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    RowIn z{d_z, z_pitch, z_type == MX_TYPE_F32};
    if (act == MX_ACT_NONE) z = {nullptr, 0, false};
    return from_cuda(launch_bias_act_backward({d_dy, dy_pitch, dy_type == MX_TYPE_F32}, z, act, T, N, d_dz, e,
                                              d_dbias, d_ws, *dev, static_cast<cudaStream_t>(stream)));
}

int64_t mx_expert_rows(int64_t T, int64_t picks, int64_t experts) {
    if (T <= 0 || picks <= 0 || experts <= 0 || T > 0x7FFFFFFF || picks > 0x7FFFFFFF) return 0;
    const int64_t n = T * picks;
    return n > 0x7FFFFFFF ? 0 : (n + 127 * std::min(experts, n)) / 128 * 128;
}

size_t mx_expert_plan_workspace_bytes(int64_t T, int64_t picks, int64_t experts) {
    return mx_expert_rows(T, picks, experts) == 0 ? 0 : align256(expert_plan_ws(T * picks, experts));
}

mx_status mx_expert_plan(const void *d_index, int index_bytes, int64_t T, int64_t picks,
                         int64_t experts, int32_t *d_offsets, int32_t *d_counts, int32_t *d_slot,
                         int32_t *d_source, void *d_ws, size_t ws_bytes, void *stream) {
    TraceRange trace("mx_expert_plan");
    if (index_bytes != 4 && index_bytes != 8) return MX_ERR_INVALID_ARG;
    const ExpertRows r{d_slot, d_source, T, picks, mx_expert_rows(T, picks, experts), 0};
    mx_status st = check_expert_rows(r);
    if (st != MX_OK) return st;
    if ((st = check_experts(experts, d_offsets)) != MX_OK) return st;
    if (d_counts == nullptr) return MX_ERR_INVALID_ARG;
    if (!aligned16(d_counts)) return MX_ERR_ALIGN;
    const int64_t n = T * picks;
    if (n > 0) {
        if (d_index == nullptr || d_slot == nullptr || d_source == nullptr) return MX_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(d_index) & static_cast<uintptr_t>(index_bytes - 1)) != 0) return MX_ERR_ALIGN;
        if (expert_plan_ws(n, experts) > 0) {
            if (d_ws == nullptr || ws_bytes < mx_expert_plan_workspace_bytes(T, picks, experts)) return MX_ERR_WORKSPACE;
            if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return MX_ERR_ALIGN;
        }
    }
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_expert_plan(d_index, index_bytes == 8, n, experts, r.rows, d_offsets, d_counts, d_slot,
                                        d_source, d_ws, *dev, static_cast<cudaStream_t>(stream)));
}

mx_status mx_expert_dispatch(const void *d_x, int x_type, int64_t x_pitch, const int32_t *d_slot,
                             const int32_t *d_source, int64_t T, int64_t picks, int64_t rows,
                             int64_t K, void *d_y, int format, void *d_codes, void *d_scales,
                             void *stream) {
    TraceRange trace("mx_expert_dispatch");
    if (!valid_type(x_type)) return MX_ERR_INVALID_ARG;
    if (rows > 0 && K > 0 && d_y == nullptr && format == MX_FORMAT_NONE) return MX_ERR_INVALID_ARG;
    const ExpertRows r{d_slot, d_source, T, picks, rows, K};
    mx_status st = check_expert_rows(r);
    if (st != MX_OK || (st = check_row_sizes(rows, K)) != MX_OK) return st;
    const RowEncode e{format, d_codes, d_scales};
    if ((st = check_row_encode(e, rows, K)) != MX_OK || rows == 0 || K == 0) return st;
    if (d_source == nullptr || (T * picks > 0 && d_slot == nullptr)) return MX_ERR_INVALID_ARG;
    if (K % 8 != 0 || !aligned16(d_y)) return MX_ERR_ALIGN;
    if (T > 0 && picks > 0 && (st = check_rows(d_x, x_pitch, K)) != MX_OK) return st;
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_expert_dispatch({d_x, x_pitch, x_type == MX_TYPE_F32}, r, d_y, e, *dev,
                                            static_cast<cudaStream_t>(stream)));
}

mx_status mx_expert_combine(const void *d_rows, int rows_type, int64_t rows_pitch,
                            const int32_t *d_slot, const float *d_weights, int64_t T,
                            int64_t picks, int64_t rows, int64_t K, const void *d_res, int res_type,
                            int64_t res_pitch, void *d_y, int y_type, void *stream) {
    TraceRange trace("mx_expert_combine");
    if (!valid_type(rows_type) || !valid_type(y_type)) return MX_ERR_INVALID_ARG;
    if (d_res != nullptr && !valid_type(res_type)) return MX_ERR_INVALID_ARG;
    const ExpertRows r{d_slot, nullptr, T, picks, rows, K};
    mx_status st = check_expert_rows(r);
    if (st != MX_OK || (st = check_row_sizes(rows, K)) != MX_OK || T == 0 || K == 0) return st;
    if (d_y == nullptr || (picks > 0 && d_slot == nullptr)) return MX_ERR_INVALID_ARG;
    if (K % 8 != 0 || !aligned16(d_y) || !aligned16(d_weights)) return MX_ERR_ALIGN;
    if (picks > 0 && rows > 0 && (st = check_rows(d_rows, rows_pitch, K)) != MX_OK) return st;
    if (d_res != nullptr && (st = check_rows(d_res, res_pitch, K)) != MX_OK) return st;
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_expert_combine({d_rows, rows_pitch, rows_type == MX_TYPE_F32}, r, d_weights,
                                           {d_res, res_pitch, res_type == MX_TYPE_F32}, d_y, y_type == MX_TYPE_F32,
                                           *dev, static_cast<cudaStream_t>(stream)));
}

mx_status mx_expert_combine_backward(const void *d_dy, int dy_type, int64_t dy_pitch,
                                     const void *d_rows, int rows_type, int64_t rows_pitch,
                                     const int32_t *d_slot, const int32_t *d_source,
                                     const float *d_weights, int64_t T, int64_t picks, int64_t rows,
                                     int64_t K, void *d_drows, int format, void *d_codes,
                                     void *d_scales, float *d_dweights, void *stream) {
    TraceRange trace("mx_expert_combine_backward");
    if (!valid_type(dy_type) || (d_dweights != nullptr && !valid_type(rows_type))) return MX_ERR_INVALID_ARG;
    if (rows > 0 && K > 0 && d_drows == nullptr && format == MX_FORMAT_NONE && d_dweights == nullptr)
        return MX_ERR_INVALID_ARG;
    const ExpertRows r{d_slot, d_source, T, picks, rows, K};
    mx_status st = check_expert_rows(r);
    if (st != MX_OK || (st = check_row_sizes(rows, K)) != MX_OK) return st;
    const RowEncode e{format, d_codes, d_scales};
    if ((st = check_row_encode(e, rows, K)) != MX_OK) return st;
    const int64_t n = T * picks;
    if (!aligned16(d_dweights) || !aligned16(d_weights) || !aligned16(d_drows) || K % 8 != 0) return MX_ERR_ALIGN;
    if (K == 0 || rows == 0)
        return d_dweights == nullptr || n == 0
                   ? MX_OK
                   : from_cuda(cudaMemsetAsync(d_dweights, 0, static_cast<size_t>(n) * sizeof(float),
                                               static_cast<cudaStream_t>(stream)));
    const bool writes = d_drows != nullptr || format != MX_FORMAT_NONE;
    if (writes && d_source == nullptr) return MX_ERR_INVALID_ARG;
    if (n > 0) {
        if (d_slot == nullptr || d_weights == nullptr) return MX_ERR_INVALID_ARG;
        if ((st = check_rows(d_dy, dy_pitch, K)) != MX_OK) return st;
        if (d_dweights != nullptr && (st = check_rows(d_rows, rows_pitch, K)) != MX_OK) return st;
    } else if (!writes) {
        return MX_OK;
    }
    const DeviceInfo *dev = nullptr;
    if ((st = device_or_error(&dev)) != MX_OK) return st;
    return from_cuda(launch_expert_combine_backward({d_dy, dy_pitch, dy_type == MX_TYPE_F32},
                                                    {d_rows, rows_pitch, rows_type == MX_TYPE_F32}, r, d_weights,
                                                    d_drows, e, d_dweights, *dev, static_cast<cudaStream_t>(stream)));
}

mx_status mx_quantize_experts(const void *d_src, int64_t experts, int64_t rows, int64_t cols,
                              int operands, int contract, int rot, int rot_block, uint64_t seed,
                              void *d_codes, void *d_scales, void *stream) {
    TraceRange trace("mx_quantize_experts");
    const bool fp8 = operands == MX_FORMAT_MXFP8;
    if (operands != MX_FORMAT_MXFP4 && !fp8) return MX_ERR_INVALID_ARG;
    if (experts < 0) return MX_ERR_SHAPE;
    mx_status st = check_encode(d_src, rows, cols, contract, rot, rot_block, MX_ROUND_RNE, d_codes, d_scales);
    if (st != MX_OK || experts == 0 || rows == 0 || cols == 0) return st;
    if (experts > MX_EXPERTS_MAX || (fp8 && (contract != MX_CONTRACT_ROWS || rot != MX_ROT_NONE)))
        return MX_ERR_UNSUPPORTED;
    const int64_t lines = contract == MX_CONTRACT_ROWS ? cols : rows, k = contract == MX_CONTRACT_ROWS ? rows : cols;
    const size_t codes = fp8 ? mx_mxfp8_codes_bytes(lines, k) : mx_codes_bytes(lines, k), scales = mx_scales_bytes(lines, k);
    if (codes % 16 != 0) return MX_ERR_ALIGN;  // the next expert's codes
    const uint8_t *src = static_cast<const uint8_t *>(d_src);
    uint8_t *c = static_cast<uint8_t *>(d_codes), *s = static_cast<uint8_t *>(d_scales);
    const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    // Whole scale groups along the rows: all experts' lines are one operand's.
    if (contract == MX_CONTRACT_COLS && rows % 128 == 0 && experts * rows <= 0x7FFFFFFF)
        return quantize_impl(d_src, experts * rows, cols, contract, rot, rot_block, MX_ROUND_RNE, seed, 1, c, s, st_);
    for (int64_t e = 0; e < experts; ++e) {
        const uint8_t *from = src + static_cast<size_t>(e) * rows * cols * 2;
        st = fp8 ? quantize_mxfp8_impl(from, rows, cols, nullptr, 0, 0, c + e * codes, s + e * scales, nullptr, nullptr, st_)
                 : quantize_impl(from, rows, cols, contract, rot, rot_block, MX_ROUND_RNE, seed, 1, c + e * codes,
                                 s + e * scales, st_);
        if (st != MX_OK) return st;
    }
    return MX_OK;
}

mx_status mx_gemm_experts(const void *d_Aq, const void *d_As, const void *d_Bq, const void *d_Bs,
                          int operands, const int32_t *d_offsets, const int32_t *d_counts,
                          int64_t experts, int64_t rows, int64_t N, int64_t K, const void *d_bias,
                          int bias_type, int act, void *d_y, int y_type, void *d_z, int format,
                          void *d_codes, void *d_scales, void *stream) {
    TraceRange trace("mx_gemm_experts");
    Product p{};
    p.mode = kProductRows;
    p.M = rows, p.N = N, p.K = K, p.experts = experts;
    p.Aq = d_Aq, p.As = d_As, p.Bq = d_Bq, p.Bs = d_Bs;
    p.offsets = d_offsets, p.counts = d_counts;
    mx_status st = check_epilogue(p, d_bias, bias_type, act, d_y, y_type, d_z, format, d_codes, d_scales);
    if (st != MX_OK) return st;
    if (rows % 128 != 0) return MX_ERR_SHAPE;
    if ((st = check_product(p, operands)) != MX_OK) return st;
    if ((st = check_experts(experts, d_offsets)) != MX_OK) return st;
    if (d_counts == nullptr) return MX_ERR_INVALID_ARG;
    if (!aligned16(d_counts)) return MX_ERR_ALIGN;
    if (rows == 0 || N == 0) return MX_OK;
    if (experts * N > 0x7FFFFFFF) return MX_ERR_SHAPE;
    return run_product(p, stream);
}

mx_status mx_gemm_experts_wgrad(const void *d_Aq, const void *d_As, const void *d_Bq,
                                const void *d_Bs, int operands, const int32_t *d_offsets,
                                int64_t experts, int64_t rows, int64_t M, int64_t N, void *d_C,
                                int c_type, void *stream) {
    TraceRange trace("mx_gemm_experts_wgrad");
    return experts_wgrad_impl(d_Aq, d_As, d_Bq, d_Bs, operands, d_offsets, experts, rows, M, N, d_C, c_type, stream);
}

size_t mx_linear_experts_wgrad_workspace_bytes(int operands, int64_t rows, int64_t N, int64_t K) {
    if (rows <= 0 || N <= 0 || K <= 0) return 0;
    const bool fp8 = operands == MX_FORMAT_MXFP8;
    const auto codes = [&](int64_t lines) { return fp8 ? mx_mxfp8_codes_bytes(lines, rows) : mx_codes_bytes(lines, rows); };
    return align256(codes(N)) + align256(mx_scales_bytes(N, rows)) + align256(codes(K)) + align256(mx_scales_bytes(K, rows));
}

mx_status mx_linear_experts_wgrad(const void *d_dY, const void *d_X, int operands,
                                  const int32_t *d_offsets, int64_t experts, int64_t rows,
                                  int64_t N, int64_t K, int rot, int rot_block, int rnd,
                                  uint64_t seed, void *d_dW, int dw_type, void *d_ws,
                                  size_t ws_bytes, void *stream) {
    TraceRange trace("mx_linear_experts_wgrad");
    const bool fp8 = operands == MX_FORMAT_MXFP8;
    if (operands != MX_FORMAT_MXFP4 && !fp8) return MX_ERR_INVALID_ARG;
    if (rows < 0 || rows % 128 != 0 || N < 0 || K < 0) return MX_ERR_SHAPE;
    if (!valid_type(dw_type)) return MX_ERR_INVALID_ARG;
    mx_status st = check_experts(experts, d_offsets);
    if (st != MX_OK || N == 0 || K == 0) return st;
    if (rows == 0)
        return experts_wgrad_impl(nullptr, nullptr, nullptr, nullptr, operands, d_offsets, experts, 0, N, K, d_dW,
                                  dw_type, stream);
    if ((st = check_encode(d_dY, rows, N, MX_CONTRACT_ROWS, rot, rot_block, rnd, d_dY, d_dY)) != MX_OK) return st;
    if ((st = check_encode(d_X, rows, K, MX_CONTRACT_ROWS, rot, rot_block, rnd, d_X, d_X)) != MX_OK) return st;
    // A rotation must not mix two experts' rows.
    if (rot != MX_ROT_NONE && (fp8 || rot_block > 128)) return MX_ERR_UNSUPPORTED;
    if (fp8 && rnd != MX_ROUND_RNE) return MX_ERR_UNSUPPORTED;
    if (d_dW == nullptr) return MX_ERR_INVALID_ARG;
    if (!aligned16(d_dW)) return MX_ERR_ALIGN;
    if (d_ws == nullptr || ws_bytes < mx_linear_experts_wgrad_workspace_bytes(operands, rows, N, K))
        return MX_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return MX_ERR_ALIGN;
    const auto codes = [&](int64_t lines) { return fp8 ? mx_mxfp8_codes_bytes(lines, rows) : mx_codes_bytes(lines, rows); };
    uint8_t *aq = static_cast<uint8_t *>(d_ws);
    uint8_t *as = aq + align256(codes(N));
    uint8_t *bq = as + align256(mx_scales_bytes(N, rows));
    uint8_t *bs = bq + align256(codes(K));
    const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    st = fp8 ? quantize_mxfp8_impl(d_dY, rows, N, d_X, rows, K, aq, as, bq, bs, st_)
             : quantize_pair_impl(d_dY, rows, N, d_X, rows, K, rot, rot_block, rnd, seed, aq, as, bq, bs, st_);
    if (st != MX_OK) return st;
    return experts_wgrad_impl(aq, as, bq, bs, operands, d_offsets, experts, rows, N, K, d_dW, dw_type, stream);
}

mx_status mx_check_status(void *stream) {
    TraceRange trace("mx_check_status");
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return MX_ERR_CUDA;
    const DeviceInfo *dev = nullptr;
    cudaError_t de = cudaSuccess;
    if ((dev = current_device(&de)) == nullptr) return MX_ERR_CUDA;
    int v = 0;
    if (cudaMemcpy(&v, dev->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
        return MX_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpy(dev->status, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
            return MX_ERR_CUDA;
        return v == kDevTimeout ? MX_ERR_TIMEOUT : v == kDevBounds ? MX_ERR_BOUNDS : MX_ERR_CUDA;
    }
    return MX_OK;
}

mx_status mx_debug_timeout_probe(int64_t limit_us, void *stream) {
    TraceRange trace("mx_debug_timeout_probe");
    if (limit_us <= 0 || limit_us > 10 * 1000 * 1000) return MX_ERR_INVALID_ARG;
    const DeviceInfo *dev = nullptr;
    mx_status st = device_or_error(&dev);
    if (st != MX_OK) return st;
    timeout_probe_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
        dev->status, static_cast<uint64_t>(limit_us) * 1000ull);
    return from_cuda(cudaGetLastError());
}

const char *mx_status_string(int status) {
    switch (status) {
        case MX_OK: return "MX_OK";
        case MX_ERR_INVALID_ARG: return "MX_ERR_INVALID_ARG";
        case MX_ERR_SHAPE: return "MX_ERR_SHAPE";
        case MX_ERR_ALIGN: return "MX_ERR_ALIGN";
        case MX_ERR_WORKSPACE: return "MX_ERR_WORKSPACE";
        case MX_ERR_CUDA: return "MX_ERR_CUDA";
        case MX_ERR_TIMEOUT: return "MX_ERR_TIMEOUT";
        case MX_ERR_UNSUPPORTED: return "MX_ERR_UNSUPPORTED";
        case MX_ERR_BOUNDS: return "MX_ERR_BOUNDS";
        default: return "MX_ERR_UNKNOWN";
    }
}

int mx_version(void) { return 100; }

}  // extern "C"
