// mx_internal.h -- host-side glue shared by the library's translation units.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mx {

struct DeviceInfo {
    int ordinal = -1;
    int sm_count = 0;
    int cc_major = 0, cc_minor = 0;
    int *status = nullptr;  // device address of the per-device status word
};

// Lazily-filled info for the current device; nullptr (and *err set) on failure.
const DeviceInfo *current_device(cudaError_t *err);

// Host wrapper of cuTensorMapEncodeTiled for a 2-D row-major tensor.
bool encode_tmap_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base,
                    uint64_t inner_elems, uint64_t outer_elems, uint64_t row_bytes,
                    uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle);

// Map of a row-major byte matrix whose lines (a multiple of 64) are loaded 64 by 64 in the order
// position 8 i + 2 c + b <- line 16 c + 2 i + b (b < 2, c < 4, i < 8): dimensions (bytes, b, c, i,
// group of 64), a box of box_inner bytes by box_lines lines.
bool encode_tmap_lines64(CUtensorMap *map, const void *base, uint64_t row_bytes, uint64_t lines,
                         uint32_t box_inner, uint32_t box_lines, CUtensorMapSwizzle swizzle);

// Scale-layout geometry (see mx.h): k-atoms (4 blocks of 32) per 128-line group.
inline int64_t scale_katoms(int64_t k) { return 2 * ((k + 255) / 256); }
inline int64_t scale_groups(int64_t mn) { return (mn + 127) / 128; }
// NVFP4 scale layout: 512-byte atoms of 128 lines x 4 blocks of 16.
inline int64_t nv_scale_katoms(int64_t k) { return 4 * ((k + 255) / 256); }

// Kernel launchers (argument validation happens before these are called).
cudaError_t launch_quantize(const void *src, int64_t rows, int64_t cols, int contract, int rot,
                            int rot_block, int rnd, uint64_t seed, uint64_t sr_tag,
                            void *codes, void *scales, const DeviceInfo &dev,
                            cudaStream_t stream);

// Both operands encoded down their rows (contraction = rows) in one launch;
// SR tags 1 and 2.
cudaError_t launch_quantize_pair_colwise(const void *src0, int64_t rows0, int64_t cols0,
                                         const void *src1, int64_t rows1, int64_t cols1, int rot,
                                         int rot_block, int rnd, uint64_t seed, void *codes0,
                                         void *scales0, void *codes1, void *scales1,
                                         const DeviceInfo &dev, cudaStream_t stream);
// One read of src [rows, cols] writes its column-direction encoding (blocks
// along rows, rotated) and its row-direction encoding (blocks along cols,
// no rotation).
// tiled scales [mx_scales_bytes(lines, k)] -> canonical [lines][k/32].
cudaError_t launch_scales_to_canonical(const void *tiled, int64_t lines, int64_t k, void *canon,
                                       const DeviceInfo &dev, cudaStream_t stream);
cudaError_t launch_quantize_dual(const void *src, int64_t rows, int64_t cols, int rot,
                                 int rot_block, int rnd, uint64_t seed, void *codes_t,
                                 void *scales_t, void *codes_n, void *scales_n,
                                 const DeviceInfo &dev, cudaStream_t stream);

// MXFP8 (E4M3 elements, the FP8 comparator) encode down the rows of one or
// two operands (src1 == nullptr: one) in one launch; no rotation, round to
// nearest.  Codes [cols][rows] bytes, scales in the tiled layout.
cudaError_t launch_quantize_mxfp8_colwise(const void *src0, int64_t rows0, int64_t cols0,
                                          const void *src1, int64_t rows1, int64_t cols1,
                                          void *codes0, void *scales0, void *codes1,
                                          void *scales1, const DeviceInfo &dev,
                                          cudaStream_t stream);

// NVFP4 encode down the rows of one or two operands (src1 == nullptr: one):
// zeroes amax[0..1], a first launch max-reduces each rotated operand's
// largest finite magnitude into it, a second encodes with the tensor scale
// 2688 / amax.  Rotation none, or Hadamard 16 / 32 (rot 1 deterministic, 2
// with random signs); round to nearest.  Codes [cols][rows/2], scales in the
// NVFP4 tiled layout.
cudaError_t launch_quantize_nvfp4_colwise(const void *src0, int64_t rows0, int64_t cols0,
                                          const void *src1, int64_t rows1, int64_t cols1, int rot,
                                          int rot_block, uint64_t seed, void *codes0,
                                          void *scales0, void *codes1, void *scales1,
                                          float *amax, const DeviceInfo &dev,
                                          cudaStream_t stream);

// Block-scaled GEMM over MXFP4 (fmt 0), MXFP8 (fmt 1) or NVFP4 (fmt 2)
// operands; NVFP4 reads the two tensor amaxes (device floats) and scales the
// result by 1 / (s_enc(a) * s_enc(b)).
enum { kGemmMXFP4 = 0, kGemmMXFP8 = 1, kGemmNVFP4 = 2 };
cudaError_t launch_gemm_fmt(int fmt, const void *Aq, const void *As, const void *Bq,
                            const void *Bs, float *C, int64_t M, int64_t N, int64_t K,
                            const float *amax_a, const float *amax_b, const DeviceInfo &dev,
                            cudaStream_t stream);

cudaError_t launch_gemm(const void *Aq, const void *As, const void *Bq, const void *Bs, float *C,
                        int64_t M, int64_t N, int64_t K, const DeviceInfo &dev,
                        cudaStream_t stream);

// Fused Wgrad: one launch whose encoder warps encode dY and X (contraction
// T) into Aq/As/Bq/Bs while the GEMM consumes them; `counters` is
// wgrad_fused_counter_bytes(T, N, K) of workspace (any contents).  Only for
// the shapes and modes wgrad_fusable() accepts.
bool wgrad_fusable(int64_t T, int64_t N, int64_t K, int rot, int rot_block, int rnd);
size_t wgrad_fused_counter_bytes(int64_t T, int64_t N, int64_t K);
cudaError_t launch_wgrad_fused(const void *dY, const void *X, float *dW, int64_t T, int64_t N,
                               int64_t K, int rot, int rot_block, void *Aq, void *As, void *Bq,
                               void *Bs, void *counters, const DeviceInfo &dev,
                               cudaStream_t stream);

// ---- row operators between the GEMMs (mx_norm.cu, mx_glu.cu)
// A row-major input: pitch in elements, f32 or bf16.
struct RowIn {
    const void *p;
    int64_t pitch;
    bool f32;
};
// Encoded output along the rows (mx_format values), or none.
enum : int { kEncNone = 0, kEncMX4 = 1, kEncMX8 = 2 };
struct RowEncode {
    int fmt;
    void *codes, *scales;
};
// h (the stream, when res.p is given; may be null), y (bf16, may be null) and the encoded y.
cudaError_t launch_rmsnorm(const RowIn &x, const RowIn &res, const void *w, int w_f32, float eps,
                           int64_t T, int64_t K, void *h, int64_t h_pitch, void *y,
                           const RowEncode &e, float *rstd, const DeviceInfo &dev,
                           cudaStream_t stream);
size_t rmsnorm_backward_ws(int64_t T, int64_t K);
cudaError_t launch_rmsnorm_backward(const RowIn &dy, const RowIn &h, const void *w, int w_f32,
                                    const float *rstd, const RowIn &dres, int64_t T, int64_t K,
                                    void *dx, int64_t dx_pitch, float *dw, void *ws,
                                    const DeviceInfo &dev, cudaStream_t stream);
cudaError_t launch_swiglu(const RowIn &gu, int64_t T, int64_t F, void *y, const RowEncode &e,
                          const DeviceInfo &dev, cudaStream_t stream);
cudaError_t launch_swiglu_backward(const RowIn &dy, const RowIn &gu, int64_t T, int64_t F,
                                   void *dgu, const DeviceInfo &dev, cudaStream_t stream);

// ---- gradient norm and clipping (mx_grad.cu)
struct GradTensor {
    const void *p;
    void *out;  // null: norm only
    int64_t n;
    bool f32, out_f32;
};
size_t grad_ws(int64_t count);
// scale == false: the norm alone.
cudaError_t launch_grad_clip(const GradTensor *t, int64_t count, bool scale, float max_norm,
                             float eps, float *norm, void *ws, const DeviceInfo &dev,
                             cudaStream_t stream);

// ---- products with an epilogue, and by expert (mx_product.cu)
// dense: [M][N] = A[M] . B[N]^T; rows: A's M rows in the experts' segments, B [experts][N];
// depth: [experts][M][N] over the experts' slices of the contraction K.
enum : int { kProductDense = 0, kProductRows = 1, kProductDepth = 2 };
struct Product {
    int mode;
    bool fp8;
    const void *Aq, *As, *Bq, *Bs;
    int64_t M, N, K, experts;
    const int32_t *offsets, *counts;
    const void *bias;
    int bias_f32;
    int act;
    RowIn res;
    void *y;
    int y_f32;
    void *z;
    RowEncode enc;
};
cudaError_t launch_product(const Product &p, const DeviceInfo &dev, cudaStream_t stream);
// Few rows of A (mx_few.cu): whether a product goes there, and its launch.
bool few_rows(const Product &p);
cudaError_t launch_few(const Product &p, const DeviceInfo &dev, cudaStream_t stream);

// ---- gradient of bias and activation (mx_act.cu)
size_t bias_act_backward_ws(int64_t T, int64_t N);
// z null: no activation.  dz (bf16), e and dbias may each be absent.
cudaError_t launch_bias_act_backward(const RowIn &dy, const RowIn &z, int act, int64_t T, int64_t N, void *dz,
                                     const RowEncode &e, float *dbias, void *ws, const DeviceInfo &dev,
                                     cudaStream_t stream);

// ---- rows by expert (mx_experts.cu)
size_t expert_plan_ws(int64_t n, int64_t experts);
// n entries; `rows`: capacity of all segments.
cudaError_t launch_expert_plan(const void *index, bool wide, int64_t n, int64_t experts, int64_t rows,
                               int32_t *offsets, int32_t *counts, int32_t *slot, int32_t *source, void *ws,
                               const DeviceInfo &dev, cudaStream_t stream);
struct ExpertRows {
    const int32_t *slot, *source;
    int64_t T, picks, rows, K;
};
cudaError_t launch_expert_dispatch(const RowIn &x, const ExpertRows &r, void *y, const RowEncode &e,
                                   const DeviceInfo &dev, cudaStream_t stream);
cudaError_t launch_expert_combine(const RowIn &rows, const ExpertRows &r, const float *weights, const RowIn &res,
                                  void *y, int y_f32, const DeviceInfo &dev, cudaStream_t stream);
cudaError_t launch_expert_combine_backward(const RowIn &dy, const RowIn &rows, const ExpertRows &r,
                                           const float *weights, void *drows, const RowEncode &e, float *dweights,
                                           const DeviceInfo &dev, cudaStream_t stream);

}  // namespace mx
