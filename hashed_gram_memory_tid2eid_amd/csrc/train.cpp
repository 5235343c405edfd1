// train.cpp -- the extern "C" entry points of the training operators in include/engram.h:
// argument checks that the host can make, then kernel launches on the caller's stream.
// None allocates or synchronises.
#include <hip/hip_runtime.h>
#include <math.h>

#include "internal.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// bf16 or f32, the types the training operators read and write
inline bool wide_type(int32_t t) { return t == ENGRAM_DTYPE_BF16 || t == ENGRAM_DTYPE_F32; }
inline bool elt_aligned(const void* p, int32_t t) { return aligned(p, t == ENGRAM_DTYPE_F32 ? 4 : 2); }

constexpr int64_t kMax32 = 0x7FFFFFFF;
// places of one lookup gradient: their sorted positions and byte sizes stay in 32 bits
constexpr int64_t kMaxPlaces = (int64_t)1 << 30;
// columns of a lookup gradient: rounded up to whole groups of lanes (2,048 columns) they stay there, too
constexpr int32_t kMaxGradDim = 0x7FFFFFFF - 2047;

int lookup_shape(int64_t rows, int32_t dim, int64_t T, int32_t cols, int64_t ids_ld, int64_t seg_pitch, int64_t ld) {
  if (rows < 1 || rows > kMax32 || dim < 1 || T < 0 || cols < 1) return ENGRAM_E_ARG;
  if (ids_ld < cols || seg_pitch < dim || ld < 0 || ld / seg_pitch < cols) return ENGRAM_E_ARG;
  if (T > kMax32) return ENGRAM_E_UNSUPPORTED;
  return ENGRAM_OK;
}

}  // namespace

extern "C" int engram_embed(const void* d_table, int32_t table_dtype, int64_t rows, int32_t dim, int64_t table_ld,
                            const int32_t* d_ids, int64_t T, int32_t cols, int64_t ids_ld, float scale, void* d_out,
                            int32_t out_dtype, int64_t out_ld, int64_t seg_pitch, hipStream_t stream) {
  if (!wide_type(table_dtype) || !wide_type(out_dtype) || !isfinite(scale)) return ENGRAM_E_ARG;
  const int rc = lookup_shape(rows, dim, T, cols, ids_ld, seg_pitch, out_ld);
  if (rc != ENGRAM_OK) return rc;
  if (table_ld < dim) return ENGRAM_E_ARG;
  if (seg_pitch > kMax32 / cols) return ENGRAM_E_UNSUPPORTED;
  if (T == 0) return ENGRAM_OK;
  if (!d_table || !d_ids || !d_out) return ENGRAM_E_ARG;
  if (!elt_aligned(d_table, table_dtype) || !elt_aligned(d_out, out_dtype) || !aligned(d_ids, 4)) return ENGRAM_E_ALIGN;
  engram::EmbedArgs a;
  a.table = d_table;
  a.rows = rows;
  a.table_ld = table_ld;
  a.dim = dim;
  a.table_f32 = table_dtype == ENGRAM_DTYPE_F32;
  a.ids = d_ids;
  a.T = T;
  a.ids_ld = ids_ld;
  a.cols = cols;
  a.scale = scale;
  a.out = d_out;
  a.out_f32 = out_dtype == ENGRAM_DTYPE_F32;
  a.out_ld = out_ld;
  a.seg_pitch = seg_pitch;
  return engram::hip_error_status(engram::launch_embed(a, stream));
}

extern "C" int engram_embed_grad_workspace(int64_t places, int64_t rows, int32_t dim, int64_t* bytes) {
  if (!bytes || places < 0 || rows < 1 || rows > kMax32 || dim < 1) return ENGRAM_E_ARG;
  if (places > kMaxPlaces || dim > kMaxGradDim) return ENGRAM_E_UNSUPPORTED;
  *bytes = engram::embed_grad_workspace_bytes(places, rows, dim);
  return ENGRAM_OK;
}

extern "C" int engram_embed_grad(const int32_t* d_ids, int64_t T, int32_t cols, int64_t ids_ld, int64_t rows,
                                 int32_t dim, float scale, const void* d_dout, int32_t dout_dtype, int64_t dout_ld,
                                 int64_t seg_pitch, int32_t mode, void* d_grad, int32_t grad_dtype, int64_t grad_ld,
                                 int32_t* d_unique, int32_t* d_count, void* d_work, int64_t work_bytes,
                                 hipStream_t stream) {
  if (!wide_type(dout_dtype) || !wide_type(grad_dtype) || !isfinite(scale)) return ENGRAM_E_ARG;
  if (mode != ENGRAM_GRAD_DENSE && mode != ENGRAM_GRAD_ACCUMULATE && mode != ENGRAM_GRAD_SPARSE) return ENGRAM_E_ARG;
  const int rc = lookup_shape(rows, dim, T, cols, ids_ld, seg_pitch, dout_ld);
  if (rc != ENGRAM_OK) return rc;
  if (grad_ld < dim) return ENGRAM_E_ARG;
  if (T > kMaxPlaces / cols || dim > kMaxGradDim) return ENGRAM_E_UNSUPPORTED;
  const int64_t n = T * cols;
  const bool sparse = mode == ENGRAM_GRAD_SPARSE;
  if (sparse && !d_count) return ENGRAM_E_ARG;
  if (n > 0 && (!d_ids || !d_dout || !d_work || (sparse && !d_unique))) return ENGRAM_E_ARG;
  if ((n > 0 || mode == ENGRAM_GRAD_DENSE) && !d_grad) return ENGRAM_E_ARG;
  if (n > 0 && work_bytes < engram::embed_grad_workspace_bytes(n, rows, dim)) return ENGRAM_E_SCRATCH;
  if (!elt_aligned(d_dout, dout_dtype) || !elt_aligned(d_grad, grad_dtype) || !aligned(d_ids, 4) ||
      !aligned(d_work, 256) || (sparse && (!aligned(d_unique, 4) || !aligned(d_count, 4))))
    return ENGRAM_E_ALIGN;
  if (n == 0 && mode == ENGRAM_GRAD_ACCUMULATE) return ENGRAM_OK;
  engram::EmbedGradArgs a;
  a.ids = d_ids;
  a.T = T;
  a.ids_ld = ids_ld;
  a.cols = cols;
  a.rows = rows;
  a.dim = dim;
  a.scale = scale;
  a.dout = d_dout;
  a.dout_f32 = dout_dtype == ENGRAM_DTYPE_F32;
  a.dout_ld = dout_ld;
  a.seg_pitch = seg_pitch;
  a.grad = d_grad;
  a.grad_f32 = grad_dtype == ENGRAM_DTYPE_F32;
  a.grad_ld = grad_ld;
  a.mode = mode;
  a.unique = d_unique;
  a.count = d_count;
  a.work = d_work;
  return engram::hip_error_status(engram::launch_embed_grad(a, stream));
}

// ---- 8-bit operands and their product -----------------------------------------------

extern "C" int engram_fp8_quantize(const void* d_x, int32_t x_dtype, int64_t M, int64_t K, int64_t x_ld,
                                   int32_t scale_kind, int32_t block_rows, uint8_t* d_q, int64_t q_ld, void* d_scales,
                                   uint8_t* d_qt, int64_t qt_ld, void* d_scales_t, hipStream_t stream) {
  if (!wide_type(x_dtype) || M < 0 || K < 0 || x_ld < K) return ENGRAM_E_ARG;
  if (scale_kind != ENGRAM_FP8_SCALE_F32 && scale_kind != ENGRAM_FP8_SCALE_E8M0) return ENGRAM_E_ARG;
  if (block_rows != 1 && block_rows != 128) return ENGRAM_E_ARG;
  if (!d_q && !d_qt) return ENGRAM_E_ARG;
  if ((d_q && !d_scales) || (d_qt && !d_scales_t)) return ENGRAM_E_ARG;
  if (M > kMax32 - 128 || K > kMax32 - 128) return ENGRAM_E_UNSUPPORTED;
  if (((K + 127) / 128) * ((M + 15) / 16) > kMax32) return ENGRAM_E_UNSUPPORTED;  // one workgroup per tile
  const int64_t k_up = (K + 127) / 128 * 128, m_up = (M + 127) / 128 * 128;
  if (d_q && (q_ld < k_up || q_ld % 16 || !aligned(d_q, 16))) return ENGRAM_E_ALIGN;
  if (d_qt && (qt_ld < m_up || qt_ld % 16 || !aligned(d_qt, 16))) return ENGRAM_E_ALIGN;
  const uintptr_t sa = scale_kind == ENGRAM_FP8_SCALE_F32 ? 4 : 1;
  if ((d_q && !aligned(d_scales, sa)) || (d_qt && !aligned(d_scales_t, sa))) return ENGRAM_E_ALIGN;
  if (M == 0 || K == 0) return ENGRAM_OK;
  if (!d_x) return ENGRAM_E_ARG;
  if (!elt_aligned(d_x, x_dtype)) return ENGRAM_E_ALIGN;
  engram::QuantizeArgs a;
  a.x = d_x;
  a.x_f32 = x_dtype == ENGRAM_DTYPE_F32;
  a.M = M;
  a.K = K;
  a.ld = x_ld;
  a.e8m0 = scale_kind == ENGRAM_FP8_SCALE_E8M0;
  a.block = block_rows;
  a.q = d_q;
  a.q_ld = q_ld;
  a.s = d_scales;
  a.qt = d_qt;
  a.qt_ld = qt_ld;
  a.st = d_scales_t;
  return engram::hip_error_status(engram::launch_fp8_quantize(a, stream));
}

namespace {

int product_shape(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 1 || K % 128 != 0) return ENGRAM_E_ARG;
  if (M > kMax32 - 256 || N > kMax32 - 256 || K > kMax32) return ENGRAM_E_UNSUPPORTED;
  return ENGRAM_OK;
}

}  // namespace

extern "C" int engram_fp8_matmul_workspace(int64_t M, int64_t N, int64_t K, int64_t* bytes) {
  if (!bytes) return ENGRAM_E_ARG;
  const int rc = product_shape(M, N, K);
  if (rc != ENGRAM_OK) return rc;
  *bytes = M == 0 || N == 0 ? 0 : engram::gemm_fp8_workspace_bytes(M, N, K / 128);
  return ENGRAM_OK;
}

extern "C" int engram_fp8_matmul(const uint8_t* d_a, int64_t a_ld, const void* d_sa, const uint8_t* d_b, int64_t b_ld,
                                 const void* d_sb, int32_t b_block_rows, int32_t scale_kind, int64_t M, int64_t N,
                                 int64_t K, void* d_c, int32_t c_dtype, int64_t c_ld, void* d_work, int64_t work_bytes,
                                 hipStream_t stream) {
  if (!wide_type(c_dtype) || (b_block_rows != 1 && b_block_rows != 128)) return ENGRAM_E_ARG;
  if (scale_kind != ENGRAM_FP8_SCALE_F32 && scale_kind != ENGRAM_FP8_SCALE_E8M0) return ENGRAM_E_ARG;
  const int rc = product_shape(M, N, K);
  if (rc != ENGRAM_OK) return rc;
  if (a_ld < K || b_ld < K || c_ld < N) return ENGRAM_E_ARG;
  if (M == 0 || N == 0) return ENGRAM_OK;
  if (!d_a || !d_sa || !d_b || !d_sb || !d_c) return ENGRAM_E_ARG;
  const uintptr_t sa = scale_kind == ENGRAM_FP8_SCALE_F32 ? 4 : 1;
  if (a_ld % 16 || b_ld % 16 || !aligned(d_a, 16) || !aligned(d_b, 16) || !aligned(d_sa, sa) || !aligned(d_sb, sa) ||
      !elt_aligned(d_c, c_dtype))
    return ENGRAM_E_ALIGN;
  // one tile's rows are addressed with 32-bit byte offsets
  if (a_ld > kMax32 / 256 || b_ld > kMax32 / 256) return ENGRAM_E_UNSUPPORTED;
  const int64_t need = engram::gemm_fp8_workspace_bytes(M, N, K / 128);
  if (need > 0 && (!d_work || work_bytes < need)) return ENGRAM_E_SCRATCH;
  if (need > 0 && !aligned(d_work, 16)) return ENGRAM_E_ALIGN;
  engram::GemmFp8Args a;
  a.A = d_a;
  a.sa = d_sa;
  a.B = d_b;
  a.sb = d_sb;
  a.lda = a_ld;
  a.ldb = b_ld;
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.KB = (int32_t)(K / 128);
  a.b_block = b_block_rows;
  a.e8m0 = scale_kind == ENGRAM_FP8_SCALE_E8M0;
  a.C = d_c;
  a.c_f32 = c_dtype == ENGRAM_DTYPE_F32;
  a.ldc = c_ld;
  a.work = static_cast<float*>(d_work);
  return engram::hip_error_status(engram::launch_gemm_fp8(a, stream));
}

// ---- the gate's backward pass --------------------------------------------------------

extern "C" int engram_gate_add_backward(const float* d_v, const void* d_streams, const uint8_t* d_keep,
                                        const void* d_dy, int32_t hidden, int32_t hc_mult, void* d_dx, float* d_dv,
                                        int32_t T, hipStream_t stream) {
  if (T < 0) return ENGRAM_E_ARG;
  if (hc_mult != 4) return ENGRAM_E_UNSUPPORTED;
  if (hidden < 8 || hidden % 8 != 0) return ENGRAM_E_ALIGN;
  if (hidden > 8192) return ENGRAM_E_UNSUPPORTED;
  if (T == 0) return ENGRAM_OK;
  if (!d_v || !d_streams || !d_dy || !d_dx || !d_dv) return ENGRAM_E_ARG;
  if (!aligned(d_v, 16) || !aligned(d_streams, 16) || !aligned(d_dy, 16) || !aligned(d_dx, 16) || !aligned(d_dv, 16))
    return ENGRAM_E_ALIGN;
  engram::GateBackwardArgs a;
  a.v = d_v;
  a.x = d_streams;
  a.dy = d_dy;
  a.keep = d_keep;
  a.dx = d_dx;
  a.dv = d_dv;
  a.T = T;
  a.hidden = hidden;
  a.inv_sqrt_hidden = (float)(1.0 / sqrt((double)hidden));
  return engram::hip_error_status(engram::launch_gate_backward(a, stream));
}
