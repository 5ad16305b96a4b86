// mx_api.cpp -- the C ABI of the MX operators (declared in include/mxfp8.h):
// host-side argument validation, then dispatch.  As in api.cpp, validation
// runs before any HIP call.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <initializer_list>

#include "../../include/mxfp8.h"
#include "mx_launch.hpp"

namespace {

// The product addresses a tile of up to 256 rows, and K along them, with
// offsets below 2^31.
constexpr int64_t kMaxGemmLd = int64_t(1) << 22;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool fp8(int fmt) { return fmt == MXFP8_E4M3 || fmt == MXFP8_E5M2; }
bool element(int fmt) { return fp8(fmt) || fmt == MXFP8_E2M1; }
bool real(int dtype) { return dtype == MXFP8_F32 || dtype == MXFP8_BF16; }
bool rule_ok(int rule) { return rule == MXFP8_RULE_CEIL || rule == MXFP8_RULE_FLOOR; }
bool extents(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= INT32_MAX && cols <= INT32_MAX / 2;
}
bool ld_ok(int64_t ld, int64_t row) { return ld >= row && ld % 16 == 0; }
int64_t code_bytes(int64_t n, int fmt) { return fmt == MXFP8_E2M1 ? n / 2 : n; }

// Whether any output equals another output or an input (null pointers aside).
bool shared(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    if (!*o) continue;
    for (auto p = outs.begin(); p != o; ++p)
      if (*p == *o) return true;
    for (const void* i : ins)
      if (i == *o) return true;
  }
  return false;
}

int launch_status() { return hipGetLastError() == hipSuccess ? MXFP8_OK : MXFP8_ERR_DEVICE; }

// Rows, adapters and their rank.
bool adapter_extents(int64_t M, int64_t adapters, int64_t rank) {
  return M >= 0 && M <= mxfp8::kMaxAdapterRows && adapters >= 0 && adapters <= INT32_MAX / 2 && rank >= 8 &&
         rank <= mxfp8::kMaxRank && rank % 8 == 0;
}
// Leading dimension of an adapter's matrix, and the stride from one to the next.
bool adapter_ld(int64_t ld, int64_t row, int64_t stride) {
  return ld >= row && ld % 8 == 0 && ld <= kMaxGemmLd && stride >= 0 && stride % 8 == 0;
}
// p in the order in which the product's tiles read it; none where the few-row kernel takes the product on every device
// (one without compute units stands for that), since the device of the workspace's query need not be the call's.
int64_t packed_bytes(int64_t M, int64_t N, int64_t K, int64_t rank) {
  return N > 0 && !mxfp8::mxfp4_few_rows(M, N, K, 0) ? mxfp8::adapter_packed_bytes(M, rank) : 0;
}
bool grad_extents(int64_t M, int64_t C, int64_t rank, int64_t adapters) {
  if (!adapter_extents(M, adapters, rank) || C < 0 || C > INT32_MAX / 2 || C % 32 != 0) return false;
  // A launch takes fewer than 2^32 threads.
  return C == 0 || adapters == 0 || mxfp8::adapter_grad_groups(M, C, rank, adapters) < (int64_t(1) << 24);
}

// Extents of the transposing quantizers.
int transposed_extents(int64_t rows, int64_t cols, int64_t rows_out, int64_t multiple) {
  if (!extents(rows, cols) || rows_out < rows || rows_out > INT32_MAX) return MXFP8_ERR_SHAPE;
  if (cols % multiple != 0 || rows_out % 32 != 0) return MXFP8_ERR_SHAPE;
  // The grid is the tiles rounded up to a multiple of 8, of at most 512 threads
  // each; a launch takes fewer than 2^32 threads.
  if (((cols + 127) / 128) * ((rows_out + 127) / 128) > (int64_t(1) << 23) - 8) return MXFP8_ERR_SHAPE;
  return MXFP8_OK;
}

}  // namespace

extern "C" {

int mxfp4_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int rule, uint8_t* q,
                   int64_t ldq, uint8_t* scales, void* stream) {
  if (!real(x_dtype) || !rule_ok(rule)) return MXFP8_ERR_ENUM;
  if (!extents(rows, cols) || cols % 32 != 0) return MXFP8_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MXFP8_OK;
  if (!x || !q || !scales) return MXFP8_ERR_NULL;
  if (!ld_ok(ldx, cols) || !ld_ok(ldq, cols / 2)) return MXFP8_ERR_LD;
  if (!aligned16(x) || !aligned16(q)) return MXFP8_ERR_ALIGN;
  if (shared({q, scales}, {x})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();  // clear any stale error so the launch status is ours
  mxfp8::launch_mxfp4_quantize(x, x_dtype, rows, cols, ldx, rule, q, ldq, scales, (hipStream_t)stream);
  return launch_status();
}

int mx_dequantize(const uint8_t* q, int64_t ldq, int fmt, const uint8_t* scales, int64_t rows, int64_t cols, void* y,
                  int y_dtype, int64_t ldy, void* stream) {
  if (!real(y_dtype) || !element(fmt)) return MXFP8_ERR_ENUM;
  if (!extents(rows, cols) || cols % 32 != 0) return MXFP8_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MXFP8_OK;
  if (!q || !scales || !y) return MXFP8_ERR_NULL;
  if (!ld_ok(ldq, code_bytes(cols, fmt)) || !ld_ok(ldy, cols)) return MXFP8_ERR_LD;
  if (!aligned16(q) || !aligned16(y)) return MXFP8_ERR_ALIGN;
  if (shared({y}, {q, scales})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_dequantize(q, ldq, fmt, scales, rows, cols, y, y_dtype, ldy, (hipStream_t)stream);
  return launch_status();
}

int mx_quantize_t(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int fmt, int rule, uint8_t* qt,
                  int64_t ldqt, int64_t rows_out, uint8_t* scales_t, void* stream) {
  if (!real(x_dtype) || !element(fmt) || !rule_ok(rule)) return MXFP8_ERR_ENUM;
  const int st = transposed_extents(rows, cols, rows_out, 16);
  if (st != MXFP8_OK || rows_out == 0 || cols == 0) return st;
  if ((!x && rows > 0) || !qt || !scales_t) return MXFP8_ERR_NULL;
  if ((rows > 0 && !ld_ok(ldx, cols)) || !ld_ok(ldqt, code_bytes(rows_out, fmt))) return MXFP8_ERR_LD;
  if (!aligned16(x) || !aligned16(qt)) return MXFP8_ERR_ALIGN;
  if (shared({qt, scales_t}, {x})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_quantize_t(x, x_dtype, rows, cols, ldx, fmt, rule, qt, ldqt, rows_out, scales_t,
                              (hipStream_t)stream);
  return launch_status();
}

int mx_requantize_t(const uint8_t* q, int64_t ldq, int q_fmt, const uint8_t* scales, int64_t rows, int64_t cols,
                    int fmt, int rule, uint8_t* qt, int64_t ldqt, int64_t rows_out, uint8_t* scales_t, void* stream) {
  if (!fp8(q_fmt) || !element(fmt) || !rule_ok(rule)) return MXFP8_ERR_ENUM;
  const int st = transposed_extents(rows, cols, rows_out, 32);
  if (st != MXFP8_OK || rows_out == 0 || cols == 0) return st;
  if ((rows > 0 && (!q || !scales)) || !qt || !scales_t) return MXFP8_ERR_NULL;
  if ((rows > 0 && !ld_ok(ldq, cols)) || !ld_ok(ldqt, code_bytes(rows_out, fmt))) return MXFP8_ERR_LD;
  if (!aligned16(q) || !aligned16(qt)) return MXFP8_ERR_ALIGN;
  if (shared({qt, scales_t}, {q, scales})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_requantize_t(q, ldq, q_fmt, scales, rows, cols, fmt, rule, qt, ldqt, rows_out, scales_t,
                                (hipStream_t)stream);
  return launch_status();
}

int mxfp4_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, int a_fmt, const uint8_t* a_scales,
               const uint8_t* b, int64_t ldb, const uint8_t* b_scales, void* c, int64_t ldc, int c_dtype,
               void* stream) {
  if (!element(a_fmt) || !real(c_dtype)) return MXFP8_ERR_ENUM;
  if (M < 0 || N < 0 || K < 0) return MXFP8_ERR_SHAPE;
  if (M > INT32_MAX / 2 || N > INT32_MAX / 2 || K > INT32_MAX / 2) return MXFP8_ERR_SHAPE;
  if (K % 128 != 0) return MXFP8_ERR_SHAPE;
  if (M == 0 || N == 0) return MXFP8_OK;
  if (!c) return MXFP8_ERR_NULL;
  if (K > 0 && (!a || !a_scales || !b || !b_scales)) return MXFP8_ERR_NULL;
  if (!ld_ok(ldc, N)) return MXFP8_ERR_LD;
  if (K > 0) {
    if (!ld_ok(lda, code_bytes(K, a_fmt)) || !ld_ok(ldb, K / 2)) return MXFP8_ERR_LD;
    if (lda > kMaxGemmLd || ldb > kMaxGemmLd) return MXFP8_ERR_LD;
    if (!aligned16(a) || !aligned16(b)) return MXFP8_ERR_ALIGN;
    if (((uintptr_t)a_scales & 3) || ((uintptr_t)b_scales & 3)) return MXFP8_ERR_ALIGN;
  }
  if (!aligned16(c)) return MXFP8_ERR_ALIGN;
  if (shared({c}, {a, b, a_scales, b_scales})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mxfp4_gemm(M, N, K, a, lda, a_fmt, a_scales, b, ldb, b_scales, c, ldc, c_dtype, (hipStream_t)stream);
  return launch_status();
}

int mx_swiglu_forward(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int fmt, int rule,
                      uint8_t* h, int64_t ldh, uint8_t* h_scales, uint8_t* kept, int64_t ldk, uint8_t* kept_scales,
                      void* stream) {
  if (!real(x_dtype) || !fp8(fmt) || !rule_ok(rule)) return MXFP8_ERR_ENUM;
  if (!extents(rows, cols) || cols % 32 != 0) return MXFP8_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MXFP8_OK;
  if (!x || !h || !h_scales || (!kept != !kept_scales)) return MXFP8_ERR_NULL;
  if (!ld_ok(ldx, 2 * cols) || !ld_ok(ldh, cols) || (kept && !ld_ok(ldk, 2 * cols))) return MXFP8_ERR_LD;
  if (!aligned16(x) || !aligned16(h) || !aligned16(kept)) return MXFP8_ERR_ALIGN;
  if (shared({h, h_scales, kept, kept_scales}, {x})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_swiglu_forward(x, x_dtype, rows, cols, ldx, fmt, rule, h, ldh, h_scales, kept, ldk, kept_scales,
                                  (hipStream_t)stream);
  return launch_status();
}

int mx_swiglu_backward(const uint8_t* kept, int64_t ldk, const uint8_t* kept_scales, int fmt, const void* dh,
                       int dtype, int64_t lddh, int64_t rows, int64_t cols, void* dx, int64_t lddx, void* stream) {
  if (!real(dtype) || !fp8(fmt)) return MXFP8_ERR_ENUM;
  if (!extents(rows, cols) || cols % 32 != 0) return MXFP8_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MXFP8_OK;
  if (!kept || !kept_scales || !dh || !dx) return MXFP8_ERR_NULL;
  if (!ld_ok(ldk, 2 * cols) || !ld_ok(lddh, cols) || !ld_ok(lddx, 2 * cols)) return MXFP8_ERR_LD;
  if (!aligned16(kept) || !aligned16(dh) || !aligned16(dx)) return MXFP8_ERR_ALIGN;
  if (shared({dx}, {kept, kept_scales, dh})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_swiglu_backward(kept, ldk, kept_scales, fmt, dh, dtype, lddh, rows, cols, dx, lddx,
                                   (hipStream_t)stream);
  return launch_status();
}

int mx_rmsnorm_forward(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const float* w, float eps,
                       int fmt, int rule, uint8_t* y, int64_t ldy, uint8_t* y_scales, uint8_t* kept, int64_t ldk,
                       uint8_t* kept_scales, float* rstd, void* stream) {
  if (!real(x_dtype) || !fp8(fmt) || !rule_ok(rule)) return MXFP8_ERR_ENUM;
  if (!extents(rows, cols) || cols % 32 != 0 || cols > mxfp8::kMaxNormCols) return MXFP8_ERR_SHAPE;
  if (!(eps >= 0.0f && eps <= 3.4e38f)) return MXFP8_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MXFP8_OK;
  if (!x || !w || !y || !y_scales || (!kept != !kept_scales) || (!kept != !rstd)) return MXFP8_ERR_NULL;
  if (!ld_ok(ldx, cols) || !ld_ok(ldy, cols) || (kept && !ld_ok(ldk, cols))) return MXFP8_ERR_LD;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(kept) || ((uintptr_t)rstd & 3))
    return MXFP8_ERR_ALIGN;
  if (shared({y, y_scales, kept, kept_scales, rstd}, {x, w})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_rmsnorm_forward(x, x_dtype, rows, cols, ldx, w, eps, fmt, rule, y, ldy, y_scales, kept, ldk,
                                   kept_scales, rstd, (hipStream_t)stream);
  return launch_status();
}

int64_t mx_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  if (!extents(rows, cols) || cols % 32 != 0 || cols > mxfp8::kMaxNormCols || cols == 0) return 0;
  return mxfp8::rmsnorm_backward_parts(rows, cols) * cols * (int64_t)sizeof(float);
}

int mx_rmsnorm_backward(const uint8_t* kept, int64_t ldk, const uint8_t* kept_scales, const float* rstd, int fmt,
                        const float* w, const void* dy, int dtype, int64_t lddy, int64_t rows, int64_t cols, void* dx,
                        int64_t lddx, float* dw, void* workspace, void* stream) {
  if (!real(dtype) || !fp8(fmt)) return MXFP8_ERR_ENUM;
  if (!extents(rows, cols) || cols % 32 != 0 || cols > mxfp8::kMaxNormCols) return MXFP8_ERR_SHAPE;
  if (cols == 0) return MXFP8_OK;
  if (!dw || (rows > 0 && (!kept || !kept_scales || !rstd || !w || !dy || !dx || !workspace))) return MXFP8_ERR_NULL;
  if (rows > 0 && (!ld_ok(ldk, cols) || !ld_ok(lddy, cols) || !ld_ok(lddx, cols))) return MXFP8_ERR_LD;
  if (!aligned16(kept) || !aligned16(dy) || !aligned16(dx) || !aligned16(w) || !aligned16(dw) ||
      !aligned16(workspace) || ((uintptr_t)rstd & 3))
    return MXFP8_ERR_ALIGN;
  if (shared({dx, dw, workspace}, {kept, kept_scales, rstd, w, dy})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_rmsnorm_backward(kept, ldk, kept_scales, rstd, fmt, w, dy, dtype, lddy, rows, cols, dx, lddx, dw,
                                    static_cast<float*>(workspace), mxfp8::rmsnorm_backward_parts(rows, cols),
                                    (hipStream_t)stream);
  return launch_status();
}

int mx_layernorm_forward(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const float* w,
                         const float* b, float eps, int fmt, int rule, uint8_t* y, int64_t ldy, uint8_t* y_scales,
                         uint8_t* kept, int64_t ldk, uint8_t* kept_scales, float* rstd, void* stream) {
  if (!real(x_dtype) || !fp8(fmt) || !rule_ok(rule)) return MXFP8_ERR_ENUM;
  if (!extents(rows, cols) || cols % 32 != 0 || cols > mxfp8::kMaxNormCols) return MXFP8_ERR_SHAPE;
  if (!(eps >= 0.0f && eps <= 3.4e38f)) return MXFP8_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MXFP8_OK;
  if (!x || !y || !y_scales || (b && !w) || (!kept != !kept_scales) || (!kept != !rstd)) return MXFP8_ERR_NULL;
  if (!ld_ok(ldx, cols) || !ld_ok(ldy, cols) || (kept && !ld_ok(ldk, cols))) return MXFP8_ERR_LD;
  if (!aligned16(x) || !aligned16(w) || !aligned16(b) || !aligned16(y) || !aligned16(kept) || ((uintptr_t)rstd & 3))
    return MXFP8_ERR_ALIGN;
  if (shared({y, y_scales, kept, kept_scales, rstd}, {x, w, b})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_layernorm_forward(x, x_dtype, rows, cols, ldx, w, b, eps, fmt, rule, y, ldy, y_scales, kept, ldk,
                                     kept_scales, rstd, (hipStream_t)stream);
  return launch_status();
}

int64_t mx_layernorm_backward_workspace(int64_t rows, int64_t cols) {
  if (!extents(rows, cols) || cols % 32 != 0 || cols > mxfp8::kMaxNormCols || cols == 0) return 0;
  return mxfp8::layernorm_backward_parts(rows, cols) * 2 * cols * (int64_t)sizeof(float);
}

int mx_layernorm_backward(const uint8_t* kept, int64_t ldk, const uint8_t* kept_scales, const float* rstd, int fmt,
                          const float* w, const void* dy, int dtype, int64_t lddy, int64_t rows, int64_t cols,
                          void* dx, int64_t lddx, float* dw, float* db, void* workspace, void* stream) {
  if (!real(dtype) || !fp8(fmt)) return MXFP8_ERR_ENUM;
  if (!extents(rows, cols) || cols % 32 != 0 || cols > mxfp8::kMaxNormCols) return MXFP8_ERR_SHAPE;
  if (cols == 0) return MXFP8_OK;
  if (!dw != !db || (rows > 0 && (!kept || !kept_scales || !rstd || !dy || !dx || (dw && !workspace))))
    return MXFP8_ERR_NULL;
  if (rows > 0 && (!ld_ok(ldk, cols) || !ld_ok(lddy, cols) || !ld_ok(lddx, cols))) return MXFP8_ERR_LD;
  if (!aligned16(kept) || !aligned16(dy) || !aligned16(dx) || !aligned16(w) || !aligned16(dw) || !aligned16(db) ||
      !aligned16(workspace) || ((uintptr_t)rstd & 3))
    return MXFP8_ERR_ALIGN;
  if (shared({dx, dw, db, workspace}, {kept, kept_scales, rstd, w, dy})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_layernorm_backward(kept, ldk, kept_scales, rstd, fmt, w, dy, dtype, lddy, rows, cols, dx, lddx, dw,
                                      db, static_cast<float*>(workspace), (hipStream_t)stream);
  return launch_status();
}

int mx_adapter_project(int64_t M, int64_t K, const uint8_t* a, int64_t lda, int a_fmt, const uint8_t* a_scales,
                       const int32_t* ids, int64_t adapters, int64_t rank, const uint16_t* down, int64_t ldd,
                       int64_t down_stride, const float* alpha, float* p, void* workspace, void* stream) {
  if (!element(a_fmt)) return MXFP8_ERR_ENUM;
  if (!adapter_extents(M, adapters, rank) || K < 0 || K > INT32_MAX / 2 || K % 128 != 0) return MXFP8_ERR_SHAPE;
  if (M == 0) return MXFP8_OK;
  if (!p || !ids || (K > 0 && (!a || !a_scales || (adapters > 0 && !down)))) return MXFP8_ERR_NULL;
  const bool work = mxfp8::adapter_project_workspace(M, K, rank) > 0;
  if (work && !workspace) return MXFP8_ERR_NULL;
  if (K > 0) {
    if (!ld_ok(lda, code_bytes(K, a_fmt)) || lda > kMaxGemmLd) return MXFP8_ERR_LD;
    if (adapters > 0 && !adapter_ld(ldd, K, down_stride)) return MXFP8_ERR_LD;
  }
  if (!aligned16(a) || !aligned16(down) || !aligned16(p) || !aligned16(workspace)) return MXFP8_ERR_ALIGN;
  if (((uintptr_t)a_scales | (uintptr_t)ids | (uintptr_t)alpha) & 3) return MXFP8_ERR_ALIGN;
  if (shared({p, work ? workspace : nullptr}, {a, a_scales, ids, down, alpha})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_adapter_project(M, K, a, lda, a_fmt, a_scales, ids, adapters, rank, down, ldd, down_stride, alpha, p,
                                   nullptr, static_cast<float*>(workspace), (hipStream_t)stream);
  return launch_status();
}

int64_t mxfp4_gemm_adapted_workspace(int64_t M, int64_t N, int64_t K, int64_t rank) {
  if (N < 0 || N > INT32_MAX / 2 || !adapter_extents(M, 0, rank) || M == 0) return 0;
  if (K < 0 || K > INT32_MAX / 2 || K % 128 != 0) return 0;
  return packed_bytes(M, N, K, rank) + mxfp8::adapter_project_workspace(M, K, rank);
}

int mxfp4_gemm_adapted(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, int a_fmt,
                       const uint8_t* a_scales, const uint8_t* b, int64_t ldb, const uint8_t* b_scales,
                       const int32_t* ids, int64_t adapters, int64_t rank, const uint16_t* down, int64_t ldd,
                       int64_t down_stride, const uint16_t* up, int64_t ldu, int64_t up_stride, const float* alpha,
                       float* p, void* c, int64_t ldc, int c_dtype, void* workspace, void* stream) {
  if (!element(a_fmt) || !real(c_dtype)) return MXFP8_ERR_ENUM;
  if (!adapter_extents(M, adapters, rank) || N < 0 || K < 0) return MXFP8_ERR_SHAPE;
  if (N > INT32_MAX / 2 || K > INT32_MAX / 2 || K % 128 != 0) return MXFP8_ERR_SHAPE;
  if (M == 0) return MXFP8_OK;
  if (!p || !ids || (N > 0 && !c)) return MXFP8_ERR_NULL;
  if (K > 0 && (!a || !a_scales || (adapters > 0 && !down) || (N > 0 && (!b || !b_scales)))) return MXFP8_ERR_NULL;
  const bool work = mxfp4_gemm_adapted_workspace(M, N, K, rank) > 0;
  if ((N > 0 && adapters > 0 && !up) || (work && !workspace)) return MXFP8_ERR_NULL;
  if (N > 0 && !ld_ok(ldc, N)) return MXFP8_ERR_LD;
  if (K > 0) {
    if (!ld_ok(lda, code_bytes(K, a_fmt)) || lda > kMaxGemmLd) return MXFP8_ERR_LD;
    if (N > 0 && (!ld_ok(ldb, K / 2) || ldb > kMaxGemmLd)) return MXFP8_ERR_LD;
    if (adapters > 0 && !adapter_ld(ldd, K, down_stride)) return MXFP8_ERR_LD;
  }
  if (N > 0 && adapters > 0 && !adapter_ld(ldu, rank, up_stride)) return MXFP8_ERR_LD;
  if (!aligned16(a) || !aligned16(b) || !aligned16(down) || !aligned16(up) || !aligned16(p) || !aligned16(c) ||
      !aligned16(workspace))
    return MXFP8_ERR_ALIGN;
  if (((uintptr_t)a_scales | (uintptr_t)b_scales | (uintptr_t)ids | (uintptr_t)alpha) & 3) return MXFP8_ERR_ALIGN;
  if (shared({c, p, work ? workspace : nullptr}, {a, b, a_scales, b_scales, ids, down, up, alpha}))
    return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  // The packed p first (a whole number of kilobytes), then the projection's runs.  It is written where the tiles read it.
  const int64_t before = packed_bytes(M, N, K, rank);
  const bool tiles = before > 0 && !mxfp8::mxfp4_few_rows(M, N, K, mxfp8::device_cus());
  uint16_t* packed = tiles ? static_cast<uint16_t*>(workspace) : nullptr;
  float* runs = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + before);
  mxfp8::launch_mx_adapter_project(M, K, a, lda, a_fmt, a_scales, ids, adapters, rank, down, ldd, down_stride, alpha, p,
                                   packed, runs, (hipStream_t)stream);
  if (N > 0)
    mxfp8::launch_mxfp4_gemm_adapted(M, N, K, a, lda, a_fmt, a_scales, b, ldb, b_scales, ids, adapters, rank, p, packed,
                                     up, ldu, up_stride, c, ldc, c_dtype, (hipStream_t)stream);
  return launch_status();
}

int64_t mx_adapter_project_workspace(int64_t M, int64_t K, int64_t rank) {
  if (!adapter_extents(M, 0, rank) || K < 0 || K > INT32_MAX / 2 || K % 128 != 0 || M == 0) return 0;
  return mxfp8::adapter_project_workspace(M, K, rank);
}

int64_t mx_adapter_grad_workspace(int64_t M, int64_t C, int64_t rank, int64_t adapters) {
  if (!grad_extents(M, C, rank, adapters) || M == 0 || C == 0 || adapters == 0) return 0;
  return mxfp8::adapter_grad_workspace(M, C, rank, adapters);
}

int mx_adapter_grad(int64_t M, int64_t C, const uint8_t* z, int64_t ldz, int z_fmt, const uint8_t* z_scales,
                    const float* p, int64_t rank, const int32_t* ids, int64_t adapters, int transposed, float* grad,
                    void* workspace, void* stream) {
  if (!element(z_fmt)) return MXFP8_ERR_ENUM;
  if (!grad_extents(M, C, rank, adapters)) return MXFP8_ERR_SHAPE;
  if (C == 0 || adapters == 0) return MXFP8_OK;
  const bool work = M > 0 && mxfp8::adapter_grad_workspace(M, C, rank, adapters) > 0;
  if (!grad || (M > 0 && (!z || !z_scales || !p || !ids)) || (work && !workspace)) return MXFP8_ERR_NULL;
  if (M > 0 && (!ld_ok(ldz, code_bytes(C, z_fmt)) || ldz > kMaxGemmLd)) return MXFP8_ERR_LD;
  if (!aligned16(z) || !aligned16(p) || !aligned16(grad) || !aligned16(workspace) || ((uintptr_t)ids & 3))
    return MXFP8_ERR_ALIGN;
  if (shared({grad, work ? workspace : nullptr}, {z, z_scales, p, ids})) return MXFP8_ERR_ALIAS;
  (void)hipGetLastError();
  mxfp8::launch_mx_adapter_grad(M, C, z, ldz, z_fmt, z_scales, p, rank, ids, adapters, transposed, grad, workspace,
                                (hipStream_t)stream);
  return launch_status();
}

}  // extern "C"
