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

}  // extern "C"
