// mx_launch.hpp -- internal host launchers of the MX operators behind the C
// ABI (arguments are checked by the caller, mx_api.cpp).
#pragma once

#include "launch.hpp"

namespace mxfp8 {

// Rows of cols elements, cols % 32 == 0, into E2M1 codes (ldq bytes a row).
void launch_mxfp4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int rule, uint8_t* q,
                           int64_t ldq, uint8_t* s, hipStream_t stream);
// Codes and scales back to values.
void launch_mx_dequantize(const uint8_t* q, int64_t ldq, int fmt, const uint8_t* s, int64_t rows, int64_t cols,
                          void* y, int y_dtype, int64_t ldy, hipStream_t stream);
// 32-token blocks down columns, transposed codes; rows_out % 32 == 0, rows_out >= rows, cols % 16 == 0.
void launch_mx_quantize_t(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int fmt, int rule,
                          uint8_t* qt, int64_t ldqt, int64_t rows_out, uint8_t* st, hipStream_t stream);
// The same from FP8 codes with scales per 32 columns; cols % 32 == 0.
void launch_mx_requantize_t(const uint8_t* q, int64_t ldq, int q_fmt, const uint8_t* s, int64_t rows, int64_t cols,
                            int fmt, int rule, uint8_t* qt, int64_t ldqt, int64_t rows_out, uint8_t* st,
                            hipStream_t stream);
// SwiGLU of x [rows][2 cols]; kept may be null.  cols % 32 == 0.
void launch_mx_swiglu_forward(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int fmt, int rule,
                              uint8_t* h, int64_t ldh, uint8_t* hs, uint8_t* kept, int64_t ldk, uint8_t* ks,
                              hipStream_t stream);
void launch_mx_swiglu_backward(const uint8_t* kept, int64_t ldk, const uint8_t* ks, int fmt, const void* dh, int dtype,
                               int64_t lddh, int64_t rows, int64_t cols, void* dx, int64_t lddx, hipStream_t stream);
// RMSNorm; kept may be null.  cols % 32 == 0, cols <= kMaxNormCols.
constexpr int64_t kMaxNormCols = 32768;
void launch_mx_rmsnorm_forward(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, const float* w,
                               float eps, int fmt, int rule, uint8_t* y, int64_t ldy, uint8_t* ys, uint8_t* kept,
                               int64_t ldk, uint8_t* ks, float* rstd, hipStream_t stream);
// Partial sums of dw that the backward pass leaves in its workspace (rows of cols floats).
int64_t rmsnorm_backward_parts(int64_t rows, int64_t cols);
void launch_mx_rmsnorm_backward(const uint8_t* kept, int64_t ldk, const uint8_t* ks, const float* rstd, int fmt,
                                const float* w, const void* dy, int dtype, int64_t lddy, int64_t rows, int64_t cols,
                                void* dx, int64_t lddx, float* dw, float* workspace, int64_t parts,
                                hipStream_t stream);
// LayerNorm; kept, b, or w and b may be null.  cols % 32 == 0, cols <= kMaxNormCols.
void launch_mx_layernorm_forward(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, const float* w,
                                 const float* b, float eps, int fmt, int rule, uint8_t* y, int64_t ldy, uint8_t* ys,
                                 uint8_t* kept, int64_t ldk, uint8_t* ks, float* rstd, hipStream_t stream);
// Partial sums of dw and db that the backward pass leaves in its workspace (rows of 2 cols floats).
int64_t layernorm_backward_parts(int64_t rows, int64_t cols);
// dw and db may both be null.
void launch_mx_layernorm_backward(const uint8_t* kept, int64_t ldk, const uint8_t* ks, const float* rstd, int fmt,
                                  const float* w, const void* dy, int dtype, int64_t lddy, int64_t rows, int64_t cols,
                                  void* dx, int64_t lddx, float* dw, float* db, float* workspace, hipStream_t stream);
// C = A B^T, B in E2M1, scales per 32 of K.  K % 128 == 0, M, N >= 1, scale pointers 4-byte aligned.
void launch_mxfp4_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, int a_fmt, const uint8_t* sa,
                       const uint8_t* b, int64_t ldb, const uint8_t* sb, void* c, int64_t ldc, int c_dtype,
                       hipStream_t stream);
// Whether the few-row kernel takes that product on a device of `cus` compute units; tiles do otherwise.  Up to 16 rows
// it is the same on every device, so what a caller's workspace holds can go by it.
constexpr int64_t kFewRowsN = int64_t(1) << 26;
bool mxfp4_few_rows(int64_t M, int64_t N, int64_t K, int64_t cus);
// The same and, for row m with a = ids[m] in 0 .. adapters - 1, up[a] p[m] added: p [M][rank], and packed, adapter
// a's [N][ldu] bf16 from up + a stride.  rank, ldu and stride are multiples of 8, ldu <= 2^22.  The few-row kernel
// does not read packed.
void launch_mxfp4_gemm_adapted(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, int a_fmt,
                               const uint8_t* sa, const uint8_t* b, int64_t ldb, const uint8_t* sb, const int32_t* ids,
                               int64_t adapters, int64_t rank, const float* p, const uint16_t* packed,
                               const uint16_t* up, int64_t ldu,
                               int64_t stride, void* c, int64_t ldc, int c_dtype, hipStream_t stream);
// p[m] = alpha[a] down[a] x[m], zeros without an adapter; adapter a's [rank][ldd] bf16 from down + a stride, alpha
// may be null (ones).  K % 128 == 0, scale pointers 4-byte aligned, M <= kMaxAdapterRows.  Bytes of workspace.
constexpr int64_t kMaxAdapterRows = int64_t(1) << 27, kMaxRank = 256;
void launch_mx_adapter_project(int64_t M, int64_t K, const uint8_t* a, int64_t lda, int a_fmt, const uint8_t* sa,
                               const int32_t* ids, int64_t adapters, int64_t rank, const uint16_t* down, int64_t ldd,
                               int64_t stride, const float* alpha, float* p, uint16_t* packed, float* workspace,
                               hipStream_t stream);
int64_t adapter_project_workspace(int64_t M, int64_t K, int64_t rank);
// p as the product's tiles read it (packed above; may be null where the few-row kernel follows).
int64_t adapter_packed_bytes(int64_t M, int64_t rank);
// out[a] = the sum over the rows m of adapter a of p[m] (x) z[m], [rank][C], or [C][rank] if transposed.  C % 32 ==
// 0, all extents >= 1.  Bytes of workspace, and workgroups (fewer than 2^24).
int64_t adapter_grad_workspace(int64_t M, int64_t C, int64_t rank, int64_t adapters);
int64_t adapter_grad_groups(int64_t M, int64_t C, int64_t rank, int64_t adapters);
void launch_mx_adapter_grad(int64_t M, int64_t C, const uint8_t* z, int64_t ldz, int z_fmt, const uint8_t* sz,
                            const float* p, int64_t rank, const int32_t* ids, int64_t adapters, int transposed,
                            float* out, void* workspace, hipStream_t stream);

}  // namespace mxfp8
