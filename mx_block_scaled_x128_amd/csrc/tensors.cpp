// tensors.cpp -- the tensor functions of the MX operators as a Python
// extension (_mx_tensors): checks of the tensors, allocation of the outputs and
// one call of the C ABI each.  The same checks in Python cost about 9 us a
// call, several times what the small kernels take; here they cost under one.
// Nothing computes here, and the C functions are those of the library that
// mx_block_scaled_x128_amd loads (bind).
#include <ATen/ATen.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/extension.h>

#include <string>

#include "../../include/mxfp8.h"

namespace {

struct Library {
  decltype(&::mxfp4_quantize) mxfp4_quantize;
  decltype(&::mx_dequantize) mx_dequantize;
  decltype(&::mx_quantize_t) mx_quantize_t;
  decltype(&::mx_requantize_t) mx_requantize_t;
  decltype(&::mxfp4_gemm) mxfp4_gemm;
  decltype(&::mx_swiglu_forward) mx_swiglu_forward;
  decltype(&::mx_swiglu_backward) mx_swiglu_backward;
  decltype(&::mx_rmsnorm_forward) mx_rmsnorm_forward;
  decltype(&::mx_rmsnorm_backward) mx_rmsnorm_backward;
  decltype(&::mx_rmsnorm_backward_workspace) mx_rmsnorm_backward_workspace;
} lib;

bool bound = false;

// All of the functions or, with an error, none.
void bind(const std::string& path) {
  void* h = dlopen(path.c_str(), RTLD_NOW);
  if (!h) throw py::import_error(dlerror());
  Library all;
  auto find = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
    if (!f) throw py::import_error(std::string(name) + " is missing from " + path);
  };
#define MXFP8_FIND(name) find(all.name, #name)
  MXFP8_FIND(mxfp4_quantize);
  MXFP8_FIND(mx_dequantize);
  MXFP8_FIND(mx_quantize_t);
  MXFP8_FIND(mx_requantize_t);
  MXFP8_FIND(mxfp4_gemm);
  MXFP8_FIND(mx_swiglu_forward);
  MXFP8_FIND(mx_swiglu_backward);
  MXFP8_FIND(mx_rmsnorm_forward);
  MXFP8_FIND(mx_rmsnorm_backward);
  MXFP8_FIND(mx_rmsnorm_backward_workspace);
#undef MXFP8_FIND
  lib = all;
  bound = true;
}

// The function, which raises while no library is bound.
template <typename R, typename... A>
auto once_bound(R (*f)(A...)) {
  return [f](A... a) -> R {
    if (!bound) throw py::import_error("libmxfp8.so is not bound to the extension");
    return f(std::forward<A>(a)...);
  };
}

// ---- checks.  The text is put together only when a check fails.

template <typename... Part>
[[noreturn]] void refuse(const Part&... part) {
  std::ostringstream s;
  (s << ... << part);
  throw py::value_error(s.str());
}
#define REQUIRE(cond, ...)             \
  do {                                 \
    if (!(cond)) refuse(__VA_ARGS__);  \
  } while (0)

void status(int st, const char* where) {
  if (st == MXFP8_OK) return;
  py::object error = py::module_::import("mx_block_scaled_x128_amd").attr("MxFp8Error");
  PyErr_SetObject(error.ptr(), error(st, where).ptr());
  throw py::error_already_set();
}

bool is_real(const at::Tensor& t) { return t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16; }
int real_type(const at::Tensor& t) { return t.scalar_type() == at::kFloat ? MXFP8_F32 : MXFP8_BF16; }
// One row has no leading dimension, whatever its stride: the least that the C functions take.
int64_t ld(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : (t.size(1) + 15) / 16 * 16; }
void* ptr(const at::Tensor& t) { return t.data_ptr(); }
uint8_t* bytes(const at::Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

// A 2-D tensor with unit column stride whose rows do not overlap.
void layout(const at::Tensor& t, const char* name) {
  REQUIRE(t.dim() == 2, name, " must be 2-D, got ", t.dim(), "-D");
  REQUIRE(t.size(1) <= 1 || t.stride(1) == 1, name, " must have unit column stride");
  REQUIRE(t.size(0) <= 1 || t.stride(0) >= t.size(1), name, " rows must not overlap");
}
void shape(const at::Tensor& t, const char* name, int64_t rows, int64_t cols) {
  REQUIRE(t.dim() == 2 && t.size(0) == rows && t.size(1) == cols, name, " must have shape (", rows, ", ", cols,
          "), got ", t.sizes());
}
void real_matrix(const at::Tensor& t, const char* name) {
  layout(t, name);
  REQUIRE(is_real(t), name, " must be float32 or bfloat16, got ", t.scalar_type());
}
bool one_byte(const at::Tensor& t, bool codes) {
  const auto s = t.scalar_type();
  return s == at::kByte || (codes ? s == at::kFloat8_e4m3fn || s == at::kFloat8_e5m2 : s == at::kFloat8_e8m0fnu);
}
// A matrix of codes; the elements of a row.
int64_t codes(const at::Tensor& t, int fmt, const char* name) {
  layout(t, name);
  REQUIRE(fmt == MXFP8_E2M1 ? t.scalar_type() == at::kByte : one_byte(t, true), name, " must hold codes (uint8",
          fmt == MXFP8_E2M1 ? "" : " or float8", "), got ", t.scalar_type());
  return fmt == MXFP8_E2M1 ? t.size(1) * 2 : t.size(1);
}
void scales(const at::Tensor& t, const char* name, int64_t rows, int64_t blocks) {
  REQUIRE(one_byte(t, false), name, " must be uint8 or float8_e8m0fnu, got ", t.scalar_type());
  shape(t, name, rows, blocks);
  REQUIRE(t.is_contiguous(), name, " must be contiguous");
}
void vector(const at::Tensor& t, const char* name, int64_t n) {
  REQUIRE(t.dim() == 1 && t.size(0) == n && t.scalar_type() == at::kFloat && t.is_contiguous(), name,
          " must be a contiguous float32 vector of ", n);
}
void blocks32(int64_t cols, const char* name) {
  REQUIRE(cols % 32 == 0, name, " must have a multiple of 32 columns, got ", cols);
}
void format(int fmt, const char* name, bool with_e2m1) {
  REQUIRE(fmt == MXFP8_E4M3 || fmt == MXFP8_E5M2 || (with_e2m1 && fmt == MXFP8_E2M1), name, " must be E4M3",
          with_e2m1 ? ", E5M2 or E2M1" : " or E5M2", ", got ", fmt);
}

// All tensors on the current device; its index.
int device_of(std::initializer_list<const at::Tensor*> all) {
  int dev = -1;
  for (const at::Tensor* t : all) {
    REQUIRE(t->is_cuda(), "expected a CUDA tensor, got device ", t->device());
    const int i = t->get_device();
    REQUIRE(dev < 0 || i == dev, "tensors are on cuda:", dev, " and cuda:", i);
    dev = i;
  }
  const int cur = c10::hip::current_device();
  REQUIRE(dev == cur, "tensors are on cuda:", dev, " but the current device is cuda:", cur);
  return dev;
}
// Where a call works: the given stream, or the current one.  A given stream is
// the current one while this lives, so what the call allocates comes from its
// memory: a block freed on another stream may still be in use there, and work
// on the given one would not wait for that.
class Place {
 public:
  Place(const py::object& stream, int dev) : dev_(dev) {
    if (stream.is_none()) {
      raw_ = c10::hip::getCurrentHIPStream(dev).stream();
      return;
    }
    const int i = stream.attr("device").attr("index").cast<int>();
    REQUIRE(i == dev, "stream is on cuda:", i, " but the tensors are on cuda:", dev);
    const c10::Stream given = c10::Stream::unpack3(stream.attr("stream_id").cast<int64_t>(), (c10::DeviceIndex)dev,
                                                   at::kCUDA);
    raw_ = reinterpret_cast<void*>(stream.attr("cuda_stream").cast<uintptr_t>());
    guard_.reset_stream(given);
    if (*guard_.original_stream() != given) caller_ = guard_.original_stream();
  }
  void* stream() const { return raw_; }
  // Uninitialized; for the length of the call.
  at::Tensor scratch(at::IntArrayRef size, at::ScalarType type) const {
    return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)dev_)));
  }
  // Uninitialized; returned to the caller, whose current stream may read it
  // until it is freed.
  at::Tensor fresh(at::IntArrayRef size, at::ScalarType type) const {
    at::Tensor t = scratch(size, type);
    if (caller_) t.record_stream(*caller_);
    return t;
  }
  // The same, [rows][cols] with rows of a multiple of 16 elements.
  at::Tensor pitched(int64_t rows, int64_t cols, at::ScalarType type) const {
    const int64_t pitch = std::max<int64_t>((cols + 15) / 16 * 16, 16);
    at::Tensor t = fresh({rows, pitch}, type);
    return pitch == cols ? t : t.narrow(1, 0, cols);
  }

 private:
  int dev_;
  void* raw_;
  c10::OptionalStreamGuard guard_;
  c10::optional<c10::Stream> caller_;
};

int64_t filled_rows(int64_t rows, const c10::optional<int64_t>& rows_out) {
  if (!rows_out.has_value()) return (rows + 127) / 128 * 128;
  REQUIRE(*rows_out % 32 == 0 && *rows_out >= rows, "rows_out must be a multiple of 32 and at least ", rows, ", got ",
          *rows_out);
  return *rows_out;
}

// ---- the functions

py::tuple quantize_mxfp4(const at::Tensor& x, int rule, const py::object& stream) {
  real_matrix(x, "x");
  const int64_t rows = x.size(0), cols = x.size(1);
  blocks32(cols, "x");
  const Place on(stream, device_of({&x}));
  at::Tensor q = on.pitched(rows, cols / 2, at::kByte), s = on.fresh({rows, cols / 32}, at::kByte);
  status(lib.mxfp4_quantize(ptr(x), real_type(x), rows, cols, ld(x), rule, bytes(q), ld(q), bytes(s),
                            on.stream()), "mxfp4_quantize");
  return py::make_tuple(q, s);
}

at::Tensor dequantize_mx(const at::Tensor& q, const at::Tensor& s, int fmt, at::ScalarType dtype,
                         const py::object& stream) {
  format(fmt, "fmt", true);
  const int64_t cols = codes(q, fmt, "q"), rows = q.size(0);
  blocks32(cols, "q");
  scales(s, "scales", rows, cols / 32);
  REQUIRE(dtype == at::kFloat || dtype == at::kBFloat16, "dtype must be float32 or bfloat16, got ", dtype);
  const Place on(stream, device_of({&q, &s}));
  at::Tensor y = on.fresh({rows, cols}, dtype);
  status(lib.mx_dequantize(bytes(q), ld(q), fmt, bytes(s), rows, cols, ptr(y), real_type(y), ld(y),
                           on.stream()), "mx_dequantize");
  return y;
}

py::tuple quantize_mx_t(const at::Tensor& x, int fmt, int rule, const c10::optional<int64_t>& rows_out,
                        const py::object& stream) {
  format(fmt, "fmt", true);
  real_matrix(x, "x");
  const int64_t rows = x.size(0), cols = x.size(1), out = filled_rows(rows, rows_out);
  REQUIRE(cols % 16 == 0, "x must have a multiple of 16 columns, got ", cols);
  const Place on(stream, device_of({&x}));
  at::Tensor qt = on.pitched(cols, fmt == MXFP8_E2M1 ? out / 2 : out, at::kByte);
  at::Tensor st = on.fresh({cols, out / 32}, at::kByte);
  status(lib.mx_quantize_t(ptr(x), real_type(x), rows, cols, ld(x), fmt, rule, bytes(qt), ld(qt), out, bytes(st),
                           on.stream()), "mx_quantize_t");
  return py::make_tuple(qt, st);
}

py::tuple requantize_mx_t(const at::Tensor& q, const at::Tensor& s, int q_fmt, int fmt, int rule,
                          const c10::optional<int64_t>& rows_out, const py::object& stream) {
  format(q_fmt, "q_fmt", false);
  format(fmt, "fmt", true);
  const int64_t cols = codes(q, q_fmt, "q"), rows = q.size(0), out = filled_rows(rows, rows_out);
  blocks32(cols, "q");
  scales(s, "scales", rows, cols / 32);
  const Place on(stream, device_of({&q, &s}));
  at::Tensor qt = on.pitched(cols, fmt == MXFP8_E2M1 ? out / 2 : out, at::kByte);
  at::Tensor st = on.fresh({cols, out / 32}, at::kByte);
  status(lib.mx_requantize_t(bytes(q), ld(q), q_fmt, bytes(s), rows, cols, fmt, rule, bytes(qt), ld(qt), out,
                             bytes(st), on.stream()), "mx_requantize_t");
  return py::make_tuple(qt, st);
}

at::Tensor mxfp4_scaled_gemm(const at::Tensor& a, const at::Tensor& sa, int a_fmt, const at::Tensor& b,
                             const at::Tensor& sb, const c10::optional<at::ScalarType>& out_dtype,
                             const c10::optional<at::Tensor>& out, const py::object& stream) {
  format(a_fmt, "a_fmt", true);
  const int64_t K = codes(a, a_fmt, "a"), kb = codes(b, MXFP8_E2M1, "b"), M = a.size(0), N = b.size(0);
  REQUIRE(kb == K, "a has K = ", K, " but b has K = ", kb);
  REQUIRE(K % 128 == 0, "mxfp4_scaled_gemm: K must be a multiple of 128, got ", K);
  scales(sa, "a_scales", M, K / 32);
  scales(sb, "b_scales", N, K / 32);
  if (out.has_value()) {
    real_matrix(*out, "out");
    shape(*out, "out", M, N);
  }
  const at::ScalarType type = out_dtype.value_or(at::kFloat);
  REQUIRE(out.has_value() || type == at::kFloat || type == at::kBFloat16,
          "out_dtype must be float32 or bfloat16, got ", type);
  const Place on(stream, out.has_value() ? device_of({&a, &sa, &b, &sb, &*out}) : device_of({&a, &sa, &b, &sb}));
  at::Tensor c = out.has_value() ? *out : on.pitched(M, N, type);
  status(lib.mxfp4_gemm(M, N, K, bytes(a), ld(a), a_fmt, bytes(sa), bytes(b), ld(b), bytes(sb), ptr(c), ld(c),
                        real_type(c), on.stream()), "mxfp4_gemm");
  return c;
}

py::tuple swiglu_mx(const at::Tensor& x, int fmt, int rule, bool keep, const py::object& stream) {
  format(fmt, "fmt", false);
  real_matrix(x, "x");
  const int64_t rows = x.size(0), wide = x.size(1), cols = wide / 2;
  REQUIRE(wide % 64 == 0, "x must have twice a multiple of 32 columns, got ", wide);
  const Place on(stream, device_of({&x}));
  at::Tensor h = on.fresh({rows, cols}, at::kByte), hs = on.fresh({rows, cols / 32}, at::kByte), k, ks;
  if (keep) {
    k = on.fresh({rows, wide}, at::kByte);
    ks = on.fresh({rows, wide / 32}, at::kByte);
  }
  status(lib.mx_swiglu_forward(ptr(x), real_type(x), rows, cols, ld(x), fmt, rule, bytes(h), cols, bytes(hs),
                               keep ? bytes(k) : nullptr, wide, keep ? bytes(ks) : nullptr, on.stream()),
         "mx_swiglu_forward");
  if (!keep) return py::make_tuple(h, hs);
  return py::make_tuple(h, hs, k, ks);
}

at::Tensor swiglu_mx_backward(const at::Tensor& k, const at::Tensor& ks, int fmt, const at::Tensor& dh,
                              const py::object& stream) {
  format(fmt, "kept.fmt", false);
  const int64_t wide = codes(k, fmt, "kept.codes"), rows = k.size(0);
  REQUIRE(wide % 64 == 0, "kept.codes must have twice a multiple of 32 columns, got ", wide);
  scales(ks, "kept.scales", rows, wide / 32);
  real_matrix(dh, "dh");
  shape(dh, "dh", rows, wide / 2);
  const Place on(stream, device_of({&k, &ks, &dh}));
  at::Tensor dx = on.fresh({rows, wide}, dh.scalar_type());
  status(lib.mx_swiglu_backward(bytes(k), ld(k), bytes(ks), fmt, ptr(dh), real_type(dh), ld(dh), rows, wide / 2,
                                ptr(dx), wide, on.stream()), "mx_swiglu_backward");
  return dx;
}

py::tuple rmsnorm_mx(const at::Tensor& x, const at::Tensor& w, double eps, int fmt, int rule, bool keep,
                     const py::object& stream) {
  format(fmt, "fmt", false);
  real_matrix(x, "x");
  const int64_t rows = x.size(0), cols = x.size(1);
  blocks32(cols, "x");
  vector(w, "w", cols);
  const Place on(stream, device_of({&x, &w}));
  at::Tensor y = on.fresh({rows, cols}, at::kByte), ys = on.fresh({rows, cols / 32}, at::kByte), k, ks, r;
  if (keep) {
    k = on.fresh({rows, cols}, at::kByte);
    ks = on.fresh({rows, cols / 32}, at::kByte);
    r = on.fresh({rows}, at::kFloat);
  }
  status(lib.mx_rmsnorm_forward(ptr(x), real_type(x), rows, cols, ld(x), static_cast<float*>(ptr(w)), (float)eps, fmt,
                                rule, bytes(y), cols, bytes(ys), keep ? bytes(k) : nullptr, cols,
                                keep ? bytes(ks) : nullptr, keep ? static_cast<float*>(ptr(r)) : nullptr,
                                on.stream()), "mx_rmsnorm_forward");
  if (!keep) return py::make_tuple(y, ys);
  return py::make_tuple(y, ys, k, ks, r);
}

py::tuple rmsnorm_mx_backward(const at::Tensor& k, const at::Tensor& ks, const at::Tensor& r, int fmt,
                              const at::Tensor& w, const at::Tensor& dy, const py::object& stream) {
  format(fmt, "kept.fmt", false);
  const int64_t cols = codes(k, fmt, "kept.codes"), rows = k.size(0);
  blocks32(cols, "kept.codes");
  scales(ks, "kept.scales", rows, cols / 32);
  vector(r, "kept.rstd", rows);
  vector(w, "w", cols);
  real_matrix(dy, "dy");
  shape(dy, "dy", rows, cols);
  const Place on(stream, device_of({&k, &ks, &r, &w, &dy}));
  at::Tensor dx = on.fresh({rows, cols}, dy.scalar_type()), dw = on.fresh({cols}, at::kFloat);
  at::Tensor work = on.scratch({lib.mx_rmsnorm_backward_workspace(rows, cols)}, at::kByte);
  status(lib.mx_rmsnorm_backward(bytes(k), ld(k), bytes(ks), static_cast<float*>(ptr(r)), fmt,
                                 static_cast<float*>(ptr(w)), ptr(dy), real_type(dy), ld(dy), rows, cols, ptr(dx),
                                 cols, static_cast<float*>(ptr(dw)), ptr(work), on.stream()), "mx_rmsnorm_backward");
  return py::make_tuple(dx, dw);
}

}  // namespace

PYBIND11_MODULE(_mx_tensors, m) {
  m.def("bind", &bind);
  m.def("quantize_mxfp4", once_bound(&quantize_mxfp4));
  m.def("dequantize_mx", once_bound(&dequantize_mx));
  m.def("quantize_mx_t", once_bound(&quantize_mx_t));
  m.def("requantize_mx_t", once_bound(&requantize_mx_t));
  m.def("mxfp4_scaled_gemm", once_bound(&mxfp4_scaled_gemm));
  m.def("swiglu_mx", once_bound(&swiglu_mx));
  m.def("swiglu_mx_backward", once_bound(&swiglu_mx_backward));
  m.def("rmsnorm_mx", once_bound(&rmsnorm_mx));
  m.def("rmsnorm_mx_backward", once_bound(&rmsnorm_mx_backward));
}
