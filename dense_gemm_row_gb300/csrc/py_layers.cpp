// py_layers.cpp -- argument marshalling of the linear-layer operators for Python
// (module dense_gemm_row_gb300._layers, used by binding.py).
//
// Each function takes CUDA tensors, checks dtypes, shapes, strides and devices,
// raises TypeError or ValueError, and otherwise calls the C entry point that the
// dtypes pick and returns its status. The checks read the tensors directly: made
// from Python attribute by attribute they took about 5 us per call, more than the
// smallest of these calls takes on the GPU. No computation happens here. The C
// library is loaded by binding.py, which passes the entry points' addresses.
#include <cstdint>
#include <cstring>
#include <exception>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "dense_gemm_row.h"

namespace {

// Entry points by name; [0] bf16, [1] fp16.
decltype(&gemm_bf16_epi) g_epi[2];
decltype(&gemm_e4m3_bf16_epi) g_epi8[2];
decltype(&gemm_bf16_dact) g_dact[2];
decltype(&gemm_act_grad_bf16) g_act_grad[2];
decltype(&gemm_rms_norm_bf16) g_norm[2];
decltype(&gemm_rms_norm_bf16_e4m3) g_norm8[2];
decltype(&gemm_rms_norm_grad_bf16) g_norm_grad[2];
decltype(&gemm_layer_norm_bf16) g_layer_norm[2];
decltype(&gemm_bf16_gated) g_gated[2];
decltype(&gemm_bf16_gated_dact) g_gated_dact[2];
decltype(&gemm_e4m3_bf16_gated) g_gated8[2];
decltype(&gemm_e4m3_block_bf16_epi) g_block[2];
decltype(&gemm_quantise_bf16_e4m3) g_quantise[2];
decltype(&gemm_layer_norm_grad_bf16) g_layer_norm_grad[2];

struct Refused {};  // a Python exception has been set

[[noreturn]] void refuse(PyObject *type, const char *format, const char *name) {
  PyErr_Format(type, format, name);
  throw Refused();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

const char *type_name(at::ScalarType t) { return c10::toString(t); }

// The CUDA device of a call: the first operand's, which has to be the current one.
int device_of(const at::Tensor &t, const char *name) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  const int dev = t.get_device();
  if (dev != c10::cuda::current_device())
    refuse(PyExc_ValueError, "%s is not on the current CUDA device", name);
  return dev;
}

cudaStream_t stream_of(PyObject *s, int dev) {
  if (s == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev));
  PyObject *v = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttrString(s, "cuda_stream");
  if (v == nullptr) throw Refused();
  void *p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (p == nullptr && PyErr_Occurred()) throw Refused();
  return static_cast<cudaStream_t>(p);
}

gemm_act_t act_of(PyObject *o) {
  if (o == Py_None) return GEMM_ACT_NONE;
  const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  static const char *const names[] = {"none", "relu", "gelu", "gelu_tanh", "silu"};
  for (int i = 0; s != nullptr && i < 5; ++i)
    if (std::strcmp(s, names[i]) == 0) return static_cast<gemm_act_t>(i);
  PyErr_Clear();
  PyErr_Format(PyExc_ValueError, "act must be one of none, relu, gelu, gelu_tanh, silu, not %R", o);
  throw Refused();
}

bool truth(PyObject *o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw Refused();
  return t != 0;
}

float number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return static_cast<float>(v);
}

struct Matrix {
  void *p = nullptr;
  int64_t ld = 0;
};

// Base address and row stride of a rows x cols matrix with unit column stride. A
// single row's stride has no meaning: it counts as the next multiple of `unit`.
Matrix matrix(const at::Tensor &t, const char *name, int64_t rows, int64_t cols,
              at::ScalarType type, int dev, int64_t unit = 1) {
  if (t.scalar_type() != type) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, not %s", name, type_name(type),
                 type_name(t.scalar_type()));
    throw Refused();
  }
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols) {
    PyErr_Format(PyExc_ValueError, "%s must be %lld x %lld", name, static_cast<long long>(rows),
                 static_cast<long long>(cols));
    throw Refused();
  }
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(PyExc_ValueError, "%s must be on the call's CUDA device", name);
  Matrix m;
  m.ld = t.stride(0);
  if (cols > 1 && rows > 0 && t.stride(1) != 1)
    refuse(PyExc_ValueError, "%s needs unit column stride (row-major)", name);
  if (rows <= 1) {
    m.ld = ((cols > 1 ? cols : 1) + unit - 1) / unit * unit;
  } else if (m.ld < cols) {
    refuse(PyExc_ValueError, "%s: rows overlap", name);
  }
  m.p = t.data_ptr();
  return m;
}
Matrix matrix_or_none(PyObject *o, const char *name, int64_t rows, int64_t cols,
                      at::ScalarType type, int dev) {
  return o == Py_None ? Matrix() : matrix(tensor(o, name), name, rows, cols, type, dev);
}

void *vector_or_none(PyObject *o, const char *name, int64_t n, at::ScalarType type, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != type) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, not %s", name, type_name(type),
                 type_name(t.scalar_type()));
    throw Refused();
  }
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous vector of %lld values", name,
                 static_cast<long long>(n));
    throw Refused();
  }
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(PyExc_ValueError, "%s must be on the call's CUDA device", name);
  return t.data_ptr();
}

// Scales of a rows x cols matrix per block of block_rows x 128, a fp32 matrix.
Matrix block_scales(PyObject *o, const char *name, int64_t rows, int64_t cols, int64_t block_rows,
                    int dev) {
  return matrix(tensor(o, name), name, (rows + block_rows - 1) / block_rows, (cols + 127) / 128,
                at::kFloat, dev);
}
bool is_matrix(PyObject *o) { return THPVariable_Check(o) && THPVariable_Unpack(o).dim() == 2; }

// 0 for bfloat16, 1 for float16.
int format_of(const at::Tensor &t, const char *name) {
  if (t.scalar_type() == at::kBFloat16) return 0;
  if (t.scalar_type() == at::kHalf) return 1;
  refuse(PyExc_TypeError, "%s must be bfloat16 or float16", name);
}

// op(A) op(B): sizes and operands of a product.
struct Product {
  int64_t m, n, k;
  Matrix a, b;
  gemm_op_t op_a, op_b;
};
Product product(const at::Tensor &A, const at::Tensor &B, PyObject *trans_a, PyObject *trans_b,
                int dev, int64_t unit) {
  if (A.dim() != 2 || B.dim() != 2) refuse(PyExc_ValueError, "%s and B must be 2-D", "A");
  const bool ta = truth(trans_a), tb = truth(trans_b);
  Product p;
  p.op_a = ta ? GEMM_OP_T : GEMM_OP_N;
  p.op_b = tb ? GEMM_OP_T : GEMM_OP_N;
  p.m = A.size(ta ? 1 : 0);
  p.k = A.size(ta ? 0 : 1);
  p.n = B.size(tb ? 0 : 1);
  if (B.size(tb ? 1 : 0) != p.k) refuse(PyExc_ValueError, "%s and B do not chain", "A");
  p.a = matrix(A, "A", A.size(0), A.size(1), A.scalar_type(), dev, unit);
  p.b = matrix(B, "B", B.size(0), B.size(1), A.scalar_type(), dev, unit);
  return p;
}

template <typename T>
T *as(void *p) {
  return static_cast<T *>(p);
}

// Runs f() -> status without the interpreter lock.
template <typename F>
int unlocked(F &&f) {
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  return static_cast<int>(st);
}

// (A, B, D, alpha, bias, act, residual, preact, trans_a, trans_b, scale_a, scale_b, stream)
int epilogue(PyObject *const *v) {
  const at::Tensor &A = tensor(v[0], "A"), &B = tensor(v[1], "B"), &D = tensor(v[2], "D");
  const int dev = device_of(A, "A");
  const bool e4m3 = A.scalar_type() == at::kFloat8_e4m3fn;
  const int f = e4m3 ? format_of(D, "D") : format_of(A, "A");
  const at::ScalarType type = e4m3 ? D.scalar_type() : A.scalar_type();
  const Product p = product(A, B, v[8], v[9], dev, e4m3 ? 16 : 8);
  const Matrix d = matrix(D, "D", p.m, p.n, type, dev);
  const Matrix r = matrix_or_none(v[6], "residual", p.m, p.n, type, dev);
  const Matrix z = matrix_or_none(v[7], "preact", p.m, p.n, type, dev);
  void *bias = vector_or_none(v[4], "bias", p.n, type, dev);
  const float alpha = number(v[3]);
  const gemm_act_t act = act_of(v[5]);
  const cudaStream_t s = stream_of(v[12], dev);
  if (e4m3) {
    if (p.op_a == GEMM_OP_T || p.op_b != GEMM_OP_T)
      refuse(PyExc_ValueError, "%s", "float8_e4m3fn takes A as M x K and B as N x K (trans_b=True)");
    if (is_matrix(v[10]) || is_matrix(v[11])) {  // a scale per block of 128
      const Matrix sa = block_scales(v[10], "scale_a", p.m, p.k, 1, dev);
      const Matrix sb = block_scales(v[11], "scale_b", p.n, p.k, 128, dev);
      return unlocked([&] {
        return g_block[f](p.m, p.n, p.k, alpha, as<uint8_t>(p.a.p), p.a.ld, as<float>(sa.p), sa.ld,
                          as<uint8_t>(p.b.p), p.b.ld, as<float>(sb.p), sb.ld, act,
                          as<uint16_t>(bias), as<uint16_t>(r.p), r.ld, as<uint16_t>(z.p), z.ld,
                          as<uint16_t>(d.p), d.ld, s);
      });
    }
    void *sa = vector_or_none(v[10], "scale_a", p.m, at::kFloat, dev);
    void *sb = vector_or_none(v[11], "scale_b", p.n, at::kFloat, dev);
    return unlocked([&] {
      return g_epi8[f](p.m, p.n, p.k, alpha, as<uint8_t>(p.a.p), p.a.ld, as<float>(sa),
                       as<uint8_t>(p.b.p), p.b.ld, as<float>(sb), act, as<uint16_t>(bias),
                       as<uint16_t>(r.p), r.ld, as<uint16_t>(z.p), z.ld, as<uint16_t>(d.p), d.ld,
                       s);
    });
  }
  if (v[10] != Py_None || v[11] != Py_None)
    refuse(PyExc_ValueError, "%s", "scales go with float8_e4m3fn operands");
  return unlocked([&] {
    return g_epi[f](p.op_a, p.op_b, p.m, p.n, p.k, alpha, as<uint16_t>(p.a.p), p.a.ld,
                    as<uint16_t>(p.b.p), p.b.ld, act, as<uint16_t>(bias), as<uint16_t>(r.p), r.ld,
                    as<uint16_t>(z.p), z.ld, as<uint16_t>(d.p), d.ld, s);
  });
}

// (A, B, Z, dZ, act, alpha, dbias, trans_a, trans_b, stream)
int dact(PyObject *const *v) {
  const at::Tensor &A = tensor(v[0], "A"), &B = tensor(v[1], "B"), &dZ = tensor(v[3], "dZ");
  const int dev = device_of(A, "A");
  const int f = format_of(A, "A");
  const at::ScalarType type = A.scalar_type();
  const Product p = product(A, B, v[7], v[8], dev, 8);
  const Matrix z = matrix_or_none(v[2], "Z", p.m, p.n, type, dev);
  const Matrix d = matrix(dZ, "dZ", p.m, p.n, type, dev);
  void *dbias = vector_or_none(v[6], "dbias", p.n, type, dev);
  const gemm_act_t act = act_of(v[4]);
  const float alpha = number(v[5]);
  const cudaStream_t s = stream_of(v[9], dev);
  return unlocked([&] {
    return g_dact[f](p.op_a, p.op_b, p.m, p.n, p.k, alpha, as<uint16_t>(p.a.p), p.a.ld,
                     as<uint16_t>(p.b.p), p.b.ld, act, as<uint16_t>(z.p), z.ld, as<uint16_t>(d.p),
                     d.ld, as<uint16_t>(dbias), s);
  });
}

// (dD, Z, dZ, act, dbias, stream)
int act_grad(PyObject *const *v) {
  const at::Tensor &dD = tensor(v[0], "dD");
  const int dev = device_of(dD, "dD");
  const int f = format_of(dD, "dD");
  const at::ScalarType type = dD.scalar_type();
  if (dD.dim() != 2) refuse(PyExc_ValueError, "%s must be 2-D", "dD");
  const int64_t m = dD.size(0), n = dD.size(1);
  const Matrix d = matrix(dD, "dD", m, n, type, dev);
  const Matrix z = matrix_or_none(v[1], "Z", m, n, type, dev);
  const Matrix o = matrix_or_none(v[2], "dZ", m, n, type, dev);
  void *dbias = vector_or_none(v[4], "dbias", n, type, dev);
  const gemm_act_t act = act_of(v[3]);
  const cudaStream_t s = stream_of(v[5], dev);
  return unlocked([&] {
    return g_act_grad[f](m, n, act, as<uint16_t>(d.p), d.ld, as<uint16_t>(z.p), z.ld,
                         as<uint16_t>(o.p), o.ld, as<uint16_t>(dbias), s);
  });
}

// (X, Y, weight, residual, h, scale, rstd, eps, stream)
int rms_norm(PyObject *const *v) {
  const at::Tensor &X = tensor(v[0], "X"), &Y = tensor(v[1], "Y");
  const int dev = device_of(X, "X");
  const int f = format_of(X, "X");
  const at::ScalarType type = X.scalar_type();
  if (X.dim() != 2) refuse(PyExc_ValueError, "%s must be 2-D", "X");
  const int64_t m = X.size(0), n = X.size(1);
  const bool e4m3 = Y.scalar_type() == at::kFloat8_e4m3fn;
  const Matrix x = matrix(X, "X", m, n, type, dev);
  const Matrix y = matrix(Y, "Y", m, n, e4m3 ? at::kFloat8_e4m3fn : type, dev);
  void *w = vector_or_none(v[2], "weight", n, type, dev);
  const Matrix r = matrix_or_none(v[3], "residual", m, n, type, dev);
  const Matrix h = matrix_or_none(v[4], "h", m, n, type, dev);
  void *scale = vector_or_none(v[5], "scale", m, at::kFloat, dev);
  void *rstd = vector_or_none(v[6], "rstd", m, at::kFloat, dev);
  const float eps = number(v[7]);
  const cudaStream_t s = stream_of(v[8], dev);
  if (e4m3) {
    if (scale == nullptr && v[5] == Py_None)
      refuse(PyExc_ValueError, "%s", "a float8_e4m3fn Y needs scale");
    return unlocked([&] {
      return g_norm8[f](m, n, eps, as<uint16_t>(x.p), x.ld, as<uint16_t>(r.p), r.ld,
                        as<uint16_t>(w), as<uint16_t>(h.p), h.ld, as<uint8_t>(y.p), y.ld,
                        as<float>(scale), as<float>(rstd), s);
    });
  }
  if (v[5] != Py_None) refuse(PyExc_ValueError, "%s", "scale goes with a float8_e4m3fn Y");
  return unlocked([&] {
    return g_norm[f](m, n, eps, as<uint16_t>(x.p), x.ld, as<uint16_t>(r.p), r.ld, as<uint16_t>(w),
                     as<uint16_t>(h.p), h.ld, as<uint16_t>(y.p), y.ld, as<float>(rstd), s);
  });
}

// (dY, H, rstd, dX, weight, dh, dweight, stream)
int rms_norm_grad(PyObject *const *v) {
  const at::Tensor &dY = tensor(v[0], "dY");
  const int dev = device_of(dY, "dY");
  const int f = format_of(dY, "dY");
  const at::ScalarType type = dY.scalar_type();
  if (dY.dim() != 2) refuse(PyExc_ValueError, "%s must be 2-D", "dY");
  const int64_t m = dY.size(0), n = dY.size(1);
  const Matrix y = matrix(dY, "dY", m, n, type, dev);
  const Matrix h = matrix(tensor(v[1], "H"), "H", m, n, type, dev);
  tensor(v[2], "rstd");
  void *rstd = vector_or_none(v[2], "rstd", m, at::kFloat, dev);
  const Matrix x = matrix(tensor(v[3], "dX"), "dX", m, n, type, dev);
  void *w = vector_or_none(v[4], "weight", n, type, dev);
  const Matrix b = matrix_or_none(v[5], "dh", m, n, type, dev);
  void *dw = vector_or_none(v[6], "dweight", n, type, dev);
  const cudaStream_t s = stream_of(v[7], dev);
  return unlocked([&] {
    return g_norm_grad[f](m, n, as<uint16_t>(y.p), y.ld, as<uint16_t>(h.p), h.ld, as<float>(rstd),
                          as<uint16_t>(w), as<uint16_t>(b.p), b.ld, as<uint16_t>(x.p), x.ld,
                          as<uint16_t>(dw), s);
  });
}

// (A, Bg, Bu, D, act, alpha, bias_gate, bias_up, gate, up, trans_a, trans_b, scale_a,
// scale_gate, scale_up, stream)
int gated(PyObject *const *v) {
  const at::Tensor &A = tensor(v[0], "A"), &Bg = tensor(v[1], "Bg"), &Bu = tensor(v[2], "Bu");
  const at::Tensor &D = tensor(v[3], "D");
  const int dev = device_of(A, "A");
  const bool e4m3 = A.scalar_type() == at::kFloat8_e4m3fn;
  const int f = e4m3 ? format_of(D, "D") : format_of(A, "A");
  const at::ScalarType type = e4m3 ? D.scalar_type() : A.scalar_type();
  const Product p = product(A, Bg, v[10], v[11], dev, e4m3 ? 16 : 8);
  const Matrix b2 =
      matrix(Bu, "Bu", Bg.size(0), Bg.size(1), A.scalar_type(), dev, e4m3 ? 16 : 8);
  const Matrix d = matrix(D, "D", p.m, p.n, type, dev);
  const Matrix g = matrix_or_none(v[8], "gate", p.m, p.n, type, dev);
  const Matrix u = matrix_or_none(v[9], "up", p.m, p.n, type, dev);
  void *bias_g = vector_or_none(v[6], "bias_gate", p.n, type, dev);
  void *bias_u = vector_or_none(v[7], "bias_up", p.n, type, dev);
  const gemm_act_t act = act_of(v[4]);
  const float alpha = number(v[5]);
  const cudaStream_t s = stream_of(v[15], dev);
  if (e4m3) {
    if (p.op_a == GEMM_OP_T || p.op_b != GEMM_OP_T)
      refuse(PyExc_ValueError, "%s",
             "float8_e4m3fn takes A as M x K, Bg and Bu as N x K (trans_b=True)");
    const Matrix sa = block_scales(v[12], "scale_a", p.m, p.k, 1, dev);
    const Matrix sg = block_scales(v[13], "scale_gate", p.n, p.k, 128, dev);
    const Matrix su = block_scales(v[14], "scale_up", p.n, p.k, 128, dev);
    return unlocked([&] {
      return g_gated8[f](p.m, p.n, p.k, alpha, as<uint8_t>(p.a.p), p.a.ld, as<float>(sa.p), sa.ld,
                         as<uint8_t>(p.b.p), p.b.ld, as<float>(sg.p), sg.ld, as<uint8_t>(b2.p),
                         b2.ld, as<float>(su.p), su.ld, act, as<uint16_t>(bias_g),
                         as<uint16_t>(bias_u), as<uint16_t>(g.p), g.ld, as<uint16_t>(u.p), u.ld,
                         as<uint16_t>(d.p), d.ld, s);
    });
  }
  if (v[12] != Py_None || v[13] != Py_None || v[14] != Py_None)
    refuse(PyExc_ValueError, "%s", "scales go with float8_e4m3fn operands");
  return unlocked([&] {
    return g_gated[f](p.op_a, p.op_b, p.m, p.n, p.k, alpha, as<uint16_t>(p.a.p), p.a.ld,
                      as<uint16_t>(p.b.p), p.b.ld, as<uint16_t>(b2.p), b2.ld, act,
                      as<uint16_t>(bias_g), as<uint16_t>(bias_u), as<uint16_t>(g.p), g.ld,
                      as<uint16_t>(u.p), u.ld, as<uint16_t>(d.p), d.ld, s);
  });
}

// (X, Y, scale, rows, stream)
int quantise_blocks(PyObject *const *v) {
  const at::Tensor &X = tensor(v[0], "X"), &Y = tensor(v[1], "Y");
  const int dev = device_of(X, "X");
  const int f = format_of(X, "X");
  if (X.dim() != 2) refuse(PyExc_ValueError, "%s must be 2-D", "X");
  const int64_t m = X.size(0), n = X.size(1);
  const long rows = PyLong_AsLong(v[3]);
  if (rows == -1 && PyErr_Occurred()) throw Refused();
  if (rows != 1 && rows != 128) refuse(PyExc_ValueError, "%s must be 1 or 128", "rows");
  const Matrix x = matrix(X, "X", m, n, X.scalar_type(), dev);
  const Matrix y = matrix(Y, "Y", m, n, at::kFloat8_e4m3fn, dev);
  const Matrix scale = block_scales(v[2], "scale", m, n, rows, dev);
  const cudaStream_t s = stream_of(v[4], dev);
  return unlocked([&] {
    return g_quantise[f](m, n, rows, as<uint16_t>(x.p), x.ld, as<uint8_t>(y.p), y.ld,
                         as<float>(scale.p), scale.ld, s);
  });
}

// (A, B, G, U, dG, dU, act, alpha, dbias_gate, dbias_up, trans_a, trans_b, stream)
int gated_dact(PyObject *const *v) {
  const at::Tensor &A = tensor(v[0], "A"), &B = tensor(v[1], "B");
  const int dev = device_of(A, "A");
  const int f = format_of(A, "A");
  const at::ScalarType type = A.scalar_type();
  const Product p = product(A, B, v[10], v[11], dev, 8);
  const Matrix g = matrix(tensor(v[2], "G"), "G", p.m, p.n, type, dev);
  const Matrix u = matrix(tensor(v[3], "U"), "U", p.m, p.n, type, dev);
  const Matrix dg = matrix(tensor(v[4], "dG"), "dG", p.m, p.n, type, dev);
  const Matrix du = matrix(tensor(v[5], "dU"), "dU", p.m, p.n, type, dev);
  void *dbg = vector_or_none(v[8], "dbias_gate", p.n, type, dev);
  void *dbu = vector_or_none(v[9], "dbias_up", p.n, type, dev);
  const gemm_act_t act = act_of(v[6]);
  const float alpha = number(v[7]);
  const cudaStream_t s = stream_of(v[12], dev);
  return unlocked([&] {
    return g_gated_dact[f](p.op_a, p.op_b, p.m, p.n, p.k, alpha, as<uint16_t>(p.a.p), p.a.ld,
                           as<uint16_t>(p.b.p), p.b.ld, act, as<uint16_t>(g.p), g.ld,
                           as<uint16_t>(u.p), u.ld, as<uint16_t>(dg.p), dg.ld,
                           as<uint16_t>(du.p), du.ld, as<uint16_t>(dbg), as<uint16_t>(dbu), s);
  });
}

// (X, Y, weight, bias, residual, h, mean, rstd, eps, stream)
int layer_norm(PyObject *const *v) {
  const at::Tensor &X = tensor(v[0], "X"), &Y = tensor(v[1], "Y");
  const int dev = device_of(X, "X");
  const int f = format_of(X, "X");
  const at::ScalarType type = X.scalar_type();
  if (X.dim() != 2) refuse(PyExc_ValueError, "%s must be 2-D", "X");
  const int64_t m = X.size(0), n = X.size(1);
  const Matrix x = matrix(X, "X", m, n, type, dev);
  const Matrix y = matrix(Y, "Y", m, n, type, dev);
  void *w = vector_or_none(v[2], "weight", n, type, dev);
  void *b = vector_or_none(v[3], "bias", n, type, dev);
  const Matrix r = matrix_or_none(v[4], "residual", m, n, type, dev);
  const Matrix h = matrix_or_none(v[5], "h", m, n, type, dev);
  void *mean = vector_or_none(v[6], "mean", m, at::kFloat, dev);
  void *rstd = vector_or_none(v[7], "rstd", m, at::kFloat, dev);
  const float eps = number(v[8]);
  const cudaStream_t s = stream_of(v[9], dev);
  return unlocked([&] {
    return g_layer_norm[f](m, n, eps, as<uint16_t>(x.p), x.ld, as<uint16_t>(r.p), r.ld,
                           as<uint16_t>(w), as<uint16_t>(b), as<uint16_t>(h.p), h.ld,
                           as<uint16_t>(y.p), y.ld, as<float>(mean), as<float>(rstd), s);
  });
}

// (dY, H, mean, rstd, dX, weight, dh, dweight, dbias, stream)
int layer_norm_grad(PyObject *const *v) {
  const at::Tensor &dY = tensor(v[0], "dY");
  const int dev = device_of(dY, "dY");
  const int f = format_of(dY, "dY");
  const at::ScalarType type = dY.scalar_type();
  if (dY.dim() != 2) refuse(PyExc_ValueError, "%s must be 2-D", "dY");
  const int64_t m = dY.size(0), n = dY.size(1);
  const Matrix y = matrix(dY, "dY", m, n, type, dev);
  const Matrix h = matrix(tensor(v[1], "H"), "H", m, n, type, dev);
  tensor(v[2], "mean"), tensor(v[3], "rstd");
  void *mean = vector_or_none(v[2], "mean", m, at::kFloat, dev);
  void *rstd = vector_or_none(v[3], "rstd", m, at::kFloat, dev);
  const Matrix x = matrix(tensor(v[4], "dX"), "dX", m, n, type, dev);
  void *w = vector_or_none(v[5], "weight", n, type, dev);
  const Matrix b = matrix_or_none(v[6], "dh", m, n, type, dev);
  void *dw = vector_or_none(v[7], "dweight", n, type, dev);
  void *db = vector_or_none(v[8], "dbias", n, type, dev);
  const cudaStream_t s = stream_of(v[9], dev);
  return unlocked([&] {
    return g_layer_norm_grad[f](m, n, as<uint16_t>(y.p), y.ld, as<uint16_t>(h.p), h.ld,
                                as<float>(mean), as<float>(rstd), as<uint16_t>(w),
                                as<uint16_t>(b.p), b.ld, as<uint16_t>(x.p), x.ld,
                                as<uint16_t>(dw), as<uint16_t>(db), s);
  });
}

// A function of exactly kArgs arguments as a Python function returning a status.
template <int (*kFunction)(PyObject *const *), Py_ssize_t kArgs>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(kFunction(args));
  } catch (const Refused &) {
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// bind(name, address) for each entry point.
PyObject *bind(PyObject *, PyObject *args) {
  const char *name;
  unsigned long long address;
  if (!PyArg_ParseTuple(args, "sK", &name, &address)) return nullptr;
  struct {
    const char *name;
    void *slot;
  } const slots[] = {
      {"gemm_bf16_epi", &g_epi[0]},
      {"gemm_f16_epi", &g_epi[1]},
      {"gemm_e4m3_bf16_epi", &g_epi8[0]},
      {"gemm_e4m3_f16_epi", &g_epi8[1]},
      {"gemm_bf16_dact", &g_dact[0]},
      {"gemm_f16_dact", &g_dact[1]},
      {"gemm_act_grad_bf16", &g_act_grad[0]},
      {"gemm_act_grad_f16", &g_act_grad[1]},
      {"gemm_rms_norm_bf16", &g_norm[0]},
      {"gemm_rms_norm_f16", &g_norm[1]},
      {"gemm_rms_norm_bf16_e4m3", &g_norm8[0]},
      {"gemm_rms_norm_f16_e4m3", &g_norm8[1]},
      {"gemm_rms_norm_grad_bf16", &g_norm_grad[0]},
      {"gemm_rms_norm_grad_f16", &g_norm_grad[1]},
      {"gemm_bf16_gated", &g_gated[0]},
      {"gemm_f16_gated", &g_gated[1]},
      {"gemm_e4m3_bf16_gated", &g_gated8[0]},
      {"gemm_e4m3_f16_gated", &g_gated8[1]},
      {"gemm_e4m3_block_bf16_epi", &g_block[0]},
      {"gemm_e4m3_block_f16_epi", &g_block[1]},
      {"gemm_quantise_bf16_e4m3", &g_quantise[0]},
      {"gemm_quantise_f16_e4m3", &g_quantise[1]},
      {"gemm_bf16_gated_dact", &g_gated_dact[0]},
      {"gemm_f16_gated_dact", &g_gated_dact[1]},
      {"gemm_layer_norm_bf16", &g_layer_norm[0]},
      {"gemm_layer_norm_f16", &g_layer_norm[1]},
      {"gemm_layer_norm_grad_bf16", &g_layer_norm_grad[0]},
      {"gemm_layer_norm_grad_f16", &g_layer_norm_grad[1]},
  };
  for (const auto &s : slots) {
    if (std::strcmp(s.name, name) == 0) {
      void *p = reinterpret_cast<void *>(static_cast<uintptr_t>(address));
      std::memcpy(s.slot, &p, sizeof p);
      Py_RETURN_NONE;
    }
  }
  PyErr_Format(PyExc_KeyError, "no entry point %s", name);
  return nullptr;
}

template <int (*kFunction)(PyObject *const *), Py_ssize_t kArgs>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&call<kFunction, kArgs>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<epilogue, 13>("gemm_epilogue"),
    method<dact, 10>("gemm_dact"),
    method<act_grad, 6>("act_grad"),
    method<rms_norm, 9>("rms_norm"),
    method<rms_norm_grad, 8>("rms_norm_grad"),
    method<gated, 16>("gemm_gated"),
    method<quantise_blocks, 5>("quantise_blocks"),
    method<gated_dact, 13>("gemm_gated_dact"),
    method<layer_norm, 10>("layer_norm"),
    method<layer_norm_grad, 10>("layer_norm_grad"),
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_layers", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers() { return PyModule_Create(&g_module); }
