// The fast path of the Python binding for the operators around the step: the
// argument checks of _lib.py on torch tensors, the current stream, and the
// C-ABI call, without the interpreter in between. A small call costs 4 us of
// host time this way (3.2 us of them the kernel launch), 6.5 to 8 us through
// ctypes, and the kernels of a decoded token take 2.
//
// Every function takes the tensors in the order of its namesake in _lib.py and
// returns the call's moe_status, or -1 if the arguments are anything but
// plainly right: then _lib.py goes through them one by one and either makes
// the call itself or says what is wrong. Nothing is decided here.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"

namespace {

decltype(&moe_permute) f_permute;
decltype(&moe_permute_grad) f_permute_grad;
decltype(&moe_unpermute) f_unpermute;
decltype(&moe_unpermute_grad) f_unpermute_grad;
decltype(&moe_mxfp_quantize) f_quantize;
decltype(&moe_mxfp_dequantize) f_dequantize;
decltype(&moe_mxfp_matmul) f_matmul;

using at::ScalarType;
using at::Tensor;

struct Args {
  PyObject* const* a;
  int dev = -1;
  bool ok = true;

  // A contiguous tensor on the current device of `type` (any if Undefined) and
  // the given sizes (any if dims < 0); null for None where that is allowed.
  const Tensor* tensor(int i, ScalarType type, bool optional = false) {
    if (optional && a[i] == Py_None) return nullptr;
    if (!THPVariable_Check(a[i])) {
      ok = false;
      return nullptr;
    }
    const Tensor* t = &THPVariable_Unpack(a[i]);
    if (!t->is_cuda() || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    if (dev < 0) dev = c10::cuda::current_device();
    if (t->get_device() != dev || (type != ScalarType::Undefined && t->scalar_type() != type)) ok = false;
    return ok ? t : nullptr;
  }
  const Tensor* sized(int i, ScalarType type, std::initializer_list<int64_t> sizes, bool optional = false) {
    const Tensor* t = tensor(i, type, optional);
    if (t && t->sizes() != at::IntArrayRef(sizes)) ok = false;
    return ok ? t : nullptr;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream(); }
};

template <typename T>
T* ptr(const Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

int dtype_code(const Tensor& t, bool bytes) {
  switch (t.scalar_type()) {
    case ScalarType::BFloat16: return MOE_DT_BF16;
    case ScalarType::Half: return MOE_DT_FP16;
    case ScalarType::Float: return MOE_DT_FP32;
    case ScalarType::Byte: return bytes ? MOE_DT_U8 : 0;
    default: return 0;
  }
}

constexpr int64_t kMaxInt = 0x7fffffff;

// The matrix a row call goes by: T, H, k (from inv_perm), element type.
struct Rows {
  int64_t T = 0, H = 0, k = 0;
  int code = 0;
  ScalarType type = ScalarType::Undefined;
  const Tensor *main = nullptr, *inv = nullptr, *ws = nullptr;
};
Rows rows(Args& g, int main, int inv, int ws, bool bytes) {
  Rows r;
  r.main = g.tensor(main, ScalarType::Undefined);
  r.inv = g.ok ? g.tensor(inv, ScalarType::Int) : nullptr;
  r.ws = g.ok ? g.tensor(ws, ScalarType::Byte) : nullptr;
  if (!g.ok || r.main->dim() != 2) {
    g.ok = false;
    return r;
  }
  r.T = r.main->size(0);
  r.H = r.main->size(1);
  r.type = r.main->scalar_type();
  r.code = dtype_code(*r.main, bytes);
  const int64_t n = r.inv->numel();
  if (r.code == 0 || r.T == 0 || n == 0 || n % r.T || r.T > kMaxInt || r.H > kMaxInt || n > kMaxInt) {
    g.ok = false;
    return r;
  }
  r.k = n / r.T;
  return r;
}

// permute(x, inv_perm, x_perm, ws)
int permute(Args& g) {
  const Rows r = rows(g, 0, 1, 3, true);
  const Tensor* xp = g.ok ? g.sized(2, r.type, {r.T * r.k, r.H}) : nullptr;
  if (!g.ok) return -1;
  return f_permute(r.main->data_ptr(), r.code, int(r.T), int(r.H), int(r.k), ptr<int32_t>(r.inv), xp->data_ptr(),
                   r.ws->data_ptr(), size_t(r.ws->numel()), g.stream());
}

// permute_grad(dx_perm, inv_perm, dx, ws)
int permute_grad(Args& g) {
  const Rows r = rows(g, 2, 1, 3, false);
  const Tensor* dxp = g.ok ? g.sized(0, r.type, {r.T * r.k, r.H}) : nullptr;
  if (!g.ok) return -1;
  return f_permute_grad(dxp->data_ptr(), r.code, int(r.T), int(r.H), int(r.k), ptr<int32_t>(r.inv),
                        r.main->data_ptr(), r.ws->data_ptr(), size_t(r.ws->numel()), g.stream());
}

// unpermute(y_perm, inv_perm, topk_w, out, ws)
int unpermute(Args& g) {
  const Rows r = rows(g, 3, 1, 4, false);
  const Tensor* y = g.ok ? g.sized(0, r.type, {r.T * r.k, r.H}) : nullptr;
  const Tensor* w = g.ok ? g.sized(2, ScalarType::Float, {r.T, r.k}) : nullptr;
  if (!g.ok) return -1;
  return f_unpermute(y->data_ptr(), r.code, int(r.T), int(r.H), int(r.k), ptr<int32_t>(r.inv), ptr<float>(w),
                     r.main->data_ptr(), r.ws->data_ptr(), size_t(r.ws->numel()), g.stream());
}

// unpermute_grad(dout, y_perm, inv_perm, topk_w, dy_perm, dtopk_w, ws)
int unpermute_grad(Args& g) {
  const Rows r = rows(g, 0, 2, 6, false);
  const Tensor* y = g.ok ? g.sized(1, r.type, {r.T * r.k, r.H}) : nullptr;
  const Tensor* w = g.ok ? g.sized(3, ScalarType::Float, {r.T, r.k}) : nullptr;
  const Tensor* dy = g.ok ? g.sized(4, r.type, {r.T * r.k, r.H}) : nullptr;
  const Tensor* dw = g.ok ? g.sized(5, ScalarType::Float, {r.T, r.k}) : nullptr;
  if (!g.ok) return -1;
  return f_unpermute_grad(r.main->data_ptr(), y->data_ptr(), r.code, int(r.T), int(r.H), int(r.k),
                          ptr<int32_t>(r.inv), ptr<float>(w), dy->data_ptr(), ptr<float>(dw), r.ws->data_ptr(),
                          size_t(r.ws->numel()), g.stream());
}

// 0 for "mx", 1 for "nv", else -1.
int format(PyObject* o) {
  if (!PyUnicode_Check(o)) return -1;
  return PyUnicode_CompareWithASCIIString(o, "mx") == 0 ? 0 : PyUnicode_CompareWithASCIIString(o, "nv") == 0 ? 1 : -1;
}
int64_t scale_bytes(int64_t cols, int nv) { return (cols / (nv ? 16 : 32) + 15) / 16 * 16; }

// quantize(x, codes, scales, fmt, tensor_scale, swiglu, rows_dev)
int quantize(Args& g) {
  const int nv = format(g.a[3]);
  const bool swiglu = g.a[5] == Py_True;
  if (nv < 0 || (!swiglu && g.a[5] != Py_False)) return -1;
  const Tensor* x = g.tensor(0, ScalarType::Undefined);
  if (!g.ok || x->dim() != 2) return -1;
  const int64_t n = x->size(0), wide = x->size(1), cols = swiglu ? wide / 2 : wide;
  const int code = dtype_code(*x, false);
  if (code == 0 || (swiglu && wide % 2) || cols > kMaxInt) return -1;
  const Tensor* codes = g.sized(1, ScalarType::Byte, {n, cols / 2});
  const Tensor* scales = g.ok ? g.sized(2, ScalarType::Byte, {n, scale_bytes(cols, nv)}) : nullptr;
  const Tensor* ts = g.ok ? g.sized(4, ScalarType::Float, {1}, true) : nullptr;
  const Tensor* rd = g.ok ? g.tensor(6, ScalarType::Int, true) : nullptr;
  if (!g.ok || (rd && rd->numel() != 1)) return -1;
  return f_quantize(x->data_ptr(), code, n, int(cols), nv ? MOE_FP_NV : MOE_FP_MX, swiglu ? MOE_FP_SWIGLU : 0u,
                    ptr<float>(ts), ptr<int32_t>(rd), ptr<uint8_t>(codes), ptr<uint8_t>(scales), g.stream());
}

// dequantize(codes, scales, out, fmt, tensor_scale, rows_dev)
int dequantize(Args& g) {
  const int nv = format(g.a[3]);
  if (nv < 0) return -1;
  const Tensor* out = g.tensor(2, ScalarType::Undefined);
  if (!g.ok || out->dim() != 2) return -1;
  const int64_t n = out->size(0), cols = out->size(1);
  const int code = dtype_code(*out, false);
  if (code == 0 || cols > kMaxInt) return -1;
  const Tensor* codes = g.sized(0, ScalarType::Byte, {n, cols / 2});
  const Tensor* scales = g.ok ? g.sized(1, ScalarType::Byte, {n, scale_bytes(cols, nv)}) : nullptr;
  const Tensor* ts = g.ok ? g.sized(4, ScalarType::Float, {1}, true) : nullptr;
  const Tensor* rd = g.ok ? g.tensor(5, ScalarType::Int, true) : nullptr;
  if (!g.ok || (rd && rd->numel() != 1)) return -1;
  return f_dequantize(ptr<uint8_t>(codes), ptr<uint8_t>(scales), n, int(cols), nv ? MOE_FP_NV : MOE_FP_MX,
                      ptr<float>(ts), ptr<int32_t>(rd), out->data_ptr(), code, g.stream());
}

// matmul(a_codes, a_scales, b_codes, b_scales, out, fmt, ws, offsets, a_tensor_scale, b_tensor_scale)
int matmul(Args& g) {
  const int nv = format(g.a[5]);
  if (nv < 0) return -1;
  const Tensor* out = g.tensor(4, ScalarType::Undefined);
  const Tensor* b = g.ok ? g.tensor(2, ScalarType::Byte) : nullptr;
  const Tensor* ws = g.ok ? g.tensor(6, ScalarType::Byte) : nullptr;
  if (!g.ok || out->dim() != 2 || b->dim() != 3) return -1;
  const int64_t R = out->size(0), N = out->size(1), E = b->size(0), half = b->size(2), S = scale_bytes(2 * half, nv);
  const int code = dtype_code(*out, false);
  if (code == 0 || b->size(1) != N || R > kMaxInt || N > kMaxInt || E > kMaxInt || 2 * half > kMaxInt) return -1;
  const Tensor* ac = g.sized(0, ScalarType::Byte, {R, half});
  const Tensor* as = g.ok ? g.sized(1, ScalarType::Byte, {R, S}) : nullptr;
  const Tensor* bs = g.ok ? g.sized(3, ScalarType::Byte, {E, N, S}) : nullptr;
  const Tensor* off = g.ok ? g.sized(7, ScalarType::Int, {E + 1}, true) : nullptr;
  const Tensor* ga = g.ok ? g.sized(8, ScalarType::Float, {1}, true) : nullptr;
  const Tensor* gb = g.ok ? g.sized(9, ScalarType::Float, {E}, true) : nullptr;
  if (!g.ok) return -1;
  return f_matmul(ptr<uint8_t>(ac), ptr<uint8_t>(as), ptr<float>(ga), int(R), int(2 * half), ptr<uint8_t>(b),
                  ptr<uint8_t>(bs), ptr<float>(gb), int(E), int(N), ptr<int32_t>(off), nv ? MOE_FP_NV : MOE_FP_MX,
                  out->data_ptr(), code, ws->data_ptr(), size_t(ws->numel()), g.stream());
}

// No C++ exception reaches the interpreter: torch's are answered like any
// other argument that is not plainly right.
template <int (*F)(Args&), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  int st = -1;
  if (n == kArgs) {
    try {
      Args g{args};
      st = F(g);
    } catch (...) {
      st = -1;
    }
  }
  return PyLong_FromLong(st);
}

template <typename Fn>
bool find(void* lib, const char* name, Fn* f) {
  *f = reinterpret_cast<Fn>(dlsym(lib, name));
  return *f != nullptr;
}

// bind(path of libmoe_b200.so)
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* lib = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (!lib || !find(lib, "moe_permute", &f_permute) || !find(lib, "moe_permute_grad", &f_permute_grad) ||
      !find(lib, "moe_unpermute", &f_unpermute) || !find(lib, "moe_unpermute_grad", &f_unpermute_grad) ||
      !find(lib, "moe_mxfp_quantize", &f_quantize) || !find(lib, "moe_mxfp_dequantize", &f_dequantize) ||
      !find(lib, "moe_mxfp_matmul", &f_matmul))
    return PyErr_Format(PyExc_ImportError, "%s does not hold the calls of include/moe.h", p);
  Py_RETURN_NONE;
}

#define MOE_FAST(name, F, kArgs) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, kArgs>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", bind, METH_O, nullptr},
    MOE_FAST("permute", permute, 4),
    MOE_FAST("permute_grad", permute_grad, 4),
    MOE_FAST("unpermute", unpermute, 5),
    MOE_FAST("unpermute_grad", unpermute_grad, 7),
    MOE_FAST("quantize", quantize, 7),
    MOE_FAST("dequantize", dequantize, 6),
    MOE_FAST("matmul", matmul, 10),
    {nullptr, nullptr, 0, nullptr},
};
#ifndef MOE_MADE_FOR
#define MOE_MADE_FOR ""
#endif
// The doc text says which torch and Python this was compiled for; the build looks for it.
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", MOE_MADE_FOR, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
