// torch_calls.cpp -- the argument marshalling of the gated feed-forward and
// Newton-Schulz bindings as a CPython module: tensors in, libfp8q's C ABI called
// on torch's current stream, result tensors out.  No step of the computation is
// here.  A small call takes longer to marshal than to run; looking at up to 18
// tensors and making up to 8 new ones costs, on a Grace core, 3.0 to 3.5 us with
// the results given (launch included) and 0.8 to 0.9 us more per new tensor,
// against 9 us and 1.6 us per tensor from Python through ctypes.
//
// Every function takes positional arguments (binding.py gives them their names
// and defaults) and returns the tuple of results, or the fp8q_status as an int
// where the call failed.  Wrong tensors raise ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <optional>
#include <string>

#include "fp8q.h"

namespace {

struct Mat {
  void *p = nullptr;
  int64_t ld = 0;
};

bool fail(const std::string &what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  return false;
}

const at::Tensor *tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

// Address and row pitch of a matrix whose shape and type must be as given; the
// strides of one-long axes do not count.
bool mat(const at::Tensor &t, int64_t rows, int64_t cols, at::ScalarType dtype, at::Device dev,
         const char *name, Mat &m) {
  if (t.scalar_type() != dtype || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    return fail(std::string(name) + " must be a " + c10::toString(dtype) + " tensor of shape (" +
                std::to_string(rows) + ", " + std::to_string(cols) + ")");
  if (!t.is_cuda()) return fail(std::string(name) + " must be on a CUDA device");
  if (t.device() != dev) return fail(std::string(name) + " must be on " + dev.str());
  if (cols > 1 && rows > 0 && t.stride(1) != 1)
    return fail(std::string(name) + " must have a contiguous last dimension");
  m.p = t.numel() ? t.data_ptr() : nullptr;
  m.ld = rows > 1 ? t.stride(0) : cols;
  return true;
}
bool mat(PyObject *o, int64_t rows, int64_t cols, at::ScalarType dtype, at::Device dev,
         const char *name, Mat &m) {
  const at::Tensor *t = tensor(o, name);
  return t && mat(*t, rows, cols, dtype, dev, name, m);
}

// Where a call runs, and where the memory that it takes for itself comes from:
// the stream of its kernels.  torch hands freed memory out again in the order of
// the stream it was taken on, so memory of the current stream would be reused
// while kernels on another one still work in it.
class Place {
 public:
  // torch's current stream, or the given stream's handle.
  bool set(PyObject *stream, at::Device device) {
    dev = device;
    // the library launches on the device that is current
    if (c10::cuda::current_device() != dev.index()) on_device_.emplace(device);
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(dev.index());
    handle = current.stream();
    if (stream == Py_None) return true;
    handle = PyLong_AsVoidPtr(stream);
    if (handle == nullptr && PyErr_Occurred()) return false;
    if (handle != current.stream()) {
      other_ = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), dev.index());
      reader_ = current;
    }
    return true;
  }
  // Scratch: nothing but this call's kernels uses it.
  at::Tensor scratch(int64_t bytes) const { return take({bytes}, at::kByte); }
  // A result: the caller may go on with it on the current stream (once that
  // stream waits for the other one) and drop it there.
  at::Tensor result(at::IntArrayRef size, at::ScalarType dtype) const {
    at::Tensor t = take(size, dtype);
    if (reader_ && t.nbytes() > 0)
      c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *reader_);
    return t;
  }

  at::Device dev{at::kCUDA, 0};
  void *handle = nullptr;

 private:
  at::Tensor take(at::IntArrayRef size, at::ScalarType dtype) const {
    std::optional<c10::cuda::CUDAStreamGuard> on;
    if (other_) on.emplace(*other_);
    return at::Tensor(at::detail::empty_cuda(size, dtype, dev, c10::nullopt));
  }
  std::optional<c10::cuda::CUDAGuard> on_device_;
  std::optional<c10::cuda::CUDAStream> other_, reader_;  // set where they differ
};

// The interpreter's other threads run while this lives: an allocation may wait
// for the device, a launch for room in its queue.
struct NoGil {
  PyThreadState *const state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

// Results of a call: the caller's tensor, checked, a new one, or None.
class Results {
 public:
  bool add(PyObject *given, bool wanted, int64_t rows, int64_t cols, at::ScalarType dtype,
           at::Device dev, const char *name, Mat &m, bool &present) {
    One &r = all_[n_++];
    present = wanted || given != Py_None;
    if (given != Py_None) {
      r.given = given;
      return mat(given, rows, cols, dtype, dev, name, m);
    }
    if (wanted) {
      m.ld = cols;
      r.rows = rows;
      r.dtype = dtype;
      r.wanted = &m;
    }
    return true;
  }
  // Make the new ones (needs no GIL).
  void make(const Place &place) {
    for (int i = 0; i < n_; ++i)
      if (Mat *m = all_[i].wanted) {
        all_[i].made = place.result({all_[i].rows, m->ld}, all_[i].dtype);
        m->p = all_[i].made.data_ptr();
      }
  }
  PyObject *tuple(fp8q_status st) {
    if (st != FP8Q_OK) return PyLong_FromLong(st);
    PyObject *t = PyTuple_New(n_);
    for (int i = 0; t && i < n_; ++i) {
      PyObject *o = all_[i].wanted ? THPVariable_Wrap(std::move(all_[i].made))
                                   : Py_NewRef(all_[i].given ? all_[i].given : Py_None);
      if (o) PyTuple_SET_ITEM(t, i, o);
      else Py_CLEAR(t);
    }
    return t;
  }

 private:
  struct One {
    PyObject *given = nullptr;
    Mat *wanted = nullptr;  // of the new one
    int64_t rows = 0;
    at::ScalarType dtype = at::kByte;
    at::Tensor made;
  };
  One all_[8];
  int n_ = 0;
};

// Flags by their truth, as Python takes them (1, a numpy bool, ...).
template <int N>
bool flags(PyObject *const *o, bool (&v)[N]) {
  for (int i = 0; i < N; ++i) {
    const int t = PyObject_IsTrue(o[i]);
    if (t < 0) return false;
    v[i] = t != 0;
  }
  return true;
}

// A Python int as a C int; what does not fit becomes the nearest that does, which
// is out of range for every argument here, and the call refuses it.
bool int_of(PyObject *o, int &v) {
  int past = 0;
  const long x = PyLong_AsLongAndOverflow(o, &past);
  if (x == -1 && past == 0 && PyErr_Occurred()) return false;
  v = past > 0 || x > INT_MAX ? INT_MAX : past < 0 || x < INT_MIN ? INT_MIN : static_cast<int>(x);
  return true;
}

PyObject *wrong_count(const char *name) {
  PyErr_Format(PyExc_TypeError, "%s: wrong number of arguments", name);
  return nullptr;
}

// (pow2, a, sa, b, sb, offs, with_h, with_gu, with_codes, scale_mode, h, gu, q, s, stream)
PyObject *swiglu_impl(PyObject *const *v, Py_ssize_t n) {
  if (n != 15) return wrong_count("swiglu");
  const bool pow2 = v[0] == Py_True;
  const at::Tensor *a = tensor(v[1], "a"), *b = tensor(v[3], "b"), *sb = tensor(v[4], "sb");
  if (!a || !b || !sb) return nullptr;
  const bool grouped = v[5] != Py_None;
  if (a->dim() != 2 || b->dim() != (grouped ? 3 : 2)) {
    fail(grouped ? "a must be [M][K] and b [G][2F][K]" : "a must be [M][K] and b [2F][K]");
    return nullptr;
  }
  const int64_t M = a->size(0), K = a->size(1), N = b->size(-2), F = N / 2;
  if (N % 2 || b->size(-1) != K) {
    fail("b must hold both projections: [2F][K] rows, with a's K");
    return nullptr;
  }
  const at::Device dev = a->device();
  Mat ma, msa, mb, msb;
  if (!mat(*a, M, K, at::kByte, dev, "a", ma) || !mat(v[2], K / 128, M, at::kFloat, dev, "sa", msa))
    return nullptr;
  const int32_t *offs = nullptr;
  int64_t G = 1;
  if (grouped) {
    G = b->size(0);
    const at::Tensor *to = tensor(v[5], "offs");
    if (!to) return nullptr;
    if (b->scalar_type() != at::kByte ||
        (b->numel() && (b->stride(2) != 1 || b->stride(0) != N * b->stride(1)))) {
      fail("b must be uint8 [G][2F][K], its last dimension contiguous and its experts back to back");
      return nullptr;
    }
    if (sb->scalar_type() != at::kFloat || sb->dim() != 3 || sb->size(0) != G ||
        sb->size(1) != N / 128 || sb->size(2) != K / 128 || !sb->is_contiguous()) {
      fail("sb must be a contiguous float32 [G][2F/128][K/128] tensor");
      return nullptr;
    }
    if (to->scalar_type() != at::kInt || to->dim() != 1 || to->size(0) != G + 1 ||
        !to->is_contiguous()) {
      fail("offs must be a contiguous int32 [G+1] tensor");
      return nullptr;
    }
    if (b->device() != dev || sb->device() != dev || to->device() != dev) {
      fail("b, sb and offs must be on a's CUDA device");
      return nullptr;
    }
    mb.p = b->numel() ? b->data_ptr() : nullptr;
    mb.ld = b->stride(1);
    msb.p = sb->numel() ? sb->data_ptr() : nullptr;
    offs = to->data_ptr<int32_t>();
  } else if (!mat(*b, N, K, at::kByte, dev, "b", mb) ||
             !mat(*sb, N / 128, K / 128, at::kFloat, dev, "sb", msb)) {
    return nullptr;
  }
  int mode = 0;
  Place place;
  bool want[3];  // h, gu, codes
  if (!int_of(v[9], mode) || !flags(v + 6, want) || !place.set(v[14], dev)) return nullptr;
  Results r;
  Mat h, gu, q, s;
  bool has_h, has_gu, has_q, has_s;
  if (!r.add(v[10], want[0], M, F, at::kBFloat16, dev, "h", h, has_h) ||
      !r.add(v[11], want[1], M, 2 * F, at::kBFloat16, dev, "gu", gu, has_gu) ||
      !r.add(v[12], want[2], M, F, at::kByte, dev, "q", q, has_q) ||
      !r.add(v[13], has_q, F / 128, M, at::kFloat, dev, "s", s, has_s))
    return nullptr;
  const float *fsa = static_cast<const float *>(msa.p), *fsb = static_cast<const float *>(msb.p);
  fp8q_status st;
  {
    NoGil free;
    r.make(place);
    float *fs = static_cast<float *>(s.p);
    if (grouped)
      st = (pow2 ? fp8q_grouped_gemm_swiglu_pow2 : fp8q_grouped_gemm_swiglu)(
          ma.p, ma.ld, fsa, msa.ld, mb.p, mb.ld, fsb, offs, static_cast<int>(G), h.p, h.ld, gu.p,
          gu.ld, q.p, q.ld, fs, s.ld, mode, M, F, K, place.handle);
    else
      st = (pow2 ? fp8q_gemm_swiglu_pow2 : fp8q_gemm_swiglu)(
          ma.p, ma.ld, fsa, msa.ld, mb.p, mb.ld, fsb, msb.ld, h.p, h.ld, gu.p, gu.ld, q.p, q.ld,
          fs, s.ld, mode, M, F, K, place.handle);
  }
  return r.tuple(st);
}

// (dh, gu, with_d, with_rows, with_cols, with_h, scale_mode, d, q, s, qT, sT, hT, shT, stream)
PyObject *bwd_impl(PyObject *const *v, Py_ssize_t n) {
  if (n != 15) return wrong_count("swiglu_bwd");
  const at::Tensor *dh = tensor(v[0], "dh");
  if (!dh) return nullptr;
  if (dh->dim() != 2) {
    fail("dh must be [T][F]");
    return nullptr;
  }
  const int64_t T = dh->size(0), F = dh->size(1), N = 2 * F;
  const at::Device dev = dh->device();
  Mat mdh, mgu;
  if (!mat(*dh, T, F, at::kBFloat16, dev, "dh", mdh) || !mat(v[1], T, N, at::kBFloat16, dev, "gu", mgu))
    return nullptr;
  int mode = 0;
  Place place;
  bool want[4];  // d, rows, cols, h
  if (!int_of(v[6], mode) || !flags(v + 2, want) || !place.set(v[14], dev)) return nullptr;
  Results r;
  Mat d, q, s, qT, sT, hT, shT;
  bool has_d, has_q, has_qT, has_hT, has;
  if (!r.add(v[7], want[0], T, N, at::kBFloat16, dev, "d", d, has_d) ||
      !r.add(v[8], want[1], T, N, at::kByte, dev, "q", q, has_q) ||
      !r.add(v[9], has_q, N / 128, T, at::kFloat, dev, "s", s, has) ||
      !r.add(v[10], want[2], N, T, at::kByte, dev, "qT", qT, has_qT) ||
      !r.add(v[11], has_qT, T / 128, N, at::kFloat, dev, "sT", sT, has) ||
      !r.add(v[12], want[3], F, T, at::kByte, dev, "hT", hT, has_hT) ||
      !r.add(v[13], has_hT, T / 128, F, at::kFloat, dev, "shT", shT, has))
    return nullptr;
  fp8q_status st;
  {
    NoGil free;
    r.make(place);
    st = fp8q_swiglu_bwd(mdh.p, mdh.ld, mgu.p, mgu.ld, d.p, d.ld, q.p, q.ld,
                         static_cast<float *>(s.p), s.ld, qT.p, qT.ld, static_cast<float *>(sT.p),
                         sT.ld, hT.p, hT.ld, static_cast<float *>(shT.p), shT.ld, T, F, mode,
                         place.handle);
  }
  return r.tuple(st);
}

// Row and matrix pitch of a matrix or a batch of matrices.
bool pitches(const at::Tensor &t, const char *name, int64_t &ld, int64_t &stride) {
  const int64_t m = t.size(-2), n = t.size(-1);
  if (n > 1 && m > 0 && t.stride(-1) != 1)
    return fail(std::string(name) + " must have a contiguous last dimension");
  ld = m > 1 ? t.stride(-2) : n;
  stride = t.dim() == 3 ? t.stride(0) : 0;
  return true;
}

// (g, steps, a, b, c, eps, out_dtype, out, workspace, stream)
PyObject *newton_schulz_impl(PyObject *const *v, Py_ssize_t n) {
  if (n != 10) return wrong_count("newton_schulz");
  const at::Tensor *g = tensor(v[0], "g");
  if (!g) return nullptr;
  if ((g->dim() != 2 && g->dim() != 3) ||
      (g->scalar_type() != at::kFloat && g->scalar_type() != at::kBFloat16) || !g->is_cuda()) {
    fail("g must be an FP32 or BF16 matrix or batch of matrices on a CUDA device");
    return nullptr;
  }
  const at::Device dev = g->device();
  int steps = 0, out_dtype = 0;
  if (!int_of(v[1], steps) || !int_of(v[6], out_dtype)) return nullptr;
  const double a = PyFloat_AsDouble(v[2]), b = PyFloat_AsDouble(v[3]), c = PyFloat_AsDouble(v[4]),
               eps = PyFloat_AsDouble(v[5]);
  Place place;
  if (PyErr_Occurred() || !place.set(v[9], dev)) return nullptr;
  const at::ScalarType od = out_dtype == FP8Q_OUT_BF16 ? at::kBFloat16 : at::kFloat;
  at::Tensor out;
  if (v[7] != Py_None) {
    const at::Tensor *t = tensor(v[7], "out");
    if (!t) return nullptr;
    if (t->sizes() != g->sizes() || t->scalar_type() != od || t->device() != dev) {
      fail("out must have g's shape and the type out_dtype names, on g's CUDA device");
      return nullptr;
    }
    out = *t;
  }
  at::Tensor ws;
  if (v[8] != Py_None) {
    const at::Tensor *t = tensor(v[8], "workspace");
    if (!t) return nullptr;
    if (t->device() != dev || !t->is_contiguous()) {
      fail("workspace must be a contiguous tensor on g's CUDA device");
      return nullptr;
    }
    ws = *t;
  }
  const int64_t B = g->dim() == 3 ? g->size(0) : 1, m = g->size(-2), nn = g->size(-1);
  int64_t ld_g, stride_g, ld_o = nn, stride_o = m * nn;
  if (!pitches(*g, "g", ld_g, stride_g) || (out.defined() && !pitches(out, "out", ld_o, stride_o)))
    return nullptr;
  const bool any = g->numel() > 0;
  fp8q_status st;
  {
    NoGil free;
    if (!out.defined()) out = place.result(g->sizes(), od);
    if (!ws.defined()) {
      const int64_t bytes = fp8q_newton_schulz_workspace_bytes(B, m, nn);
      ws = place.scratch(bytes > 0 ? bytes : 1);
    }
    st = fp8q_newton_schulz(
        any ? g->data_ptr() : nullptr, ld_g, stride_g,
        g->scalar_type() == at::kFloat ? FP8Q_OUT_FP32 : FP8Q_OUT_BF16,
        any ? out.data_ptr() : nullptr, ld_o, stride_o, out_dtype, B, m, nn, steps,
        static_cast<float>(a), static_cast<float>(b), static_cast<float>(c),
        static_cast<float>(eps), ws.data_ptr(), static_cast<int64_t>(ws.nbytes()), place.handle);
  }
  if (st != FP8Q_OK) return PyLong_FromLong(st);
  if (v[7] != Py_None) {
    Py_INCREF(v[7]);
    return v[7];
  }
  return THPVariable_Wrap(std::move(out));
}

// No C++ exception (an allocation that fails, say) leaves through CPython.
template <PyObject *(*kImpl)(PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *, PyObject *const *v, Py_ssize_t n) {
  try {
    return kImpl(v, n);
  } catch (const c10::OutOfMemoryError &e) {
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyMethodDef methods[] = {
    {"swiglu", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<swiglu_impl>)),
     METH_FASTCALL, nullptr},
    {"swiglu_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<bwd_impl>)),
     METH_FASTCALL, nullptr},
    {"newton_schulz",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<newton_schulz_impl>)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&module); }
