// torch_calls.cpp -- the argument marshalling of the gated feed-forward,
// Newton-Schulz, norm, AdamW and router bindings as a CPython module: tensors in,
// libfp8q's C ABI called on torch's current stream, result tensors out.  No step of
// the computation is here.  A small call takes longer to marshal than to run; looking
// at up to 18 tensors and making up to 8 new ones costs, on a Grace core, 2.7 to 3.5 us
// with the results given (launch included) and 0.8 to 0.9 us more per new tensor, against
// 9 us and 1.6 us per tensor from Python through ctypes.  Small results of the norm and
// router calls share an allocation: eight cost 3.6 us more, three 1.9.
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
#include <vector>

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

// Address of a vector whose length and type must be as given.
bool vec(const at::Tensor &t, int64_t n, at::ScalarType dtype, at::Device dev, const char *name,
         void *&p) {
  if (t.scalar_type() != dtype || t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    return fail(std::string(name) + " must be a contiguous " + c10::toString(dtype) +
                " tensor of shape (" + std::to_string(n) + ",)");
  if (t.device() != dev || !t.is_cuda())
    return fail(std::string(name) + " must be on " + (dev.is_cuda() ? dev.str() : "a CUDA device"));
  p = n ? t.data_ptr() : nullptr;
  return true;
}

// FP8Q_OUT_BF16 or FP8Q_OUT_FP32 for a tensor of either type.
bool kind_of(const at::Tensor &t, const char *name, int &kind) {
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
    return fail(std::string(name) + " must be BFloat16 or Float");
  kind = t.scalar_type() == at::kFloat ? FP8Q_OUT_FP32 : FP8Q_OUT_BF16;
  return true;
}

// One value in device memory (a tensor of one element), or null for None.
bool scalar(PyObject *o, at::ScalarType dtype, at::Device dev, const char *name, const void *&p) {
  p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor *t = tensor(o, name);
  if (!t) return false;
  if (t->scalar_type() != dtype || t->numel() != 1 || t->device() != dev)
    return fail(std::string(name) + " must be a " + c10::toString(dtype) + " tensor of one element on " +
                dev.str());
  p = t->data_ptr();
  return true;
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

// Results of a call: the caller's tensor, checked, a new one, or None.  With
// `together` new ones are parts of an allocation, 256 bytes apart at least: it takes
// longer to ask the allocator for each than to run a small call.  A part keeps the whole
// alive, so what is little (a loss, a few rows' statistics) shares with no more than
// kFew bytes, however many of it a program keeps.
class Results {
 public:
  explicit Results(bool together = false) : together_(together) {}
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
  // The same for a vector of n elements.
  bool add_vec(PyObject *given, bool wanted, int64_t n, at::ScalarType dtype, at::Device dev,
               const char *name, Mat &m) {
    One &r = all_[n_++];
    if (given != Py_None) {
      r.given = given;
      const at::Tensor *t = tensor(given, name);
      return t && vec(*t, n, dtype, dev, name, m.p);
    }
    if (wanted) {
      r.rows = n;
      r.dtype = dtype;
      r.vector = true;
      r.wanted = &m;
    }
    return true;
  }
  // The call's own scratch, made with the results; `p` is set by make().
  void scratch(int64_t bytes, void *&p) {
    scratch_bytes_ = bytes;
    scratch_ = &p;
  }
  // Make the new ones (needs no GIL).
  void make(const Place &place) {
    if (together_) make_together(place);
    if (scratch_ && !*scratch_) {
      scratch_made_ = place.scratch(scratch_bytes_);
      *scratch_ = scratch_made_.data_ptr();
    }
    for (int i = 0; i < n_; ++i)
      if (Mat *m = all_[i].wanted; m && !all_[i].made.defined()) {
        One &r = all_[i];
        r.made = r.vector ? place.result({r.rows}, r.dtype) : place.result({r.rows, m->ld}, r.dtype);
        m->p = r.made.data_ptr();
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
    bool vector = false;
    at::Tensor made;
  };
  static constexpr int64_t kLittle = 4 << 10, kFew = 64 << 10, kMost = 2 << 20;  // bytes
  int64_t room(const One &r) const {
    const int64_t n = r.vector ? r.rows : r.rows * r.wanted->ld;
    return (n * static_cast<int64_t>(c10::elementSize(r.dtype)) + 255) / 256 * 256;
  }
  void make_together(const Place &place) {
    int64_t all = scratch_bytes_;
    for (int i = 0; i < n_; ++i)
      if (all_[i].wanted) all += room(all_[i]);
    if (all <= kFew) {
      make_block(place, -1, kFew, kFew, true);
    } else {
      make_block(place, -1, kLittle, kFew, false);
      make_block(place, kLittle, kMost, kMost, true);
    }
  }
  // Those of more than `over` and at most `upto` bytes, and the scratch, in one allocation, if
  // there are two at least and `most` bytes hold them.
  void make_block(const Place &place, int64_t over, int64_t upto, int64_t most, bool with_scratch) {
    int64_t at[8], bytes = 0;
    int count = 0;
    for (int i = 0; i < n_; ++i) {
      at[i] = -1;
      if (!all_[i].wanted) continue;
      const int64_t size = room(all_[i]);
      if (size <= over || size > upto) continue;
      at[i] = bytes;
      bytes += size;
      ++count;
    }
    with_scratch = with_scratch && scratch_;
    const int64_t scratch_at = bytes;
    if (with_scratch) {
      bytes += scratch_bytes_;
      ++count;
    }
    if (count < 2 || bytes > most) return;
    const at::Tensor block = place.result({bytes}, at::kByte);
    char *base = static_cast<char *>(block.data_ptr());
    for (int i = 0; i < n_; ++i) {
      if (at[i] < 0) continue;
      One &r = all_[i];
      r.made = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(block.storage()), block.key_set(),
                                                        c10::scalarTypeToTypeMeta(r.dtype));
      c10::TensorImpl *impl = r.made.unsafeGetTensorImpl();
      impl->set_storage_offset(at[i] / static_cast<int64_t>(c10::elementSize(r.dtype)));
      if (r.vector) impl->set_sizes_contiguous({r.rows});
      else impl->set_sizes_contiguous({r.rows, r.wanted->ld});
      r.wanted->p = base ? base + at[i] : nullptr;
    }
    if (with_scratch) {
      scratch_made_ = block;
      *scratch_ = base + scratch_at;
    }
  }
  One all_[8];
  void **scratch_ = nullptr;
  int64_t scratch_bytes_ = 0;
  at::Tensor scratch_made_;
  int n_ = 0;
  const bool together_;
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

// A tensor argument of either type as rows x cols.
bool mat_any(PyObject *o, int64_t rows, int64_t cols, at::Device dev, const char *name, Mat &m,
             int &kind) {
  const at::Tensor *t = tensor(o, name);
  return t && kind_of(*t, name, kind) && mat(*t, rows, cols, t->scalar_type(), dev, name, m);
}
bool vec_any(PyObject *o, int64_t n, at::Device dev, const char *name, Mat &m, int &kind) {
  const at::Tensor *t = tensor(o, name);
  return t && kind_of(*t, name, kind) && vec(*t, n, t->scalar_type(), dev, name, m.p);
}
// The caller's workspace.
bool workspace(PyObject *o, at::Device dev, void *&p, int64_t &bytes) {
  const at::Tensor *t = tensor(o, "workspace");
  if (!t) return false;
  if (t->device() != dev || !t->is_contiguous())
    return fail("workspace must be a contiguous tensor on " + dev.str());
  p = t->numel() ? t->data_ptr() : nullptr;
  bytes = static_cast<int64_t>(t->nbytes());
  return true;
}

at::ScalarType type_of(int kind) { return kind == FP8Q_OUT_FP32 ? at::kFloat : at::kBFloat16; }

// (x, w, residual, eps, with_r, with_y, with_codes, with_rstd, scale_mode, r, y, q, s, rstd, stream)
PyObject *rmsnorm_impl(PyObject *const *v, Py_ssize_t n) {
  if (n != 15) return wrong_count("rmsnorm");
  const at::Tensor *x = tensor(v[0], "x");
  if (!x) return nullptr;
  if (x->dim() != 2) {
    fail("x must be [T][C]");
    return nullptr;
  }
  const int64_t T = x->size(0), C = x->size(1);
  const at::Device dev = x->device();
  Mat mx, mw, mres;
  int kx = 0, kw = 0, kres = 0, mode = 0;
  const bool has_res = v[2] != Py_None;
  if (!mat_any(v[0], T, C, dev, "x", mx, kx) || !vec_any(v[1], C, dev, "w", mw, kw) ||
      (has_res && !mat_any(v[2], T, C, dev, "residual", mres, kres)))
    return nullptr;
  const double eps = PyFloat_AsDouble(v[3]);
  Place place;
  bool want[4];  // r, y, codes, rstd
  if (PyErr_Occurred() || !int_of(v[8], mode) || !flags(v + 4, want) || !place.set(v[14], dev))
    return nullptr;
  if (!has_res && v[9] != Py_None) {
    fail("r is the sum with the residual: it needs one");
    return nullptr;
  }
  Results out(true);
  Mat r, y, q, s, rstd;
  bool has_r, has_y, has_q, has_s;
  if (!out.add(v[9], want[0] && has_res, T, C, type_of(kres), dev, "r", r, has_r) ||
      !out.add(v[10], want[1], T, C, at::kBFloat16, dev, "y", y, has_y) ||
      !out.add(v[11], want[2], T, C, at::kByte, dev, "q", q, has_q) ||
      !out.add(v[12], has_q, C / 128, T, at::kFloat, dev, "s", s, has_s) ||
      !out.add_vec(v[13], want[3], T, at::kFloat, dev, "rstd", rstd))
    return nullptr;
  fp8q_status st;
  {
    NoGil free;
    out.make(place);
    st = fp8q_rmsnorm(mx.p, mx.ld, kx, mres.p, mres.ld, kres, mw.p, kw, static_cast<float>(eps), r.p,
                      r.ld, y.p, y.ld, q.p, q.ld, static_cast<float *>(s.p), s.ld,
                      static_cast<float *>(rstd.p), mode, T, C, place.handle);
  }
  return out.tuple(st);
}

// (dy, x, rstd, w, dres, with_dx, with_dw, out_dtype, dx, dw, accumulate, workspace, stream)
PyObject *rmsnorm_bwd_impl(PyObject *const *v, Py_ssize_t n) {
  if (n != 13) return wrong_count("rmsnorm_bwd");
  const at::Tensor *dy = tensor(v[0], "dy");
  if (!dy) return nullptr;
  if (dy->dim() != 2) {
    fail("dy must be [T][C]");
    return nullptr;
  }
  const int64_t T = dy->size(0), C = dy->size(1);
  const at::Device dev = dy->device();
  Mat mdy, mx, mrstd, mw, mdres;
  int kdy = 0, kx = 0, kw = 0, kd = 0;
  const at::Tensor *rstd = tensor(v[2], "rstd");
  if (!rstd || !mat_any(v[0], T, C, dev, "dy", mdy, kdy) || !mat_any(v[1], T, C, dev, "x", mx, kx) ||
      !vec(*rstd, T, at::kFloat, dev, "rstd", mrstd.p) || !vec_any(v[3], C, dev, "w", mw, kw) ||
      !int_of(v[7], kd))
    return nullptr;
  const at::ScalarType od = type_of(kd);
  if (v[4] != Py_None && !mat(v[4], T, C, od, dev, "dres", mdres)) return nullptr;
  Place place;
  bool want[2], accumulate[1];  // dx, dw
  if (!flags(v + 5, want) || !flags(v + 10, accumulate) || !place.set(v[12], dev)) return nullptr;
  if (accumulate[0] && v[9] == Py_None) {
    fail("accumulate adds to the dw that is given");
    return nullptr;
  }
  Results out(true);
  Mat dx, dw;
  bool has_dx;
  if (!out.add(v[8], want[0], T, C, od, dev, "dx", dx, has_dx) ||
      !out.add_vec(v[9], want[1], C, at::kFloat, dev, "dw", dw))
    return nullptr;
  void *ws = nullptr;
  int64_t ws_bytes = 0;
  if (v[11] != Py_None) {
    if (!workspace(v[11], dev, ws, ws_bytes)) return nullptr;
  } else if (want[1] || v[9] != Py_None) {
    ws_bytes = fp8q_rmsnorm_bwd_workspace_bytes(T, C);
    if (ws_bytes > 0) out.scratch(ws_bytes, ws);
  }
  fp8q_status st;
  {
    NoGil free;
    out.make(place);
    st = fp8q_rmsnorm_bwd(mdy.p, mdy.ld, kdy, mx.p, mx.ld, kx, static_cast<float *>(mrstd.p), mw.p, kw,
                          mdres.p, mdres.ld, dx.p, dx.ld, kd, static_cast<float *>(dw.p),
                          accumulate[0], T, C, ws, ws_bytes, place.handle);
  }
  return out.tuple(st);
}

// A list or tuple of tensors.
class List {
 public:
  ~List() { Py_XDECREF(items_); }
  bool take(PyObject *o, const char *name) {
    name_ = name;
    items_ = PySequence_Fast(o, "");
    if (!items_) {
      PyErr_Format(PyExc_TypeError, "%s must be a list of tensors", name);
      return false;
    }
    return true;
  }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(items_); }
  const at::Tensor *at(Py_ssize_t i) const { return tensor(PySequence_Fast_GET_ITEM(items_, i), name_); }

 private:
  PyObject *items_ = nullptr;
  const char *name_ = "";
};

// Address of entry i of a list: as many values as its parameter has, dense.
bool entry(const List &l, Py_ssize_t i, const char *name, int64_t count, at::ScalarType dtype,
           at::Device dev, void *&p) {
  const at::Tensor *t = l.at(i);
  if (!t) return false;
  if (t->scalar_type() != dtype || t->numel() != count || !t->is_contiguous() || t->device() != dev)
    return fail(std::string(name) + "[" + std::to_string(i) + "] must be a contiguous " +
                c10::toString(dtype) + " tensor of " + std::to_string(count) + " elements on " +
                dev.str());
  p = count ? t->data_ptr() : nullptr;
  return true;
}

// (params, grads, m, v, m_scales, v_scales, copies, lr, beta1, beta2, eps, weight_decay, step,
//  lr tensor, step tensor, grad_scale, stream); betas of None: what the moments' type can follow
PyObject *adamw_impl(PyObject *const *v, Py_ssize_t n) {
  if (n != 17) return wrong_count("adamw");
  List params, grads, ms, vs, mscales, vscales, copies;
  if (!params.take(v[0], "params") || !grads.take(v[1], "grads") || !ms.take(v[2], "m") ||
      !vs.take(v[3], "v"))
    return nullptr;
  const Py_ssize_t count = params.size();
  const bool has_scales = v[4] != Py_None, has_copies = v[6] != Py_None;
  if (has_scales != (v[5] != Py_None)) {
    fail("m_scales and v_scales go together");
    return nullptr;
  }
  if ((has_scales && (!mscales.take(v[4], "m_scales") || !vscales.take(v[5], "v_scales"))) ||
      (has_copies && !copies.take(v[6], "copies")))
    return nullptr;
  if (grads.size() != count || ms.size() != count || vs.size() != count ||
      (has_scales && (mscales.size() != count || vscales.size() != count)) ||
      (has_copies && copies.size() != count)) {
    fail("the lists must be as long as params");
    return nullptr;
  }
  double num[5];
  const bool own_betas = v[8] != Py_None || v[9] != Py_None;
  for (int i = 0; i < 5; ++i)
    if (own_betas || (i != 1 && i != 2)) num[i] = PyFloat_AsDouble(v[7 + i]);
  const long long step = PyLong_AsLongLong(v[12]);
  if (PyErr_Occurred()) return nullptr;
  if (count == 0) return PyLong_FromLong(FP8Q_OK);
  const at::Tensor *p0 = params.at(0), *g0 = p0 ? grads.at(0) : nullptr, *m0 = g0 ? ms.at(0) : nullptr;
  if (!m0) return nullptr;
  int kp = 0, kg = 0, state = FP8Q_STATE_E4M3;
  if (!kind_of(*p0, "params", kp) || !kind_of(*g0, "grads", kg)) return nullptr;
  const bool codes = m0->scalar_type() == at::kByte;
  if (!codes && !kind_of(*m0, "m", state)) return nullptr;
  if (codes != has_scales) {
    fail(codes ? "uint8 moments need m_scales and v_scales" : "only uint8 moments have scales");
    return nullptr;
  }
  if (!own_betas) {
    num[1] = 0.9;
    num[2] = state == FP8Q_STATE_FP32 ? 0.999 : 0.95;
  }
  const at::Device dev = p0->device();
  if (!dev.is_cuda()) {
    fail("params must be on a CUDA device");
    return nullptr;
  }
  const at::ScalarType tp = p0->scalar_type(), tg = g0->scalar_type(), tm = m0->scalar_type();
  const void *lr_dev, *step_dev, *scale;
  Place place;
  if (!scalar(v[13], at::kFloat, dev, "lr", lr_dev) || !scalar(v[14], at::kLong, dev, "step", step_dev) ||
      !scalar(v[15], at::kFloat, dev, "grad_scale", scale) || !place.set(v[16], dev))
    return nullptr;
  std::vector<fp8q_adamw_tensor> list(static_cast<size_t>(count));
  for (Py_ssize_t i = 0; i < count; ++i) {
    fp8q_adamw_tensor &t = list[static_cast<size_t>(i)];
    const at::Tensor *p = params.at(i);
    if (!p) return nullptr;
    t.n = p->numel();
    const int64_t groups = (t.n + 127) / 128;
    void *g = nullptr, *msc = nullptr, *vsc = nullptr;
    t.copy = nullptr;
    if (!entry(params, i, "params", t.n, tp, dev, t.p) || !entry(grads, i, "grads", t.n, tg, dev, g) ||
        !entry(ms, i, "m", t.n, tm, dev, t.m) || !entry(vs, i, "v", t.n, tm, dev, t.v) ||
        (codes && (!entry(mscales, i, "m_scales", groups, at::kFloat, dev, msc) ||
                   !entry(vscales, i, "v_scales", groups, at::kFloat, dev, vsc))) ||
        (has_copies && !entry(copies, i, "copies", t.n, at::kBFloat16, dev, t.copy)))
      return nullptr;
    t.g = g;
    t.m_scale = static_cast<float *>(msc);
    t.v_scale = static_cast<float *>(vsc);
  }
  fp8q_status st;
  {
    NoGil free;
    st = fp8q_adamw(list.data(), count, kp, kg, state, num[0], num[1], num[2], num[3], num[4], step,
                    static_cast<const float *>(lr_dev), static_cast<const int64_t *>(step_dev),
                    static_cast<const float *>(scale), place.handle);
  }
  return PyLong_FromLong(st);
}

// The logits of a router and the tokens that count.
bool router_in(PyObject *ol, PyObject *ovalid, Mat &l, int &kind, const uint8_t *&valid, int64_t &T,
               int64_t &E, std::optional<at::Device> &dev) {
  const at::Tensor *t = tensor(ol, "logits");
  if (!t) return false;
  if (t->dim() != 2) return fail("logits must be [T][E]");
  T = t->size(0);
  E = t->size(1);
  dev = t->device();
  if (!mat_any(ol, T, E, *dev, "logits", l, kind)) return false;
  valid = nullptr;
  if (ovalid == Py_None) return true;
  const at::Tensor *m = tensor(ovalid, "valid");
  if (!m) return false;
  if (m->scalar_type() != at::kBool && m->scalar_type() != at::kByte)
    return fail("valid must be a Bool or Byte tensor");
  void *p = nullptr;
  if (!vec(*m, T, m->scalar_type(), *dev, "valid", p)) return false;
  valid = static_cast<const uint8_t *>(p);
  return true;
}

// A result of T x k values without gaps.
bool dense(const Mat &m, int64_t T, int64_t k, const char *name) {
  return T <= 1 || m.ld == k || fail(std::string(name) + " must be contiguous");
}

// (logits, k, score, normalise, scale, valid, idx, weight, counts, offs, order, slot, tokens, loss,
//  workspace, stream)
PyObject *route_impl(PyObject *const *v, Py_ssize_t n) {
  if (n != 16) return wrong_count("route");
  Mat l;
  int kind = 0, k = 0, score = 0;
  const uint8_t *valid;
  int64_t T, E;
  std::optional<at::Device> at_dev;
  if (!router_in(v[0], v[5], l, kind, valid, T, E, at_dev)) return nullptr;
  const at::Device dev = *at_dev;
  bool normalise[1];
  if (!int_of(v[1], k) || !int_of(v[2], score) || !flags(v + 3, normalise)) return nullptr;
  const double scale = PyFloat_AsDouble(v[4]);
  Place place;
  if (PyErr_Occurred() || !place.set(v[15], dev)) return nullptr;
  if (E < 1 || E > 1024 || k < 1 || k > E || k > 32 || T > (int64_t{1} << 26) || T * k > 0x7FFFFFFFll)
    return PyLong_FromLong(FP8Q_ERR_SHAPE);  // before results of such sizes are made
  Results out(true);
  Mat idx, weight, counts, offs, order, slot, tokens, loss;
  bool has;
  if (!out.add(v[6], true, T, k, at::kInt, dev, "idx", idx, has) ||
      !out.add(v[7], true, T, k, at::kFloat, dev, "weight", weight, has) ||
      !out.add_vec(v[8], true, E, at::kInt, dev, "counts", counts) ||
      !out.add_vec(v[9], true, E + 1, at::kInt, dev, "offs", offs) ||
      !out.add_vec(v[10], true, T * k, at::kInt, dev, "order", order) ||
      !out.add(v[11], true, T, k, at::kInt, dev, "slot", slot, has) ||
      !out.add_vec(v[12], true, 1, at::kInt, dev, "tokens", tokens) ||
      !out.add_vec(v[13], true, 1, at::kFloat, dev, "loss", loss) || !dense(idx, T, k, "idx") ||
      !dense(weight, T, k, "weight") || !dense(slot, T, k, "slot"))
    return nullptr;
  void *ws = nullptr;
  int64_t ws_bytes = 0;
  if (v[14] != Py_None) {
    if (!workspace(v[14], dev, ws, ws_bytes)) return nullptr;
  } else {
    ws_bytes = fp8q_route_workspace_bytes(T, E);
    if (ws_bytes > 0) out.scratch(ws_bytes, ws);
  }
  fp8q_status st;
  {
    NoGil free;
    out.make(place);
    st = fp8q_route(l.p, l.ld, kind, valid, score, normalise[0], static_cast<float>(scale),
                    static_cast<int32_t *>(idx.p), static_cast<float *>(weight.p),
                    static_cast<int32_t *>(counts.p), static_cast<int32_t *>(offs.p),
                    static_cast<int32_t *>(order.p), static_cast<int32_t *>(slot.p),
                    static_cast<int32_t *>(tokens.p), static_cast<float *>(loss.p), T, E, k, ws, ws_bytes,
                    place.handle);
  }
  return out.tuple(st);
}

// (logits, idx, counts, tokens, dweight, dloss, score, normalise, scale, valid, dlogits, stream)
PyObject *route_bwd_impl(PyObject *const *v, Py_ssize_t n) {
  if (n != 12) return wrong_count("route_bwd");
  Mat l, midx, mcounts, mtokens, mdw;
  int kind = 0, score = 0;
  const uint8_t *valid;
  int64_t T, E;
  std::optional<at::Device> at_dev;
  if (!router_in(v[0], v[9], l, kind, valid, T, E, at_dev)) return nullptr;
  const at::Device dev = *at_dev;
  const at::Tensor *idx = tensor(v[1], "idx"), *counts = tensor(v[2], "counts"),
                   *tokens = tensor(v[3], "tokens");
  if (!idx || !counts || !tokens) return nullptr;
  if (idx->dim() != 2) {
    fail("idx must be [T][k]");
    return nullptr;
  }
  const int64_t k = idx->size(1);
  const void *dloss;
  bool normalise[1];
  if (!mat(*idx, T, k, at::kInt, dev, "idx", midx) || !dense(midx, T, k, "idx") ||
      !vec(*counts, E, at::kInt, dev, "counts", mcounts.p) ||
      !vec(*tokens, 1, at::kInt, dev, "tokens", mtokens.p) ||
      (v[4] != Py_None && (!mat(v[4], T, k, at::kFloat, dev, "dweight", mdw) || !dense(mdw, T, k, "dweight"))) ||
      !scalar(v[5], at::kFloat, dev, "dloss", dloss) || !int_of(v[6], score) || !flags(v + 7, normalise))
    return nullptr;
  const double scale = PyFloat_AsDouble(v[8]);
  Place place;
  if (PyErr_Occurred() || !place.set(v[11], dev)) return nullptr;
  Results out(true);
  Mat d;
  bool has;
  if (!out.add(v[10], true, T, E, type_of(kind), dev, "dlogits", d, has)) return nullptr;
  fp8q_status st;
  {
    NoGil free;
    out.make(place);
    st = fp8q_route_bwd(l.p, l.ld, kind, valid, score, normalise[0], static_cast<float>(scale),
                        static_cast<const int32_t *>(midx.p), static_cast<const int32_t *>(mcounts.p),
                        static_cast<const int32_t *>(mtokens.p), static_cast<const float *>(mdw.p),
                        static_cast<const float *>(dloss), d.p, d.ld, T, E, k, place.handle);
  }
  return out.tuple(st);
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
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<rmsnorm_impl>)),
     METH_FASTCALL, nullptr},
    {"rmsnorm_bwd",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<rmsnorm_bwd_impl>)),
     METH_FASTCALL, nullptr},
    {"adamw", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<adamw_impl>)),
     METH_FASTCALL, nullptr},
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<route_impl>)),
     METH_FASTCALL, nullptr},
    {"route_bwd",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<route_bwd_impl>)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&module); }
