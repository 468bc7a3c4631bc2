// Python binding of the operators on rows: argument checks and marshalling, in C++ because a
// decode step makes four of these calls per layer and the same checks in Python cost more
// host time (9-20 us a call) than the kernels take on the device.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "ula.h"

namespace {

constexpr int64_t kLatent = ULA_ROW_LATENT, kRope = ULA_ROW_ROPE, kRow = ULA_ROW_BYTES;

struct Refused {  // becomes a ValueError
  const char *why;
};
struct Failed {  // an error of the C ABI: becomes an UlaError
  int code;
  const char *what;
};

void need(bool ok, const char *why) {
  if (!ok) throw Refused{why};
}
void check(int code, const char *what) {
  if (code != ULA_OK) throw Failed{code, what};
}

// What the objects hold (references, borrowed for the call).  The operators record nothing for
// autograd: a gradient that is expected would be missing without a word.
const at::Tensor &tensor(PyObject *o) {
  need(THPVariable_Check(o), "the arguments are tensors");
  const at::Tensor &t = THPVariable_Unpack(o);
  need(!t.requires_grad() || !at::GradMode::is_enabled(),
       "no gradient is recorded: detach the tensors that require one, or call under torch.no_grad()");
  return t;
}
bool given(PyObject *o) { return o != Py_None; }

// The ula_rotary that an object (the ctypes struct) holds, read through its buffer: no address is
// kept in Python, where a copied or unpickled rotary would bring another object's.
ula_rotary rotary_of(PyObject *o) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw python_error();
  ula_rotary r;
  const bool whole = b.len == (Py_ssize_t)sizeof r;
  if (whole) memcpy(&r, b.buf, sizeof r);
  PyBuffer_Release(&b);
  need(whole, "the rotary is a ula_rotary");
  return r;
}

// What one step along a dimension adds; a dimension of one element has no steps, whatever its stride.
int64_t step_of(const at::Tensor &t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }

int type_of(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return ULA_TYPE_BF16;
    case at::kHalf: return ULA_TYPE_F16;
    case at::kFloat: return ULA_TYPE_F32;
    default: return -1;
  }
}

// The current stream of the tensors' device, which has to be the current device.
class On {
 public:
  explicit On(const at::Tensor &t) : device_(t.device()) {
    need(device_.is_cuda() && device_.index() == c10::cuda::current_device(),
         "the tensors must be on the current CUDA device");
  }
  void same(const at::Tensor &t) const { need(t.device() == device_, "the tensors must be on one device"); }
  at::Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::detail::empty_cuda(size, type, device_, std::nullopt);
  }
  void *stream() const { return c10::cuda::getCurrentCUDAStream(device_.index()).stream(); }

 private:
  c10::Device device_;
};

struct Positions {
  at::Tensor held;
  const int32_t *data;
  uint64_t stride;
  Positions(const On &on, const at::Tensor &t, const ula_rotary &rotary, int64_t n) : held(t) {
    need(t.scalar_type() == at::kInt, "positions are int32");
    on.same(t);
    const bool one = t.dim() == 1;
    need((one || t.dim() == 2) && (one ? 1 : t.size(0)) >= rotary.n_axes && t.size(-1) == n,
         "positions are [axes][tokens]");
    if (n > 1 && t.stride(-1) != 1) held = t.contiguous();
    data = held.data_ptr<int32_t>();
    stride = one ? 0 : held.stride(0);
  }
};

// The result: a new tensor, or the caller's, whose version then says that it was written.
PyObject *wrap(PyObject *as_given, const at::Tensor &t) {
  if (!given(as_given)) return THPVariable_Wrap(t);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  Py_INCREF(as_given);
  return as_given;
}

PyObject *wrap2(PyObject *oa, const at::Tensor &a, PyObject *ob, const at::Tensor &b) {
  PyObject *x = wrap(oa, a), *y = x ? wrap(ob, b) : nullptr, *both = y ? PyTuple_New(2) : nullptr;
  if (!both) {
    Py_XDECREF(x);
    Py_XDECREF(y);
    return nullptr;
  }
  PyTuple_SET_ITEM(both, 0, x);
  PyTuple_SET_ITEM(both, 1, y);
  return both;
}

// rotate(x, pos, rotary, out or None, inverse) -> out
PyObject *rotate(PyObject *const *a) {
  at::Tensor x = tensor(a[0]);
  const ula_rotary rotary = rotary_of(a[2]);
  const int type = type_of(x);
  need((x.dim() == 2 || x.dim() == 3) && x.size(-1) == kRope && type >= 0,
       "x is [tokens][heads][64] of bf16, f16 or f32");
  const On on(x);
  const bool three = x.dim() == 3;
  const int64_t n = x.size(0), heads = three ? x.size(1) : 1;
  const Positions pos(on, tensor(a[1]), rotary, n);
  const at::Tensor out = given(a[3]) ? tensor(a[3]) : on.empty(x.sizes(), x.scalar_type());
  on.same(out);
  need(out.sizes() == x.sizes() && out.scalar_type() == x.scalar_type() && out.stride(-1) == 1,
       "out has x's shape and type, and dense channels");
  need(n <= INT32_MAX && heads <= INT32_MAX, "too many tokens or heads");
  if (x.stride(-1) != 1) x = x.contiguous();
  check(ula_rows_rotate(&rotary, a[4] == Py_True ? ULA_ROTATE_INVERSE : 0, pos.data, pos.stride, n, heads, type,
                        x.data_ptr(), step_of(x, 0), three ? step_of(x, 1) : 0, out.data_ptr(), step_of(out, 0),
                        three ? step_of(out, 1) : 0, on.stream()),
        "ula_rows_rotate");
  return wrap(a[3], out);
}

// pack(latent, rope, pos, rotary, rows or None) -> rows
PyObject *pack(PyObject *const *a) {
  at::Tensor latent = tensor(a[0]), rope = tensor(a[1]);
  const ula_rotary rotary = rotary_of(a[3]);
  const int type = type_of(latent);
  need(latent.dim() == 2 && latent.size(1) == kLatent && type >= 0, "latent is [tokens][512] of bf16, f16 or f32");
  const On on(latent);
  const int64_t n = latent.size(0);
  need(rope.scalar_type() == latent.scalar_type() && rope.dim() == 2 && rope.size(0) == n && rope.size(1) == kRope,
       "rope is [tokens][64] of the latent's type");
  on.same(rope);
  const Positions pos(on, tensor(a[2]), rotary, n);
  const at::Tensor rows = given(a[4]) ? tensor(a[4]) : on.empty({n, kRow}, at::kByte);
  on.same(rows);
  need(rows.scalar_type() == at::kByte && rows.dim() == 2 && rows.size(0) == n && rows.size(1) == kRow &&
           rows.stride(1) == 1 && (n < 2 || rows.stride(0) >= kRow),
       "rows is uint8 [tokens][656]");
  need(n <= INT32_MAX, "too many tokens");
  if (latent.stride(1) != 1) latent = latent.contiguous();
  if (rope.stride(1) != 1) rope = rope.contiguous();
  check(ula_rows_pack(&rotary, pos.data, pos.stride, n, type, latent.data_ptr(), step_of(latent, 0), rope.data_ptr(),
                      step_of(rope, 0), rows.data_ptr(), n > 1 ? rows.stride(0) : kRow, on.stream()),
        "ula_rows_pack");
  return wrap(a[4], rows);
}

// attend(q, rows, entry_row, scale, own_rows or None, out or None, lse or None) -> (out, lse)
PyObject *attend(PyObject *const *a) {
  at::Tensor q = tensor(a[0]), entry = tensor(a[2]);
  const at::Tensor &rows = tensor(a[1]);
  const double scale = PyFloat_AsDouble(a[3]);
  if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  need(q.dim() == 4 && q.size(3) == kLatent + kRope && q.scalar_type() == at::kBFloat16,
       "q is bf16 [requests][query tokens][heads][576]");
  const On on(q);
  const int64_t R = q.size(0), Q = q.size(1), H = q.size(2);
  need(rows.scalar_type() == at::kByte && rows.dim() == 2 && rows.size(1) == kRow && rows.is_contiguous(),
       "rows is contiguous uint8 [rows][656]");
  on.same(rows);
  need(entry.scalar_type() == at::kInt && entry.dim() == 3 && entry.size(0) == R && entry.size(1) == Q,
       "entry_row is int32 [requests][query tokens][k]");
  on.same(entry);
  const int64_t K = entry.size(2);
  need(R <= INT32_MAX && Q <= INT32_MAX && H <= INT32_MAX && K <= INT32_MAX && rows.size(0) <= INT32_MAX,
       "too many requests, query tokens, heads, entries or rows");
  if (!entry.is_contiguous()) entry = entry.contiguous();
  if (q.stride(3) != 1 || step_of(q, 0) % 8 || step_of(q, 1) % 8 || step_of(q, 2) % 8 ||
      reinterpret_cast<uintptr_t>(q.data_ptr()) % 16)
    q = q.clone(at::MemoryFormat::Contiguous);
  ula_attend_args args{};
  if (given(a[4])) {
    const at::Tensor &own = tensor(a[4]);
    need(own.scalar_type() == at::kByte && own.dim() == 3 && own.size(0) == R && own.size(1) == Q &&
             own.size(2) == kRow && own.stride(2) == 1,
         "own_rows is uint8 [requests][query tokens][656]");
    on.same(own);
    args.own_rows = own.data_ptr();
    args.own_req_stride = step_of(own, 0), args.own_tok_stride = step_of(own, 1);
  }
  const at::Tensor out = given(a[5]) ? tensor(a[5]) : on.empty({R, Q, H, kLatent}, at::kBFloat16);
  if (given(a[5])) {
    on.same(out);
    need(out.scalar_type() == at::kBFloat16 && out.dim() == 4 && out.sizes() == at::IntArrayRef({R, Q, H, kLatent}) &&
             out.is_contiguous(),
         "out is contiguous bf16 [requests][query tokens][heads][512]");
  }
  const at::Tensor lse = given(a[6]) ? tensor(a[6]) : on.empty({R, Q, H}, at::kFloat);
  if (given(a[6])) {
    on.same(lse);
    need(lse.scalar_type() == at::kFloat && lse.dim() == 3 && lse.sizes() == at::IntArrayRef({R, Q, H}) &&
             lse.is_contiguous(),
         "lse is contiguous float32 [requests][query tokens][heads]");
  }
  at::Tensor space;
  args.workspace_bytes = ula_rows_attend_workspace(R, Q, H, K, args.own_rows != nullptr);
  if (args.workspace_bytes) {
    space = on.empty({(int64_t)args.workspace_bytes}, at::kByte);
    args.workspace = space.data_ptr();
  }
  args.q = q.data_ptr();
  args.q_req_stride = step_of(q, 0), args.q_tok_stride = step_of(q, 1), args.q_head_stride = step_of(q, 2);
  args.rows = rows.data_ptr(), args.n_rows = rows.size(0);
  args.entry_row = entry.data_ptr<int32_t>();
  args.out = out.data_ptr(), args.lse = lse.data_ptr<float>();
  args.n_req = R, args.n_q = Q, args.heads = H, args.k = K, args.softmax_scale = (float)scale;
  check(ula_rows_attend(&args, on.stream()), "ula_rows_attend");
  return wrap2(a[5], out, a[6], lse);
}

// join(outs, lses, out or None, lse or None) -> (out, lse)
PyObject *join(PyObject *const *a) {
  need((PyList_Check(a[0]) || PyTuple_Check(a[0])) && (PyList_Check(a[1]) || PyTuple_Check(a[1])),
       "the parts' outs and lses are lists");
  const Py_ssize_t parts = PySequence_Fast_GET_SIZE(a[0]);
  need(parts >= 1 && parts <= (Py_ssize_t)ULA_MAX_PARTS && parts == PySequence_Fast_GET_SIZE(a[1]),
       "1 to 8 parts, an out and an lse of each");
  const void *outs[ULA_MAX_PARTS];
  const float *lses[ULA_MAX_PARTS];
  const at::Tensor &first = tensor(PySequence_Fast_GET_ITEM(a[0], 0));
  need(first.dim() >= 1 && first.size(-1) == kLatent, "a part's out is [...][512]");
  const On on(first);
  const at::IntArrayRef shape = first.sizes(), heads = shape.slice(0, shape.size() - 1);
  for (Py_ssize_t i = 0; i < parts; ++i) {
    const at::Tensor &o = tensor(PySequence_Fast_GET_ITEM(a[0], i)), &z = tensor(PySequence_Fast_GET_ITEM(a[1], i));
    need(o.scalar_type() == at::kBFloat16 && o.sizes() == shape && o.is_contiguous(),
         "a part's out is contiguous bf16 [...][512], all of one shape");
    need(z.scalar_type() == at::kFloat && z.sizes() == heads && z.is_contiguous(),
         "a part's lse is contiguous float32 of its out's shape without the channels");
    on.same(o);
    on.same(z);
    outs[i] = o.data_ptr();
    lses[i] = z.data_ptr<float>();
  }
  const at::Tensor out = given(a[2]) ? tensor(a[2]) : on.empty(shape, at::kBFloat16);
  const at::Tensor lse = given(a[3]) ? tensor(a[3]) : on.empty(heads, at::kFloat);
  on.same(out);
  on.same(lse);
  need(out.scalar_type() == at::kBFloat16 && out.sizes() == shape && out.is_contiguous(),
       "out is contiguous bf16 of the parts' shape");
  need(lse.scalar_type() == at::kFloat && lse.sizes() == heads && lse.is_contiguous(),
       "lse is contiguous float32 of the parts' shape without the channels");
  check(ula_rows_join(outs, lses, parts, lse.numel(), out.data_ptr(), lse.data_ptr<float>(), on.stream()),
        "ula_rows_join");
  return wrap2(a[2], out, a[3], lse);
}

void raise_failed(const Failed &f) {
  PyObject *module = PyImport_ImportModule("serving_step_sparse_gb300.ula");
  PyObject *type = module ? PyObject_GetAttrString(module, "UlaError") : nullptr;
  PyObject *error = type ? PyObject_CallFunction(type, "is", f.code, f.what) : nullptr;
  if (error) PyErr_SetObject(type, error);
  Py_XDECREF(error);
  Py_XDECREF(type);
  Py_XDECREF(module);
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t kArgs>
PyObject *entry_point(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused &r) {
    PyErr_SetString(PyExc_ValueError, r.why);
  } catch (const Failed &f) {
    raise_failed(f);
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t kArgs>
PyMethodDef method(const char *name) {
  return {name, (PyCFunction)(void (*)())entry_point<F, kArgs>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rotate, 5>("rotate"), method<pack, 5>("pack"), method<attend, 7>("attend"),
                         method<join, 4>("join"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rows", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rows() { return PyModule_Create(&module); }
