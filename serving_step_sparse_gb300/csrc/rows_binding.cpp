// Python binding of the operators on rows: argument checks and marshalling, in C++ because a
// decode step makes four of these calls per layer and the same checks in Python cost more
// host time (9-20 us a call) than the kernels take on the device.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <optional>

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
// autograd: a gradient that is expected, or a forward tangent, would be missing without a word.
const at::Tensor &tensor(PyObject *o) {
  need(THPVariable_Check(o), "the arguments are tensors");
  const at::Tensor &t = THPVariable_Unpack(o);
  need(!t.requires_grad() || !at::GradMode::is_enabled(),
       "no gradient is recorded: detach the tensors that require one, or call under torch.no_grad()");
  need(!t._fw_grad(/*level=*/0).defined() || !c10::AutogradState::get_tls_state().get_fw_grad_mode(),
       "no tangent is computed: call on the primals of dual tensors");
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

// What pack and pack_norm share: the arguments' checks and copies, and the rows.
struct Pack {
  at::Tensor latent, rope, rows;
  int type;
  On on;
  int64_t n;
  Positions pos;

  Pack(PyObject *olatent, PyObject *orope, PyObject *opos, const ula_rotary &rotary, PyObject *orows)
      : latent(tensor(olatent)), rope(tensor(orope)), type(type_of(latent)), on((check_latent(latent, type), latent)),
        n(latent.size(0)), pos((check_rope(), on), tensor(opos), rotary, n) {
    rows = given(orows) ? tensor(orows) : on.empty({n, kRow}, at::kByte);
    on.same(rows);
    need(rows.scalar_type() == at::kByte && rows.dim() == 2 && rows.size(0) == n && rows.size(1) == kRow &&
             rows.stride(1) == 1 && (n < 2 || rows.stride(0) >= kRow),
         "rows is uint8 [tokens][656]");
    need(n <= INT32_MAX, "too many tokens");
    if (latent.stride(1) != 1) latent = latent.contiguous();
    if (rope.stride(1) != 1) rope = rope.contiguous();
  }
  static void check_latent(const at::Tensor &t, int type) {
    need(t.dim() == 2 && t.size(1) == kLatent && type >= 0, "latent is [tokens][512] of bf16, f16 or f32");
  }
  void check_rope() const {
    need(rope.scalar_type() == latent.scalar_type() && rope.dim() == 2 && rope.size(0) == n && rope.size(1) == kRope,
         "rope is [tokens][64] of the latent's type");
    on.same(rope);
  }
  int64_t row_step() const { return n > 1 ? rows.stride(0) : kRow; }
};

// pack(latent, rope, pos, rotary, rows or None) -> rows
PyObject *pack(PyObject *const *a) {
  const ula_rotary rotary = rotary_of(a[3]);
  Pack c(a[0], a[1], a[2], rotary, a[4]);
  check(ula_rows_pack(&rotary, c.pos.data, c.pos.stride, c.n, c.type, c.latent.data_ptr(), step_of(c.latent, 0),
                      c.rope.data_ptr(), step_of(c.rope, 0), c.rows.data_ptr(), c.row_step(), c.on.stream()),
        "ula_rows_pack");
  return wrap(a[4], c.rows);
}

// A norm's weight: [n] of the operand's type or float32.
struct Weight {
  at::Tensor held;
  uint32_t type;
  Weight(const On &on, const at::Tensor &t, int64_t n, int operand, const char *why) : held(t) {
    const int own = type_of(t);
    need(t.dim() == 1 && t.size(0) == n && own >= 0 && (own == operand || own == ULA_TYPE_F32), why);
    on.same(t);
    if (t.stride(0) != 1) held = t.contiguous();
    type = own;
  }
};

float eps_of(PyObject *o) {
  const double eps = PyFloat_AsDouble(o);
  if (eps == -1.0 && PyErr_Occurred()) throw python_error();
  need(eps >= 0.0 && eps <= 3.0e38, "eps is finite and not negative");
  return (float)eps;
}

// norm_rotate(x, weight, pos, rotary, eps, at or None, out or None) -> out
PyObject *norm_rotate(PyObject *const *a) {
  at::Tensor x = tensor(a[0]);
  const ula_rotary rotary = rotary_of(a[3]);
  const int type = type_of(x);
  need((x.dim() == 2 || x.dim() == 3) && x.size(-1) >= kRope && x.size(-1) <= (int64_t)ULA_MAX_WIDTH && type >= 0,
       "x is [tokens][heads][64 to 1024] of bf16, f16 or f32");
  const On on(x);
  const bool three = x.dim() == 3;
  const int64_t n = x.size(0), heads = three ? x.size(1) : 1, width = x.size(-1);
  const Weight weight(on, tensor(a[1]), width, type, "weight is [width] of x's type or float32");
  const Positions pos(on, tensor(a[2]), rotary, n);
  const float eps = eps_of(a[4]);
  int64_t at = width - kRope;
  if (given(a[5])) {
    at = PyLong_AsLongLong(a[5]);
    if (at == -1 && PyErr_Occurred()) throw python_error();
  }
  need(at >= 0 && at <= width - kRope, "the rope channels lie within the head: 0 <= at <= width - 64");
  const at::Tensor out = given(a[6]) ? tensor(a[6]) : on.empty(x.sizes(), x.scalar_type());
  on.same(out);
  need(out.sizes() == x.sizes() && out.scalar_type() == x.scalar_type() && out.stride(-1) == 1,
       "out has x's shape and type, and dense channels");
  need(n <= INT32_MAX && heads <= INT32_MAX, "too many tokens or heads");
  if (x.stride(-1) != 1) x = x.contiguous();
  check(ula_rows_norm_rotate(&rotary, pos.data, pos.stride, n, heads, width, at, type, x.data_ptr(), step_of(x, 0),
                             three ? step_of(x, 1) : 0, weight.held.data_ptr(), weight.type, eps, out.data_ptr(),
                             step_of(out, 0), three ? step_of(out, 1) : 0, on.stream()),
        "ula_rows_norm_rotate");
  return wrap(a[6], out);
}

// pack_norm(latent, rope, latent_weight, pos, rotary, eps, rope_weight or None, rows or None) -> rows
PyObject *pack_norm(PyObject *const *a) {
  const ula_rotary rotary = rotary_of(a[4]);
  Pack c(a[0], a[1], a[3], rotary, a[7]);
  const Weight latent_weight(c.on, tensor(a[2]), kLatent, c.type, "latent_weight is [512] of the latent's type or float32");
  const float eps = eps_of(a[5]);
  std::optional<Weight> rope_weight;
  if (given(a[6])) rope_weight.emplace(c.on, tensor(a[6]), kRope, c.type, "rope_weight is [64] of the latent's type or float32");
  check(ula_rows_pack_norm(&rotary, c.pos.data, c.pos.stride, c.n, c.type, c.latent.data_ptr(), step_of(c.latent, 0),
                           c.rope.data_ptr(), step_of(c.rope, 0), latent_weight.held.data_ptr(), latent_weight.type,
                           rope_weight ? rope_weight->held.data_ptr() : nullptr, rope_weight ? rope_weight->type : 0, eps,
                           c.rows.data_ptr(), c.row_step(), c.on.stream()),
        "ula_rows_pack_norm");
  return wrap(a[7], c.rows);
}

// What attend and attend_tree share: the arguments' checks and copies, the outputs and the struct.
struct Attend {
  at::Tensor q, entry, out, lse, space;
  On on;
  ula_attend_args args{};
  int64_t R, Q, H, K;

  // `shared`: entry_row may be [requests][k] as well
  Attend(PyObject *oq, PyObject *orows, PyObject *oentry, PyObject *oscale, PyObject *oown, PyObject *oout, PyObject *olse, bool shared)
      : q(tensor(oq)), entry(tensor(oentry)), on((check_q(q), q)) {
    const at::Tensor &rows = tensor(orows);
    const double scale = PyFloat_AsDouble(oscale);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    R = q.size(0), Q = q.size(1), H = q.size(2);
    need(rows.scalar_type() == at::kByte && rows.dim() == 2 && rows.size(1) == kRow && rows.is_contiguous(),
         "rows is contiguous uint8 [rows][656]");
    on.same(rows);
    need(entry.scalar_type() == at::kInt && (entry.dim() == 3 || (shared && entry.dim() == 2)) && entry.size(0) == R &&
             (entry.dim() == 2 || entry.size(1) == Q),
         shared ? "entry_row is int32 [requests][query tokens][k] or [requests][k]"
                : "entry_row is int32 [requests][query tokens][k]");
    on.same(entry);
    K = entry.size(-1);
    need(R <= INT32_MAX && Q <= INT32_MAX && H <= INT32_MAX && K <= INT32_MAX && rows.size(0) <= INT32_MAX,
         "too many requests, query tokens, heads, entries or rows");
    if (!entry.is_contiguous()) entry = entry.contiguous();
    if (q.stride(3) != 1 || step_of(q, 0) % 8 || step_of(q, 1) % 8 || step_of(q, 2) % 8 ||
        reinterpret_cast<uintptr_t>(q.data_ptr()) % 16)
      q = q.clone(at::MemoryFormat::Contiguous);
    if (given(oown)) {
      const at::Tensor &own = tensor(oown);
      need(own.scalar_type() == at::kByte && own.dim() == 3 && own.size(0) == R && own.size(1) == Q &&
               own.size(2) == kRow && own.stride(2) == 1,
           "own_rows is uint8 [requests][query tokens][656]");
      on.same(own);
      args.own_rows = own.data_ptr();
      args.own_req_stride = step_of(own, 0), args.own_tok_stride = step_of(own, 1);
    }
    out = given(oout) ? tensor(oout) : on.empty({R, Q, H, kLatent}, at::kBFloat16);
    if (given(oout)) {
      on.same(out);
      need(out.scalar_type() == at::kBFloat16 && out.dim() == 4 && out.sizes() == at::IntArrayRef({R, Q, H, kLatent}) &&
               out.is_contiguous(),
           "out is contiguous bf16 [requests][query tokens][heads][512]");
    }
    lse = given(olse) ? tensor(olse) : on.empty({R, Q, H}, at::kFloat);
    if (given(olse)) {
      on.same(lse);
      need(lse.scalar_type() == at::kFloat && lse.dim() == 3 && lse.sizes() == at::IntArrayRef({R, Q, H}) &&
               lse.is_contiguous(),
           "lse is contiguous float32 [requests][query tokens][heads]");
    }
    args.q = q.data_ptr();
    args.q_req_stride = step_of(q, 0), args.q_tok_stride = step_of(q, 1), args.q_head_stride = step_of(q, 2);
    args.rows = rows.data_ptr(), args.n_rows = rows.size(0);
    args.entry_row = entry.data_ptr<int32_t>();
    args.out = out.data_ptr(), args.lse = lse.data_ptr<float>();
    args.n_req = R, args.n_q = Q, args.heads = H, args.k = K, args.softmax_scale = (float)scale;
  }
  void workspace(uint64_t bytes) {
    args.workspace_bytes = bytes;
    if (!bytes) return;
    space = on.empty({(int64_t)bytes}, at::kByte);
    args.workspace = space.data_ptr();
  }
  static void check_q(const at::Tensor &q) {
    need(q.dim() == 4 && q.size(3) == kLatent + kRope && q.scalar_type() == at::kBFloat16,
         "q is bf16 [requests][query tokens][heads][576]");
  }
};

// attend(q, rows, entry_row, scale, own_rows or None, out or None, lse or None) -> (out, lse)
PyObject *attend(PyObject *const *a) {
  Attend c(a[0], a[1], a[2], a[3], a[4], a[5], a[6], false);
  c.workspace(ula_rows_attend_workspace(c.R, c.Q, c.H, c.K, c.args.own_rows != nullptr));
  check(ula_rows_attend(&c.args, c.on.stream()), "ula_rows_attend");
  return wrap2(a[5], c.out, a[6], c.lse);
}

// attend_tree(q, rows, entry_row, scale, own_rows, parent, out or None, lse or None) -> (out, lse)
PyObject *attend_tree(PyObject *const *a) {
  need(given(a[4]), "a tree's nodes have rows of their own");
  Attend c(a[0], a[1], a[2], a[3], a[4], a[6], a[7], true);
  at::Tensor parent = tensor(a[5]);
  need(parent.scalar_type() == at::kInt && parent.dim() == 2 && parent.size(0) == c.R && parent.size(1) == c.Q,
       "parent is int32 [requests][nodes]");
  need(c.Q <= (int64_t)ULA_MAX_TREE, "a tree has at most 64 nodes");
  c.on.same(parent);
  if (!parent.is_contiguous()) parent = parent.contiguous();
  const uint32_t flags = c.entry.dim() == 2 ? ULA_TREE_SHARED_LIST : 0;
  c.workspace(ula_rows_attend_tree_workspace(c.R, c.Q, c.H, c.K, flags));
  check(ula_rows_attend_tree(&c.args, parent.data_ptr<int32_t>(), flags, c.on.stream()), "ula_rows_attend_tree");
  return wrap2(a[6], c.out, a[7], c.lse);
}

// score(scores, q, rows, entry_row, address, lse, scale) -> scores
PyObject *score(PyObject *const *a) {
  const at::Tensor &scores = tensor(a[0]), &rows = tensor(a[2]);
  at::Tensor q = tensor(a[1]), entry = tensor(a[3]), address = tensor(a[4]), lse = tensor(a[5]);
  const double scale = PyFloat_AsDouble(a[6]);
  if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  Attend::check_q(q);
  const On on(q);
  const int64_t R = q.size(0), Q = q.size(1), H = q.size(2);
  need(scores.scalar_type() == at::kFloat && scores.dim() == 1 && scores.is_contiguous(), "scores is contiguous float32 [addresses]");
  need(rows.scalar_type() == at::kByte && rows.dim() == 2 && rows.size(1) == kRow && rows.is_contiguous(),
       "rows is contiguous uint8 [rows][656]");
  need(entry.scalar_type() == at::kInt && (entry.dim() == 2 || (entry.dim() == 3 && entry.size(1) == Q)) && entry.size(0) == R,
       "entry_row is int32 [requests][query tokens][k] or [requests][k]");
  need(address.scalar_type() == at::kInt && address.sizes() == entry.sizes(), "address is int32 of entry_row's shape");
  need(lse.scalar_type() == at::kFloat && lse.dim() == 3 && lse.sizes() == at::IntArrayRef({R, Q, H}),
       "lse is float32 [requests][query tokens][heads]");
  on.same(scores);
  on.same(rows);
  on.same(entry);
  on.same(address);
  on.same(lse);
  const int64_t K = entry.size(-1);
  need(R <= INT32_MAX && Q <= INT32_MAX && H <= INT32_MAX && K <= INT32_MAX && rows.size(0) <= INT32_MAX && scores.size(0) <= INT32_MAX,
       "too many requests, query tokens, heads, entries, rows or addresses");
  if (!entry.is_contiguous()) entry = entry.contiguous();
  if (!address.is_contiguous()) address = address.contiguous();
  if (!lse.is_contiguous()) lse = lse.contiguous();
  if (q.stride(3) != 1 || step_of(q, 0) % 8 || step_of(q, 1) % 8 || step_of(q, 2) % 8 ||
      reinterpret_cast<uintptr_t>(q.data_ptr()) % 16)
    q = q.clone(at::MemoryFormat::Contiguous);
  ula_score_args args{};
  args.flags = entry.dim() == 2 ? ULA_TREE_SHARED_LIST : 0;
  args.workspace_bytes = ula_rows_score_workspace(R, Q, H, args.flags, scores.size(0));
  const at::Tensor space = on.empty({(int64_t)args.workspace_bytes}, at::kByte);
  args.workspace = space.data_ptr();
  args.q = q.data_ptr();
  args.q_req_stride = step_of(q, 0), args.q_tok_stride = step_of(q, 1), args.q_head_stride = step_of(q, 2);
  args.rows = rows.data_ptr(), args.n_rows = rows.size(0);
  args.entry_row = entry.data_ptr<int32_t>(), args.address = address.data_ptr<int32_t>();
  args.lse = lse.data_ptr<float>();
  args.scores = scores.data_ptr<float>(), args.n_scores = scores.size(0);
  args.n_req = R, args.n_q = Q, args.heads = H, args.k = K, args.softmax_scale = (float)scale;
  check(ula_rows_score(&args, on.stream()), "ula_rows_score");
  return wrap(a[0], scores);
}

int64_t count_of(PyObject *o, const char *why) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  need(v >= 0 && v <= INT32_MAX, why);
  return v;
}

// evict(scores, address, length, budget, first, last, kept or None, dropped or None) -> (kept, dropped)
PyObject *evict(PyObject *const *a) {
  at::Tensor scores = tensor(a[0]), address = tensor(a[1]), length = tensor(a[2]);
  need(scores.scalar_type() == at::kFloat && scores.dim() == 1, "scores is float32 [addresses]");
  const On on(scores);
  need(address.scalar_type() == at::kInt && address.dim() == 2, "address is int32 [requests][longest]");
  const int64_t R = address.size(0), N = address.size(1);
  need(length.scalar_type() == at::kInt && length.dim() == 1 && length.size(0) == R, "length is int32 [requests]");
  on.same(address);
  on.same(length);
  need(R <= INT32_MAX && N <= INT32_MAX && scores.size(0) <= INT32_MAX, "too many requests or addresses");
  const int64_t budget = count_of(a[3], "budget is not negative"), first = count_of(a[4], "first is not negative"),
                last = count_of(a[5], "last is not negative"), room = N > budget ? N - budget : 0;
  need(first + last <= budget, "what stays in any case (first + last) is within the budget");
  if (!scores.is_contiguous()) scores = scores.contiguous();
  if (!address.is_contiguous()) address = address.contiguous();
  if (!length.is_contiguous()) length = length.contiguous();
  const at::Tensor kept = given(a[6]) ? tensor(a[6]) : on.empty({R, budget}, at::kInt);
  const at::Tensor dropped = given(a[7]) ? tensor(a[7]) : on.empty({R, room}, at::kInt);
  on.same(kept);
  on.same(dropped);
  need(kept.scalar_type() == at::kInt && kept.dim() == 2 && kept.size(0) == R && kept.size(1) == budget && kept.is_contiguous(),
       "kept is contiguous int32 [requests][budget]");
  need(dropped.scalar_type() == at::kInt && dropped.dim() == 2 && dropped.size(0) == R && dropped.size(1) == room && dropped.is_contiguous(),
       "dropped is contiguous int32 [requests][longest - budget]");
  check(ula_rows_evict(scores.data_ptr<float>(), scores.size(0), address.data_ptr<int32_t>(), length.data_ptr<int32_t>(),
                       R, N, budget, first, last, kept.data_ptr<int32_t>(), dropped.data_ptr<int32_t>(), on.stream()),
        "ula_rows_evict");
  return wrap2(a[6], kept, a[7], dropped);
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
                         method<attend_tree, 8>("attend_tree"), method<norm_rotate, 7>("norm_rotate"),
                         method<pack_norm, 8>("pack_norm"), method<score, 7>("score"), method<evict, 8>("evict"),
                         method<join, 4>("join"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rows", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rows() { return PyModule_Create(&module); }
