// The per-layer calls as Python sees them: checks of torch tensors, the argument
// structs of the C ABI, and the call.  They run once per layer and step, so
// their host time is a small call's time; in Python the same checks cost 6 to
// 12 us a call.  No step of the computation is here.
#include <Python.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/empty.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>
#include <type_traits>

#include "spec_verify.h"

namespace {

struct Api {
  decltype(&sv_tree_mask) tree_mask;
  decltype(&kv_append) append;
  decltype(&kv_read) read;
  decltype(&sv_attention_workspace_size) attention_size;
  decltype(&sv_tree_attention) attention;
  decltype(&sv_adjust_logits) logits;
  decltype(&sv_prefix_groups) prefix_groups;
} api;
PyObject* g_error = nullptr;  // SvError(function, code)

constexpr int kTail = 16;

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused();
}

void done(const char* fn, sv_status code) {
  if (code == SV_OK) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "si", fn, (int)code)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused();
}

// An argument: a tensor, or nothing.
struct Arg {
  const at::Tensor* t = nullptr;
  Arg(PyObject* o, const char* name) {
    if (o == Py_None) return;
    if (!THPVariable_Check(o)) refuse(std::string(name) + ": tensor expected");
    t = &THPVariable_Unpack(o);
  }
  explicit operator bool() const { return t != nullptr; }
  const at::Tensor* operator->() const { return t; }
};

Arg need(PyObject* o, const char* name) {
  Arg a(o, name);
  if (!a) refuse(std::string(name) + ": tensor expected");
  return a;
}

template <class T = void>
T* ptr(const at::Tensor& t) {
  if (!t.is_cuda()) refuse("device tensor expected");
  return static_cast<T*>(t.data_ptr());
}

// Whether a tensor holds what a call reads: fp32, int32, or words of bits.
template <class T>
bool holds(const at::Tensor& t) {
  if (std::is_same_v<std::remove_const_t<T>, float>) return t.scalar_type() == at::kFloat;
  return t.scalar_type() == at::kInt || (std::is_same_v<std::remove_const_t<T>, uint32_t> && t.scalar_type() == at::kUInt32);
}
template <class T>
std::string type_name() {
  return std::is_same_v<std::remove_const_t<T>, float> ? "fp32" : std::is_same_v<std::remove_const_t<T>, uint32_t> ? "int32 or uint32" : "int32";
}

// An optional contiguous array of at least n values.
template <class T>
T* vec(PyObject* o, int64_t n, const char* name) {
  Arg t(o, name);
  if (!t) return nullptr;
  if (!holds<T>(*t.t) || !t->is_contiguous() || t->numel() < n)
    refuse(std::string(name) + ": a contiguous " + type_name<T>() + " tensor of at least " + std::to_string(n) + " values expected");
  return ptr<T>(*t.t);
}

// An optional contiguous [rows][cols] array: one row of another width would shift
// all that follow.
template <class T>
T* grid(PyObject* o, int64_t rows, int64_t cols, const char* name) {
  Arg t(o, name);
  if (!t) return nullptr;
  if (!holds<T>(*t.t) || !t->is_contiguous() || t->numel() != rows * cols || (t->dim() > 1 && t->size(-1) != cols))
    refuse(std::string(name) + ": a contiguous " + type_name<T>() + " [" + std::to_string(rows) + "][" + std::to_string(cols) + "] tensor expected");
  return ptr<T>(*t.t);
}

// An optional contiguous [rows][ld] (or [..][ld]) table.
template <class T>
T* table(PyObject* o, int64_t rows, int64_t* ld, const char* name) {
  Arg t(o, name);
  *ld = 0;
  if (!t) return nullptr;
  if (!holds<T>(*t.t) || !t->is_contiguous() || t->dim() < 2 || t->numel() != rows * t->size(-1))
    refuse(std::string(name) + ": a contiguous " + type_name<T>() + " [" + std::to_string(rows) + "][..] tensor expected");
  *ld = t->size(-1);
  return ptr<T>(*t.t);
}

int dtype_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return SV_BF16;
  if (t.scalar_type() != at::kFloat) refuse(std::string(name) + ": bf16 or fp32 expected");
  return SV_FP32;
}

int format_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return SV_KV_BF16;
    case at::kFloat: return SV_KV_FP32;
    case at::kByte: return SV_KV_E4M3;
    default: refuse(std::string(name) + ": bf16, fp32 or uint8 (8-bit entries) expected");
  }
}

void paged(sv_kv_place* p, PyObject* okv, PyObject* otable, int layer, int64_t B) {
  Arg kv = need(okv, "kv"), t = need(otable, "block_table");
  if (kv->dim() != 6 || kv->size(2) != 2 || !kv->is_contiguous())
    refuse("kv must be a contiguous [num_blocks, layers, 2, heads, BS, row] tensor");
  if (t->dim() != 2 || t->size(0) != B || t->scalar_type() != at::kInt || !t->is_contiguous())
    refuse("block_table must be a contiguous int32 [B][max_blocks]");
  p->format = format_of(*kv.t, "kv");
  p->data = ptr(*kv.t), p->block_table = ptr<int32_t>(*t.t);
  p->layers = (int)kv->size(1), p->heads = (int)kv->size(3);
  p->head_dim = (int)kv->size(5) - (p->format == SV_KV_E4M3 ? kTail : 0);
  p->layer = layer, p->num_blocks = (int)kv->size(0), p->block_size = (int)kv->size(4);
  p->max_blocks = (int)t->size(1);
}

void staged(sv_kv_place* p, PyObject* o, int layer, int64_t B) {
  Arg s = need(o, "stage");
  if (s->dim() != 6 || s->size(3) != 2 || s->size(0) != B || !s->is_contiguous())
    refuse("stage must be a contiguous [B, R, layers, 2, heads, row] tensor");
  p->format = format_of(*s.t, "stage");
  p->data = ptr(*s.t);
  p->layers = (int)s->size(2), p->heads = (int)s->size(4);
  p->head_dim = (int)s->size(5) - (p->format == SV_KV_E4M3 ? kTail : 0);
  p->layer = layer, p->rows = (int)s->size(1);
}

void place(sv_kv_place* p, PyObject* kv, PyObject* otable, PyObject* stage, int layer, int64_t B) {
  if ((kv == Py_None) == (stage == Py_None) || (kv == Py_None) != (otable == Py_None))
    refuse("give either kv with block_table, or stage");
  if (kv == Py_None)
    staged(p, stage, layer, B);
  else
    paged(p, kv, otable, layer, B);
}

// [B, R, H, D] with a contiguous last dimension: pointer and strides.
template <class T>
T* heads(const at::Tensor& t, int64_t B, int64_t R, int64_t H, int64_t D, int64_t (&st)[3], const char* name) {
  if (t.dim() != 4 || t.size(0) != B || t.size(1) != R || t.size(2) != H || t.size(3) != D || t.stride(3) != 1)
    refuse(std::string(name) + ": expected [" + std::to_string(B) + ", " + std::to_string(R) + ", " + std::to_string(H) +
           ", " + std::to_string(D) + "] with a contiguous last dimension");
  st[0] = t.stride(0), st[1] = t.stride(1), st[2] = t.stride(2);
  return ptr<T>(t);
}

sv_handle* handle_of(PyObject* o) {
  return o == Py_None ? nullptr : static_cast<sv_handle*>(PyLong_AsVoidPtr(o));
}
sv_stream_t stream_of(PyObject* o) { return static_cast<sv_stream_t>(PyLong_AsVoidPtr(o)); }
int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  if (v != (int)v) refuse("integer out of range");
  return (int)v;
}

PyObject* none() { Py_RETURN_NONE; }

// A reference that the call owns: what the caller gave, or a new output.
class Owned {
 public:
  explicit Owned(PyObject* given) : o_(given) { Py_INCREF(o_); }
  ~Owned() { Py_XDECREF(o_); }
  Owned(const Owned&) = delete;
  Owned& operator=(const Owned&) = delete;
  void allocate(const at::Tensor& like) {
    PyObject* made = THPVariable_Wrap(at::empty(like.sizes(), like.options()));
    Py_DECREF(o_);
    o_ = made;
  }
  PyObject* get() const { return o_; }
  PyObject* release() {
    PyObject* o = o_;
    o_ = nullptr;
    return o;
  }

 private:
  PyObject* o_;
};

// (handle, parent, n_nodes, mask, depth, stream) -> (mask, depth)
PyObject* tree_mask(PyObject* const* a) {
  Arg parent = need(a[1], "parent");
  if (parent->dim() != 2 || parent->scalar_type() != at::kInt || !parent->is_contiguous())
    refuse("parent must be a contiguous int32 [B][N]");
  const int64_t B = parent->size(0), N = parent->size(1), W = (N + 32) / 32, n = B * (N + 1);
  if ((a[3] == Py_None) != (a[4] == Py_None)) refuse("mask and depth: give both or neither");
  at::Tensor mask, depth;
  int64_t ld = W;
  if (a[3] == Py_None) {
    at::AutoDispatchBelowADInplaceOrView plain;  // no gradients are kept here
    const at::Tensor both = at::empty({n * (W + 1)}, parent->options());  // one allocation
    mask = both.as_strided({B, N + 1, W}, {(N + 1) * W, W, 1}, 0);
    depth = both.as_strided({B, N + 1}, {N + 1, 1}, n * W);
  } else {
    table<uint32_t>(a[3], n, &ld, "mask");
    grid<int32_t>(a[4], B, N + 1, "depth");
    mask = THPVariable_Unpack(a[3]), depth = THPVariable_Unpack(a[4]);
  }
  done("sv_tree_mask", api.tree_mask(handle_of(a[0]), (int)B, (int)N, ptr<int32_t>(*parent.t), vec<int32_t>(a[2], B, "n_nodes"),
                                     ptr<uint32_t>(mask), ld, ptr<int32_t>(depth), stream_of(a[5])));
  if (a[3] != Py_None) return PyTuple_Pack(2, a[3], a[4]);
  PyObject *m = THPVariable_Wrap(mask), *d = THPVariable_Wrap(depth), *r = PyTuple_Pack(2, m, d);
  Py_DECREF(m), Py_DECREF(d);
  return r;
}

// (handle, k, v, seq_len, kv, block_table, stage, layer, q, q_out, rope, pairs, depth, n_nodes, stream) -> q_out
PyObject* append(PyObject* const* a) {
  Arg k = need(a[1], "k"), v = need(a[2], "v"), q(a[8], "q"), rope(a[10], "rope");
  if (k->dim() != 4) refuse("k: expected [B, R, heads, head_dim]");
  const int64_t B = k->size(0), R = k->size(1), H = k->size(2), D = k->size(3);
  sv_append_args p = {};
  place(&p.dst, a[4], a[5], a[6], integer(a[7]), B);
  p.B = (int)B, p.R = (int)R, p.dtype = dtype_of(*k.t, "k");
  if (H != p.dst.heads || D != p.dst.head_dim || v->scalar_type() != k->scalar_type())
    refuse("k and v do not match the cache");
  p.k = heads<const void>(*k.t, B, R, H, D, p.k_stride, "k");
  p.v = heads<const void>(*v.t, B, R, H, D, p.v_stride, "v");
  Owned out(a[9]);
  if (q) {
    if (out.get() == Py_None) out.allocate(*q.t);
    Arg o = need(out.get(), "q_out");
    if (q->scalar_type() != k->scalar_type() || o->scalar_type() != k->scalar_type() || q->dim() != 4)
      refuse("q and q_out need k's dtype");
    p.Hq = (int)q->size(2);
    p.q = heads<const void>(*q.t, B, R, p.Hq, D, p.q_stride, "q");
    p.q_out = heads<void>(*o.t, B, R, p.Hq, D, p.q_out_stride, "q_out");
  }
  if (rope) {
    if (rope->dim() != 3 || rope->size(2) != 2 || rope->scalar_type() != at::kFloat || !rope->is_contiguous())
      refuse("rope must be a contiguous fp32 [max_pos, rot_dim / 2, 2] tensor");
    p.rope = ptr<float>(*rope.t), p.max_pos = (int)rope->size(0), p.rot_dim = 2 * (int)rope->size(1);
  }
  if (PyObject_IsTrue(a[11])) p.flags = SV_APPEND_PAIRS;
  p.depth = grid<int32_t>(a[12], B, R, "depth");
  p.seq_len = vec<int32_t>(a[3], B, "seq_len");
  p.n_nodes = vec<int32_t>(a[13], B, "n_nodes");
  done("kv_append", api.append(handle_of(a[0]), &p, stream_of(a[14])));
  return out.release();
}

// (handle, out, seq_len, kv, block_table, stage, layer, n_nodes, stream)
PyObject* read(PyObject* const* a) {
  Arg out = need(a[1], "out");
  if (out->dim() != 5) refuse("out must be a contiguous bf16 or fp32 [B, R, 2, heads, head_dim] tensor");
  const int64_t B = out->size(0), R = out->size(1);
  sv_kv_place p = {};
  place(&p, a[3], a[4], a[5], integer(a[6]), B);
  if (out->size(2) != 2 || out->size(3) != p.heads || out->size(4) != p.head_dim || !out->is_contiguous())
    refuse("out must be a contiguous bf16 or fp32 [B, R, 2, heads, head_dim] tensor");
  done("kv_read", api.read(handle_of(a[0]), (int)B, (int)R, vec<int32_t>(a[2], B, "seq_len"), vec<int32_t>(a[7], B, "n_nodes"),
                           &p, ptr(*out.t), dtype_of(*out.t, "out"), stream_of(a[8])));
  return none();
}

// q, kv, block_table, seq_len, out, stage, mask, n_nodes, scale, layer at a[0..9]
void fill(sv_attention_args* p, PyObject* const* a, const at::Tensor& out) {
  Arg q = need(a[0], "q"), mask(a[6], "mask");
  if (q->dim() != 4) refuse("q: expected [B, R, Hq, head_dim]");
  const int64_t B = q->size(0), R = q->size(1), Hq = q->size(2), D = q->size(3);
  const int layer = integer(a[9]);
  paged(&p->cache, a[1], a[2], layer, B);
  if (D != p->cache.head_dim || out.scalar_type() != q->scalar_type()) refuse("q and out do not match the cache");
  if (a[5] != Py_None) staged(&p->stage, a[5], layer, B);
  p->B = (int)B, p->R = (int)R, p->Hq = (int)Hq, p->dtype = dtype_of(*q.t, "q");
  p->q = heads<const void>(*q.t, B, R, Hq, D, p->q_stride, "q");
  p->out = heads<void>(out, B, R, Hq, D, p->out_stride, "out");
  p->mask = table<const uint32_t>(a[6], B * R, &p->mask_ld, "mask");
  p->seq_len = vec<int32_t>(a[3], B, "seq_len");
  p->n_nodes = vec<int32_t>(a[7], B, "n_nodes");
  const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AsDouble(a[8]);
  if (scale == -1.0 && PyErr_Occurred()) throw Refused();
  p->scale = (float)scale;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}

// softcap, slopes, window, depth, shared_len, shared_members at a[0..5], after fill
void fill_forms(sv_attention_args* p, PyObject* const* a) {
  if (a[0] != Py_None) {
    const double cap = number(a[0]);
    if (!(cap >= 0x1p-60 && cap <= 0x1p60)) refuse("softcap: 2^-60 .. 2^60 expected");
    p->softcap = (float)cap;
  }
  if (Arg slopes(a[1], "slopes"); slopes && slopes->numel() != p->Hq) refuse("slopes: one value per query head expected");
  p->slopes = vec<float>(a[1], p->Hq, "slopes");
  if (a[2] != Py_None && (p->window = integer(a[2])) < 1) refuse("window: at least one position expected");
  p->depth = grid<int32_t>(a[3], p->B, p->R, "depth");
  if ((a[4] == Py_None) != (a[5] == Py_None)) refuse("groups: length and members: give both or neither");
  p->shared_len = vec<int32_t>(a[4], p->B, "length");
  p->shared_members = vec<int32_t>(a[5], p->B, "members");
}

// (address of an sv_attention_args, q, kv, block_table, seq_len, out, stage, mask, n_nodes, scale, layer)
PyObject* attention_args(PyObject* const* a) {
  sv_attention_args p = {};
  fill(&p, a + 1, *need(a[5], "out").t);
  *static_cast<sv_attention_args*>(PyLong_AsVoidPtr(a[0])) = p;
  return none();
}

// The same and softcap, slopes, window, depth, shared_len, shared_members.
PyObject* attention_args_forms(PyObject* const* a) {
  sv_attention_args p = {};
  fill(&p, a + 1, *need(a[5], "out").t);
  fill_forms(&p, a + 11);
  *static_cast<sv_attention_args*>(PyLong_AsVoidPtr(a[0])) = p;
  return none();
}

// (handle, workspace, stream, q, kv, block_table, seq_len, out, stage, mask, n_nodes, scale, layer)
// -> out, or the bytes of workspace that the call needs and was not given
template <bool kForms>
PyObject* attend(PyObject* const* a) {
  Arg ws(a[1], "workspace"), q = need(a[3], "q");
  Owned out(a[7]);
  if (out.get() == Py_None) out.allocate(*q.t);
  sv_attention_args p = {};
  fill(&p, a + 3, *need(out.get(), "out").t);
  if (kForms) fill_forms(&p, a + 13);
  size_t bytes = 0;
  done("sv_attention_workspace_size", api.attention_size(handle_of(a[0]), &p, &bytes));
  if (!ws || (size_t)ws->nbytes() < bytes) return PyLong_FromSize_t(bytes);
  done("sv_tree_attention", api.attention(handle_of(a[0]), &p, ptr(*ws.t), ws->nbytes(), stream_of(a[2])));
  return out.release();
}
PyObject* attention(PyObject* const* a) { return attend<false>(a); }
// The same and softcap, slopes, window, depth, shared_len, shared_members.
PyObject* attention_forms(PyObject* const* a) { return attend<true>(a); }

// (handle, block_table, seq_len, block_size, least, shared_len, shared_members, stream) -> (shared_len, shared_members)
PyObject* prefix_groups(PyObject* const* a) {
  Arg t = need(a[1], "block_table"), len = need(a[2], "seq_len");
  if (t->dim() != 2 || t->scalar_type() != at::kInt || !t->is_contiguous())
    refuse("block_table must be a contiguous int32 [B][max_blocks]");
  const int64_t B = t->size(0);
  if (B > INT32_MAX || t->size(1) > INT32_MAX) refuse("block_table: too large");
  if ((a[5] == Py_None) != (a[6] == Py_None)) refuse("length and members: give both or neither");
  at::Tensor length, members;
  if (a[5] == Py_None) {
    at::AutoDispatchBelowADInplaceOrView plain;  // no gradients are kept here
    const at::Tensor both = at::empty({2 * B}, t->options());  // one allocation
    length = both.as_strided({B}, {1}, 0), members = both.as_strided({B}, {1}, B);
  } else {
    grid<int32_t>(a[5], 1, B, "length"), grid<int32_t>(a[6], 1, B, "members");
    length = THPVariable_Unpack(a[5]), members = THPVariable_Unpack(a[6]);
  }
  done("sv_prefix_groups", api.prefix_groups(handle_of(a[0]), (int)B, vec<int32_t>(a[2], B, "seq_len"), ptr<int32_t>(*t.t),
                                             (int)t->size(1), integer(a[3]), integer(a[4]), ptr<int32_t>(length),
                                             ptr<int32_t>(members), stream_of(a[7])));
  if (a[5] != Py_None) return PyTuple_Pack(2, a[5], a[6]);
  PyObject *l = THPVariable_Wrap(length), *m = THPVariable_Wrap(members), *r = PyTuple_Pack(2, l, m);
  Py_DECREF(l), Py_DECREF(m);
  return r;
}

// (handle, logits, out, V, history, tokens, mask, n_nodes, rep, presence, frequency, bias_ids, bias_values, allowed, stream)
PyObject* logits(PyObject* const* a) {
  Arg x = need(a[1], "logits"), y = need(a[2], "out");
  if (x->dim() != 3 || y->dim() != 3 || x->size(0) != y->size(0) || x->size(1) != y->size(1) ||
      x->scalar_type() != y->scalar_type())
    refuse("out does not match logits");
  const int64_t B = x->size(0), R = x->size(1);
  if (x->stride(2) != 1 || y->stride(2) != 1 ||
      (B > 1 && R > 1 && (x->stride(0) != R * x->stride(1) || y->stride(0) != R * y->stride(1))))
    refuse("logits and out must be whole [B][R][ld] rows");
  sv_logits_args p = {};
  p.B = (int)B, p.R = (int)R, p.V = a[3] == Py_None ? (int)x->size(2) : integer(a[3]), p.dtype = dtype_of(*x.t, "logits");
  if (p.V > x->size(2) || p.V > y->size(2)) done("sv_adjust_logits", SV_ERR_INVALID);  // ld alone may reach past a view's end
  // one row a request: the requests' distance; one row in all: anything that holds it
  const auto ld = [&](const Arg& t) { return R > 1 ? t->stride(1) : B > 1 ? t->stride(0) : (t->size(2) + 7) / 8 * 8; };
  p.logits = ptr(*x.t), p.out = ptr(*y.t), p.ld = ld(x), p.out_ld = ld(y);
  int64_t values;
  p.history = table<int32_t>(a[4], B, &p.history_ld, "history");
  p.tokens = grid<int32_t>(a[5], B, R - 1, "tokens");
  p.mask = table<uint32_t>(a[6], B * R, &p.mask_ld, "mask");
  p.n_nodes = vec<int32_t>(a[7], B, "n_nodes");
  p.rep_penalty = vec<float>(a[8], B, "rep_penalty");
  p.presence = vec<float>(a[9], B, "presence");
  p.frequency = vec<float>(a[10], B, "frequency");
  p.bias_ids = table<int32_t>(a[11], B, &p.bias_ld, "bias_ids");
  p.bias_values = table<float>(a[12], B, &values, "bias_values");
  if (values != p.bias_ld) refuse("bias_ids and bias_values differ in shape");
  p.allowed = table<uint32_t>(a[13], B * R, &p.allowed_ld, "allowed");
  done("sv_adjust_logits", api.logits(handle_of(a[0]), &p, stream_of(a[14])));
  return none();
}

// No C++ exception leaves a call; torch's keep their Python types.
template <PyObject* (*fn)(PyObject* const*), int kArgs>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return fn(a);
  } catch (const Refused&) {
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// open(path of the library, error class)
PyObject* open_library(PyObject*, PyObject* args) {
  const char* path;
  PyObject* cls;
  if (!PyArg_ParseTuple(args, "sO", &path, &cls)) return nullptr;
  void* lib = dlopen(path, RTLD_NOW);
  if (!lib) {
    PyErr_SetString(PyExc_ImportError, dlerror());
    return nullptr;
  }
  const auto sym = [&](const char* name, auto& f) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(lib, name));
    if (!f) PyErr_Format(PyExc_ImportError, "%s has no %s", path, name);
    return f != nullptr;
  };
  decltype(&sv_append_args_size) append_size, attention_size, logits_size;
  if (!sym("sv_tree_mask", api.tree_mask) || !sym("kv_append", api.append) || !sym("kv_read", api.read) ||
      !sym("sv_attention_workspace_size", api.attention_size) || !sym("sv_tree_attention", api.attention) ||
      !sym("sv_adjust_logits", api.logits) || !sym("sv_prefix_groups", api.prefix_groups) || !sym("sv_append_args_size", append_size) ||
      !sym("sv_attention_args_size", attention_size) || !sym("sv_logits_args_size", logits_size))
    return nullptr;
  if (append_size() != sizeof(sv_append_args) || attention_size() != sizeof(sv_attention_args) ||
      logits_size() != sizeof(sv_logits_args)) {
    PyErr_Format(PyExc_ImportError, "%s was built from another header", path);
    return nullptr;
  }
  Py_INCREF(cls);
  g_error = cls;
  return none();
}

#define SV_CALL(name, fn, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&call<fn, n>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {{"open", open_library, METH_VARARGS, nullptr},
                          SV_CALL("tree_mask", tree_mask, 6),
                          SV_CALL("append", append, 15),
                          SV_CALL("read", read, 9),
                          SV_CALL("attention_args", attention_args, 11),
                          SV_CALL("attention", attention, 13),
                          SV_CALL("attention_args_forms", attention_args_forms, 17),
                          SV_CALL("attention_forms", attention_forms, 19),
                          SV_CALL("prefix_groups", prefix_groups, 8),
                          SV_CALL("logits", logits, 15),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
