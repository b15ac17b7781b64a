// Python binding of the gated feed-forward block and of the optimizer step (see
// binding.h; train.py passes the arguments by position, the current stream last).
#include <ATen/ops/new_empty.h>

#include <algorithm>
#include <memory>
#include <vector>

#include "../../include/libfp8blk_train.h"
#include "binding.h"

namespace {

using namespace fp8blk_py;

// --- the gated feed-forward block ----------------------------------------------

// Codes and scales of a product's operands, checked; G = 0: one B, otherwise one for every expert.
struct Product {
  const Tensor *A, *sA, *B, *sB, *offsets;
  int64_t G = 0, M, N, K, lda, ldb, strideB = 0, stride_sB = 0, max_rows = 0;
  int act, opB;
};

// a[0 .. 8]: offsets, A, sA, B, sB, act, opB, pow2_scales, max_group_rows
Product product(PyObject* const* a) {
  Product p;
  p.offsets = maybe(a[0], "offsets");
  p.A = &given(a[1], "A");
  p.sA = &given(a[2], "sA");
  p.B = &given(a[3], "B");
  p.sB = &given(a[4], "sB");
  p.act = static_cast<int>(integer(a[5]));
  p.opB = static_cast<int>(integer(a[6]));
  if (p.opB != FP8BLK_OP_N && p.opB != FP8BLK_OP_T) value_error("opB must be OP_N or OP_T");
  need(*p.A, at::kByte, "A");
  need(*p.B, at::kByte, "B");
  need(*p.sB, at::kFloat, "sB");
  two_d(*p.A, "A");
  p.M = p.A->size(0);
  p.K = p.A->size(1);
  p.lda = pitch(*p.A, "A");
  const bool grouped = p.offsets != nullptr;
  if (p.B->dim() != (grouped ? 3 : 2)) value_error(std::string("B must have ") + (grouped ? "3" : "2") + " dimensions, got " + sizes(*p.B));
  const Tensor one = grouped && p.B->size(0) > 0 ? p.B->select(0, 0) : grouped ? p.B->new_empty({p.B->size(1), p.B->size(2)}) : *p.B;
  const int64_t rows = one.size(0), cols = one.size(1);
  p.ldb = pitch(one, "B");
  p.N = p.opB == FP8BLK_OP_N ? cols : rows;
  if ((p.opB == FP8BLK_OP_N ? rows : cols) != p.K)
    value_error("B must have " + std::to_string(p.K) + (p.opB == FP8BLK_OP_N ? " rows" : " columns") + ", as A has columns, got " + sizes(*p.B));
  if (p.K % 128 != 0 || p.N % 128 != 0) value_error("sizes of B must be multiples of 128, got " + sizes(*p.B));
  dense(*p.sA, at::kFloat, {p.K / 128, p.M}, "sA");
  if (!grouped) {
    dense(*p.sB, at::kFloat, {rows / 128, cols / 128}, "sB");
  } else {
    need(*p.offsets, at::kInt, "offsets");
    if (p.offsets->dim() != 1 || p.offsets->size(0) != p.B->size(0) + 1 || !p.offsets->is_contiguous())
      value_error("offsets must be a contiguous vector of one more than the experts of B, got " + sizes(*p.offsets));
    p.G = p.B->size(0);
    if (p.sB->dim() != 3 || p.sB->size(0) != p.G) value_error("sB has the wrong shape: " + sizes(*p.sB));
    if (p.G > 0) dense(p.sB->select(0, 0), at::kFloat, {rows / 128, cols / 128}, "sB");
    p.strideB = p.G > 1 ? p.B->stride(0) : rows * p.ldb;
    p.stride_sB = p.G > 1 ? p.sB->stride(0) : rows / 128 * (cols / 128);
    p.max_rows = a[8] == Py_None ? p.M : integer(a[8]);
  }
  if (truth(a[7])) p.opB |= FP8BLK_GEMM_POW2_SCALES;
  return p;
}

uint16_t* bits(const Tensor& t) { return t.defined() ? static_cast<uint16_t*>(addr(t)) : nullptr; }

// q and s of `cols` columns where they are asked for.
void quantized(const Product& p, int64_t cols, const Tensor* oq, const Tensor* os, Tensor& q, Tensor& s, int64_t& ldq) {
  q = output(oq, p.M, cols, at::kByte, *p.A, "q", ldq);
  if (os != nullptr) dense(*os, at::kFloat, {cols / 128, p.M}, "s");
  s = os != nullptr ? *os : vec({cols / 128, p.M}, at::kFloat, *p.A);
}

// A tensor of a call by its name, and the bytes it covers: `pieces` times rows, `apart` bytes from one to the next.
struct Named {
  const Tensor* t;
  const char* name;
};
struct Bytes {
  Span at;
  int64_t pieces = 1, apart = 0;
  int64_t end() const { return at.end() + (pieces - 1) * apart; }
  explicit Bytes(const Tensor& t) {
    const int64_t size = t.element_size(), d = t.dim();
    at.base = static_cast<int64_t>(reinterpret_cast<uintptr_t>(addr(t)));
    const auto reach = [&](int64_t i) { return (t.size(i) - 1) * t.stride(i) * size; };
    at.width = size + (d > 0 ? reach(d - 1) : 0);
    at.pitch = at.width;
    at.rows = 1;
    if (d > 1 && t.size(d - 2) > 1) {
      at.pitch = t.stride(d - 2) * size;
      at.rows = t.size(d - 2);
    }
    if (d > 2) {
      pieces = t.size(d - 3);
      apart = t.stride(d - 3) * size;
    }
    if (d <= 3 && at.pitch >= at.width) return;
    at.width = size;  // of another kind, refused by its shape or strides: all that it reaches over
    for (int64_t i = 0; i < d; ++i) at.width += reach(i);
    at.pitch = at.width;
    at.rows = pieces = 1;
  }
};
bool meet(const Bytes& a, const Bytes& b) {
  if (a.at.base >= b.end() || b.at.base >= a.end()) return false;
  for (int64_t i = 0; i < a.pieces; ++i)
    for (int64_t j = 0; j < b.pieces; ++j) {
      Span p = a.at, q = b.at;
      p.base += i * a.apart;
      q.base += j * b.apart;
      if (p.base < q.end() && q.base < p.end() && fp8blk_py::meet(p, q)) return true;
    }
  return false;
}

// What a call writes, among itself and with what it reads: workgroups run in
// any order, so none of it may lie in another's memory.  `onto`: an output that
// may be that input element for element (each lane reads its own before it writes).
void apart(std::initializer_list<Named> outs, std::initializer_list<Named> ins, const Tensor* onto = nullptr) {
  const auto real = [](const Named& n) { return n.t != nullptr && n.t->numel() != 0; };
  for (const Named* o = outs.begin(); o != outs.end(); ++o) {
    if (!real(*o)) continue;
    const Bytes a(*o->t);
    const auto check = [&](const Named& n, bool may_be_same) {
      if (!real(n)) return;
      const Bytes b(*n.t);
      if (may_be_same && n.t == onto && o->t->scalar_type() == n.t->scalar_type() && a.at.base == b.at.base &&
          a.at.width == b.at.width && a.at.pitch == b.at.pitch && a.at.rows == b.at.rows)
        return;
      if (meet(a, b)) value_error(std::string(o->name) + " shares memory with " + n.name);
    };
    for (const Named& n : ins) check(n, o == outs.begin());
    for (const Named* n = outs.begin(); n != o; ++n) check(*n, false);
  }
}

// The given workspace, or a new one of that size (none for 0 bytes).
Tensor room(const Tensor* given, size_t bytes, const Tensor& like) {
  if (given != nullptr) return *given;
  return bytes != 0 ? vec({static_cast<int64_t>((bytes + 3) / 4)}, at::kFloat, like) : Tensor();
}

// product's arguments, then quantize, pow2, want_h, want_u, split_k, workspace, u, h, q, s, stream
PyObject* gated_gemm(PyObject* const* a) {
  const Product p = product(a);
  a += 9;
  const bool quantize = truth(a[0]), pow2 = truth(a[1]), want_h = truth(a[2]), want_u = truth(a[3]), split = truth(a[4]);
  const Tensor *w = maybe(a[5], "workspace"), *ou = maybe(a[6], "u"), *oh = maybe(a[7], "h"), *oq = maybe(a[8], "q");
  const Tensor* os = maybe(a[9], "s");
  if (p.N % 256 != 0) value_error("B must have the gate's columns and as many of the up projection, got " + sizes(*p.B));
  if (!quantize && (oq != nullptr || os != nullptr)) value_error("q and s need quantize");
  scratch(w);
  own({w, ou, oh, oq, os});
  apart({{ou, "u"}, {oh, "h"}, {oq, "q"}, {os, "s"}, {split ? w : nullptr, "workspace"}},
        {{p.A, "A"}, {p.sA, "sA"}, {p.B, "B"}, {p.sB, "sB"}, {p.offsets, "offsets"}});
  void* stream = stream_of(a[10], *p.A, {p.offsets, p.sA, p.B, p.sB, w, ou, oh, oq, os});
  Unlocked unlocked;
  const int64_t H = p.N / 2;
  int64_t ldu = 0, ldh = 0, ldq = 0;
  Tensor u, h, q, s;
  if (ou != nullptr || want_u) u = output(ou, p.M, 2 * H, at::kBFloat16, *p.A, "u", ldu);
  if (oh != nullptr || want_h || !quantize) h = output(oh, p.M, H, at::kBFloat16, *p.A, "h", ldh);
  if (quantize) quantized(p, H, oq, os, q, s, ldq);
  const uint32_t flags = pow2 ? FP8BLK_SCALE_POW2 : 0;
  auto* qp = q.defined() ? static_cast<uint8_t*>(addr(q)) : nullptr;
  auto* sp = s.defined() ? static_cast<float*>(addr(s)) : nullptr;
  const auto *A = static_cast<uint8_t*>(addr(p.A)), *B = static_cast<uint8_t*>(addr(p.B));
  const auto *sA = static_cast<float*>(addr(p.sA)), *sB = static_cast<float*>(addr(p.sB));
  if (p.offsets != nullptr) {
    ok(fp8blk_grouped_gated_gemm_fp8_blockscaled(p.G, static_cast<int32_t*>(addr(p.offsets)), p.M, p.max_rows, H, p.K, A,
                                                 p.lda, sA, B, p.ldb, p.strideB, p.opB, sB, p.stride_sB, p.act, bits(u),
                                                 ldu, bits(h), ldh, qp, ldq, sp, flags, stream),
       "grouped_gated_gemm_fp8_blockscaled");
  } else {
    const Tensor ws = room(w, split ? fp8blk_gated_gemm_workspace_bytes(p.M, H, p.K) : 0, *p.A);
    ok(fp8blk_gated_gemm_fp8_blockscaled(p.M, H, p.K, A, p.lda, sA, B, p.ldb, p.opB, sB, p.act, bits(u), ldu, bits(h),
                                         ldh, qp, ldq, sp, flags, split && ws.defined() ? addr(ws) : nullptr,
                                         split && ws.defined() ? ws.nbytes() : 0, stream),
       "gated_gemm_fp8_blockscaled");
  }
  unlocked.end();
  wrote({ou, oh, oq, os});
  return tuple({&u, &h, &q, &s});
}

// product's arguments, then u, quantize, pow2, want_h, want_du, split_k, workspace, du, h, q, s, stream
PyObject* gated_gemm_backward(PyObject* const* a) {
  const Product p = product(a);
  a += 9;
  const Tensor& u = given(a[0], "u");
  const bool quantize = truth(a[1]), pow2 = truth(a[2]), want_h = truth(a[3]), want_du = truth(a[4]), split = truth(a[5]);
  const Tensor *w = maybe(a[6], "workspace"), *od = maybe(a[7], "du"), *oh = maybe(a[8], "h"), *oq = maybe(a[9], "q");
  const Tensor* os = maybe(a[10], "s");
  if (!quantize && (oq != nullptr || os != nullptr)) value_error("q and s need quantize");
  const int64_t H = p.N, ldu = pitch(u, at::kBFloat16, p.M, 2 * H, "u");
  scratch(w);
  own({w, od, oh, oq, os});
  apart({{od, "du"}, {oh, "h"}, {oq, "q"}, {os, "s"}, {split ? w : nullptr, "workspace"}},
        {{&u, "u"}, {p.A, "A"}, {p.sA, "sA"}, {p.B, "B"}, {p.sB, "sB"}, {p.offsets, "offsets"}}, &u);
  void* stream = stream_of(a[11], *p.A, {p.offsets, p.sA, p.B, p.sB, &u, w, od, oh, oq, os});
  Unlocked unlocked;
  int64_t lddu = 0, ldh = 0, ldq = 0;
  Tensor du, h, q, s;
  if (od != nullptr || want_du || !quantize) du = output(od, p.M, 2 * H, at::kBFloat16, *p.A, "du", lddu);
  if (oh != nullptr || want_h) h = output(oh, p.M, H, at::kBFloat16, *p.A, "h", ldh);
  if (quantize) quantized(p, 2 * H, oq, os, q, s, ldq);
  const uint32_t flags = pow2 ? FP8BLK_SCALE_POW2 : 0;
  auto* qp = q.defined() ? static_cast<uint8_t*>(addr(q)) : nullptr;
  auto* sp = s.defined() ? static_cast<float*>(addr(s)) : nullptr;
  const auto *A = static_cast<uint8_t*>(addr(p.A)), *B = static_cast<uint8_t*>(addr(p.B));
  const auto *sA = static_cast<float*>(addr(p.sA)), *sB = static_cast<float*>(addr(p.sB));
  if (p.offsets != nullptr) {
    ok(fp8blk_grouped_gated_gemm_backward_fp8_blockscaled(
           p.G, static_cast<int32_t*>(addr(p.offsets)), p.M, p.max_rows, H, p.K, A, p.lda, sA, B, p.ldb, p.strideB, p.opB,
           sB, p.stride_sB, p.act, bits(u), ldu, bits(du), lddu, bits(h), ldh, qp, ldq, sp, flags, stream),
       "grouped_gated_gemm_backward_fp8_blockscaled");
  } else {
    const Tensor ws = room(w, split ? fp8blk_gated_gemm_backward_workspace_bytes(p.M, H, p.K) : 0, *p.A);
    ok(fp8blk_gated_gemm_backward_fp8_blockscaled(p.M, H, p.K, A, p.lda, sA, B, p.ldb, p.opB, sB, p.act, bits(u), ldu,
                                                  bits(du), lddu, bits(h), ldh, qp, ldq, sp, flags,
                                                  split && ws.defined() ? addr(ws) : nullptr,
                                                  split && ws.defined() ? ws.nbytes() : 0, stream),
       "gated_gemm_backward_fp8_blockscaled");
  }
  unlocked.end();
  wrote({od, oh, oq, os});
  return tuple({&du, &h, &q, &s});
}

// --- AdamW -------------------------------------------------------------------

// A list or tuple of n tensors (or None, where that may be).
struct Tensors {
  PyObject* fast;
  const char* what;
  Tensors(PyObject* o, const char* what_) : fast(PySequence_Fast(o, "a state's tensors must be lists")), what(what_) {
    if (fast == nullptr) throw python_error();
  }
  Tensors(const Tensors&) = delete;
  Tensors& operator=(const Tensors&) = delete;
  ~Tensors() { Py_DECREF(fast); }
  int64_t size() const { return PySequence_Fast_GET_SIZE(fast); }
  const Tensor* at(int64_t i) const { return maybe(PySequence_Fast_GET_ITEM(fast, i), what); }
};

// That a state's tensors fit each other.  A table asks it anew: a parameter's
// memory may be another one, of another size, type or device, since the state
// was built (a module moved or sharded under its parameters), as may what its
// lists hold, and the kernel takes every size from the parameter.
PyObject* adamw_check(PyObject* const* a) {  // params, ms, vs, m_scales, v_scales, copies, state
  const Tensors params(a[0], "parameters"), copies(a[5], "copies");
  const Tensors moments[2] = {{a[1], "moments"}, {a[2], "moments"}}, scales[2] = {{a[3], "scales"}, {a[4], "scales"}};
  const int64_t state = integer(a[6]), n = params.size();
  for (const Tensors* t : {&moments[0], &moments[1], &scales[0], &scales[1], &copies})
    if (t->size() != n)
      value_error(std::to_string(n) + " parameters, " + std::to_string(t->size()) + " " + t->what);
  const ScalarType kind = state == FP8BLK_ADAMW_F32 ? at::kFloat : state == FP8BLK_ADAMW_BF16 ? at::kBFloat16 : at::kByte;
  const auto none = [](const char* what, const std::string& of) { type_error(std::string(what) + of + " must be tensors"); };
  for (int64_t i = 0; i < n; ++i) {
    const auto of = [&] { return " of parameter " + std::to_string(i); };
    if (params.at(i) == nullptr) type_error("parameter " + std::to_string(i) + " must be a tensor");
    const Tensor& p = *params.at(i);
    is_f32(p, "parameters");
    if (p.device() != params.at(0)->device())
      value_error("parameter " + std::to_string(i) + " is on " + p.device().str() + ", the first one on " +
                  params.at(0)->device().str());
    const auto fits = [&](const Tensors& list, ScalarType dtype, int64_t count, const char* counted) {
      const Tensor* t = list.at(i);
      if (t == nullptr) none(list.what, of());
      if (t->scalar_type() != dtype)
        type_error(list.what + of() + " must be " + c10::toString(dtype) + ", got " + c10::toString(t->scalar_type()));
      if (t->numel() != count || !t->is_contiguous() || t->device() != p.device())
        value_error(list.what + of() + " must be contiguous, " + counted + " (" + std::to_string(count) + "), on " +
                    p.device().str());
    };
    for (const Tensors& list : moments) fits(list, kind, p.numel(), "one for each element");
    if (state == FP8BLK_ADAMW_E4M3)
      for (const Tensors& list : scales) fits(list, at::kFloat, (p.numel() + 127) / 128, "one for 128 elements");
    const Tensor* c = copies.at(i);
    if (c == nullptr) continue;
    if (c->scalar_type() != at::kBFloat16)
      type_error("copy " + std::to_string(i) + " must be bfloat16, got " + c10::toString(c->scalar_type()));
    if (c->sizes() != p.sizes() || c->device() != p.device())
      value_error("copy " + std::to_string(i) + " must have the parameter's shape and device");
  }
  Py_RETURN_NONE;
}

// Two tensors of a list that a step must not take together: memory that one of
// them writes is the other's too.  Returns None, or (entry, name, entry, name).
PyObject* adamw_shared(PyObject* const* a) {  // address of the entries, their number, state
  const auto* list = reinterpret_cast<const fp8blk_adamw_t*>(static_cast<uintptr_t>(integer(a[0])));
  const int64_t n = integer(a[1]), state = integer(a[2]);
  struct Item {
    Span at;
    int64_t entry;
    const char* what;
    bool written;
  };
  std::vector<Item> items, open;
  auto add = [&](const void* p, int64_t rows, int64_t width, int64_t pitch, int64_t entry, const char* what, bool written) {
    if (p != nullptr)
      items.push_back({{static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)), width, pitch, rows}, entry, what, written});
  };
  for (int64_t i = 0; i < n; ++i) {
    const fp8blk_adamw_t& t = list[i];
    const int64_t pe = t.flags & FP8BLK_ADAMW_PARAM_F32 ? 4 : 2, ge = t.flags & FP8BLK_ADAMW_GRAD_F32 ? 4 : 2;
    const int64_t me = state == FP8BLK_ADAMW_F32 ? 4 : state == FP8BLK_ADAMW_BF16 ? 2 : 1;
    const int64_t count = t.rows * t.cols, scales = (count + 127) / 128 * 4;
    add(t.param, t.rows, t.cols * pe, t.ldp * pe, i, "parameter", true);
    add(t.grad, t.rows, t.cols * ge, t.ldg * ge, i, "gradient", false);
    add(t.copy, t.rows, t.cols * 2, t.ldc * 2, i, "copy", true);
    add(t.m, 1, count * me, count * me, i, "first moment", true);
    add(t.v, 1, count * me, count * me, i, "second moment", true);
    add(t.m_scale, 1, scales, scales, i, "first moment's scales", true);
    add(t.v_scale, 1, scales, scales, i, "second moment's scales", true);
  }
  std::sort(items.begin(), items.end(), [](const Item& p, const Item& q) { return p.at.base < q.at.base; });
  for (const Item& q : items) {  // against the extents that reach past its start
    size_t kept = 0;
    for (const Item& p : open) {
      if (p.at.end() <= q.at.base) continue;
      if ((p.written || q.written) && meet(p.at, q.at))
        return Py_BuildValue("LsLs", static_cast<long long>(p.entry), p.what, static_cast<long long>(q.entry), q.what);
      open[kept++] = p;
    }
    open.resize(kept);
    open.push_back(q);
  }
  Py_RETURN_NONE;
}

// The memory that a table names, kept as long as the table: a step looks whether
// the tensors still have it.  (One whose memory was replaced since would be left
// as it is, and what it had be written behind its next owner's back.)
struct Place {
  c10::Storage memory;
  const void* at;
  int64_t entry;
  const char* what;
  bool written;
};
const void* place_of(const Tensor& t, bool written) {
  return written ? t.mutable_data_ptr() : t.const_data_ptr();  // a copy-on-write clone that is written gets its own
}
std::vector<Place>& places_of(PyObject* held) {
  if (!PyTuple_Check(held) || PyTuple_GET_SIZE(held) != 2) type_error("held must be what adamw_hold returned");
  auto* p = static_cast<std::vector<Place>*>(PyCapsule_GetPointer(PyTuple_GET_ITEM(held, 1), "fp8blk.places"));
  if (p == nullptr) throw python_error();
  return *p;
}

// Returns (the tensors that a table names, their places).
PyObject* adamw_hold(PyObject* const* a) {  // params, grads, ms, vs, m_scales, v_scales, copies
  static const char* const names[] = {"parameter",      "gradient", "first moment", "second moment", "first moment's scales",
                                      "second moment's scales", "copy"};
  std::vector<PyObject*> tensors;
  auto places = std::make_unique<std::vector<Place>>();
  const Tensors params(a[0], names[0]);
  for (int k = 0; k < 7; ++k) {
    const Tensors list(a[k], names[k]);
    for (int64_t i = 0; i < std::min(list.size(), params.size()); ++i) {
      const Tensor* t = list.at(i);
      if (t == nullptr || t->numel() == 0) continue;
      const bool written = k != 1;
      const void* at = place_of(*t, written);
      tensors.push_back(PySequence_Fast_GET_ITEM(list.fast, i));
      places->push_back({t->storage(), at, i, names[k], written});
    }
  }
  PyObject* capsule = PyCapsule_New(places.get(), "fp8blk.places", [](PyObject* c) {
    delete static_cast<std::vector<Place>*>(PyCapsule_GetPointer(c, "fp8blk.places"));
  });
  if (capsule == nullptr) throw python_error();
  places.release();
  PyObject* kept = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  if (kept == nullptr) {
    Py_DECREF(capsule);
    throw python_error();
  }
  for (size_t i = 0; i < tensors.size(); ++i) {
    Py_INCREF(tensors[i]);
    PyTuple_SET_ITEM(kept, static_cast<Py_ssize_t>(i), tensors[i]);
  }
  return Py_BuildValue("NN", kept, capsule);
}

// Refuses a step whose tensors have other memory than when the table was built.
void still_there(PyObject* held) {
  const std::vector<Place>& places = places_of(held);
  PyObject* kept = PyTuple_GET_ITEM(held, 0);
  for (size_t i = 0; i < places.size(); ++i) {
    const Place& p = places[i];
    if (place_of(THPVariable_Unpack(PyTuple_GET_ITEM(kept, static_cast<Py_ssize_t>(i))), p.written) != p.at)
      value_error(std::string(p.what) + " " + std::to_string(p.entry) +
                  " has other memory than when the table was built: build it anew");
  }
}

// A step has written what the table names, but for the gradients.
void wrote_all(PyObject* held) {
  const std::vector<Place>& places = places_of(held);
  PyObject* kept = PyTuple_GET_ITEM(held, 0);
  for (size_t i = 0; i < places.size(); ++i)
    if (places[i].written) wrote(THPVariable_Unpack(PyTuple_GET_ITEM(kept, static_cast<Py_ssize_t>(i))));
}

// One value on the device that a captured step reads anew at every replay, or NULL.
const Tensor* device_value(PyObject* o, ScalarType dtype, const char* what) {
  if (!THPVariable_Check(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  need(t, dtype, what);
  if (t.numel() != 1) value_error(std::string(what) + " must be one value");
  return &t;
}

// table, n, chunks, state, lr, step, beta1, beta2, eps, norm, max_norm, clip_eps, seed, held, stream
PyObject* adamw_step(PyObject* const* a) {
  const Tensor& table = given(a[0], "table");
  const int64_t n = integer(a[1]), chunks = integer(a[2]);
  const int state = static_cast<int>(integer(a[3]));
  fp8blk_adamw_step_t s{};
  const Tensor *lr = device_value(a[4], at::kFloat, "lr"), *step = device_value(a[5], at::kLong, "step");
  const Tensor *norm = maybe(a[9], "norm"), *seed = device_value(a[12], at::kLong, "seed");
  if (lr == nullptr) s.lr = number(a[4]);
  if (step == nullptr) s.step = integer(a[5]);
  s.beta1 = number(a[6]);
  s.beta2 = number(a[7]);
  s.eps = number(a[8]);
  if (norm != nullptr) {
    need(*norm, at::kFloat, "norm");
    if (norm->numel() != 1) value_error("norm must be one value");
    if (a[10] == Py_None) value_error("norm without max_norm");
    s.max_norm = static_cast<float>(number(a[10]));
    s.clip_eps = static_cast<float>(number(a[11]));
  } else if (a[10] != Py_None) {
    value_error("max_norm without norm: give grad_norm of the table");
  }
  if (a[12] != Py_None) {
    s.flags = FP8BLK_ADAMW_RANDOM;
    if (seed == nullptr) {
      const uint64_t v = PyLong_AsUnsignedLongLongMask(a[12]);
      if (PyErr_Occurred()) throw python_error();
      s.seed = static_cast<uint32_t>(v);
    }
  }
  still_there(a[13]);
  void* stream = stream_of(a[14], table, {lr, step, norm, seed});
  s.lr_at = static_cast<float*>(addr(lr));
  s.step_at = static_cast<int64_t*>(addr(step));
  s.seed_at = static_cast<int64_t*>(addr(seed));
  s.norm = static_cast<float*>(addr(norm));
  Unlocked unlocked;
  ok(fp8blk_adamw_step(addr(table), n, chunks, state, &s, stream), "adamw_step");
  unlocked.end();
  wrote_all(a[13]);
  Py_RETURN_NONE;
}

}  // namespace

PyMethodDef fp8blk_train_methods[] = {FP8BLK_METHOD(gated_gemm, 20),
                                      FP8BLK_METHOD(gated_gemm_backward, 21),
                                      FP8BLK_METHOD(adamw_check, 7),
                                      FP8BLK_METHOD(adamw_hold, 7),
                                      FP8BLK_METHOD(adamw_shared, 3),
                                      FP8BLK_METHOD(adamw_step, 15),
                                      {nullptr, nullptr, 0, nullptr}};
