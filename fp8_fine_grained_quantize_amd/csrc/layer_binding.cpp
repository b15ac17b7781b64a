// Python binding of the operators around the GEMMs: argument checks, output
// allocation and the call of the C entry point, in C++ because a small call
// spent most of its time on them in Python: host time of residual_norm of 16
// rows 9.5 us, 18 through ctypes, moe_combine 5.4 / 9.6, moe_sort 7.0 / 10.9,
// clip_grad_norm (two launches) 9.2 / 11.3, where a launch takes about 4.
//
// Functions of this module take their arguments by position, as layer.py passes
// them, with the current stream's handle last (None if the first tensor is not
// on the current GPU).
#include <algorithm>
#include <utility>
#include <vector>

#include "../../include/libfp8blk_layer.h"
#include "binding.h"

namespace {

using namespace fp8blk_py;

// K of the pairs' map [T][K].
int64_t pairs(const Tensor& row_of, int64_t T) {
  need(row_of, at::kInt, "row_of");
  if (row_of.dim() != 2 || row_of.size(0) != T)
    value_error("row_of must be [T][K] with T = " + std::to_string(T) + ", got " + sizes(row_of));
  if (!row_of.is_contiguous()) value_error("row_of must be contiguous");
  return row_of.size(1);
}

// --- tokens by expert ------------------------------------------------------

PyObject* moe_sort(PyObject* const* a) {  // ids, E, offsets, row_of, slot_of, workspace, stream
  Tensor ids = given(a[0], "expert_ids");
  const int64_t E = integer(a[1]);
  const Tensor *o = maybe(a[2], "offsets"), *r = maybe(a[3], "row_of"), *s = maybe(a[4], "slot_of");
  const Tensor* w = maybe(a[5], "workspace");
  if ((ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong) || ids.dim() != 2)
    type_error("expert_ids must be an int32 or int64 matrix [T][K]");
  scratch(w);
  void* stream = stream_of(a[6], ids, {o, r, s, w});
  Unlocked unlocked;
  own({o, r, s, w});
  const int64_t T = ids.size(0), K = ids.size(1);
  if ((K > 1 && ids.stride(1) != 1) || (T > 1 && ids.stride(0) < K)) ids = ids.contiguous();
  const int64_t bounds = std::clamp<int64_t>(E, 0, 1 << 16) + 1;  // the library refuses far fewer: no memory for those
  if (o != nullptr) dense(*o, at::kInt, {bounds}, "offsets");
  if (r != nullptr) dense(*r, at::kInt, {T, K}, "row_of");
  if (s != nullptr) dense(*s, at::kInt, {T * K}, "slot_of");
  const Tensor off = o != nullptr ? *o : vec({bounds}, at::kInt, ids);
  const Tensor row = r != nullptr ? *r : vec({T, K}, at::kInt, ids);
  const Tensor slot = s != nullptr ? *s : vec({T * K}, at::kInt, ids);
  const size_t bytes = fp8blk_moe_sort_workspace_bytes(T, K, E);
  Tensor ws;
  if (w != nullptr) ws = *w;
  else if (bytes != 0) ws = vec({static_cast<int64_t>(bytes / 4)}, at::kInt, ids);
  ok(fp8blk_moe_sort(addr(ids), T, K, T > 1 ? ids.stride(0) : K, E, static_cast<int32_t*>(addr(off)),
                     static_cast<int32_t*>(addr(row)), static_cast<int32_t*>(addr(slot)),
                     ws.defined() ? addr(ws) : nullptr, ws.defined() ? ws.nbytes() : 0,
                     ids.scalar_type() == at::kLong ? FP8BLK_MOE_IDS_I64 : 0, stream),
     "moe_sort");
  unlocked.end();
  return tuple({&off, &row, &slot});
}

PyObject* moe_dispatch(PyObject* const* a) {  // x, row_of, out, stream
  const Tensor &x = given(a[0], "x"), &row_of = given(a[1], "row_of");
  const Tensor* o = maybe(a[2], "out");
  need(x, at::kBFloat16, "x");
  two_d(x, "x");
  const int64_t T = x.size(0), C = x.size(1), K = pairs(row_of, T), ldx = pitch(x, "x");
  void* stream = stream_of(a[3], x, {&row_of, o});
  Unlocked unlocked;
  own({o});
  int64_t ldo;
  const Tensor out = output(o, T * K, C, at::kBFloat16, x, "out", ldo);
  ok(fp8blk_moe_dispatch(static_cast<uint16_t*>(addr(x)), T, C, ldx, K, static_cast<int32_t*>(addr(row_of)),
                         static_cast<uint16_t*>(addr(out)), ldo, stream),
     "moe_dispatch");
  unlocked.end();
  return wrap(out);
}

PyObject* moe_dispatch_fp8(PyObject* const* a) {  // q, s, row_of, slot_of, qr, sr, stream
  const Tensor &q = given(a[0], "q"), &s = given(a[1], "s"), &row_of = given(a[2], "row_of");
  const Tensor& slot_of = given(a[3], "slot_of");
  const Tensor *oq = maybe(a[4], "qr"), *os = maybe(a[5], "sr");
  need(q, at::kByte, "q");
  two_d(q, "q");
  const int64_t T = q.size(0), C = q.size(1), K = pairs(row_of, T), G = (C + 127) / 128, ldq = pitch(q, "q");
  dense(s, at::kFloat, {G, T}, "s");
  dense(slot_of, at::kInt, {T * K}, "slot_of");
  if (os != nullptr) dense(*os, at::kFloat, {G, T * K}, "sr");
  void* stream = stream_of(a[6], q, {&s, &row_of, &slot_of, oq, os});
  Unlocked unlocked;
  own({oq, os});
  int64_t ldqr;
  const Tensor qr = output(oq, T * K, C, at::kByte, q, "qr", ldqr);
  const Tensor sr = os != nullptr ? *os : vec({G, T * K}, at::kFloat, q);
  ok(fp8blk_moe_dispatch_fp8(static_cast<uint8_t*>(addr(q)), T, C, ldq, static_cast<float*>(addr(s)), K,
                             static_cast<int32_t*>(addr(row_of)), static_cast<int32_t*>(addr(slot_of)),
                             static_cast<uint8_t*>(addr(qr)), ldqr, static_cast<float*>(addr(sr)), stream),
     "moe_dispatch_fp8");
  unlocked.end();
  return tuple({&qr, &sr});
}

PyObject* moe_combine(PyObject* const* a) {  // rows, row_of, weights, out_dtype, out, stream
  const Tensor &rows = given(a[0], "rows"), &row_of = given(a[1], "row_of");
  const Tensor *w = maybe(a[2], "weights"), *o = maybe(a[4], "out");
  two_d(row_of, "row_of");
  two_d(rows, "rows");
  const int64_t T = row_of.size(0), K = pairs(row_of, T), C = rows.size(1);
  uint32_t flags = is_f32(rows, "rows") ? FP8BLK_MOE_ROWS_F32 : 0;
  matrix(rows, T * K, C, "rows");
  const int64_t ldr = pitch(rows, "rows");
  if (w != nullptr) dense(*w, at::kFloat, {T, K}, "weights");
  if (o != nullptr) is_f32(*o, "out");
  const ScalarType dt = o != nullptr ? o->scalar_type() : dtype_of(a[3]);
  void* stream = stream_of(a[5], rows, {&row_of, w, o});
  Unlocked unlocked;
  own({o});
  int64_t ldo;
  const Tensor out = output(o, T, C, dt, rows, "out", ldo);
  if (out.scalar_type() == at::kFloat) flags |= FP8BLK_MOE_TOKENS_F32;
  ok(fp8blk_moe_combine(addr(rows), T, K, C, ldr, static_cast<int32_t*>(addr(row_of)), static_cast<float*>(addr(w)),
                        addr(out), ldo, flags, stream),
     "moe_combine");
  unlocked.end();
  return wrap(out);
}

PyObject* moe_combine_backward(PyObject* const* a) {  // dy, rows, row_of, weights, drows_dtype, drows, dweights, stream
  const Tensor &dy = given(a[0], "dy"), &rows = given(a[1], "rows"), &row_of = given(a[2], "row_of");
  const Tensor& w = given(a[3], "weights");
  const Tensor *od = maybe(a[5], "drows"), *ow = maybe(a[6], "dweights");
  two_d(dy, "dy");
  const int64_t T = dy.size(0), C = dy.size(1), K = pairs(row_of, T);
  uint32_t flags = (is_f32(dy, "dy") ? FP8BLK_MOE_TOKENS_F32 : 0) | (is_f32(rows, "rows") ? FP8BLK_MOE_ROWS_F32 : 0);
  matrix(rows, T * K, C, "rows");
  dense(w, at::kFloat, {T, K}, "weights");
  const int64_t lddy = pitch(dy, "dy"), ldr = pitch(rows, "rows");
  if (od != nullptr) is_f32(*od, "drows");
  if (ow != nullptr) dense(*ow, at::kFloat, {T, K}, "dweights");
  const ScalarType dt = od != nullptr ? od->scalar_type() : a[4] == Py_None ? rows.scalar_type() : dtype_of(a[4]);
  void* stream = stream_of(a[7], dy, {&rows, &row_of, &w, od, ow});
  Unlocked unlocked;
  own({od, ow});
  int64_t lddr;
  const Tensor drows = output(od, T * K, C, dt, dy, "drows", lddr);
  if (dt == at::kFloat) flags |= FP8BLK_MOE_DROWS_F32;
  const Tensor dw = ow != nullptr ? *ow : vec({T, K}, at::kFloat, dy);
  ok(fp8blk_moe_combine_backward(addr(dy), lddy, addr(rows), ldr, T, K, C, static_cast<int32_t*>(addr(row_of)),
                                 static_cast<float*>(addr(w)), addr(drows), lddr, static_cast<float*>(addr(dw)), flags,
                                 stream),
     "moe_combine_backward");
  unlocked.end();
  return tuple({&drows, &dw});
}

// --- norms around a block ----------------------------------------------------

// The flag of the parameters' common type, checked.
uint32_t params(int64_t C, std::initializer_list<const Tensor*> ts) {
  int type = -1;
  for (const Tensor* t : ts) {
    if (t == nullptr) continue;
    if (t->dim() != 1 || t->size(0) != C || !t->is_contiguous())
      value_error("w_pre, w_post and a gate per channel must be contiguous vectors of " + std::to_string(C) + ", got " +
                  sizes(*t));
    const int f = is_f32(*t, "w_pre, w_post and a gate per channel") ? 1 : 0;
    if (type >= 0 && f != type) type_error("w_pre, w_post and a gate per channel must have one type");
    type = f;
  }
  return type == 1 ? FP8BLK_NORM_PARAM_F32 : 0;
}

// Flags of x's type, the parameters' and the gate; ldg: the pitch of a gate per token.
uint32_t norm_flags(const Tensor& x, const Tensor* w_pre, const Tensor* w_post, const Tensor* gate, int64_t& ldg) {
  const int64_t M = x.size(0), C = x.size(1);
  const bool row = gate != nullptr && gate->dim() == 2;
  ldg = row ? pitch(*gate, at::kBFloat16, M, C, "a gate per token") : 0;
  return (row ? FP8BLK_NORM_GATE_ROW : 0) | params(C, {w_pre, w_post, row ? nullptr : gate}) |
         (is_f32(x, "x") ? FP8BLK_NORM_RES_F32 : 0);
}

// x, w_pre, f, w_post, gate, alpha, eps, quantize, pow2, want_n, x_out, n, q, s, stream
PyObject* residual_norm(PyObject* const* a) {
  const Tensor& x = given(a[0], "x");
  const Tensor *wn = maybe(a[1], "w_pre"), *f = maybe(a[2], "f"), *wp = maybe(a[3], "w_post"), *g = maybe(a[4], "gate");
  const double alpha = number(a[5]), eps = number(a[6]);
  const bool quantize = truth(a[7]), pow2 = truth(a[8]), want_n = truth(a[9]);
  const Tensor *ox = maybe(a[10], "x_out"), *on = maybe(a[11], "n"), *oq = maybe(a[12], "q"), *os = maybe(a[13], "s");
  two_d(x, "x");
  const int64_t M = x.size(0), C = x.size(1), G = (C + 127) / 128, ldx = pitch(x, "x");
  int64_t ldg, ldf = 0, ldxo = 0, ldn = 0, ldq = 0;
  uint32_t flags = norm_flags(x, wn, wp, g, ldg);
  if ((wp != nullptr || g != nullptr) && f == nullptr) value_error("w_post and gate need f");
  if (f == nullptr && wn == nullptr) value_error("nothing to do: neither f nor w_pre is given");
  if (wn == nullptr && (quantize || on != nullptr)) value_error("n and its quantization need w_pre");
  if (f == nullptr && ox != nullptr) value_error("x_out without f: x would not change");
  if (f != nullptr) ldf = pitch(*f, at::kBFloat16, M, C, "f");
  void* stream = stream_of(a[14], x, {wn, f, wp, g, ox, on, oq, os});
  Unlocked unlocked;
  own({ox, on, oq, os});
  Tensor xo, n, q, s, r_post, r_pre;
  if (f != nullptr) {
    xo = output(ox, M, C, x.scalar_type(), x, "x_out", ldxo);
    if (wp != nullptr) r_post = vec({M}, at::kFloat, x);
  }
  if (wn != nullptr) {
    r_pre = vec({M}, at::kFloat, x);
    if (on != nullptr || want_n || !quantize) n = output(on, M, C, at::kBFloat16, x, "n", ldn);
    if (quantize) {
      q = output(oq, M, C, at::kByte, x, "q", ldq);
      if (os != nullptr) dense(*os, at::kFloat, {G, M}, "s");
      s = os != nullptr ? *os : vec({G, M}, at::kFloat, x);
      if (pow2) flags |= FP8BLK_SCALE_POW2;
    }
  }
  auto at_ = [](const Tensor& t) { return t.defined() ? addr(t) : nullptr; };
  ok(fp8blk_residual_norm(M, C, addr(x), ldx, static_cast<uint16_t*>(addr(f)), ldf, addr(wp), addr(g), ldg,
                          static_cast<float>(alpha), addr(wn), static_cast<float>(eps), at_(xo), ldxo,
                          static_cast<uint16_t*>(at_(n)), ldn, static_cast<uint8_t*>(at_(q)), ldq,
                          static_cast<float*>(at_(s)), static_cast<float*>(at_(r_post)),
                          static_cast<float*>(at_(r_pre)), flags, stream),
     "residual_norm");
  unlocked.end();
  return tuple({f == nullptr ? &x : &xo, &n, &q, &s, &r_post, &r_pre});
}

// x_out, dx_out, dn, rstd_pre, w_pre, f, rstd_post, w_post, gate, alpha, dx, df, workspace, stream
PyObject* residual_norm_backward(PyObject* const* a) {
  const Tensor& x = given(a[0], "x_out");
  const Tensor *dxo = maybe(a[1], "dx_out"), *dn = maybe(a[2], "dn"), *r_pre = maybe(a[3], "rstd_pre");
  const Tensor *wn = maybe(a[4], "w_pre"), *f = maybe(a[5], "f"), *r_post = maybe(a[6], "rstd_post");
  const Tensor *wp = maybe(a[7], "w_post"), *g = maybe(a[8], "gate");
  const double alpha = number(a[9]);
  const Tensor *ox = maybe(a[10], "dx"), *of = maybe(a[11], "df"), *w = maybe(a[12], "workspace");
  two_d(x, "x_out");
  const int64_t M = x.size(0), C = x.size(1), ldx = pitch(x, "x_out");
  int64_t ldg, lddxo = 0, lddn = 0, ldf = 0, lddx = 0, lddf = 0, lddg = 0;
  const uint32_t flags = norm_flags(x, wn, wp, g, ldg);
  if (dxo == nullptr && dn == nullptr) value_error("neither dx_out nor dn is given");
  if ((wp != nullptr || g != nullptr) && f == nullptr) value_error("w_post and gate need f");
  if ((dn == nullptr) != (wn == nullptr) || (r_pre == nullptr) != (wn == nullptr))
    value_error("dn, rstd_pre and w_pre go together");
  if ((r_post == nullptr) != (wp == nullptr)) value_error("rstd_post and w_post go together");
  if (dxo != nullptr) lddxo = pitch(*dxo, x.scalar_type(), M, C, "dx_out");
  if (wn != nullptr) {
    lddn = pitch(*dn, at::kBFloat16, M, C, "dn");
    dense(*r_pre, at::kFloat, {M}, "rstd_pre");
  }
  if (f != nullptr) ldf = pitch(*f, at::kBFloat16, M, C, "f");
  if (wp != nullptr) dense(*r_post, at::kFloat, {M}, "rstd_post");
  scratch(w);
  void* stream = stream_of(a[13], x, {dxo, dn, r_pre, wn, f, r_post, wp, g, ox, of, w});
  Unlocked unlocked;
  own({ox, of, w});
  Tensor dx, df, dw_pre, dw_post, dgate, ws;
  if (wn != nullptr || ox != nullptr) dx = output(ox, M, C, x.scalar_type(), x, "dx", lddx);
  if (wn != nullptr) dw_pre = vec({C}, at::kFloat, x);
  if (f != nullptr) df = output(of, M, C, at::kBFloat16, x, "df", lddf);
  if (wp != nullptr) dw_post = vec({C}, at::kFloat, x);
  const bool row = flags & FP8BLK_NORM_GATE_ROW;
  if (g != nullptr) dgate = row ? output(nullptr, M, C, at::kBFloat16, x, "dgate", lddg) : vec({C}, at::kFloat, x);
  if (w != nullptr)
    ws = *w;
  else if (dw_pre.defined() || dw_post.defined() || (dgate.defined() && !row))
    ws = vec({static_cast<int64_t>((fp8blk_residual_norm_backward_workspace_bytes(M, C) + 3) / 4)}, at::kFloat, x);
  auto at_ = [](const Tensor& t) { return t.defined() ? addr(t) : nullptr; };
  if (dx.defined() || f != nullptr)
    ok(fp8blk_residual_norm_backward(
           M, C, addr(x), ldx, addr(dxo), lddxo, static_cast<uint16_t*>(addr(dn)), lddn,
           static_cast<float*>(addr(r_pre)), addr(wn), static_cast<uint16_t*>(addr(f)), ldf,
           static_cast<float*>(addr(r_post)), addr(wp), addr(g), ldg, static_cast<float>(alpha), at_(dx), lddx,
           static_cast<uint16_t*>(at_(df)), lddf, static_cast<float*>(at_(dw_pre)), static_cast<float*>(at_(dw_post)),
           at_(dgate), lddg, at_(ws), ws.defined() ? ws.nbytes() : 0, flags, stream),
       "residual_norm_backward");
  unlocked.end();
  return tuple({dx.defined() ? &dx : dxo, &df, &dw_pre, &dw_post, &dgate});
}

// --- gradient norm and clipping ------------------------------------------------

Span span(const void* p, const fp8blk_grad_t& g, int64_t ld, bool f32) {
  const int64_t size = f32 ? 4 : 2;
  return {static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)), g.cols * size, ld * size, g.rows};
}
Span grad_span(const fp8blk_grad_t& g) { return span(g.grad, g, g.ld, g.flags & FP8BLK_GRAD_F32); }
Span out_span(const fp8blk_grad_t& g) { return span(g.out, g, g.ldo, g.flags & FP8BLK_GRAD_OUT_F32); }
// Clipped in place: every element is read and written by one lane.
bool in_place(const fp8blk_grad_t& g) {
  return g.grad == g.out && (g.rows == 1 || g.ld == g.ldo) &&
         !(g.flags & FP8BLK_GRAD_F32) == !(g.flags & FP8BLK_GRAD_OUT_F32);
}

// Two gradients of a list that clipping must not take together: an output of
// one shares memory with the other's gradient or output, or with its own
// gradient other than in place, so that values would be scaled twice or read
// while they are written.  Gradients that are only read may share theirs.
// first[t] .. first[t + 1]: the entries of tensor t.
PyObject* grad_shared(PyObject* const* a) {  // address of the entries, of `first`, tensors
  const auto* list = reinterpret_cast<const fp8blk_grad_t*>(static_cast<uintptr_t>(integer(a[0])));
  const auto* first = reinterpret_cast<const int64_t*>(static_cast<uintptr_t>(integer(a[1])));
  struct Item {  // the extent of a tensor's gradient or output
    int64_t lo, hi, t;
    bool out;
  };
  std::vector<Item> items, open;
  const int64_t tensors = integer(a[2]);
  for (int64_t t = 0; t < tensors; ++t) {
    if (first[t] == first[t + 1]) continue;
    Item g{INT64_MAX, INT64_MIN, t, false}, o{INT64_MAX, INT64_MIN, t, true};
    bool all_in_place = true;
    for (int64_t e = first[t]; e < first[t + 1]; ++e) {
      const Span gs = grad_span(list[e]), os = out_span(list[e]);
      g = {std::min(g.lo, gs.base), std::max(g.hi, gs.end()), t, false};
      o = {std::min(o.lo, os.base), std::max(o.hi, os.end()), t, true};
      all_in_place = all_in_place && in_place(list[e]);
    }
    items.push_back(o);
    if (!all_in_place) items.push_back(g);
  }
  auto shared = [&](const Item& p, const Item& q) {
    for (int64_t e = first[p.t]; e < first[p.t + 1]; ++e)
      for (int64_t f = first[q.t]; f < first[q.t + 1]; ++f) {
        if (e == f && in_place(list[e])) continue;
        if (meet(p.out ? out_span(list[e]) : grad_span(list[e]), q.out ? out_span(list[f]) : grad_span(list[f])))
          return true;
      }
    return false;
  };
  std::sort(items.begin(), items.end(), [](const Item& p, const Item& q) { return p.lo < q.lo; });
  for (const Item& q : items) {  // against the extents that reach past its start
    size_t kept = 0;
    for (const Item& p : open) {
      if (p.hi <= q.lo) continue;
      if ((p.out || q.out) && shared(p, q))
        return Py_BuildValue("LL", static_cast<long long>(std::min(p.t, q.t)), static_cast<long long>(std::max(p.t, q.t)));
      open[kept++] = p;
    }
    open.resize(kept);
    open.push_back(q);
  }
  Py_RETURN_NONE;
}

// The table tensor (undefined address for n = 0), n, chunks, ...

PyObject* grad_norm(PyObject* const* a) {  // table, n, chunks, stream
  const Tensor& table = given(a[0], "table");
  const int64_t n = integer(a[1]), chunks = integer(a[2]);
  void* stream = stream_of(a[3], table, {});
  Unlocked unlocked;
  const Tensor norm = vec({}, at::kFloat, table);
  const Tensor ws = vec({static_cast<int64_t>(FP8BLK_GRAD_WORKSPACE_BYTES / 8)}, at::kDouble, table);
  ok(fp8blk_grad_norm(addr(table), n, chunks, static_cast<float*>(addr(norm)), addr(ws), ws.nbytes(), stream),
     "grad_norm");
  unlocked.end();
  return wrap(norm);
}

PyObject* grad_clip(PyObject* const* a) {  // table, n, chunks, norm, max_norm, eps, stream
  const Tensor &table = given(a[0], "table"), &norm = given(a[3], "norm");
  need(norm, at::kFloat, "norm");
  if (norm.numel() != 1) value_error("norm must be one value");
  const int64_t n = integer(a[1]), chunks = integer(a[2]);
  const float max_norm = static_cast<float>(number(a[4])), eps = static_cast<float>(number(a[5]));
  void* stream = stream_of(a[6], table, {&norm});
  Unlocked unlocked;
  ok(fp8blk_grad_clip(addr(table), n, chunks, static_cast<float*>(addr(norm)), max_norm, eps, stream), "grad_clip");
  unlocked.end();
  Py_RETURN_NONE;
}

PyObject* clip_grad_norm(PyObject* const* a) {  // table, n, chunks, max_norm, eps, stream
  const Tensor& table = given(a[0], "table");
  const int64_t n = integer(a[1]), chunks = integer(a[2]);
  const float max_norm = static_cast<float>(number(a[3])), eps = static_cast<float>(number(a[4]));
  void* stream = stream_of(a[5], table, {});
  Unlocked unlocked;
  const Tensor norm = vec({}, at::kFloat, table);
  const Tensor ws = vec({static_cast<int64_t>(FP8BLK_GRAD_WORKSPACE_BYTES / 8)}, at::kDouble, table);
  ok(fp8blk_grad_clip_norm(addr(table), n, chunks, max_norm, eps, static_cast<float*>(addr(norm)), addr(ws),
                           ws.nbytes(), stream),
     "clip_grad_norm");
  unlocked.end();
  return wrap(norm);
}

PyObject* set_error(PyObject* const* a) {  // the exception of a failed call
  Py_INCREF(a[0]);
  Py_XDECREF(g_error);
  g_error = a[0];
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {FP8BLK_METHOD(moe_sort, 7),
                         FP8BLK_METHOD(moe_dispatch, 4),
                         FP8BLK_METHOD(moe_dispatch_fp8, 7),
                         FP8BLK_METHOD(moe_combine, 6),
                         FP8BLK_METHOD(moe_combine_backward, 8),
                         FP8BLK_METHOD(residual_norm, 15),
                         FP8BLK_METHOD(residual_norm_backward, 14),
                         FP8BLK_METHOD(grad_shared, 3),
                         FP8BLK_METHOD(grad_norm, 4),
                         FP8BLK_METHOD(grad_clip, 7),
                         FP8BLK_METHOD(clip_grad_norm, 6),
                         FP8BLK_METHOD(set_error, 1),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern PyMethodDef fp8blk_train_methods[];  // train_binding.cpp

PyMODINIT_FUNC PyInit__layer_ext() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddFunctions(m, fp8blk_train_methods) != 0) Py_CLEAR(m);
  return m;
}
