// Python binding of the gated feed-forward block and of the optimizer step (see
// binding.h; train.py passes the arguments by position, the current stream last).
#include <algorithm>
#include <vector>

#include "../../include/libfp8blk_train.h"
#include "binding.h"

namespace {

using namespace fp8blk_py;

// --- AdamW -------------------------------------------------------------------

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

// One value on the device that a captured step reads anew at every replay, or NULL.
const Tensor* device_value(PyObject* o, ScalarType dtype, const char* what) {
  if (!THPVariable_Check(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  need(t, dtype, what);
  if (t.numel() != 1) value_error(std::string(what) + " must be one value");
  return &t;
}

// table, n, chunks, state, lr, step, beta1, beta2, eps, norm, max_norm, clip_eps, seed, stream
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
  void* stream = stream_of(a[13], table, {lr, step, norm, seed});
  s.lr_at = static_cast<float*>(addr(lr));
  s.step_at = static_cast<int64_t*>(addr(step));
  s.seed_at = static_cast<int64_t*>(addr(seed));
  s.norm = static_cast<float*>(addr(norm));
  Unlocked unlocked;
  ok(fp8blk_adamw_step(addr(table), n, chunks, state, &s, stream), "adamw_step");
  unlocked.end();
  Py_RETURN_NONE;
}

}  // namespace

PyMethodDef fp8blk_train_methods[] = {FP8BLK_METHOD(adamw_shared, 3),
                                      FP8BLK_METHOD(adamw_step, 14),
                                      {nullptr, nullptr, 0, nullptr}};
