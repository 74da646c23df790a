// Argument marshalling for Python of the calls that a serving loop makes every
// step: decode on both schedules, the append to INT8 pages, packed prompts. As
// marshal.cpp: each function does what binding.py's function of the same purpose
// does, checks included, and returns its status, or None, having done nothing, for
// arguments that binding.py has to refuse. Through ctypes these calls took 12 to 30
// us of a Grace core; they take 4 (append, packed prompts) and 8 to 9 (decode: two
// launches and two tensor maps).
#include <ATen/ops/empty.h>

#include "marshal_args.h"

namespace {

// Rows of heads that lie side by side: bf16 [rows, heads, head_dim], contiguous or
// a part of wider rows.
struct Heads {
  void* p = nullptr;
  int64_t rows = 0, heads = 0, d = 0, stride = 0;
};
Heads heads_rows(Args& g, int i) {
  Heads h;
  if (!THPVariable_CheckExact(g.a[i])) {
    g.ok = false;
    return h;
  }
  const at::Tensor& t = THPVariable_Unpack(g.a[i]);
  if (t.device().type() != PD_MARSHAL_DEVICE || t.layout() != at::kStrided || t.dim() != 3 ||
      t.scalar_type() != kBf16 || (g.dev >= 0 && t.get_device() != g.dev)) {
    g.ok = false;
    return h;
  }
  g.dev = static_cast<int>(t.get_device());
  h.rows = t.size(0);
  h.heads = t.size(1);
  h.d = t.size(2);
  const int64_t s0 = t.stride(0);
  if ((h.d > 1 && t.stride(2) != 1) || (h.heads > 1 && t.stride(1) != h.d) ||
      (h.rows > 1 && s0 < h.heads * h.d) || h.rows > kMost || h.heads > kMost || h.d > kMost)
    g.ok = false;
  h.stride = h.rows > 1 ? s0 : 0;
  h.p = t.data_ptr();
  return h;
}
int32_t i32_of(int64_t v) { return static_cast<int32_t>(v); }

// The workspace of a call: the caller's (argument i), or for None one of `bytes`
// bytes from the current stream's memory (the call runs on that stream then).
struct Work {
  at::Tensor own;
  void* p = nullptr;
  size_t bytes = 0;
};
Work workspace(Args& g, int i, const at::Tensor& like, size_t bytes) {
  Work w;
  if (g.a[i] != Py_None) {
    const at::Tensor* t = g.tensor(i);
    if (t) {
      w.p = t->data_ptr();
      w.bytes = t->nbytes();
    }
    return w;
  }
  if (!g.ok) return w;
  w.bytes = bytes < 16 ? 16 : bytes;
  w.own = at::empty({static_cast<int64_t>(w.bytes)}, like.options().dtype(at::kByte));
  w.p = w.own.data_ptr();
  return w;
}

// (qkv, q_out or None: in place, num_q_heads, head_dim (read in place only), k_cache, v_cache,
//  block_tables, seq_lens, cu_q, cos_sin, max_q_len, num_kv_heads, block_size, num_blocks,
//  positions, k_out, interleaved, stream)
PyObject* rope_append(PyObject* const* args) {
  Args g{args};
  const at::Tensor* qkv = g.tensor(0);
  if (!qkv || qkv->scalar_type() != kBf16 || qkv->dim() != 2) Py_RETURN_NONE;
  const int64_t T = qkv->size(0), row = qkv->size(1);
  const int64_t hkv = g.i64(11);
  Heads q, k;
  if (args[1] != Py_None) {
    q = heads_rows(g, 1);
    if (args[15] != Py_None) {
      k = heads_rows(g, 15);
      if (k.rows != T || k.heads != hkv || k.d != q.d) g.ok = false;
    }
  } else {
    if (args[15] != Py_None) Py_RETURN_NONE;
    q = {qkv->data_ptr(), T, g.i64(2), g.i64(3), row};
    if (!g.ok || q.heads < 0 || q.d < 0 || q.heads > kMost || q.d > kMost) Py_RETURN_NONE;
    k = q;
    k.p = static_cast<char*>(q.p) + 2 * q.heads * q.d;
  }
  void* kc = g.bytes(4);
  void* vc = g.bytes(5);
  const at::Tensor* bt = g.tensor(6);
  if (!g.ok || bt->scalar_type() != kI32 || bt->dim() != 2) Py_RETURN_NONE;
  const int64_t B = bt->size(0), mbs = bt->size(1);
  const void* lens = g.ptr(7, kI32, B);
  const void* cu = g.ptr(8, kI32, B + 1);
  const at::Tensor* cs = g.tensor(9);
  if (!g.ok || cs->scalar_type() != at::kFloat || cs->dim() != 2) Py_RETURN_NONE;
  const int32_t most_q = g.i32(10), bs = g.i32(12);
  const int64_t nb = g.i64(13);
  const void* pos = g.optional(14, kI32, T);
  const int inter = PyObject_IsTrue(args[16]);
  void* st = g.stream(17);
  if (!g.ok || inter < 0 || q.rows != T || hkv < 0 || hkv > kMost || T > kMost || B > kMost ||
      mbs > kMost || cs->size(0) > kMost || cs->size(1) > kMost ||
      row < (q.heads + 2 * hkv) * q.d) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const size_t need = pd_cache_bytes(PD_KV_INT8, nb, bs, i32_of(hkv), i32_of(q.d));
  if (THPVariable_Unpack(args[4]).nbytes() < need || THPVariable_Unpack(args[5]).nbytes() < need)
    Py_RETURN_NONE;
  const void* rows = qkv->data_ptr();
  const float* table = static_cast<const float*>(cs->data_ptr());
  const int32_t top = i32_of(cs->size(0)), rot = i32_of(cs->size(1));
  const void* tables = bt->data_ptr();
  return status([&] {
    return pd_rope_append_int8(rows, row, static_cast<const int32_t*>(cu),
                               static_cast<const int32_t*>(lens), static_cast<const int32_t*>(pos),
                               table, top, rot, inter, q.p, q.stride, k.p, k.stride, kc, vc,
                               static_cast<const int32_t*>(tables), i32_of(B), i32_of(T), most_q,
                               i32_of(q.heads), i32_of(hkv), i32_of(q.d), bs, i32_of(mbs), nb, st);
  });
}

// (q, k, v, cu_q, out, max_q_len, scale, causal, sliding_window, stream)
PyObject* prefill_packed(PyObject* const* args) {
  Args g{args};
  const Heads q = heads_rows(g, 0), k = heads_rows(g, 1), v = heads_rows(g, 2);
  const at::Tensor* cu = g.tensor(3);
  const Heads o = heads_rows(g, 4);
  const int32_t most_q = g.i32(5), window = g.i32(8);
  const float scale = g.f32(6);
  const int causal = PyObject_IsTrue(args[7]);
  void* st = g.stream(9);
  if (!g.ok || causal < 0 || cu->scalar_type() != kI32 || cu->dim() != 1 || cu->size(0) < 1 ||
      cu->size(0) > kMost || o.rows != q.rows || o.heads != q.heads || o.d != q.d ||
      k.rows != q.rows || v.rows != q.rows || k.d != q.d || v.d != q.d || v.heads != k.heads) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const int32_t* offsets = static_cast<const int32_t*>(cu->data_ptr());
  const int32_t B = i32_of(cu->size(0) - 1);
  return status([&] {
    return pd_prefill_packed(q.p, q.stride, k.p, k.stride, v.p, v.stride, offsets, o.p, o.stride, B,
                             i32_of(q.rows), most_q, i32_of(q.heads), i32_of(k.heads), i32_of(q.d),
                             scale, causal, window, st);
  });
}

// What both schedules of decode take first: (q, k_cache, v_cache, block_tables, ..., out).
struct DecodeTensors {
  const void *q, *tables;
  void *kc, *vc, *out;
  int64_t B, hq, d, mbs;
};
bool decode_tensors(Args& g, int out_at, DecodeTensors& t) {
  const at::Tensor* q = g.tensor(0);
  t.kc = g.bytes(1);
  t.vc = g.bytes(2);
  const at::Tensor* bt = g.tensor(3);
  const at::Tensor* o = g.tensor(out_at);
  if (!g.ok || q->scalar_type() != kBf16 || q->dim() != 3 || o->scalar_type() != kBf16 ||
      !o->sizes().equals(q->sizes()) || bt->scalar_type() != kI32 || bt->dim() != 2 ||
      bt->size(0) != q->size(0))
    return false;
  t.q = q->data_ptr();
  t.out = o->data_ptr();
  t.tables = bt->data_ptr();
  t.B = q->size(0);
  t.hq = q->size(1);
  t.d = q->size(2);
  t.mbs = bt->size(1);
  return t.B <= kMost && t.hq <= kMost && t.d <= kMost && t.mbs <= kMost;
}

// (q, k_cache, v_cache, block_tables, seq_lens, out, num_kv_heads, block_size, num_blocks, scale,
//  num_splits, sliding_window, kv_dtype, k_scale, v_scale, workspace or None: from the current
//  stream's memory, stream)
PyObject* decode(PyObject* const* args) {
  Args g{args};
  DecodeTensors t;
  if (!decode_tensors(g, 5, t)) Py_RETURN_NONE;
  const void* lens = g.ptr(4, kI32, t.B);
  const int32_t hkv = g.i32(6), bs = g.i32(7), window = g.i32(11);
  int32_t splits = g.i32(10);
  const int64_t nb = g.i64(8);
  const float scale = g.f32(9), ks = g.f32(13), vs = g.f32(14);
  const int32_t code = g.i32(12);
  void* st = g.stream(16);
  size_t need = 0;
  if (g.ok && args[15] == Py_None) {
    if (splits == 0)
      splits = pd_choose_num_splits(i32_of(t.B), hkv, i32_of(t.mbs), bs, window, i32_of(t.d), code,
                                    g.dev);
    if (splits < 1) Py_RETURN_NONE;  // a shape that binding.py says what is wrong with
    need = pd_decode_workspace_bytes(i32_of(t.B), i32_of(t.hq), i32_of(t.d), splits);
  }
  const Work ws = workspace(g, 15, THPVariable_Unpack(args[0]), need);
  if (!g.ok) Py_RETURN_NONE;
  void* work = ws.p;
  const size_t work_bytes = ws.bytes;
  return status([&] {
    return pd_decode(t.q, t.kc, t.vc, static_cast<const int32_t*>(t.tables),
                     static_cast<const int32_t*>(lens), t.out, i32_of(t.B), i32_of(t.hq), hkv,
                     i32_of(t.d), bs, i32_of(t.mbs), nb, scale, splits, window, code, ks, vs, work,
                     work_bytes, st);
  });
}

// (q, k_cache, v_cache, block_tables, plan, out, num_kv_heads, block_size, num_blocks, scale,
//  sliding_window, kv_dtype, k_scale, v_scale, num_ctas, num_pieces, workspace or None, the plan's
//  workspace_bytes, stream)
PyObject* decode_balanced(PyObject* const* args) {
  Args g{args};
  DecodeTensors t;
  if (!decode_tensors(g, 5, t)) Py_RETURN_NONE;
  const at::Tensor* plan = g.tensor(4);
  const int32_t hkv = g.i32(6), bs = g.i32(7), window = g.i32(10), code = g.i32(11);
  const int64_t nb = g.i64(8);
  const float scale = g.f32(9), ks = g.f32(12), vs = g.f32(13);
  const int32_t ctas = g.i32(14), pieces = g.i32(15);
  const int64_t need = g.i64(17);
  void* st = g.stream(18);
  if (!g.ok || plan->scalar_type() != kI32 || need < 0) Py_RETURN_NONE;
  const Work ws = workspace(g, 16, THPVariable_Unpack(args[0]), static_cast<size_t>(need));
  if (!g.ok) Py_RETURN_NONE;
  const void* words = plan->data_ptr();
  const size_t plan_bytes = plan->nbytes();
  void* work = ws.p;
  const size_t work_bytes = ws.bytes;
  return status([&] {
    return pd_decode_balanced(t.q, t.kc, t.vc, static_cast<const int32_t*>(t.tables), words,
                              plan_bytes, t.out, i32_of(t.B), i32_of(t.hq), hkv, i32_of(t.d), bs,
                              i32_of(t.mbs), nb, scale, window, code, ks, vs, ctas, pieces, work,
                              work_bytes, st);
  });
}

PyMethodDef kMethods[] = {method<rope_append, 18>("rope_append"),
                          method<prefill_packed, 10>("prefill_packed"),
                          method<decode, 17>("decode"),
                          method<decode_balanced, 19>("decode_balanced"),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal_serve", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal_serve() { return PyModule_Create(&kModule); }
