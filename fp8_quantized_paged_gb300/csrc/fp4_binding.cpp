// fp4_binding.cpp -- Python binding of include/kvq_fp4.h: argument checks and
// marshalling, nothing else; and the module, which has the functions of
// step_binding.cpp too.
//
// A call of a small batch takes a few microseconds on the GPU; reading the
// twelve tensors of a decode call (type, shape, layout, device, address) from
// Python and passing them through ctypes took 14.7 us on the host, here 2.5.
// The checks are what the C ABI cannot see from a pointer.  The library is
// bound at run time (bind), so this file links against torch alone.
#include "binding.h"

#include <dlfcn.h>

#include "../../include/kvq_fp4.h"

PyObject* binding::g_error = nullptr;

namespace {

using namespace binding;

decltype(&kvq_fp4_write) p_write = nullptr;
decltype(&kvq_fp4_read) p_read = nullptr;
decltype(&kvq_fp4_decode_attn) p_decode = nullptr;
decltype(&kvq_fp4_prefill_attn) p_prefill = nullptr;

struct Caches {
  void *k, *v;
  int64_t blocks, heads, dh;
};

// Both caches, uint8 [blocks][heads][9 * head_dim]; dh 0: any.
Caches caches(const char* where, Tensors& ts, PyObject* k, PyObject* v, int64_t dh) {
  const at::Tensor& t = ts.tensor("k_cache", k);
  Caches c;
  c.k = ts.dense("k_cache", t, at::kByte);
  if (t.dim() != 3) fail(where, "caches must have shape [num_blocks][Hkv][9 * head_dim]", KVQ_ERR_SHAPE);
  c.blocks = t.size(0);
  c.heads = t.size(1);
  if (t.size(2) % 9 || (dh && t.size(2) != 9 * dh))
    fail(where, "a cache page of " + std::to_string(t.size(2)) + " bytes is not 9 * head_dim", KVQ_ERR_SHAPE);
  c.dh = t.size(2) / 9;
  c.v = ts.dense("v_cache", v, at::kByte, t.sizes());
  return c;
}

struct Scales {
  float *k, *v;
  int nk, nv;
};
Scales scales(const char* where, Tensors& ts, PyObject* k, PyObject* v) {
  int64_t nk, nv;
  Scales s;
  s.k = static_cast<float*>(ts.dense("k_scale", k, at::kFloat, &nk));
  s.v = static_cast<float*>(ts.dense("v_scale", v, at::kFloat, &nv));
  s.nk = narrow(where, "scales", nk);
  s.nv = narrow(where, "scales", nv);
  return s;
}

void bound(const char* where) {
  if (!g_error || !p_write) {
    PyErr_Format(PyExc_RuntimeError, "%s: the library is not bound", where);
    throw Raised();
  }
}

PyObject* fp4_write(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"k", "v", "slot_mapping", "k_cache", "v_cache", "k_scale", "v_scale",
                                      "scale_granularity", "dev_status", "stream"};
  const char* where = "kvq_fp4_write";
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 8, args, nargs, kw);
    Tensors ts(where);
    const at::Tensor &k = ts.tensor("k", a[0]), &v = ts.tensor("v", a[1]);
    if (k.dim() != 3) fail(where, "k must have shape [num_tokens][Hkv][head_dim]", KVQ_ERR_SHAPE);
    const int64_t n = k.size(0), heads = k.size(1), dh = k.size(2);
    int64_t sk, sv;
    void *kp = ts.rows("k", k, n, heads, dh, sk), *vp = ts.rows("v", v, n, heads, dh, sv);
    if (sk != sv) fail(where, "k and v must have the same row distance", KVQ_ERR_SHAPE);
    const Caches c = caches(where, ts, a[3], a[4], dh);
    if (c.heads != heads) fail(where, "the caches and k must hold the same number of KV heads", KVQ_ERR_SHAPE);
    auto* slots = static_cast<int64_t*>(ts.dense("slot_mapping", a[2], at::kLong, at::IntArrayRef(&n, 1)));
    const Scales s = scales(where, ts, a[5], a[6]);
    const int gran = int32(where, "scale_granularity", a[7]);
    uint32_t* st = ts.status(a[8]);
    const int h = narrow(where, "KV heads", heads), d = narrow(where, "head dims", dh);
    kvq_stream_t stream = ts.stream(a[9]);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = p_write(kp, vp, sk, slots, n, h, d, c.k, c.v, c.blocks, kBlockSize, s.k, s.nk, s.v, s.nv, gran, st, stream);
    Py_END_ALLOW_THREADS
    return result(where, r);
  });
}

PyObject* fp4_read(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"k_cache", "v_cache", "block_tables", "starts", "cu_lens", "k_scale", "v_scale",
                                      "scale_granularity", "k_out", "v_out", "dev_status", "stream"};
  const char* where = "kvq_fp4_read";
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 10, args, nargs, kw);
    Tensors ts(where);
    const Caches c = caches(where, ts, a[0], a[1], 0);
    const at::Tensor &ko = ts.tensor("k_out", a[8]), &vo = ts.tensor("v_out", a[9]);
    if (ko.dim() != 3) fail(where, "k_out must have shape [num_rows][Hkv][head_dim]", KVQ_ERR_SHAPE);
    const int64_t n = ko.size(0);
    int64_t sk, sv;
    void *kp = ts.rows("k_out", ko, n, c.heads, c.dh, sk), *vp = ts.rows("v_out", vo, n, c.heads, c.dh, sv);
    if (sk != sv) fail(where, "k_out and v_out must have the same row distance", KVQ_ERR_SHAPE);
    const at::Tensor& bt = ts.tensor("block_tables", a[2]);
    auto* table = static_cast<int32_t*>(ts.dense("block_tables", bt, at::kInt));
    if (bt.dim() != 2) fail(where, "block_tables must have shape [num_seqs][max_blocks_per_seq]", KVQ_ERR_SHAPE);
    const int64_t B = bt.size(0), B1 = B + 1;
    int32_t* starts = nullptr;
    if (a[3] != Py_None) starts = static_cast<int32_t*>(ts.dense("starts", a[3], at::kInt, at::IntArrayRef(&B, 1)));
    auto* cu = static_cast<int32_t*>(ts.dense("cu_lens", a[4], at::kInt, at::IntArrayRef(&B1, 1)));
    const Scales s = scales(where, ts, a[5], a[6]);
    const int gran = int32(where, "scale_granularity", a[7]);
    uint32_t* st = ts.status(a[10]);
    const int h = narrow(where, "KV heads", c.heads), d = narrow(where, "head dims", c.dh);
    const int mb = narrow(where, "blocks per sequence", bt.size(1)), b = narrow(where, "sequences", B);
    kvq_stream_t stream = ts.stream(a[11]);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = p_read(c.k, c.v, c.blocks, kBlockSize, h, d, table, mb, starts, cu, b, n, s.k, s.nk, s.v, s.nv, gran, kp, vp, sk,
               st, stream);
    Py_END_ALLOW_THREADS
    return result(where, r);
  });
}

// What both attentions take after their queries.
struct Attn {
  Caches c;
  int32_t *table, *lens;
  int mb, B, window, sinks, gran;
  Scales s;
  void *ws, *out;
  int64_t ws_bytes;
  uint32_t* st;
};
Attn attn(const char* where, Tensors& ts, PyObject* const* a, const at::Tensor& q, int64_t num_seqs, PyObject* status) {
  // a: k_cache v_cache block_tables seq_lens k_scale v_scale scale_granularity sliding_window
  //    num_sinks workspace out; num_seqs < 0: as many as seq_lens holds
  Attn r;
  r.c = caches(where, ts, a[0], a[1], q.size(2));
  const at::Tensor &bt = ts.tensor("block_tables", a[2]), &sl = ts.tensor("seq_lens", a[3]);
  r.table = static_cast<int32_t*>(ts.dense("block_tables", bt, at::kInt));
  r.lens = static_cast<int32_t*>(ts.dense("seq_lens", sl, at::kInt));
  if (sl.dim() != 1 || (num_seqs >= 0 && sl.size(0) != num_seqs))
    fail(where, "seq_lens must have shape [" + (num_seqs < 0 ? "num_seqs" : std::to_string(num_seqs)) + "]", KVQ_ERR_SHAPE);
  if (bt.dim() != 2 || bt.size(0) != sl.size(0))
    fail(where, "block_tables must have shape [" + std::to_string(sl.size(0)) + "][max_blocks_per_seq]", KVQ_ERR_SHAPE);
  r.B = narrow(where, "sequences", sl.size(0));
  r.mb = narrow(where, "blocks per sequence", bt.size(1));
  r.s = scales(where, ts, a[4], a[5]);
  r.gran = int32(where, "scale_granularity", a[6]);
  r.window = int32(where, "sliding_window", a[7]);
  r.sinks = int32(where, "num_sinks", a[8]);
  r.ws = ts.dense("workspace", a[9], at::kByte, &r.ws_bytes);
  r.out = ts.dense("out", a[10], at::kBFloat16, q.sizes());
  r.st = ts.status(status);
  return r;
}

PyObject* fp4_decode(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"q", "k_cache", "v_cache", "block_tables", "seq_lens", "k_scale", "v_scale",
                                      "scale_granularity", "sliding_window", "num_sinks", "workspace", "out",
                                      "dev_status", "stream"};
  const char* where = "kvq_fp4_decode_attn";
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 12, args, nargs, kw);
    Tensors ts(where);
    const at::Tensor& q = ts.tensor("q", a[0]);
    void* qp = ts.dense("q", q, at::kBFloat16);
    if (q.dim() != 3) fail(where, "q must have shape [num_seqs][Hq][head_dim]", KVQ_ERR_SHAPE);
    const Attn r = attn(where, ts, a.data() + 1, q, q.size(0), a[12]);
    const int hq = narrow(where, "query heads", q.size(1)), h = narrow(where, "KV heads", r.c.heads);
    kvq_stream_t stream = ts.stream(a[13]);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = p_decode(qp, r.c.k, r.c.v, r.table, r.mb, r.lens, r.B, hq, h, static_cast<int>(r.c.dh), r.c.blocks, kBlockSize,
                  r.s.k, r.s.nk, r.s.v, r.s.nv, r.gran, r.window, r.sinks, r.ws, static_cast<size_t>(r.ws_bytes), r.out,
                  r.st, stream);
    Py_END_ALLOW_THREADS
    return result(where, st);
  });
}

PyObject* fp4_prefill(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"q", "cu_q_lens", "max_q_len", "k_cache", "v_cache", "block_tables", "seq_lens",
                                      "k_scale", "v_scale", "scale_granularity", "sliding_window", "num_sinks",
                                      "workspace", "out", "dev_status", "stream"};
  const char* where = "kvq_fp4_prefill_attn";
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 14, args, nargs, kw);
    Tensors ts(where);
    const at::Tensor& q = ts.tensor("q", a[0]);
    void* qp = ts.dense("q", q, at::kBFloat16);
    if (q.dim() != 3) fail(where, "q must have shape [num_q_tokens][Hq][head_dim]", KVQ_ERR_SHAPE);
    const Attn r = attn(where, ts, a.data() + 3, q, -1, a[14]);
    const int64_t B1 = static_cast<int64_t>(r.B) + 1;
    auto* cu = static_cast<int32_t*>(ts.dense("cu_q_lens", a[1], at::kInt, at::IntArrayRef(&B1, 1)));
    const int most = int32(where, "max_q_len", a[2]);
    const int hq = narrow(where, "query heads", q.size(1)), h = narrow(where, "KV heads", r.c.heads);
    kvq_stream_t stream = ts.stream(a[15]);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = p_prefill(qp, cu, q.size(0), most, r.c.k, r.c.v, r.table, r.mb, r.lens, r.B, hq, h, static_cast<int>(r.c.dh),
                   r.c.blocks, kBlockSize, r.s.k, r.s.nk, r.s.v, r.s.nv, r.gran, r.window, r.sinks, r.ws,
                   static_cast<size_t>(r.ws_bytes), r.out, r.st, stream);
    Py_END_ALLOW_THREADS
    return result(where, st);
  });
}

// bind(path, KvqError): the library to call and the error to raise.
PyObject* fp4_bind(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&]() -> PyObject* {
    const char* path = nargs == 2 ? PyUnicode_AsUTF8(args[0]) : nullptr;
    if (!path) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "bind(path, error)");
      throw Raised();
    }
    void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!h) {
      PyErr_SetString(PyExc_ImportError, dlerror());
      throw Raised();
    }
    auto w = reinterpret_cast<decltype(p_write)>(dlsym(h, "kvq_fp4_write"));
    auto r = reinterpret_cast<decltype(p_read)>(dlsym(h, "kvq_fp4_read"));
    auto d = reinterpret_cast<decltype(p_decode)>(dlsym(h, "kvq_fp4_decode_attn"));
    auto f = reinterpret_cast<decltype(p_prefill)>(dlsym(h, "kvq_fp4_prefill_attn"));
    if (!w || !r || !d || !f) {
      PyErr_Format(PyExc_ImportError, "%s lacks an entry point of kvq_fp4.h", path);
      throw Raised();
    }
    if (!step_bind(h, path)) throw Raised();
    p_write = w;
    p_read = r;
    p_decode = d;
    p_prefill = f;
    Py_XSETREF(g_error, Py_NewRef(args[1]));
    Py_RETURN_NONE;
  });
}

#define KVQ_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {
    {"bind", KVQ_FAST(fp4_bind), METH_FASTCALL, "bind(path, error): the library to call, the error to raise."},
    {"kvq_fp4_write", KVQ_FAST(fp4_write), METH_FASTCALL | METH_KEYWORDS,
     "kvq_fp4_write(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, scale_granularity, dev_status=None, "
     "stream=None)\n\nQuantize-and-scatter: k, v bf16 [N][Hkv][dh] (rows may lie further apart than Hkv * dh), "
     "slot_mapping int64 [N] (negative: skipped)."},
    {"kvq_fp4_read", KVQ_FAST(fp4_read), METH_FASTCALL | METH_KEYWORDS,
     "kvq_fp4_read(k_cache, v_cache, block_tables, starts, cu_lens, k_scale, v_scale, scale_granularity, k_out, v_out, "
     "dev_status=None, stream=None)\n\nGather tokens back to bf16: rows cu_lens[b] .. cu_lens[b + 1] of k_out and v_out "
     "[num_rows][Hkv][dh] are the tokens of sequence b from starts[b] on (starts None: from its first).  cu_lens int32 "
     "[B + 1]; rows from cu_lens[B] on are left as they were."},
    {"kvq_fp4_decode_attn", KVQ_FAST(fp4_decode), METH_FASTCALL | METH_KEYWORDS,
     "kvq_fp4_decode_attn(q, k_cache, v_cache, block_tables, seq_lens, k_scale, v_scale, scale_granularity, "
     "sliding_window, num_sinks, workspace, out, dev_status=None, stream=None)\n\nDecode attention: q bf16 [B][Hq][dh] "
     "-> out; each query sees its sequence's last sliding_window tokens (0: all) and its first num_sinks."},
    {"kvq_fp4_prefill_attn", KVQ_FAST(fp4_prefill), METH_FASTCALL | METH_KEYWORDS,
     "kvq_fp4_prefill_attn(q, cu_q_lens, max_q_len, k_cache, v_cache, block_tables, seq_lens, k_scale, v_scale, "
     "scale_granularity, sliding_window, num_sinks, workspace, out, dev_status=None, stream=None)\n\nPrefill attention: "
     "q bf16 [total_q][Hq][dh], cu_q_lens int32 [B + 1] (device), max_q_len a host bound of the chunks' lengths; a chunk "
     "is its sequence's last tokens, each of which sees what kvq_fp4_decode_attn shows it."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvq_fp4", "Binding of kvq_fp4.h and kvq_step.h.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvq_fp4() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddFunctions(m, step_methods) < 0) Py_CLEAR(m);
  return m;
}
