// step_binding.cpp -- Python binding of include/kvq_step.h: argument checks and
// marshalling, nothing else.  Part of fp4_binding.cpp's module.
#include "binding.h"

#include <dlfcn.h>

#include <vector>

#include "../../include/kvq_step.h"

namespace {

using namespace binding;

decltype(&kvq_rope_write) p_rope = nullptr;
decltype(&kvq_tree_attn) p_tree = nullptr;
decltype(&kvq_tree_commit) p_commit = nullptr;
decltype(&kvq_copy_pages) p_copy = nullptr;
decltype(&kvq_pages_init) p_init = nullptr;
decltype(&kvq_pages_alloc) p_alloc = nullptr;
decltype(&kvq_pages_free) p_free = nullptr;
decltype(&kvq_pages_fork) p_fork = nullptr;

void bound(const char* where) {
  if (!g_error || !p_rope) {
    PyErr_Format(PyExc_RuntimeError, "%s: the library is not bound", where);
    throw Raised();
  }
}

bool given(PyObject* o) { return o && o != Py_None; }

double real(const char* where, const char* name, PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    fail(where, std::string(name) + " must be a number", KVQ_ERR_ARG);
  }
  return v;
}

// Both caches [blocks][heads][16][head_dim], of the format's element size.
struct Paged {
  void *k, *v;
  int64_t blocks, heads, dh;
};
Paged paged(const char* where, Tensors& ts, PyObject* k, PyObject* v, int fmt) {
  const at::Tensor &a = ts.tensor("k_cache", k), &b = ts.tensor("v_cache", v);
  if (a.dim() != 4 || a.size(2) != kBlockSize)
    fail(where, "k_cache must have shape [num_blocks][Hkv][16][head_dim]", KVQ_ERR_SHAPE);
  if (b.sizes() != a.sizes())
    fail(where, "v_cache must have shape " + shape_text(a.sizes()) + ", got " + shape_text(b.sizes()), KVQ_ERR_SHAPE);
  if (fmt < KVQ_FMT_BF16 || fmt > KVQ_FMT_E5M2) fail(where, "unknown format", KVQ_ERR_ARG);
  for (const at::Tensor* t : {&a, &b}) {
    const char* name = t == &a ? "k_cache" : "v_cache";
    if (fmt == KVQ_FMT_BF16 ? t->scalar_type() != at::kBFloat16 : t->element_size() != 1)
      fail(where, std::string(name) + " must have the format's elements, got " + c10::toString(t->scalar_type()), KVQ_ERR_ARG);
    if (!t->is_contiguous()) fail(where, std::string(name) + " must be contiguous", KVQ_ERR_SHAPE);
  }
  return {a.data_ptr(), b.data_ptr(), a.size(0), a.size(1), a.size(3)};
}

// Scales, fp32; None is NULL.
float* scale(const char* where, Tensors& ts, const char* name, PyObject* o, int& n) {
  n = 0;
  if (!given(o)) return nullptr;
  int64_t numel;
  float* p = static_cast<float*>(ts.dense(name, o, at::kFloat, &numel));
  n = narrow(where, "scales", numel);
  return p;
}

int32_t* ints(Tensors& ts, const char* name, PyObject* o, at::IntArrayRef shape) {
  return static_cast<int32_t*>(ts.dense(name, o, at::kInt, shape));
}

// int32 [rows][columns]; rows < 0: any.
struct Table {
  int32_t* p;
  int64_t rows, columns;
};
Table table(const char* where, Tensors& ts, const char* name, PyObject* o, int64_t rows) {
  const at::Tensor& t = ts.tensor(name, o);
  Table r = {static_cast<int32_t*>(ts.dense(name, t, at::kInt)), 0, 0};
  if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows))
    fail(where, std::string(name) + " must have " + (rows < 0 ? "two dims" : std::to_string(rows) + " rows") + ", got shape " +
                    shape_text(t.sizes()), KVQ_ERR_SHAPE);
  r.rows = t.size(0);
  r.columns = t.size(1);
  return r;
}

PyObject* rope_write(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"q", "k", "v", "positions", "turns", "axis", "q_weight", "k_weight", "eps", "interleaved",
                                      "slot_mapping", "k_cache", "v_cache", "k_scale", "v_scale", "scale_granularity", "fmt",
                                      "q_out", "dev_status", "stream"};
  const char* where = "kvq_rope_write";
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 18, args, nargs, kw);
    Tensors ts(where);
    const at::Tensor &q = ts.tensor("q", a[0]), &k = ts.tensor("k", a[1]), &v = ts.tensor("v", a[2]);
    if (q.dim() != 3) fail(where, "q must have shape [num_tokens][Hq][head_dim]", KVQ_ERR_SHAPE);
    const int64_t n = q.size(0), hq = q.size(1), dh = q.size(2);
    const int fmt = int32(where, "fmt", a[16]);
    const Paged c = paged(where, ts, a[11], a[12], fmt);
    if (c.dh != dh) fail(where, "the caches and q must have the same head_dim", KVQ_ERR_SHAPE);
    int64_t sq, sk, sv, so;
    void *qp = ts.rows("q", q, n, hq, dh, sq), *kp = ts.rows("k", k, n, c.heads, dh, sk), *vp = ts.rows("v", v, n, c.heads, dh, sv);
    const at::Tensor& pos = ts.tensor("positions", a[3]);
    auto* pp = static_cast<int32_t*>(ts.dense("positions", pos, at::kInt));
    if ((pos.dim() != 1 && pos.dim() != 2) || pos.size(-1) != n)
      fail(where, "positions must have shape [num_axes][" + std::to_string(n) + "], got " + shape_text(pos.sizes()), KVQ_ERR_SHAPE);
    const int axes = narrow(where, "axes", pos.dim() == 2 ? pos.size(0) : 1);
    int64_t pairs;
    auto* turns = static_cast<int64_t*>(ts.dense("turns", a[4], at::kLong, &pairs));
    uint8_t* axis = given(a[5]) ? static_cast<uint8_t*>(ts.dense("axis", a[5], at::kByte, at::IntArrayRef(&pairs, 1))) : nullptr;
    void* w[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i)
      if (given(a[6 + i])) w[i] = ts.dense(names[6 + i], a[6 + i], at::kBFloat16, at::IntArrayRef(&dh, 1));
    const double eps = real(where, "eps", a[8]);
    const int inter = PyObject_IsTrue(a[9]);
    if (inter < 0) throw Raised();
    auto* slots = static_cast<int64_t*>(ts.dense("slot_mapping", a[10], at::kLong, at::IntArrayRef(&n, 1)));
    int nk, nv;
    float *ks = scale(where, ts, "k_scale", a[13], nk), *vs = scale(where, ts, "v_scale", a[14], nv);
    const int gran = int32(where, "scale_granularity", a[15]);
    void* op = ts.rows("q_out", ts.tensor("q_out", a[17]), n, hq, dh, so);
    uint32_t* st = ts.status(a[18]);
    const int h = narrow(where, "query heads", hq), g = narrow(where, "KV heads", c.heads), d = narrow(where, "head dims", dh);
    const int np = narrow(where, "pairs", pairs);
    kvq_stream_t stream = ts.stream(a[19]);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = p_rope(qp, sq, kp, sk, vp, sv, n, h, g, d, pp, axes, turns, axis, np, inter, w[0], w[1], static_cast<float>(eps), slots,
               c.k, c.v, c.blocks, kBlockSize, ks, nk, vs, nv, gran, fmt, op, so, st, stream);
    Py_END_ALLOW_THREADS
    return result(where, r);
  });
}

PyObject* tree_attn(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"q", "cu_q_lens", "parents", "k_cache", "v_cache", "block_tables", "seq_lens", "k_scale",
                                      "v_scale", "scale_granularity", "fmt", "sliding_window", "workspace", "out", "dev_status",
                                      "stream", "q_scale", "flags"};
  const char* where = "kvq_tree_attn";
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 14, args, nargs, kw);
    Tensors ts(where);
    const at::Tensor& q = ts.tensor("q", a[0]);
    void* qp = ts.dense("q", q, at::kBFloat16);
    if (q.dim() != 3) fail(where, "q must have shape [num_q_tokens][Hq][head_dim]", KVQ_ERR_SHAPE);
    const int64_t n = q.size(0);
    const int fmt = int32(where, "fmt", a[10]);
    const Paged c = paged(where, ts, a[3], a[4], fmt);
    if (c.dh != q.size(2)) fail(where, "the caches and q must have the same head_dim", KVQ_ERR_SHAPE);
    const Table bt = table(where, ts, "block_tables", a[5], -1);
    const int64_t B1 = bt.rows + 1;
    int32_t *lens = ints(ts, "seq_lens", a[6], at::IntArrayRef(&bt.rows, 1)), *cu = ints(ts, "cu_q_lens", a[1], at::IntArrayRef(&B1, 1));
    int32_t* parents = given(a[2]) ? ints(ts, "parents", a[2], at::IntArrayRef(&n, 1)) : nullptr;
    int nq, nk, nv;
    float *ks = scale(where, ts, "k_scale", a[7], nk), *vs = scale(where, ts, "v_scale", a[8], nv);
    float* qs = scale(where, ts, "q_scale", a[16], nq);
    const int gran = int32(where, "scale_granularity", a[9]), window = int32(where, "sliding_window", a[11]);
    int64_t ws_bytes;
    void* ws = ts.dense("workspace", a[12], at::kByte, &ws_bytes);
    void* out = ts.dense("out", a[13], at::kBFloat16, q.sizes());
    uint32_t* st = ts.status(a[14]);
    const int flags = a[17] ? int32(where, "flags", a[17]) : 0;
    const int hq = narrow(where, "query heads", q.size(1)), h = narrow(where, "KV heads", c.heads), d = narrow(where, "head dims", c.dh);
    const int B = narrow(where, "sequences", bt.rows), mb = narrow(where, "blocks per sequence", bt.columns);
    kvq_stream_t stream = ts.stream(a[15]);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = p_tree(qp, cu, n, parents, c.k, c.v, bt.p, mb, lens, B, hq, h, d, c.blocks, kBlockSize, qs, nq, ks, nk, vs, nv, gran, fmt,
               window, static_cast<unsigned>(flags), ws, static_cast<size_t>(ws_bytes), out, st, stream);
    Py_END_ALLOW_THREADS
    return result(where, r);
  });
}

// A sequence of cache tensors, all of the same blocks and heads; at least one.
struct Rows {
  std::vector<kvq_rows> c;
  int64_t blocks = 0, heads = 0;
};
Rows rows_of(const char* where, Tensors& ts, PyObject* list) {
  PyObject* seq = PySequence_Fast(list, "caches must be a sequence of tensors");
  if (!seq) throw Raised();
  struct Hold {
    PyObject* o;
    ~Hold() { Py_DECREF(o); }
  } hold = {seq};
  Rows r;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  if (n == 0) fail(where, "caches must not be empty", KVQ_ERR_ARG);
  if (n > (1 << 20)) fail(where, "too many caches", KVQ_ERR_UNSUPPORTED);
  r.c.reserve(n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor& t = ts.tensor("caches", PySequence_Fast_GET_ITEM(seq, i));
    if (!t.is_contiguous()) fail(where, "a cache must be contiguous", KVQ_ERR_SHAPE);
    kvq_rows c = {t.data_ptr(), 0, 0};
    const bool fp8 = t.element_size() == 1, bf16 = t.scalar_type() == at::kBFloat16;
    if (t.dim() == 4 && t.size(2) == kBlockSize && (fp8 || bf16) && (t.size(3) == 64 || t.size(3) == 128)) {
      c.row_bytes = static_cast<int32_t>(t.size(3) * t.element_size());
    } else if (t.dim() == 3 && t.scalar_type() == at::kFloat && t.size(2) == kBlockSize) {
      c.row_bytes = 4;
    } else if (t.dim() == 3 && t.scalar_type() == at::kByte && (t.size(2) == 9 * 64 || t.size(2) == 9 * 128)) {
      c.row_bytes = static_cast<int32_t>(t.size(2) / 18);
      c.sub_bytes = static_cast<int32_t>(t.size(2) / 144);
    } else {
      fail(where, "a cache must have shape [num_blocks][Hkv][16][head_dim] (FP8 or bf16), [num_blocks][Hkv][16] (fp32 scales) or "
                  "[num_blocks][Hkv][9 * head_dim] (4 bits), got " + shape_text(t.sizes()) + " of " + c10::toString(t.scalar_type()),
           KVQ_ERR_SHAPE);
    }
    if (i == 0) {
      r.blocks = t.size(0);
      r.heads = t.size(1);
    } else if (t.size(0) != r.blocks || t.size(1) != r.heads) {
      fail(where, "the caches must hold the same blocks and KV heads", KVQ_ERR_SHAPE);
    }
    r.c.push_back(c);
  }
  return r;
}

PyObject* tree_commit(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"caches", "cu_q_lens", "block_tables", "seq_lens", "accepted", "num_accepted", "new_lens",
                                      "dev_status", "stream"};
  const char* where = "kvq_tree_commit";
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 7, args, nargs, kw);
    Tensors ts(where);
    const Rows c = rows_of(where, ts, a[0]);
    const Table bt = table(where, ts, "block_tables", a[2], -1), path = table(where, ts, "accepted", a[4], bt.rows);
    const int64_t B1 = bt.rows + 1;
    const at::IntArrayRef one(&bt.rows, 1);
    int32_t *cu = ints(ts, "cu_q_lens", a[1], at::IntArrayRef(&B1, 1)), *lens = ints(ts, "seq_lens", a[3], one);
    int32_t *taken = ints(ts, "num_accepted", a[5], one), *out = ints(ts, "new_lens", a[6], one);
    uint32_t* st = ts.status(a[7]);
    const int B = narrow(where, "sequences", bt.rows), mb = narrow(where, "blocks per sequence", bt.columns);
    const int most = narrow(where, "places of a path", path.columns), h = narrow(where, "KV heads", c.heads);
    kvq_stream_t stream = ts.stream(a[8]);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = p_commit(c.c.data(), static_cast<int>(c.c.size()), c.blocks, h, kBlockSize, cu, bt.p, mb, lens, B, path.p, most, taken, out,
                 st, stream);
    Py_END_ALLOW_THREADS
    return result(where, r);
  });
}

PyObject* copy_pages(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"caches", "copies", "dev_status", "stream"};
  const char* where = "kvq_copy_pages";
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 2, args, nargs, kw);
    Tensors ts(where);
    const Rows c = rows_of(where, ts, a[0]);
    const Table t = table(where, ts, "copies", a[1], -1);
    if (t.columns != 2) fail(where, "copies must have shape [num_copies][2]", KVQ_ERR_SHAPE);
    uint32_t* st = ts.status(a[2]);
    const int n = narrow(where, "copies", t.rows), h = narrow(where, "KV heads", c.heads);
    kvq_stream_t stream = ts.stream(a[3]);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = p_copy(c.c.data(), static_cast<int>(c.c.size()), c.blocks, h, kBlockSize, t.p, n, st, stream);
    Py_END_ALLOW_THREADS
    return result(where, r);
  });
}

// A pool's words, and how many pages it is of.
int32_t* pool_of(const char* where, Tensors& ts, PyObject* o, int64_t& blocks) {
  int64_t n;
  auto* p = static_cast<int32_t*>(ts.dense("pool", o, at::kInt, &n));
  blocks = (n - KVQ_POOL_HEADER) * 32 / 33;
  while (blocks > 0 && KVQ_POOL_WORDS(blocks) > n) --blocks;
  if (blocks <= 0 || KVQ_POOL_WORDS(blocks) != n) fail(where, "pool has no pool's size: see new_page_pool", KVQ_ERR_SHAPE);
  return p;
}

PyObject* pages_init(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"pool", "stream"};
  const char* where = "kvq_pages_init";
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 1, args, nargs, kw);
    Tensors ts(where);
    int64_t blocks;
    int32_t* pool = pool_of(where, ts, a[0], blocks);
    kvq_stream_t stream = ts.stream(a[1]);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = p_init(pool, blocks, stream);
    Py_END_ALLOW_THREADS
    return result(where, r);
  });
}

PyObject* pages_call(const char* where, const decltype(&kvq_pages_alloc)& f, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"pool", "block_tables", "old_lens", "new_lens", "dev_status", "stream"};
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 4, args, nargs, kw);
    Tensors ts(where);
    int64_t blocks;
    int32_t* pool = pool_of(where, ts, a[0], blocks);
    const Table bt = table(where, ts, "block_tables", a[1], -1);
    const at::IntArrayRef one(&bt.rows, 1);
    int32_t *old_lens = ints(ts, "old_lens", a[2], one), *new_lens = ints(ts, "new_lens", a[3], one);
    uint32_t* st = ts.status(a[4]);
    const int B = narrow(where, "sequences", bt.rows), mb = narrow(where, "blocks per sequence", bt.columns);
    kvq_stream_t stream = ts.stream(a[5]);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = f(pool, blocks, bt.p, mb, old_lens, new_lens, B, st, stream);
    Py_END_ALLOW_THREADS
    return result(where, r);
  });
}

PyObject* pages_alloc(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  return pages_call("kvq_pages_alloc", p_alloc, args, nargs, kw);
}
PyObject* pages_free(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  return pages_call("kvq_pages_free", p_free, args, nargs, kw);
}

PyObject* pages_fork(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"pool", "block_tables", "seq_lens", "parents", "out_tables", "out_lens", "copies",
                                      "dev_status", "stream"};
  const char* where = "kvq_pages_fork";
  return guarded([&]() -> PyObject* {
    bound(where);
    auto a = take(where, names, 7, args, nargs, kw);
    Tensors ts(where);
    int64_t blocks;
    int32_t* pool = pool_of(where, ts, a[0], blocks);
    const Table src = table(where, ts, "block_tables", a[1], -1), out = table(where, ts, "out_tables", a[4], -1);
    if (out.columns != src.columns) fail(where, "out_tables and block_tables must have the same columns", KVQ_ERR_SHAPE);
    const at::IntArrayRef one(&out.rows, 1);
    const int64_t pair[2] = {out.rows, 2};
    int32_t *lens = ints(ts, "seq_lens", a[2], at::IntArrayRef(&src.rows, 1)), *parents = ints(ts, "parents", a[3], one);
    int32_t *out_lens = ints(ts, "out_lens", a[5], one), *copies = ints(ts, "copies", a[6], at::IntArrayRef(pair, 2));
    uint32_t* st = ts.status(a[7]);
    const int ns = narrow(where, "sequences", src.rows), no = narrow(where, "sequences", out.rows);
    const int mb = narrow(where, "blocks per sequence", src.columns);
    kvq_stream_t stream = ts.stream(a[8]);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = p_fork(pool, blocks, src.p, lens, ns, mb, parents, no, out.p, out_lens, copies, st, stream);
    Py_END_ALLOW_THREADS
    return result(where, r);
  });
}

}  // namespace

namespace binding {

bool step_bind(void* handle, const char* path) {
  bool all = true;
  auto sym = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(handle, name));
    all = all && f;
  };
  sym(p_tree, "kvq_tree_attn");
  sym(p_commit, "kvq_tree_commit");
  sym(p_copy, "kvq_copy_pages");
  sym(p_init, "kvq_pages_init");
  sym(p_alloc, "kvq_pages_alloc");
  sym(p_free, "kvq_pages_free");
  sym(p_fork, "kvq_pages_fork");
  sym(p_rope, "kvq_rope_write");
  if (!all) {
    p_rope = nullptr;
    PyErr_Format(PyExc_ImportError, "%s lacks an entry point of kvq_step.h", path);
  }
  return all;
}

#define KVQ_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef step_methods[] = {
    {"kvq_rope_write", KVQ_FAST(rope_write), METH_FASTCALL | METH_KEYWORDS,
     "kvq_rope_write(q, k, v, positions, turns, axis, q_weight, k_weight, eps, interleaved, slot_mapping, k_cache, v_cache, "
     "k_scale, v_scale, scale_granularity, fmt, q_out, dev_status=None, stream=None)\n\nNorm (with a weight of [head_dim], None: "
     "none) and rotate q and k bf16 [N][heads][dh], write q to q_out and quantize k and v into their slots.  positions int32 [N] "
     "or [axes][N]; turns int64 [pairs] (rope_turns); axis uint8 [pairs] or None.  q_out may be q."},
    {"kvq_tree_attn", KVQ_FAST(tree_attn), METH_FASTCALL | METH_KEYWORDS,
     "kvq_tree_attn(q, cu_q_lens, parents, k_cache, v_cache, block_tables, seq_lens, k_scale, v_scale, scale_granularity, fmt, "
     "sliding_window, workspace, out, dev_status=None, stream=None, q_scale=None, flags=0)\n\nAttention of trees of drafted tokens, "
     "each sequence's last ones: q bf16 [total_q][Hq][dh], cu_q_lens int32 [B + 1], parents int32 [total_q] (a node of the same "
     "tree before it, -1: none; None: drafts in a row).  A node sees the tokens before the tree, its ancestors and itself."},
    {"kvq_tree_commit", KVQ_FAST(tree_commit), METH_FASTCALL | METH_KEYWORDS,
     "kvq_tree_commit(caches, cu_q_lens, block_tables, seq_lens, accepted, num_accepted, new_lens, dev_status=None, stream=None)"
     "\n\nMove the rows of each sequence's accepted path (int32 [B][max_path] nodes, the first num_accepted[b] of them) together "
     "behind the tokens before its tree, in every cache; new_lens int32 [B] gets the lengths."},
    {"kvq_copy_pages", KVQ_FAST(copy_pages), METH_FASTCALL | METH_KEYWORDS,
     "kvq_copy_pages(caches, copies, dev_status=None, stream=None)\n\nCopy page copies[i][0] onto copies[i][1] (int32 [n][2], "
     "negative: nothing) in every cache."},
    {"kvq_pages_init", KVQ_FAST(pages_init), METH_FASTCALL | METH_KEYWORDS,
     "kvq_pages_init(pool, stream=None)\n\nEvery page of the pool free."},
    {"kvq_pages_alloc", KVQ_FAST(pages_alloc), METH_FASTCALL | METH_KEYWORDS,
     "kvq_pages_alloc(pool, block_tables, old_lens, new_lens, dev_status=None, stream=None)\n\nTake pages for the tokens from "
     "old_lens to new_lens (int32 [B]), the lowest free ones, sequence by sequence; all or none of them."},
    {"kvq_pages_free", KVQ_FAST(pages_free), METH_FASTCALL | METH_KEYWORDS,
     "kvq_pages_free(pool, block_tables, old_lens, new_lens, dev_status=None, stream=None)\n\nGive back the pages past new_lens."},
    {"kvq_pages_fork", KVQ_FAST(pages_fork), METH_FASTCALL | METH_KEYWORDS,
     "kvq_pages_fork(pool, block_tables, seq_lens, parents, out_tables, out_lens, copies, dev_status=None, stream=None)\n\nRow b of "
     "out_tables goes on from row parents[b]: full pages are shared, a last one that is not full is to be copied as copies[b] says "
     "(kvq_copy_pages)."},
    {nullptr, nullptr, 0, nullptr}};

}  // namespace binding
