// Compiled part of the Python binding for the serving step's calls: checks
// the tensors (type, device, layout, shapes) and passes their addresses and
// the stream to the C ABI.
//
// A decode step's small calls run 3-15 us on the GPU; the same checks and a
// ctypes call with up to 22 arguments took 10-25 us on the host (GB300's
// Grace CPU), so the host set the step's time.  Here a tensor's check is a
// few loads.  Every function takes its arguments by position and returns the
// library's status; a tensor that does not fit raises TypeError (its type)
// or ValueError (anything else).  No C++ exception leaves a function.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/smla.h"

namespace {

// Raised after a Python error has been set.
struct PyError {};

[[noreturn]] void refuse(PyObject* type, const char* format, const char* name, const char* more = "") {
  PyErr_Format(type, format, name, more);
  throw PyError{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

void need_dtype(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s", name, c10::toString(type));
}

// A contiguous tensor of a type, on a device.
const at::Tensor& need(PyObject* o, const char* name, at::ScalarType type, at::Device dev) {
  const at::Tensor& t = tensor(o, name);
  need_dtype(t, name, type);
  if (t.device() != dev) refuse(PyExc_ValueError, "%s is on another device than the other tensors", name);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}

const at::Tensor& vec(PyObject* o, const char* name, at::ScalarType type, at::Device dev, int64_t n) {
  const at::Tensor& t = need(o, name, type, dev);
  if (t.dim() != 1 || (n >= 0 && t.size(0) != n))
    refuse(PyExc_ValueError, "%s must be 1-D, with one entry for each of its kind", name);
  return t;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}

int32_t i32(PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "an integer argument does not fit 32 bits");
    throw PyError{};
  }
  return int32_t(v);
}

int32_t size32(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(PyExc_ValueError, "%s has too many entries", name);
  return int32_t(v);
}

float f32(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError{};
  return float(v);
}

template <class T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// Runs `call(stream)` on the tensors' device and the given or current stream.
template <class F>
PyObject* launch(at::Device dev, PyObject* stream, F&& call) {
  if (!dev.is_cuda()) {
    PyErr_SetString(PyExc_ValueError, "tensors must be on a CUDA device");
    throw PyError{};
  }
  void* s = nullptr;
  if (stream != Py_None) {
    PyObject* v = PyObject_GetAttrString(stream, "cuda_stream");
    if (!v) throw PyError{};
    s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!s && PyErr_Occurred()) throw PyError{};
  }
  const c10::cuda::CUDAGuard guard(dev);
  if (stream == Py_None) s = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  smla_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = call(s);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const PyError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// A packed cache: its format by its rows' bytes.
int32_t cache_format(const at::Tensor& kv, const char* name, at::Device dev) {
  need_dtype(kv, name, at::kByte);
  const int64_t row = kv.dim() == 2 ? kv.size(1) : 0;
  if (kv.device() != dev || (row != SMLA_ROW_BYTES && row != SMLA_FP4_ROW_BYTES) || !kv.is_contiguous())
    refuse(PyExc_ValueError, "%s must be a contiguous uint8 [num_slots, 656 or 416] tensor on the other tensors' device", name);
  return row == SMLA_ROW_BYTES ? SMLA_CACHE_FP8 : SMLA_CACHE_FP4;
}

struct Table {
  const int32_t* data;
  int64_t rows, stride;
  int32_t width;
};

// A block table with contiguous rows; width: its meaningful columns (None:
// all).  A one-row table's stride means nothing and may be anything.
Table block_table(const at::Tensor& t, const char* name, at::Device dev, PyObject* width) {
  if (t.scalar_type() != at::kInt || t.device() != dev || t.dim() != 2 ||
      (t.stride(1) != 1 && t.size(1) > 1))
    refuse(PyExc_ValueError, "%s must be 2-D int32 with contiguous rows", name);
  Table r{ptr<int32_t>(t), t.size(0), t.size(0) > 1 ? t.stride(0) : t.size(1),
          width == Py_None ? size32(t.size(1), name) : i32(width)};
  if (r.width > t.size(1)) refuse(PyExc_ValueError, "%s has fewer columns than its width", name);
  return r;
}

// The D shards' pools and tables (None where not used).
struct Pools {
  int32_t D = 0, format = -1;
  int64_t rows = INT64_MAX;  // of the smallest table
  const uint8_t* kv[SMLA_MAX_DCP] = {};
  int64_t slots[SMLA_MAX_DCP] = {};
  const int32_t* bt[SMLA_MAX_DCP] = {};
  int64_t stride[SMLA_MAX_DCP] = {};
  int32_t width[SMLA_MAX_DCP] = {};
};

struct Seq {  // a list or tuple, kept for as long as its items are read
  PyObject* fast;
  Seq(PyObject* o, const char* message) : fast(PySequence_Fast(o, message)) {
    if (!fast) throw PyError{};
  }
  ~Seq() { Py_DECREF(fast); }
  Seq(const Seq&) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

Pools pools_of(PyObject* kv_caches, PyObject* block_tables, PyObject* widths, at::Device dev,
               int32_t rank) {
  const Seq kvs(kv_caches, "kv_caches must be a sequence");
  const Seq bts(block_tables, "block_tables must be a sequence");
  const bool given = widths != Py_None;
  const Seq ws(given ? widths : kv_caches, "bt_widths must be a sequence");
  if (kvs.size() < 1 || kvs.size() != bts.size() || ws.size() != kvs.size())
    refuse(PyExc_ValueError, "need one block table%s per KV pool (>= 1)", given ? " and width" : "");
  if (kvs.size() > SMLA_MAX_DCP) refuse(PyExc_ValueError, "too many %s", "kv_caches");
  Pools p;
  p.D = int32_t(kvs.size());
  if (rank < -1 || rank >= p.D) refuse(PyExc_ValueError, "%s must be -1 or one of the pools", "rank");
  for (int32_t d = 0; d < p.D; ++d) {
    if (rank >= 0 && d != rank) continue;
    const at::Tensor& kv = tensor(kvs[d], "kv_caches[d]");
    const int32_t f = cache_format(kv, "kv_caches[d]", dev);
    if (p.format >= 0 && f != p.format) refuse(PyExc_ValueError, "%s must share one row format", "kv_caches");
    p.format = f;
    const Table t =
        block_table(tensor(bts[d], "block_tables[d]"), "block_tables[d]", dev, given ? ws[d] : Py_None);
    p.kv[d] = ptr<uint8_t>(kv);
    p.slots[d] = kv.size(0);
    p.bt[d] = t.data;
    p.stride[d] = t.stride;
    p.width[d] = t.width;
    p.rows = t.rows < p.rows ? t.rows : p.rows;
  }
  return p;
}

// q [T, H, 576], its outputs, and the optional workspace.
struct Query {
  at::Device dev{at::kCPU};
  int32_t T, H;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  void* ws = nullptr;
  size_t ws_bytes = 0;
};

Query query_of(PyObject* q_, PyObject* out_, PyObject* lse_, PyObject* ws_) {
  const at::Tensor& q = tensor(q_, "q");
  Query r;
  r.dev = q.device();
  need(q_, "q", at::kBFloat16, r.dev);
  if (q.dim() != 3 || q.size(2) != SMLA_QK_DIM) refuse(PyExc_ValueError, "%s must be [T, H, 576]", "q");
  r.T = size32(q.size(0), "q");
  r.H = size32(q.size(1), "q");
  const at::Tensor& out = need(out_, "out", at::kBFloat16, r.dev);
  const at::Tensor& lse = need(lse_, "lse", at::kFloat, r.dev);
  if (out.dim() != 3 || out.size(0) != r.T || out.size(1) != r.H || out.size(2) != SMLA_V_DIM)
    refuse(PyExc_ValueError, "%s must be [T, H, 512]", "out");
  if (lse.dim() != 2 || lse.size(0) != r.T || lse.size(1) != r.H)
    refuse(PyExc_ValueError, "%s must be [T, H]", "lse");
  r.q = ptr<uint16_t>(q);
  r.out = ptr<uint16_t>(out);
  r.lse = ptr<float>(lse);
  if (ws_ != Py_None) {
    const at::Tensor& ws = need(ws_, "workspace", at::kByte, r.dev);
    r.ws = ws.data_ptr();
    r.ws_bytes = size_t(ws.numel());
  }
  return r;
}

// ids [T, K] of a row's entries.
struct Entries {
  const int32_t* data;
  int32_t K;
};

Entries entries(PyObject* o, const char* name, const Query& q) {
  const at::Tensor& t = need(o, name, at::kInt, q.dev);
  if (t.dim() != 2 || t.size(0) != q.T) refuse(PyExc_ValueError, "%s must be [T, K]", name);
  return {ptr<int32_t>(t), size32(t.size(1), name)};
}

// (q, kv_cache, local_slots, sm_scale, out, lse, workspace, stream)
PyObject* decode_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Query q = query_of(a[0], a[4], a[5], a[6]);
    const at::Tensor& kv = tensor(a[1], "kv_cache");
    if (cache_format(kv, "kv_cache", q.dev) != SMLA_CACHE_FP4)
      refuse(PyExc_ValueError, "%s must be [num_slots, 416]", "kv_cache");
    const Entries slots = entries(a[2], "local_slots", q);
    const float scale = f32(a[3]);
    return launch(q.dev, a[7], [&](void* s) {
      return smla_sparse_mla_decode_fp4(q.q, ptr<uint8_t>(kv), kv.size(0), slots.data, q.T, q.H, slots.K,
                                        scale, q.out, q.lse, q.ws, q.ws_bytes, s);
    });
  });
}

// (q, req_id, topk, kv_caches, block_tables, block_size, sm_scale, interleave,
//  bt_widths, out, lse, workspace, stream)
PyObject* decode_fused_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Query q = query_of(a[0], a[9], a[10], a[11]);
    const at::Tensor& req = vec(a[1], "req_id_per_token", at::kInt, q.dev, q.T);
    const Entries topk = entries(a[2], "topk_global", q);
    const Pools p = pools_of(a[3], a[4], a[8], q.dev, -1);
    if (p.format != SMLA_CACHE_FP4) refuse(PyExc_ValueError, "%s must be [num_slots, 416]", "kv_caches[d]");
    const int32_t bs = i32(a[5]), I = i32(a[7]), reqs = size32(p.rows, "block_tables");
    const float scale = f32(a[6]);
    return launch(q.dev, a[12], [&](void* s) {
      return smla_dcp_sparse_mla_decode_fused_fp4(
          q.q, q.T, q.H, topk.K, scale, ptr<int32_t>(req), topk.data, reqs, p.D, bs, I, p.kv, p.slots,
          p.bt, p.stride, p.width, q.out, q.lse, q.ws, q.ws_bytes, s);
    });
  });
}

// (q, ctx_lens, max_ctx, S, window, sinks, kv_caches, block_tables, block_size,
//  sm_scale, rank, interleave, bt_widths, out, lse, workspace, stream)
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&] {
    const Query q = query_of(a[0], a[13], a[14], a[15]);
    const at::Tensor& ctx = vec(a[1], "ctx_lens", at::kInt, q.dev, -1);
    const int32_t max_ctx = i32(a[2]), S = i32(a[3]), window = i32(a[4]), sinks = i32(a[5]);
    const int32_t bs = i32(a[8]), rank = i32(a[10]), I = i32(a[11]);
    const float scale = f32(a[9]);
    if (q.T != ctx.size(0) * S) refuse(PyExc_ValueError, "%s must be [B*S, H, 576] with B = len(ctx_lens)", "q");
    const Pools p = pools_of(a[6], a[7], a[12], q.dev, rank);
    if (p.rows < ctx.size(0)) refuse(PyExc_ValueError, "%s need a row per request", "block_tables");
    return launch(q.dev, a[16], [&](void* s) {
      return smla_dcp_window_mla_decode(q.q, int32_t(ctx.size(0)), S, q.H, scale, ptr<int32_t>(ctx), max_ctx,
                                        window, sinks, p.D, rank, bs, I, p.format, p.kv, p.slots, p.bt,
                                        p.stride, p.width, q.out, q.lse, q.ws, q.ws_bytes, s);
    });
  });
}

// (ctx_lens, q_lens, free_blocks, block_table, T, D, rank, block_size,
//  interleave, bt_width, (row_start, req_id, positions, slots, local_lens,
//  blocks_taken), stream)
PyObject* step_maps(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const at::Device dev = tensor(a[0], "ctx_lens").device();
    const at::Tensor& ctx = vec(a[0], "ctx_lens", at::kInt, dev, -1);
    const int32_t B = size32(ctx.size(0), "ctx_lens"), T = i32(a[4]);
    const at::Tensor& ql = vec(a[1], "q_lens", at::kInt, dev, B);
    const at::Tensor& free = vec(a[2], "free_blocks", at::kInt, dev, -1);
    const Table t = block_table(tensor(a[3], "block_table"), "block_table", dev, a[9]);
    if (t.rows < B) refuse(PyExc_ValueError, "%s needs a row per request", "block_table");
    const Seq out(a[10], "out must be a sequence");
    if (out.size() != 6) refuse(PyExc_ValueError, "%s must hold six tensors", "out");
    const char* names[6] = {"row_start", "req_id", "positions", "slots", "local_lens", "blocks_taken"};
    const int64_t sizes[6] = {int64_t(B) + 1, T, T, T, B, 1};
    int32_t* o[6];
    for (int i = 0; i < 6; ++i) o[i] = ptr<int32_t>(vec(out[i], names[i], at::kInt, dev, sizes[i]));
    const int32_t D = i32(a[5]), rank = i32(a[6]), bs = i32(a[7]), I = i32(a[8]);
    const int32_t nf = size32(free.size(0), "free_blocks");
    return launch(dev, a[11], [&](void* s) {
      return smla_dcp_step_maps(ptr<int32_t>(ctx), ptr<int32_t>(ql), B, T, D, rank, bs, I, ptr<int32_t>(free),
                                nf, const_cast<int32_t*>(t.data), t.stride, t.width, o[0], o[1], o[2], o[3],
                                o[4], o[5], s);
    });
  });
}

// (kv, slots, kv_cache, gamma, eps, positions, cos_sin, rope_pairs, stream)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const at::Tensor& cache = tensor(a[2], "kv_cache");
    const at::Device dev = cache.device();
    const int32_t fmt = cache_format(cache, "kv_cache", dev);
    const at::Tensor& kv = tensor(a[0], "kv");
    if (kv.scalar_type() != at::kBFloat16 || kv.device() != dev || kv.dim() != 2 ||
        kv.size(1) != SMLA_QK_DIM || kv.stride(1) != 1)
      refuse(PyExc_ValueError, "%s must be a bf16 [T, 576] tensor with contiguous rows", "kv");
    const int32_t T = size32(kv.size(0), "kv");
    const at::Tensor& slots = vec(a[1], "slots", at::kInt, dev, T);
    const uint16_t* gamma =
        a[3] == Py_None ? nullptr : ptr<uint16_t>(vec(a[3], "gamma", at::kBFloat16, dev, SMLA_V_DIM));
    const int32_t* pos = nullptr;
    const float* cs = nullptr;
    int32_t P = 0;
    if (a[6] != Py_None) {
      if (a[5] == Py_None) refuse(PyExc_ValueError, "%s needs positions", "cos_sin");
      pos = ptr<int32_t>(vec(a[5], "positions", at::kInt, dev, T));
      const at::Tensor& t = need(a[6], "cos_sin", at::kFloat, dev);
      if (t.dim() != 2 || t.size(1) != 64) refuse(PyExc_ValueError, "%s must be [P, 64]", "cos_sin");
      cs = ptr<float>(t);
      P = size32(t.size(0), "cos_sin");
    }
    const float eps = f32(a[4]);
    const int32_t pairs = i32(a[7]);
    return launch(dev, a[8], [&](void* s) {
      return smla_mla_cache_write(ptr<uint16_t>(kv), T > 1 ? kv.stride(0) : SMLA_QK_DIM, T, gamma, eps, pos,
                                  cs, P, pairs, ptr<int32_t>(slots), fmt, ptr<uint8_t>(cache), cache.size(0),
                                  s);
    });
  });
}

// (kv_cache, slots, out, stream)
PyObject* cache_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    const at::Tensor& cache = tensor(a[0], "kv_cache");
    const at::Device dev = cache.device();
    const int32_t fmt = cache_format(cache, "kv_cache", dev);
    const at::Tensor& slots = vec(a[1], "slots", at::kInt, dev, -1);
    const int32_t N = size32(slots.size(0), "slots");
    const at::Tensor& out = tensor(a[2], "out");
    const bool fp32 = out.scalar_type() == at::kFloat;
    if ((!fp32 && out.scalar_type() != at::kBFloat16) || out.device() != dev || out.dim() != 2 ||
        out.size(0) != N || out.size(1) != SMLA_QK_DIM || out.stride(1) != 1)
      refuse(PyExc_ValueError, "%s must be a bf16 or fp32 [N, 576] tensor with contiguous rows", "out");
    return launch(dev, a[3], [&](void* s) {
      return smla_mla_cache_gather(ptr<uint8_t>(cache), cache.size(0), fmt, ptr<int32_t>(slots), N,
                                   out.data_ptr(), N > 1 ? out.stride(0) : SMLA_QK_DIM, fp32, s);
    });
  });
}

// (parents, row_start, prefix_lens, max_nodes, (masks, positions), stream)
PyObject* tree_maps(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const at::Device dev = tensor(a[0], "parents").device();
    const at::Tensor& parents = vec(a[0], "parents", at::kInt, dev, -1);
    const int32_t T = size32(parents.size(0), "parents");
    const at::Tensor& prefix = vec(a[2], "prefix_lens", at::kInt, dev, -1);
    const int32_t B = size32(prefix.size(0), "prefix_lens"), nodes = i32(a[3]);
    const at::Tensor& starts = vec(a[1], "row_start", at::kInt, dev, int64_t(B) + 1);
    const Seq out(a[4], "out must be a sequence");
    if (out.size() != 2) refuse(PyExc_ValueError, "%s must hold two tensors", "out");
    const at::Tensor& masks = need(out[0], "masks", at::kLong, dev);
    if (masks.dim() != 2 || masks.size(0) != T || masks.size(1) != (int64_t(nodes) + 63) / 64)
      refuse(PyExc_ValueError, "%s must be [T, ceil(max_nodes / 64)]", "masks");
    const at::Tensor& pos = vec(out[1], "positions", at::kInt, dev, T);
    return launch(dev, a[5], [&](void* s) {
      return smla_tree_maps(ptr<int32_t>(parents), ptr<int32_t>(starts), ptr<int32_t>(prefix), B, T, nodes,
                            ptr<uint64_t>(masks), ptr<int32_t>(pos), s);
    });
  });
}

// (q, row_start, prefix_lens, max_prefix, masks, max_nodes, draft_slots,
//  kv_caches, block_tables, block_size, sm_scale, rank, interleave, bt_widths,
//  out, lse, workspace, stream, window or None, sinks, positions (with a window))
PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 21, [&] {
    const Query q = query_of(a[0], a[14], a[15], a[16]);
    const at::Tensor& prefix = vec(a[2], "prefix_lens", at::kInt, q.dev, -1);
    const int32_t B = size32(prefix.size(0), "prefix_lens");
    const at::Tensor& starts = vec(a[1], "row_start", at::kInt, q.dev, int64_t(B) + 1);
    const int32_t max_prefix = i32(a[3]), nodes = i32(a[5]), bs = i32(a[9]), rank = i32(a[11]), I = i32(a[12]);
    const float scale = f32(a[10]);
    const at::Tensor& masks = need(a[4], "masks", at::kLong, q.dev);
    if (masks.dim() != 2 || masks.size(0) != q.T || masks.size(1) != (int64_t(nodes) + 63) / 64)
      refuse(PyExc_ValueError, "%s must be [T, ceil(max_nodes / 64)]", "masks");
    const Pools p = pools_of(a[7], a[8], a[13], q.dev, rank);
    if (p.rows < B) refuse(PyExc_ValueError, "%s need a row per request", "block_tables");
    const Seq drafts(a[6], "draft_slots must be a sequence");
    if (drafts.size() != p.D) refuse(PyExc_ValueError, "%s must have an entry for each pool", "draft_slots");
    const int32_t* slots[SMLA_MAX_DCP] = {};
    for (int32_t d = 0; d < p.D; ++d)
      if (rank < 0 || d == rank) slots[d] = ptr<int32_t>(vec(drafts[d], "draft_slots[d]", at::kInt, q.dev, q.T));
    if (a[18] != Py_None) {
      const int32_t window = i32(a[18]), sinks = i32(a[19]);
      const at::Tensor& positions = vec(a[20], "positions", at::kInt, q.dev, q.T);
      return launch(q.dev, a[17], [&](void* s) {
        return smla_dcp_tree_window_mla_decode(
            q.q, q.T, q.H, scale, ptr<int32_t>(starts), ptr<int32_t>(prefix), ptr<int32_t>(positions), B, max_prefix,
            ptr<uint64_t>(masks), nodes, window, sinks, slots, p.D, rank, bs, I, p.format, p.kv, p.slots, p.bt,
            p.stride, p.width, q.out, q.lse, q.ws, q.ws_bytes, s);
      });
    }
    return launch(q.dev, a[17], [&](void* s) {
      return smla_dcp_tree_mla_decode(q.q, q.T, q.H, scale, ptr<int32_t>(starts), ptr<int32_t>(prefix), B,
                                      max_prefix, ptr<uint64_t>(masks), nodes, slots, p.D, rank, bs, I, p.format,
                                      p.kv, p.slots, p.bt, p.stride, p.width, q.out, q.lse, q.ws, q.ws_bytes, s);
    });
  });
}

// (parents, tokens, targets, row_start, (accepted, rows, next_tokens), stream)
PyObject* tree_accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const at::Device dev = tensor(a[0], "parents").device();
    const at::Tensor& parents = vec(a[0], "parents", at::kInt, dev, -1);
    const int32_t T = size32(parents.size(0), "parents");
    const at::Tensor& tokens = vec(a[1], "tokens", at::kInt, dev, T);
    const at::Tensor& targets = vec(a[2], "targets", at::kInt, dev, T);
    const at::Tensor& starts = vec(a[3], "row_start", at::kInt, dev, -1);
    if (starts.size(0) < 1) refuse(PyExc_ValueError, "%s must be [B + 1]", "row_start");
    const int32_t B = size32(starts.size(0) - 1, "row_start");
    const Seq out(a[4], "out must be a sequence");
    if (out.size() != 3) refuse(PyExc_ValueError, "%s must hold three tensors", "out");
    const at::Tensor& accepted = vec(out[0], "accepted", at::kInt, dev, B);
    const at::Tensor& rows = vec(out[1], "rows", at::kInt, dev, T);
    const at::Tensor& next = vec(out[2], "next_tokens", at::kInt, dev, B);
    return launch(dev, a[5], [&](void* s) {
      return smla_tree_accept(ptr<int32_t>(parents), ptr<int32_t>(tokens), ptr<int32_t>(targets),
                              ptr<int32_t>(starts), B, T, ptr<int32_t>(accepted), ptr<int32_t>(rows),
                              ptr<int32_t>(next), s);
    });
  });
}

// (kv_cache, rows, src_slots, dst_slots, stream)
PyObject* cache_move(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    const at::Tensor& cache = tensor(a[0], "kv_cache");
    const at::Device dev = cache.device();
    const int32_t fmt = cache_format(cache, "kv_cache", dev);
    const at::Tensor& rows = vec(a[1], "rows", at::kInt, dev, -1);
    const int32_t N = size32(rows.size(0), "rows");
    const at::Tensor& src = vec(a[2], "src_slots", at::kInt, dev, -1);
    const int32_t T = size32(src.size(0), "src_slots");
    const at::Tensor& dst = vec(a[3], "dst_slots", at::kInt, dev, N);
    return launch(dev, a[4], [&](void* s) {
      return smla_mla_cache_move(fmt, ptr<uint8_t>(cache), cache.size(0), ptr<int32_t>(rows), N,
                                 ptr<int32_t>(src), T, ptr<int32_t>(dst), s);
    });
  });
}

// A matrix [M, K] or a batch of them [G, M, K]; strides of one-entry
// dimensions mean nothing.
struct Matrix {
  void* data;
  int64_t G, rows, cols, batch, row, col;
};

Matrix matrix(PyObject* o, const char* name, at::Device dev, int64_t dims) {
  const at::Tensor& t = tensor(o, name);
  if (t.device() != dev) refuse(PyExc_ValueError, "%s is on another device than the other tensors", name);
  if (t.dim() != dims) refuse(PyExc_ValueError, "%s must have as many dimensions as the other tensors", name);
  Matrix m{};
  m.data = t.data_ptr();
  m.G = dims == 3 ? t.size(0) : 1;
  m.rows = t.size(dims - 2);
  m.cols = t.size(dims - 1);
  m.col = m.cols > 1 ? t.stride(dims - 1) : 1;
  m.row = m.rows > 1 ? t.stride(dims - 2) : (m.cols * m.col + 15) / 16 * 16;
  m.batch = m.G > 1 ? t.stride(0) : (m.rows * m.row + 15) / 16 * 16;
  return m;
}

Matrix rows_of(PyObject* o, const char* name, at::ScalarType type, at::Device dev, int64_t dims) {
  need_dtype(tensor(o, name), name, type);
  const Matrix m = matrix(o, name, dev, dims);
  if (m.col != 1) refuse(PyExc_ValueError, "%s must have contiguous rows", name);
  return m;
}

Matrix scales_of(PyObject* o, const char* name, at::Device dev, int64_t dims, int64_t G, int64_t rows,
                 int64_t cols) {
  need_dtype(tensor(o, name), name, at::kFloat);
  const Matrix m = matrix(o, name, dev, dims);
  if (m.G != G || m.rows != rows || m.cols != cols)
    refuse(PyExc_ValueError, "%s must have one entry for each block of 128", name);
  return m;
}

int64_t dims_of(PyObject* o, const char* name) {
  const int64_t d = tensor(o, name).dim();
  if (d != 2 && d != 3) refuse(PyExc_ValueError, "%s must be a matrix or a batch of them", name);
  return d;
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// (x, codes, scales, stream)
PyObject* fp8_quantise(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    const at::Device dev = tensor(a[0], "x").device();
    const int64_t dims = dims_of(a[0], "x");
    const Matrix x = rows_of(a[0], "x", at::kBFloat16, dev, dims);
    const Matrix c = rows_of(a[1], "codes", at::kFloat8_e4m3fn, dev, dims);
    if (c.G != x.G || c.rows != x.rows || c.cols != x.cols) refuse(PyExc_ValueError, "%s must be x's shape", "codes");
    const Matrix s = scales_of(a[2], "scales", dev, dims, x.G, x.rows, blocks(x.cols));
    const int32_t G = size32(x.G, "x"), M = size32(x.rows, "x"), K = size32(x.cols, "x");
    return launch(dev, a[3], [&](void* st) {
      return smla_fp8_quantise(static_cast<uint16_t*>(x.data), x.batch, x.row, G, M, K,
                               static_cast<uint8_t*>(c.data), c.batch, c.row, static_cast<float*>(s.data),
                               s.batch, s.row, s.col, st);
    });
  });
}

// (a, a_scales, b, b_scales, out, stream)
PyObject* fp8_matmul(PyObject*, PyObject* const* p, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const at::Device dev = tensor(p[0], "a").device();
    const int64_t dims = dims_of(p[0], "a");
    const Matrix a = rows_of(p[0], "a", at::kFloat8_e4m3fn, dev, dims);
    const Matrix b = rows_of(p[2], "b", at::kFloat8_e4m3fn, dev, dims);
    if (b.G != a.G || b.cols != a.cols) refuse(PyExc_ValueError, "%s must have a's batches and columns", "b");
    const Matrix as = scales_of(p[1], "a_scales", dev, dims, a.G, a.rows, blocks(a.cols));
    const Matrix bs = scales_of(p[3], "b_scales", dev, dims, a.G, blocks(b.rows), blocks(a.cols));
    const bool fp32 = tensor(p[4], "out").scalar_type() == at::kFloat;
    const Matrix o = rows_of(p[4], "out", fp32 ? at::kFloat : at::kBFloat16, dev, dims);
    if (o.G != a.G || o.rows != a.rows || o.cols != b.rows)
      refuse(PyExc_ValueError, "%s must be [.., M, N]", "out");
    const int32_t G = size32(a.G, "a"), M = size32(a.rows, "a"), N = size32(b.rows, "b"),
                  K = size32(a.cols, "a");
    return launch(dev, p[5], [&](void* st) {
      return smla_fp8_matmul(static_cast<uint8_t*>(a.data), a.batch, a.row, static_cast<float*>(as.data),
                             as.batch, as.row, as.col, static_cast<uint8_t*>(b.data), b.batch, b.row,
                             static_cast<float*>(bs.data), bs.batch, bs.row, bs.col, G, M, N, K, o.data,
                             o.batch, o.row, fp32, st);
    });
  });
}

#define SMLA_FN(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {SMLA_FN(decode_fp4), SMLA_FN(decode_fused_fp4), SMLA_FN(decode_window),
                          SMLA_FN(step_maps),  SMLA_FN(cache_write),      SMLA_FN(cache_gather),
                          SMLA_FN(tree_maps),  SMLA_FN(tree_accept),      SMLA_FN(cache_move),
                          SMLA_FN(decode_tree), SMLA_FN(fp8_quantise),    SMLA_FN(fp8_matmul),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_smla_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__smla_torch() { return PyModule_Create(&kModule); }
