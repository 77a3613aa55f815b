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

#define SMLA_FN(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {SMLA_FN(decode_fp4), SMLA_FN(decode_fused_fp4), SMLA_FN(decode_window),
                          SMLA_FN(step_maps),  SMLA_FN(cache_write),      SMLA_FN(cache_gather),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_smla_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__smla_torch() { return PyModule_Create(&kModule); }
