// Torch tensors to the paged cache's entry points, without Python's share of the
// work: a decode step makes these calls once a layer, and reading some forty
// tensor properties through Python costs more (5 to 13 us a call) than the
// launch (2 us).  Each function checks in one pass that its tensors are what
// the call takes as they stand and returns None where they are not; the Python
// functions of the same name then name the fault, or handle what is legal but
// unusual (strides of dims of one entry, another device than the current one).
// Otherwise the result is the entry point's status, or the outputs.
#include <Python.h>

#include <vector>

#include <ATen/Context.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "smla.h"

namespace {

constexpr int64_t kDim = 512;
constexpr int64_t kInt32Max = 0x7fffffff;

struct Unusual {};                          // not plain: for the Python functions

void need(bool ok) {
  if (!ok) throw Unusual{};
}

// The call's tensors: all on one CUDA device, the current one.
struct Call {
  int device = -1;

  const at::Tensor& tensor(PyObject* o) {
    need(THPVariable_Check(o));
    const at::Tensor& t = THPVariable_Unpack(o);
    need(t.is_cuda() && t.layout() == c10::kStrided);
    if (device < 0) {
      device = t.get_device();
      need(device == c10::cuda::current_device());
    }
    need(t.get_device() == device);
    return t;
  }
  // An array that the kernels index: contiguous, of this type and at least this long; nullptr for None.
  void* array(PyObject* o, c10::ScalarType type, int64_t entries, bool optional) {
    if (optional && o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == type && t.is_contiguous() && t.numel() >= entries);
    return t.data_ptr();
  }
  void* words(PyObject* o, int64_t entries, bool optional = false) { return array(o, c10::kInt, entries, optional); }
  void* bytes(PyObject* o, size_t* n) {     // a workspace
    *n = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    need(t.is_contiguous());
    *n = t.nbytes();
    return t.data_ptr();
  }
  void* stream(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    need(PyLong_Check(o));
    void* s = PyLong_AsVoidPtr(o);
    if (s == nullptr && PyErr_Occurred()) {
      PyErr_Clear();
      throw Unusual{};
    }
    return s;
  }
};

int32_t int32(int64_t v) {
  need(v >= -kInt32Max - 1 && v <= kInt32Max);
  return (int32_t)v;
}

int32_t int32(PyObject* o) {
  need(PyLong_Check(o));
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  need(overflow == 0);
  return int32(v);
}

smla_cache cache(Call& call, PyObject* rows_o, PyObject* scales_o, PyObject* tables_o, PyObject* seq_lens, PyObject* cum) {
  const at::Tensor &rows = call.tensor(rows_o), &scales = call.tensor(scales_o), &tables = call.tensor(tables_o);
  need(rows.dim() == 3 && scales.dim() == 2 && tables.dim() == 2);
  const auto rs = rows.sizes(), rt = rows.strides(), ss = scales.sizes(), st = scales.strides(), ts = tables.sizes(),
             tt = tables.strides();
  need((rows.scalar_type() == c10::kFloat8_e4m3fn || rows.scalar_type() == c10::kByte) &&
       scales.scalar_type() == c10::kFloat && tables.scalar_type() == c10::kInt);
  need(rs[2] == kDim && rt[2] == 1 && st[1] == 1 && tt[1] == 1 && ss[0] == rs[0] && rs[0] > 0 && ss[1] > 0 && rs[1] > 0 &&
       rs[1] % ss[1] == 0 && rt[0] > 0 && rt[1] > 0 && st[0] >= ss[1] && ts[0] > 0 && ts[1] > 0 && tt[0] >= ts[1]);
  smla_cache c = {};
  c.rows = rows.data_ptr();
  c.row_stride = rs[1] > 1 ? rt[1] : kDim;
  c.page_stride = rs[0] > 1 ? rt[0] : 0;
  c.scales = static_cast<float*>(scales.data_ptr());
  c.scale_stride = rs[0] > 1 ? st[0] : ss[1];
  c.num_pages = rs[0];
  c.page_size = int32(rs[1]);
  c.block_rows = int32(rs[1] / ss[1]);
  c.block_tables = static_cast<const int32_t*>(tables.data_ptr());
  c.block_table_stride = ts[0] > 1 ? tt[0] : ts[1];
  c.max_pages = int32(ts[1]);
  c.batch = int32(ts[0]);
  c.seq_lens = static_cast<const int32_t*>(call.words(seq_lens, ts[0]));
  c.cum_seq_lens_q = static_cast<const int32_t*>(call.words(cum, ts[0] + 1, true));
  return c;
}

// A scale that is a number, or a float32 on the device.
void scale(Call& call, PyObject* o, float* value, const float** dev) {
  *value = 1.f;
  if (PyFloat_Check(o)) *value = (float)PyFloat_AS_DOUBLE(o);
  else *dev = static_cast<const float*>(call.array(o, c10::kFloat, 1, false));
}

// Runs f, which gives the result or throws; the entry point itself is called
// without the interpreter's lock (a launch may wait for room in the queue).
template <class F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd needed", given, wanted);
    return nullptr;
  }
  try {
    return f();
  } catch (...) {                           // not plain, or torch's own complaint, which the Python functions meet again
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

template <class F>
smla_status unlocked(F f) {
  smla_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f();
  Py_END_ALLOW_THREADS
  return s;
}

// A new output.  at::empty without its dispatch (1 us a tensor), but where that does
// more than allocate: it fills new memory where deterministic algorithms are asked
// for (calls leave the outputs of tokens of no request alone), and modes see it.
at::Tensor new_output(at::IntArrayRef sizes, c10::ScalarType type, c10::Device device) {
  const at::Context& context = at::globalContext();
  if ((context.deterministicAlgorithms() && context.deterministicFillUninitializedMemory()) ||
      c10::impl::TorchDispatchModeTLS::any_modes_set())
    return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
  return at::detail::empty_cuda(sizes, type, device, std::nullopt);
}

// What the two attention calls have alike: (q, rows, scales, block_tables, seq_lens, workspace, cum_seq_lens_q, sinks,
// then what the caller sets, then from a[at] on bmm1_scale, bmm2_scale, out, out_lse, error_word, stream) ->
// (out, out_lse), a status that is not 0, or None
template <class Args, class Set, class Run>
PyObject* attention(PyObject* const* a, int at, Set set, Run run) {
  Call call;
  Args w = {};
  const at::Tensor& q = call.tensor(a[0]);
  need(q.scalar_type() == c10::kBFloat16 && q.dim() == 3);
  const int64_t T = q.size(0), H = q.size(1);
  need(T > 0 && H > 0 && q.size(2) == kDim && q.stride(2) == 1 && (H == 1 || q.stride(1) == kDim) &&
       (T == 1 || q.stride(0) > 0));
  w.cache = cache(call, a[1], a[2], a[3], a[4], a[6]);
  w.workspace = call.bytes(a[5], &w.workspace_bytes);
  w.sinks = static_cast<const float*>(call.array(a[7], c10::kFloat, H, true));
  set(call, w);
  a += at;
  scale(call, a[0], &w.bmm1_scale, &w.bmm1_scale_dev);
  scale(call, a[1], &w.bmm2_scale, &w.bmm2_scale_dev);
  w.sum_q = int32(T);
  w.num_heads = int32(H);
  w.q = q.data_ptr();
  w.q_stride_token = T > 1 ? q.stride(0) : 0;
  w.error_word = static_cast<int32_t*>(call.words(a[4], 1, true));
  void* const stream = call.stream(a[5]);
  // (outputs of a call on another stream than the current one have to be that stream's memory)
  need((a[2] != Py_None && a[3] != Py_None) || stream == call.stream(Py_None));
  at::Tensor out, lse;                      // those that are not given
  if (a[2] == Py_None) {
    out = new_output({T, H, kDim}, c10::kBFloat16, q.device());
    w.out = out.data_ptr();
  } else {
    w.out = call.array(a[2], c10::kBFloat16, T * H * kDim, false);
    need(THPVariable_Unpack(a[2]).numel() == T * H * kDim);
  }
  if (a[3] == Py_None) {
    lse = new_output({T, H}, c10::kFloat, q.device());
    w.out_lse = static_cast<float*>(lse.data_ptr());
  } else {
    w.out_lse = static_cast<float*>(call.array(a[3], c10::kFloat, T * H, false));
    need(THPVariable_Unpack(a[3]).numel() == T * H);
  }
  const smla_status s = unlocked([&] { return run(&w, stream); });
  if (s != SMLA_OK) return PyLong_FromLong(s);
  PyObject* o = out.defined() ? THPVariable_Wrap(out) : Py_NewRef(a[2]);
  PyObject* l = lse.defined() ? THPVariable_Wrap(lse) : Py_NewRef(a[3]);
  PyObject* both = o != nullptr && l != nullptr ? PyTuple_Pack(2, o, l) : nullptr;
  Py_XDECREF(o);
  Py_XDECREF(l);
  return both;
}

// (.., window, first_tokens, num_splits, ..)
PyObject* window_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    return attention<smla_window_args>(
        a, 11,
        [&](Call&, smla_window_args& w) {
          w.window = int32(a[8]);
          w.first_tokens = int32(a[9]);
          w.num_splits = int32(a[10]);
        },
        smla_window_attention);
  });
}

// (.., group_starts, prefix_lens, ..)
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    return attention<smla_prefix_args>(
        a, 10,
        [&](Call& call, smla_prefix_args& w) {
          w.group_starts = static_cast<const int32_t*>(call.words(a[8], 1));
          w.num_groups = int32(THPVariable_Unpack(a[8]).numel() - 1);
          w.prefix_lens = static_cast<const int32_t*>(call.words(a[9], w.num_groups));
        },
        smla_prefix_attention);
  });
}

// (latent, rows, scales, block_tables, seq_lens, cum_seq_lens_q, error_word, stream) -> status or None
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    Call call;
    smla_append_args p = {};
    const at::Tensor& x = call.tensor(a[0]);
    need(x.scalar_type() == c10::kBFloat16 && x.dim() == 2 && x.size(0) > 0 && x.size(1) == kDim && x.stride(1) == 1 &&
         (x.size(0) == 1 || x.stride(0) > 0));
    p.cache = cache(call, a[1], a[2], a[3], a[4], a[5]);
    p.sum_q = int32(x.size(0));
    p.latent = x.data_ptr();
    p.latent_stride = x.size(0) > 1 ? x.stride(0) : kDim;
    p.error_word = static_cast<int32_t*>(call.words(a[6], 1, true));
    void* const stream = call.stream(a[7]);
    return PyLong_FromLong(unlocked([&] { return smla_cache_append(&p, stream); }));
  });
}

int32_t* table(Call& call, PyObject* o, int32_t* rows, int32_t* max_pages, int64_t* stride) {
  const at::Tensor& t = call.tensor(o);
  need(t.scalar_type() == c10::kInt && t.dim() == 2 && t.size(0) > 0 && t.size(1) > 0 && t.stride(1) == 1 &&
       t.stride(0) >= t.size(1));
  *rows = int32(t.size(0));
  *max_pages = int32(t.size(1));
  *stride = *rows > 1 ? t.stride(0) : *max_pages;
  return static_cast<int32_t*>(t.data_ptr());
}

smla_pages_args pages(Call& call, PyObject* tables_o, PyObject* refs, PyObject* lens, PyObject* page_size, PyObject* error) {
  smla_pages_args p = {};
  p.block_tables = table(call, tables_o, &p.rows, &p.max_pages, &p.block_table_stride);
  p.page_size = int32(page_size);
  p.ref_counts = static_cast<int32_t*>(call.words(refs, 1));
  p.num_pages = THPVariable_Unpack(refs).numel();
  p.lens = static_cast<const int32_t*>(call.words(lens, p.rows));
  p.error_word = static_cast<int32_t*>(call.words(error, 1, true));
  return p;
}

void moves_of(Call& call, PyObject* o, smla_pages_args* p) {
  need(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 3);
  p->move_src = static_cast<int32_t*>(call.words(PyTuple_GET_ITEM(o, 0), 0));
  p->move_capacity = THPVariable_Unpack(PyTuple_GET_ITEM(o, 0)).numel();
  p->move_dst = static_cast<int32_t*>(call.words(PyTuple_GET_ITEM(o, 1), p->move_capacity));
  p->move_count = static_cast<int32_t*>(call.words(PyTuple_GET_ITEM(o, 2), 1));
}

// (block_tables, ref_counts, lens, new_lens, workspace, page_size, moves, error_word, stream) -> status or None
PyObject* pages_resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Call call;
    smla_pages_args p = pages(call, a[0], a[1], a[2], a[5], a[7]);
    p.new_lens = static_cast<const int32_t*>(call.words(a[3], p.rows));
    p.workspace = call.bytes(a[4], &p.workspace_bytes);
    moves_of(call, a[6], &p);
    void* const stream = call.stream(a[8]);
    return PyLong_FromLong(unlocked([&] { return smla_pages_resize(&p, stream); }));
  });
}

// (block_tables, ref_counts, lens, parents, out_lens, page_size, error_word, stream) -> status or None
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    Call call;
    smla_pages_args p = pages(call, a[0], a[1], a[2], a[5], a[6]);
    p.parents = static_cast<const int32_t*>(call.words(a[3], p.rows));
    p.out_lens = static_cast<int32_t*>(call.words(a[4], p.rows));
    void* const stream = call.stream(a[7]);
    return PyLong_FromLong(unlocked([&] { return smla_pages_fork(&p, stream); }));
  });
}

// (block_tables, ref_counts, lens, parents, out_lens, workspace, page_size, error_word, stream) -> status or None
PyObject* pages_reorder(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Call call;
    smla_pages_args p = pages(call, a[0], a[1], a[2], a[6], a[7]);
    p.parents = static_cast<const int32_t*>(call.words(a[3], p.rows));
    p.out_lens = static_cast<int32_t*>(call.words(a[4], p.rows));
    p.workspace = call.bytes(a[5], &p.workspace_bytes);
    void* const stream = call.stream(a[8]);
    return PyLong_FromLong(unlocked([&] { return smla_pages_reorder(&p, stream); }));
  });
}

// (block_tables, lens, group_starts, prefix_lens, page_size, error_word, stream) -> status or None
PyObject* pages_shared_prefix(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Call call;
    smla_pages_args p = {};
    p.block_tables = table(call, a[0], &p.rows, &p.max_pages, &p.block_table_stride);
    p.lens = static_cast<const int32_t*>(call.words(a[1], p.rows));
    int32_t* const prefix = static_cast<int32_t*>(call.words(a[3], 1));
    const int32_t groups = int32(THPVariable_Unpack(a[3]).numel());
    const int32_t* const starts = static_cast<const int32_t*>(call.words(a[2], groups + 1));
    p.page_size = int32(a[4]);
    p.error_word = static_cast<int32_t*>(call.words(a[5], 1, true));
    void* const stream = call.stream(a[6]);
    return PyLong_FromLong(unlocked([&] { return smla_pages_shared_prefix(&p, starts, groups, prefix, stream); }));
  });
}

// (block_tables, ref_counts, lens, workspace, page_size, moves, error_word, stream) -> status or None
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    Call call;
    smla_pages_args p = pages(call, a[0], a[1], a[2], a[4], a[6]);
    p.workspace = call.bytes(a[3], &p.workspace_bytes);
    moves_of(call, a[5], &p);
    void* const stream = call.stream(a[7]);
    return PyLong_FromLong(unlocked([&] { return smla_pages_compact(&p, stream); }));
  });
}

// (pools, moves, error_word, stream) -> status or None
PyObject* pages_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    need(PyList_Check(a[0]) || PyTuple_Check(a[0]));
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[0]);
    need(count > 0);
    Call call;
    smla_pages_args p = {};
    moves_of(call, a[1], &p);
    std::vector<smla_pool> pool((size_t)count);
    int64_t num_pages = 0;
    for (Py_ssize_t i = 0; i < count; ++i) {
      const at::Tensor& t = call.tensor(PySequence_Fast_GET_ITEM(a[0], i));
      need(t.dim() > 0 && t.numel() > 0);
      if (i == 0) num_pages = t.size(0);
      need(t.size(0) == num_pages);
      int64_t page = 1;                     // entries of one, if they are contiguous
      for (int64_t d = t.dim() - 1; d > 0; --d) {
        need(t.size(d) == 1 || t.stride(d) == page);
        page *= t.size(d);
      }
      const int64_t size = (int64_t)t.element_size();
      pool[i].base = t.data_ptr();
      pool[i].page_bytes = page * size;
      pool[i].page_stride = (num_pages > 1 ? t.stride(0) : page) * size;
    }
    int32_t* const error = static_cast<int32_t*>(call.words(a[2], 1, true));
    void* const stream = call.stream(a[3]);
    const int32_t pools = int32((int64_t)count);
    return PyLong_FromLong(unlocked([&] {
      return smla_pages_copy(pool.data(), pools, num_pages, p.move_src, p.move_dst, p.move_count, p.move_capacity, error,
                             stream);
    }));
  });
}

// A tensor or a new one of this type and these sizes; its memory.
struct Output {
  at::Tensor fresh;
  PyObject* given = nullptr;
  void* data = nullptr;

  void set(Call& call, PyObject* o, c10::ScalarType type, at::IntArrayRef sizes, int64_t entries, const at::Tensor& like) {
    if (o != nullptr) {
      data = call.array(o, type, entries, false);
      given = o;
    } else {
      fresh = new_output(sizes, type, like.device());
      data = fresh.data_ptr();
    }
  }
  PyObject* wrap() const { return fresh.defined() ? THPVariable_Wrap(fresh) : Py_NewRef(given != nullptr ? given : Py_None); }
};

PyObject* tuple_of(const Output* outputs, Py_ssize_t n) {
  PyObject* all = PyTuple_New(n);
  for (Py_ssize_t i = 0; all != nullptr && i < n; ++i) {
    PyObject* o = outputs[i].wrap();
    if (o == nullptr) {
      Py_CLEAR(all);
      break;
    }
    PyTuple_SET_ITEM(all, i, o);
  }
  return all;
}

// Outputs that a call allocates are the current stream's memory.
void need_own_stream(Call& call, bool allocates, void* stream) { need(!allocates || stream == call.stream(Py_None)); }

// (lens, new_lens, block_tables, max_tokens, page_size, out, error_word, stream) ->
// (cum_seq_lens_q, requests, positions, slots), a status that is not 0, or None
PyObject* token_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    Call call;
    smla_token_slots_args p = {};
    const at::Tensor& lens = call.tensor(a[0]);
    p.batch = int32(lens.numel());
    p.lens = static_cast<const int32_t*>(call.words(a[0], 0));
    p.new_lens = static_cast<const int32_t*>(call.words(a[1], p.batch));
    p.max_tokens = int32(a[3]);
    need(p.max_tokens >= 0);
    const bool tables = a[2] != Py_None, given = a[5] != Py_None;
    if (tables) {
      int32_t rows = 0;
      p.block_tables = table(call, a[2], &rows, &p.max_pages, &p.block_table_stride);
      p.page_size = int32(a[4]);
      need(rows >= p.batch);
    }
    need(!given || (PyTuple_Check(a[5]) && PyTuple_GET_SIZE(a[5]) == 4));
    const auto item = [&](Py_ssize_t i) { return given ? PyTuple_GET_ITEM(a[5], i) : nullptr; };
    p.error_word = static_cast<int32_t*>(call.words(a[6], 1, true));
    void* const stream = call.stream(a[7]);
    need_own_stream(call, !given, stream);
    Output out[4];
    out[0].set(call, item(0), c10::kInt, {p.batch + (int64_t)1}, p.batch + (int64_t)1, lens);
    out[1].set(call, item(1), c10::kInt, {p.max_tokens}, p.max_tokens, lens);
    out[2].set(call, item(2), c10::kInt, {p.max_tokens}, p.max_tokens, lens);
    if (tables) out[3].set(call, item(3), c10::kLong, {p.max_tokens}, p.max_tokens, lens);
    else need(!given || item(3) == Py_None);
    p.cum_seq_lens_q = static_cast<int32_t*>(out[0].data);
    p.requests = static_cast<int32_t*>(out[1].data);
    p.positions = static_cast<int32_t*>(out[2].data);
    p.slots = static_cast<int64_t*>(out[3].data);
    const smla_status s = unlocked([&] { return smla_token_slots(&p, stream); });
    return s != SMLA_OK ? PyLong_FromLong(s) : tuple_of(out, 4);
  });
}

// (seq_lens, swa_tables, num_tokens, page_size, cum_seq_lens_q, selected, num_selected, compressed_tables,
//  compressed_page_size, compress_ratio, sparse_indices, topk_lens, error_word, stream) ->
// (sparse_indices, topk_lens), a status that is not 0, or None
PyObject* sparse_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    Call call;
    smla_sparse_slots_args p = {};
    p.swa_tables = table(call, a[1], &p.batch, &p.swa_max_pages, &p.swa_table_stride);
    p.seq_lens = static_cast<const int32_t*>(call.words(a[0], p.batch));
    p.sum_q = int32(a[2]);
    need(p.sum_q > 0);
    p.swa_page_size = int32(a[3]);
    p.cum_seq_lens_q = static_cast<const int32_t*>(call.words(a[4], p.batch + (int64_t)1, true));
    p.num_selected = int32(a[6]);
    if (a[5] != Py_None) {
      const at::Tensor& t = call.tensor(a[5]);
      need(t.scalar_type() == c10::kInt && t.dim() == 2 && t.size(0) == p.sum_q && t.size(1) > 0 && t.stride(1) == 1 &&
           (p.sum_q == 1 || t.stride(0) >= t.size(1)));
      p.selected = static_cast<const int32_t*>(t.data_ptr());
      p.num_selected = int32(t.size(1));
      p.selected_stride = p.sum_q > 1 ? t.stride(0) : 0;
    }
    need(p.num_selected >= 0 && (p.num_selected == 0 || a[7] != Py_None));
    if (a[7] != Py_None) {
      int32_t rows = 0;
      p.comp_tables = table(call, a[7], &rows, &p.comp_max_pages, &p.comp_table_stride);
      p.comp_page_size = int32(a[8]);
      need(rows == p.batch);
    }
    p.compress_ratio = int32(a[9]);
    p.error_word = static_cast<int32_t*>(call.words(a[12], 1, true));
    void* const stream = call.stream(a[13]);
    need_own_stream(call, a[10] == Py_None || a[11] == Py_None, stream);
    const int64_t columns = SMLA_SWA_COLS + (int64_t)p.num_selected;
    Output out[2];
    if (a[10] == Py_None) {
      out[0].set(call, nullptr, c10::kInt, {p.sum_q, columns}, 0, call.tensor(a[1]));
      p.indices_row_stride = columns;
    } else {
      const at::Tensor& t = call.tensor(a[10]);
      need(t.scalar_type() == c10::kInt && t.dim() == 2 && t.size(0) == p.sum_q && t.size(1) == columns && t.stride(1) == 1 &&
           (p.sum_q == 1 || t.stride(0) >= columns));
      out[0].given = a[10];
      out[0].data = t.data_ptr();
      p.indices_row_stride = p.sum_q > 1 ? t.stride(0) : columns;
    }
    out[1].set(call, a[11] == Py_None ? nullptr : a[11], c10::kInt, {p.sum_q}, p.sum_q, call.tensor(a[1]));
    p.sparse_indices = static_cast<int32_t*>(out[0].data);
    p.topk_lens = static_cast<int32_t*>(out[1].data);
    const smla_status s = unlocked([&] { return smla_sparse_slots(&p, stream); });
    return s != SMLA_OK ? PyLong_FromLong(s) : tuple_of(out, 2);
  });
}

// (logits, scores, workspace, num_out, finished, end_token, out, error_word, stream) ->
// (scores, parents, tokens), a status that is not 0, or None
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Call call;
    smla_beam_args p = {};
    const at::Tensor &logits = call.tensor(a[0]), &scores = call.tensor(a[1]);
    need(logits.dim() == 2 && scores.dim() == 2 && scores.scalar_type() == c10::kFloat && scores.is_contiguous() &&
         logits.size(0) == scores.numel() && logits.size(0) > 0 && logits.size(1) > 0 && logits.stride(1) == 1 &&
         (logits.size(0) == 1 || logits.stride(0) >= logits.size(1)));
    switch (logits.scalar_type()) {
      case c10::kBFloat16: p.dtype = SMLA_LOGITS_BF16; break;
      case c10::kHalf: p.dtype = SMLA_LOGITS_FP16; break;
      case c10::kFloat: p.dtype = SMLA_LOGITS_FP32; break;
      default: need(false);
    }
    p.batch = int32(scores.size(0));
    p.beams = int32(scores.size(1));
    p.vocab = int32(logits.size(1));
    p.num_out = a[3] == Py_None ? p.beams : int32(a[3]);
    need(p.num_out > 0 && p.num_out <= SMLA_MAX_BEAM_OUT);
    p.logits = logits.data_ptr();
    p.logits_stride = logits.size(0) > 1 ? logits.stride(0) : p.vocab;
    p.scores = static_cast<const float*>(scores.data_ptr());
    p.workspace = call.bytes(a[2], &p.workspace_bytes);
    if (a[4] != Py_None) {
      const at::Tensor& t = call.tensor(a[4]);
      need((t.scalar_type() == c10::kBool || t.scalar_type() == c10::kByte) && t.is_contiguous() &&
           t.numel() == scores.numel());
      p.finished = static_cast<const uint8_t*>(t.data_ptr());
    }
    p.end_token = int32(a[5]);
    const bool given = a[6] != Py_None;
    need(!given || (PyTuple_Check(a[6]) && PyTuple_GET_SIZE(a[6]) == 3));
    p.error_word = static_cast<int32_t*>(call.words(a[7], 1, true));
    void* const stream = call.stream(a[8]);
    need_own_stream(call, !given, stream);
    const int64_t entries = (int64_t)p.batch * p.num_out;
    Output out[3];
    for (int i = 0; i < 3; ++i)
      out[i].set(call, given ? PyTuple_GET_ITEM(a[6], i) : nullptr, i == 0 ? c10::kFloat : c10::kInt, {p.batch, p.num_out},
                 entries, scores);
    p.out_scores = static_cast<float*>(out[0].data);
    p.out_parents = static_cast<int32_t*>(out[1].data);
    p.out_tokens = static_cast<int32_t*>(out[2].data);
    const smla_status s = unlocked([&] { return smla_beam_select(&p, stream); });
    return s != SMLA_OK ? PyLong_FromLong(s) : tuple_of(out, 3);
  });
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {
    {"window_attention", fast(window_attention), METH_FASTCALL, nullptr},
    {"prefix_attention", fast(prefix_attention), METH_FASTCALL, nullptr},
    {"append", fast(append), METH_FASTCALL, nullptr},
    {"pages_resize", fast(pages_resize), METH_FASTCALL, nullptr},
    {"pages_fork", fast(pages_fork), METH_FASTCALL, nullptr},
    {"pages_reorder", fast(pages_reorder), METH_FASTCALL, nullptr},
    {"pages_shared_prefix", fast(pages_shared_prefix), METH_FASTCALL, nullptr},
    {"pages_compact", fast(pages_compact), METH_FASTCALL, nullptr},
    {"pages_copy", fast(pages_copy), METH_FASTCALL, nullptr},
    {"token_slots", fast(token_slots), METH_FASTCALL, nullptr},
    {"sparse_slots", fast(sparse_slots), METH_FASTCALL, nullptr},
    {"beam_select", fast(beam_select), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "smla_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_smla_torch() { return PyModule_Create(&module); }
