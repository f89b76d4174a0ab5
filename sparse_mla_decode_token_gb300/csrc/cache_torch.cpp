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

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
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

// (q, rows, scales, block_tables, seq_lens, workspace, cum_seq_lens_q, sinks, window, first_tokens, num_splits,
//  bmm1_scale, bmm2_scale, out, out_lse, error_word, stream) -> (out, out_lse), a status that is not 0, or None
PyObject* window_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    Call call;
    smla_window_args w = {};
    const at::Tensor& q = call.tensor(a[0]);
    need(q.scalar_type() == c10::kBFloat16 && q.dim() == 3);
    const int64_t T = q.size(0), H = q.size(1);
    need(T > 0 && H > 0 && q.size(2) == kDim && q.stride(2) == 1 && (H == 1 || q.stride(1) == kDim) &&
         (T == 1 || q.stride(0) > 0));
    w.cache = cache(call, a[1], a[2], a[3], a[4], a[6]);
    w.workspace = call.bytes(a[5], &w.workspace_bytes);
    w.sinks = static_cast<const float*>(call.array(a[7], c10::kFloat, H, true));
    w.window = int32(a[8]);
    w.first_tokens = int32(a[9]);
    w.num_splits = int32(a[10]);
    scale(call, a[11], &w.bmm1_scale, &w.bmm1_scale_dev);
    scale(call, a[12], &w.bmm2_scale, &w.bmm2_scale_dev);
    w.sum_q = int32(T);
    w.num_heads = int32(H);
    w.q = q.data_ptr();
    w.q_stride_token = T > 1 ? q.stride(0) : 0;
    w.error_word = static_cast<int32_t*>(call.words(a[15], 1, true));
    void* const stream = call.stream(a[16]);
    // (outputs of a call on another stream than the current one have to be that stream's memory)
    need((a[13] != Py_None && a[14] != Py_None) || stream == call.stream(Py_None));
    at::Tensor out, lse;                    // those that are not given
    if (a[13] == Py_None) {
      out = at::empty_like(q, q.options(), c10::MemoryFormat::Contiguous);
      w.out = out.data_ptr();
    } else {
      w.out = call.array(a[13], c10::kBFloat16, T * H * kDim, false);
      need(THPVariable_Unpack(a[13]).numel() == T * H * kDim);
    }
    if (a[14] == Py_None) {
      lse = at::empty({T, H}, q.options().dtype(c10::kFloat));
      w.out_lse = static_cast<float*>(lse.data_ptr());
    } else {
      w.out_lse = static_cast<float*>(call.array(a[14], c10::kFloat, T * H, false));
      need(THPVariable_Unpack(a[14]).numel() == T * H);
    }
    const smla_status s = unlocked([&] { return smla_window_attention(&w, stream); });
    if (s != SMLA_OK) return PyLong_FromLong(s);
    PyObject* o = out.defined() ? THPVariable_Wrap(out) : Py_NewRef(a[13]);
    PyObject* l = lse.defined() ? THPVariable_Wrap(lse) : Py_NewRef(a[14]);
    PyObject* both = o != nullptr && l != nullptr ? PyTuple_Pack(2, o, l) : nullptr;
    Py_XDECREF(o);
    Py_XDECREF(l);
    return both;
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

smla_pages_args pages(Call& call, PyObject* tables_o, PyObject* refs, PyObject* lens, PyObject* page_size, PyObject* error) {
  smla_pages_args p = {};
  const at::Tensor& tables = call.tensor(tables_o);
  need(tables.scalar_type() == c10::kInt && tables.dim() == 2 && tables.size(0) > 0 && tables.size(1) > 0 &&
       tables.stride(1) == 1 && tables.stride(0) >= tables.size(1));
  p.block_tables = static_cast<int32_t*>(tables.data_ptr());
  p.rows = int32(tables.size(0));
  p.max_pages = int32(tables.size(1));
  p.block_table_stride = p.rows > 1 ? tables.stride(0) : p.max_pages;
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

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {
    {"window_attention", fast(window_attention), METH_FASTCALL, nullptr},
    {"append", fast(append), METH_FASTCALL, nullptr},
    {"pages_resize", fast(pages_resize), METH_FASTCALL, nullptr},
    {"pages_fork", fast(pages_fork), METH_FASTCALL, nullptr},
    {"pages_compact", fast(pages_compact), METH_FASTCALL, nullptr},
    {"pages_copy", fast(pages_copy), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "smla_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_smla_torch() { return PyModule_Create(&module); }
