// layer_binding.h — the host side of the calls around the projections and the
// paged cache of a served layer (include/bq.h: bq_paged_extend, bq_add_rms_norm,
// bq_rotary, bq_lora), a part of paged_binding.cpp's extension and in its manner.
// A failed call of the library returns (status, message).
#pragma once

#include "binding_common.h"

namespace {

PyObject *failed(int r) { return Py_BuildValue("(is)", r, bq_last_error()); }

bool flag(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Wrong{PyExc_TypeError};
  return v != 0;
}

void on(const at::Tensor &t, const at::Device &d, const char *name) {
  if (t.device() != d) wrong(PyExc_ValueError, "%s is on another device than the first tensor", name);
}

// A contiguous tensor of a type and shape on a device; sizes < 0: any.
const at::Tensor &plain(PyObject *o, const char *name, const at::Device &d, at::ScalarType type, std::initializer_list<int64_t> shape) {
  const at::Tensor &t = cuda_tensor(o, name);
  if (t.scalar_type() != type) wrong(PyExc_TypeError, "%s must be %s", name, at::toString(type));
  bool fits = t.dim() == int64_t(shape.size());
  int i = 0;
  for (const int64_t s : shape) {
    fits = fits && (s < 0 || t.size(i) == s);
    ++i;
  }
  if (!fits) wrong(PyExc_ValueError, "%s has the wrong shape", name);
  if (!t.is_contiguous()) wrong(PyExc_ValueError, "%s must be contiguous", name);
  on(t, d, name);
  return t;
}

// (rows, n) of a float type, the last axis contiguous; sizes < 0: any.
const at::Tensor &matrix(PyObject *o, const char *name, const at::Device *d, int64_t rows, int64_t n) {
  const at::Tensor &t = cuda_tensor(o, name);
  if (elem_of(t.scalar_type()) < 0) wrong(PyExc_TypeError, "%s must be float32, float16 or bfloat16", name);
  if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || (n >= 0 && t.size(1) != n)) wrong(PyExc_ValueError, "%s has the wrong shape", name);
  if (t.size(1) > 1 && t.stride(1) != 1) wrong(PyExc_ValueError, "the rows of %s must be contiguous", name);
  if (d) on(t, *d, name);
  return t;
}

at::ScalarType type_of(int64_t elem) {
  if (elem < 0 || elem > 2) wrong(PyExc_TypeError, "dtype must be float32, float16 or bfloat16");
  return elem == BQ_ELEM_F32 ? at::kFloat : elem == BQ_ELEM_F16 ? at::kHalf : at::kBFloat16;
}

// New references; nullptr entries become None.
PyObject *tuple_of(std::initializer_list<const at::Tensor *> tensors) {
  PyObject *r = PyTuple_New(Py_ssize_t(tensors.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor *t : tensors) {
    if (t && t->defined()) {
      PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(*t));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(r, i++, Py_None);
    }
  }
  return r;
}

// n elements of `type` from int32 element `from` of an allocation, as a tensor of
// its own (a view made through the dispatcher takes a microsecond, this a tenth).
at::Tensor part(const at::Tensor &all, at::ScalarType type, int64_t from, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), at::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  t.unsafeGetTensorImpl()->set_storage_offset(from * 4 / int64_t(at::elementSize(type)));
  return t;
}

// page_size, n_pages, kv_len, n_new, page_table, free_pages, n_slots
PyObject *paged_extend(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != 7) wrong(PyExc_TypeError, "paged_extend: wrong number of arguments");
    const int64_t page = to_int(args[0], "page_size"), pages = to_int(args[1], "n_pages"), n_slots = to_int(args[6], "n_slots");
    const at::Device d = cuda_tensor(args[2], "kv_len").device();
    const at::Tensor &kv = plain(args[2], "kv_len", d, at::kInt, {-1});
    const int64_t B = kv.size(0);
    const at::Tensor &fresh = plain(args[3], "n_new", d, at::kInt, {B}), &table = plain(args[4], "page_table", d, at::kInt, {B, -1}),
                     &free = plain(args[5], "free_pages", d, at::kInt, {-1});
    if (n_slots < 0) wrong(PyExc_ValueError, "n_slots is negative");
    const c10::cuda::CUDAGuard guard(d);
    // one allocation for the five outputs, each 16-byte aligned
    const int64_t a1 = 2 * ((n_slots + 1) / 2 * 2), a2 = a1 + (B + 4) / 4 * 4, a3 = a2 + (B + 3) / 4 * 4, a4 = a3 + (n_slots + 3) / 4 * 4;
    const at::Tensor all = at::empty({a4 + 4}, kv.options());
    const at::Tensor slots = part(all, at::kLong, 0, n_slots), q_start = part(all, at::kInt, a1, B + 1), kv_out = part(all, at::kInt, a2, B),
                     positions = part(all, at::kInt, a3, n_slots), taken = part(all, at::kInt, a4, 2);
    use_stream();
    const int r = bq_paged_extend(page, pages, kv.data_ptr<int>(), fresh.data_ptr<int>(), B, free.data_ptr<int>(), free.size(0),
                                  table.data_ptr<int>(), table.size(1), q_start.data_ptr<int>(), kv_out.data_ptr<int>(),
                                  slots.data_ptr<int64_t>(), positions.data_ptr<int>(), n_slots, taken.data_ptr<int>());
    if (r) return failed(r);
    return tuple_of({&q_start, &kv_out, &slots, &positions, &taken});
  } catch (const Wrong &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// x, weight, eps, residual, out, q8 (True, False or a tensor each), sum (None or a tensor)
PyObject *add_rms_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != 7) wrong(PyExc_TypeError, "add_rms_norm: wrong number of arguments");
    const at::Tensor &x = matrix(args[0], "x", nullptr, -1, -1);
    const at::Device d = x.device();
    const int64_t rows = x.size(0), cols = x.size(1);
    const at::Tensor &weight = plain(args[1], "weight", d, at::kFloat, {cols});
    const double eps = PyFloat_AsDouble(args[2]);
    if (eps == -1.0 && PyErr_Occurred()) throw Wrong{PyExc_TypeError};
    auto like_x = [&](PyObject *o, const char *name) -> const at::Tensor & {
      const at::Tensor &t = matrix(o, name, &d, rows, cols);
      if (t.scalar_type() != x.scalar_type()) wrong(PyExc_TypeError, "%s must have x's type", name);
      return t;
    };
    const at::Tensor res = args[3] == Py_None ? at::Tensor() : like_x(args[3], "residual");
    const c10::cuda::CUDAGuard guard(d);
    at::Tensor out, q8, sum;
    const int64_t q8_bytes = cols / 32 * 34;
    if (THPVariable_Check(args[4])) out = like_x(args[4], "out");
    else if (flag(args[4])) out = at::empty({rows, cols}, x.options());
    if (THPVariable_Check(args[5])) q8 = plain(args[5], "q8", d, at::kByte, {rows, q8_bytes});
    else if (flag(args[5])) q8 = at::empty({rows, q8_bytes}, x.options().dtype(at::kByte));
    if (args[6] != Py_None) {
      if (!res.defined()) wrong(PyExc_ValueError, "sum without a residual");
      sum = like_x(args[6], "sum");
    } else if (res.defined()) {
      sum = at::empty({rows, cols}, x.options());
    }
    use_stream();
    auto ptr = [](const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
    auto stride = [](const at::Tensor &t) { return t.defined() ? t.stride(0) : 0; };
    const int r = bq_add_rms_norm(elem_of(x.scalar_type()), x.data_ptr(), x.stride(0), ptr(res), stride(res), weight.data_ptr<float>(), eps,
                                  ptr(sum), stride(sum), ptr(out), stride(out), ptr(q8), rows, cols);
    if (r) return failed(r);
    return tuple_of({&out, &sum, &q8});
  } catch (const Wrong &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// q, k, positions, inv_freq, axis, interleaved, inverse, elem (-1: as given), out_q, out_k
PyObject *rotary(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != 10) wrong(PyExc_TypeError, "rotary: wrong number of arguments");
    const at::Tensor &q = cuda_tensor(args[0], "q");
    const at::Device d = q.device();
    if (q.dim() != 3) wrong(PyExc_ValueError, "q must be (tokens, heads, head_dim)");
    const int64_t T = q.size(0), D = q.size(2);
    auto rows = [&](PyObject *o, const char *name, at::ScalarType type, int64_t heads) -> const at::Tensor & {
      const at::Tensor &t = cuda_tensor(o, name);
      if (elem_of(t.scalar_type()) < 0) wrong(PyExc_TypeError, "%s must be float32, float16 or bfloat16", name);
      if (t.scalar_type() != type) wrong(PyExc_TypeError, "%s must be %s", name, at::toString(type));
      if (t.dim() != 3 || t.size(0) != T || t.size(2) != D || (heads >= 0 && t.size(1) != heads))
        wrong(PyExc_ValueError, "%s has the wrong shape", name);
      if (t.stride(2) != 1) wrong(PyExc_ValueError, "the channels of %s must be contiguous", name);
      on(t, d, name);
      return t;
    };
    rows(args[0], "q", q.scalar_type(), -1);
    const at::Tensor k = args[1] == Py_None ? at::Tensor() : rows(args[1], "k", q.scalar_type(), -1);
    const at::Tensor &pos = cuda_tensor(args[2], "positions");
    if (pos.scalar_type() != at::kInt) wrong(PyExc_TypeError, "positions must be Int");
    if (pos.dim() < 1 || pos.dim() > 2 || pos.size(-1) != T) wrong(PyExc_ValueError, "positions must be (axes, tokens) or (tokens)");
    if (T > 1 && pos.stride(-1) != 1) wrong(PyExc_ValueError, "an axis of positions must be contiguous");
    on(pos, d, "positions");
    const int64_t axes = pos.dim() == 2 ? pos.size(0) : 1;
    const at::Tensor &freq = plain(args[3], "inv_freq", d, at::kDouble, {-1});
    const int64_t pairs = freq.size(0);
    const int *axis = args[4] == Py_None ? nullptr : plain(args[4], "axis", d, at::kInt, {pairs}).data_ptr<int>();
    const bool interleaved = flag(args[5]), inverse = flag(args[6]);
    const int64_t code = to_int(args[7], "elem");
    const at::ScalarType type = code == -1 ? q.scalar_type() : type_of(code);
    const c10::cuda::CUDAGuard guard(d);
    at::Tensor out_q, out_k;
    out_q = args[8] == Py_None ? at::empty({T, q.size(1), D}, q.options().dtype(type)) : rows(args[8], "out_q", type, q.size(1));
    if (k.defined())
      out_k = args[9] == Py_None ? at::empty({T, k.size(1), D}, q.options().dtype(type)) : rows(args[9], "out_k", type, k.size(1));
    use_stream();
    const bool has_k = k.defined();
    const int r = bq_rotary(elem_of(q.scalar_type()), q.data_ptr(), q.stride(0), q.stride(1), q.size(1), has_k ? k.data_ptr() : nullptr,
                            has_k ? k.stride(0) : 0, has_k ? k.stride(1) : 0, has_k ? k.size(1) : 0, elem_of(type), out_q.data_ptr(),
                            out_q.stride(0), out_q.stride(1), has_k ? out_k.data_ptr() : nullptr, has_k ? out_k.stride(0) : 0,
                            has_k ? out_k.stride(1) : 0, pos.data_ptr<int>(), pos.dim() == 2 ? pos.stride(0) : 0, axes,
                            freq.data_ptr<double>(), axis, 2 * pairs, D, T, interleaved, inverse);
    if (r) return failed(r);
    return tuple_of({&out_q, &out_k});
  } catch (const Wrong &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// x, a, b, adapter, y, scale, out, elem of out where there is neither y nor out (-1: x's)
PyObject *lora(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != 8) wrong(PyExc_TypeError, "lora: wrong number of arguments");
    const at::Tensor &x = matrix(args[0], "x", nullptr, -1, -1);
    const at::Device d = x.device();
    const int64_t T = x.size(0), K = x.size(1);
    const at::Tensor &first = cuda_tensor(args[1], "a");
    if (first.scalar_type() != at::kHalf && first.scalar_type() != at::kBFloat16) wrong(PyExc_TypeError, "a must be float16 or bfloat16");
    const at::Tensor &a = plain(args[1], "a", d, first.scalar_type(), {-1, -1, K});
    const at::Tensor &b = plain(args[2], "b", d, first.scalar_type(), {a.size(0), -1, a.size(1)});
    const int64_t M = b.size(1);
    const at::Tensor &adapter = plain(args[3], "adapter", d, at::kInt, {T});
    const at::Tensor y = args[4] == Py_None ? at::Tensor() : matrix(args[4], "y", &d, T, M);
    const float *scale = args[5] == Py_None ? nullptr : plain(args[5], "scale", d, at::kFloat, {a.size(0)}).data_ptr<float>();
    const int64_t code = to_int(args[7], "elem");
    const at::ScalarType type = y.defined() ? y.scalar_type() : args[6] != Py_None ? matrix(args[6], "out", &d, T, M).scalar_type()
                                                             : code == -1 ? x.scalar_type() : type_of(code);
    const c10::cuda::CUDAGuard guard(d);
    at::Tensor out;
    if (args[6] == Py_None) {
      out = at::empty({T, M}, x.options().dtype(type));
    } else {
      out = matrix(args[6], "out", &d, T, M);
      if (out.scalar_type() != type) wrong(PyExc_TypeError, "out must have y's type");
    }
    CallWorkspace ws(bq_lora_workspace_size(T, a.size(0), a.size(1), K, M), d);
    use_stream();
    const int r = bq_lora(elem_of(x.scalar_type()), x.data_ptr(), x.stride(0), elem_of(a.scalar_type()), a.data_ptr(), b.data_ptr(), scale,
                          a.size(0), a.size(1), adapter.data_ptr<int>(), elem_of(type), y.defined() ? y.data_ptr() : nullptr,
                          y.defined() ? y.stride(0) : 0, out.data_ptr(), out.stride(0), T, M, K);
    if (r) return ws.failed(r);
    return THPVariable_Wrap(out);
  } catch (const Wrong &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// type, blocks, rows, cols, out
PyObject *dequantize_rows(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != 5) wrong(PyExc_TypeError, "dequantize_rows: wrong number of arguments");
    const int type = to_code(args[0], "t");
    const at::Tensor &blocks = cuda_tensor(args[1], "blocks");
    const at::Device d = blocks.device();
    if (blocks.scalar_type() != at::kByte) wrong(PyExc_TypeError, "blocks must be Byte");
    const int64_t rows = to_int(args[2], "rows"), cols = to_int(args[3], "cols");
    at::Tensor out;
    if (args[4] != Py_None) {
      out = cuda_tensor(args[4], "out");
      if (out.scalar_type() != at::kFloat) wrong(PyExc_TypeError, "out must be Float");
      if (!out.is_contiguous()) wrong(PyExc_ValueError, "out must be contiguous");
      on(out, d, "out");
      if (out.numel() < rows * cols) wrong(PyExc_ValueError, "out must have rows * cols values");
    }
    const c10::cuda::CUDAGuard guard(d);
    if (!out.defined()) out = at::empty({rows, cols}, blocks.options().dtype(at::kFloat));
    use_stream();
    const int r = bq_dequantize_rows(type, blocks.data_ptr(), static_cast<float *>(out.data_ptr()), rows, cols);
    if (r) return failed(r);
    return THPVariable_Wrap(out);
  } catch (const Wrong &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define BQ_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
#define BQ_LAYER_METHODS BQ_METHOD(paged_extend), BQ_METHOD(add_rms_norm), BQ_METHOD(rotary), BQ_METHOD(lora), BQ_METHOD(dequantize_rows)

}  // namespace
