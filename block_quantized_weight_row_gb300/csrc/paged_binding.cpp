// paged_binding.cpp — the host side of the paged KV-cache calls from Python:
// checks of the tensors, outputs, the workspace and the call into libbq.so, as
// one CPython function each. A decode step makes these calls once per layer
// and their kernels take ~10 us, so the host's share counts: attribute by
// attribute from Python the checks and the foreign call took 30 us of an
// attention call; here they take ~2 beside its two launches.
// The functions return the outputs, or the library's status as an int, which
// the Python wrapper turns into its exception. Wrong tensors raise TypeError
// or ValueError. (The C ABI itself stays free of torch types: include/bq.h.)
#include "binding_common.h"
#include "layer_binding.h"

namespace {

int block_bytes(int type) { return type == BQ_TYPE_Q4_0 ? 18 : type == BQ_TYPE_Q8_0 ? 34 : 0; }

// args[0..6]: k_pages, v_pages, page_size, head_dim, k_type, v_type, k_basis
struct Cache {
  bq_paged_cache c;
  at::Device device;
};
constexpr int kCacheArgs = 7;

Cache cache_of(PyObject *const *args) {
  const int64_t page = to_int(args[2], "page_size"), dim = to_int(args[3], "head_dim");
  const int types[2] = {to_code(args[4], "k_type"), to_code(args[5], "v_type")}, basis = to_code(args[6], "k_basis");
  const at::Tensor &k = cuda_tensor(args[0], "k_pages"), &v = cuda_tensor(args[1], "v_pages");
  const at::Tensor *pools[2] = {&k, &v};
  const char *names[2] = {"k_pages", "v_pages"};
  for (int i = 0; i < 2; ++i) {
    const at::Tensor &t = *pools[i];
    if (t.scalar_type() != at::kByte || t.dim() != 3)
      wrong(PyExc_TypeError, "%s must be uint8 (n_pages, n_kv_heads, bytes)", names[i]);
    if (!t.is_contiguous()) wrong(PyExc_ValueError, "%s must be contiguous", names[i]);
    const int bb = block_bytes(types[i]);
    if (bb && page > 0 && dim > 0 && page <= (1 << 20) && dim <= (1 << 20) && t.size(2) * 32 != page * dim * bb)
      wrong(PyExc_ValueError, "%s has %lld bytes per head page, not page_size * head_dim / 32 blocks", names[i],
            (long long)t.size(2));
  }
  if (k.size(0) != v.size(0) || k.size(1) != v.size(1) || k.device() != v.device())
    wrong(PyExc_ValueError, "k_pages and v_pages must have the same pages, heads and device");
  return Cache{bq_paged_cache{k.data_ptr(), v.data_ptr(), k.size(0), page, k.size(1), dim, types[0], types[1], basis}, k.device()};
}

void same_device(const at::Tensor &t, const at::Device &d, const char *name) {
  if (t.device() != d) wrong(PyExc_ValueError, "%s is on another device than the cache", name);
}

// (tokens, heads, head_dim) of an element type the calls take, channels
// contiguous; other strides are free. heads < 0: any.
const at::Tensor &rows(PyObject *o, const char *name, const Cache &c, int64_t heads) {
  const at::Tensor &t = cuda_tensor(o, name);
  if (elem_of(t.scalar_type()) < 0) wrong(PyExc_TypeError, "%s must be float32, float16 or bfloat16", name);
  same_device(t, c.device, name);
  if (t.dim() != 3 || t.size(2) != c.c.head_dim || (heads >= 0 && t.size(1) != heads))
    wrong(PyExc_ValueError, "%s must be (tokens, %lld, %lld)", name, (long long)heads, (long long)c.c.head_dim);
  if (t.stride(2) != 1) wrong(PyExc_ValueError, "the channels of %s must be contiguous", name);
  return t;
}

const at::Tensor &exact(PyObject *o, const char *name, const Cache &c, at::ScalarType type, at::IntArrayRef shape) {
  const at::Tensor &t = cuda_tensor(o, name);
  if (t.scalar_type() != type) wrong(PyExc_TypeError, "%s must be %s", name, at::toString(type));
  if (t.sizes() != shape) wrong(PyExc_TypeError, "%s has the wrong shape", name);
  if (!t.is_contiguous()) wrong(PyExc_ValueError, "%s must be contiguous", name);
  same_device(t, c.device, name);
  return t;
}

const float *bias_of(PyObject *o, const Cache &c) {
  return o == Py_None ? nullptr : exact(o, "bias", c, at::kFloat, {c.c.n_kv_heads, c.c.head_dim}).data_ptr<float>();
}

// None as the bias's basis: the cache's
int basis_of(PyObject *o, const Cache &c) { return o == Py_None ? c.c.k_basis : to_code(o, "bias_basis"); }

// cache, k, v, slots, bias, bias_basis
PyObject *kv_write(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != kCacheArgs + 5) wrong(PyExc_TypeError, "paged_kv_write: wrong number of arguments");
    const Cache c = cache_of(args);
    args += kCacheArgs;
    const at::Tensor &k = rows(args[0], "k", c, c.c.n_kv_heads), &v = rows(args[1], "v", c, c.c.n_kv_heads);
    if (v.scalar_type() != k.scalar_type()) wrong(PyExc_TypeError, "k and v must have the same type");
    if (v.size(0) != k.size(0)) wrong(PyExc_ValueError, "k and v must have the same shape");
    const at::Tensor &slots = exact(args[2], "slots", c, at::kLong, {k.size(0)});
    const float *bias = bias_of(args[3], c);
    const int basis = basis_of(args[4], c);
    const c10::cuda::CUDAGuard guard(c.device);
    use_stream();
    const int r = bq_paged_kv_write(&c.c, elem_of(k.scalar_type()), k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                                    v.stride(0), v.stride(1), bias, basis, slots.data_ptr<int64_t>(), k.size(0));
    return r ? status(r) : none();
  } catch (const Wrong &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// cache, slots, elem, bias, bias_basis, out_k, out_v
PyObject *kv_read(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != kCacheArgs + 6) wrong(PyExc_TypeError, "paged_kv_read: wrong number of arguments");
    const Cache c = cache_of(args);
    args += kCacheArgs;
    const at::Tensor &some = cuda_tensor(args[0], "slots");
    const at::Tensor &slots = exact(args[0], "slots", c, at::kLong, {some.numel()});
    const int64_t elem = to_int(args[1], "elem"), T = slots.size(0);
    if (elem < 0 || elem > 2) wrong(PyExc_TypeError, "dtype must be float32, float16 or bfloat16");
    const at::ScalarType type = elem == BQ_ELEM_F32 ? at::kFloat : elem == BQ_ELEM_F16 ? at::kHalf : at::kBFloat16;
    const float *bias = bias_of(args[2], c);
    const int basis = basis_of(args[3], c);
    const c10::cuda::CUDAGuard guard(c.device);
    const std::array<int64_t, 3> shape = {T, c.c.n_kv_heads, c.c.head_dim};
    const auto options = at::TensorOptions().dtype(type).device(c.device);
    const char *names[2] = {"out_k", "out_v"};
    at::Tensor out[2];
    for (int i = 0; i < 2; ++i)
      out[i] = args[4 + i] == Py_None ? at::empty(shape, options) : exact(args[4 + i], names[i], c, type, shape);
    use_stream();
    const int r = bq_paged_kv_read(&c.c, int(elem), out[0].data_ptr(), out[1].data_ptr(), bias, basis, slots.data_ptr<int64_t>(), T);
    if (r) return status(r);
    PyObject *pair = PyTuple_New(2);
    if (!pair) return nullptr;
    for (int i = 0; i < 2; ++i) PyTuple_SET_ITEM(pair, i, THPVariable_Wrap(out[i]));
    return pair;
  } catch (const Wrong &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// cache, q, q_start, kv_len, page_table, scale, max_q_len, max_kv_len, causal, window, out, lse
PyObject *attn(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != kCacheArgs + 11) wrong(PyExc_TypeError, "paged_attn: wrong number of arguments");
    const Cache c = cache_of(args);
    args += kCacheArgs;
    const at::Tensor &q = rows(args[0], "q", c, -1);
    const int64_t n_q = q.size(0), H = q.size(1), D = c.c.head_dim;
    const int64_t B = cuda_tensor(args[2], "kv_len").numel();
    const at::Tensor &start = exact(args[1], "q_start", c, at::kInt, {B + 1}), &lens = exact(args[2], "kv_len", c, at::kInt, {B});
    const at::Tensor &any = cuda_tensor(args[3], "page_table");
    const int64_t pages = any.dim() == 2 ? any.size(1) : -1;
    const at::Tensor &table = exact(args[3], "page_table", c, at::kInt, {B, pages});
    const double scale = PyFloat_AsDouble(args[4]);
    if (scale == -1.0 && PyErr_Occurred()) throw Wrong{PyExc_TypeError};
    const int64_t max_q = to_int(args[5], "max_q_len"), max_kv = to_int(args[6], "max_kv_len"), window = to_int(args[8], "window");
    const int causal = PyObject_IsTrue(args[7]);
    if (causal < 0) throw Wrong{PyExc_TypeError};
    const int elem = elem_of(q.scalar_type());
    const c10::cuda::CUDAGuard guard(c.device);
    at::Tensor out;
    if (args[9] == Py_None) {
      out = at::empty({n_q, H, D}, q.options());
    } else {
      out = rows(args[9], "out", c, H);
      if (out.scalar_type() != q.scalar_type()) wrong(PyExc_TypeError, "out must have q's type");
      if (out.size(0) != n_q) wrong(PyExc_ValueError, "out must have q's shape");
    }
    float *lse = args[10] == Py_None ? nullptr : exact(args[10], "lse", c, at::kFloat, {n_q, H}).data_ptr<float>();
    CallWorkspace ws(bq_paged_attn_workspace_size(&c.c, elem, B, n_q, max_q, max_kv, H, causal, window), c.device);
    use_stream();
    const int r = bq_paged_attn(&c.c, elem, q.data_ptr(), q.stride(0), q.stride(1), out.data_ptr(), out.stride(0), out.stride(1), lse,
                                start.data_ptr<int>(), lens.data_ptr<int>(), table.data_ptr<int>(), pages, B, n_q, max_q, max_kv, H,
                                float(scale), causal, window);
    if (r) return ws.failed(r);
    return THPVariable_Wrap(out);
  } catch (const Wrong &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"kv_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_write)), METH_FASTCALL, nullptr},
    {"kv_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_read)), METH_FASTCALL, nullptr},
    {"attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attn)), METH_FASTCALL, nullptr},
    BQ_LAYER_METHODS,
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged", "Paged KV-cache calls of libbq.so on torch tensors.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&kModule); }
