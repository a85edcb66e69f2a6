// The argument side of the binding of a drafted tree's operators (tree.py):
// checks torch tensors, allocates the outputs that the caller did not give, and
// calls the C ABI on the current stream.  In C++ because these calls take a few
// microseconds on the device and the same checks in Python took 11 to 18.
//
// Every function returns its outputs, a pair; an int, the C status, if the
// library refused the call; None if the tensors are not on the current device
// (nothing was done: the caller goes there and calls again).

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <string>

#include "specverify.h"

namespace {

decltype(&spec_append_nodes) append_fn;
decltype(&spec_tree_attention) attention_fn;
decltype(&spec_keep_path) keep_fn;
decltype(&spec_process_logits) process_fn;
decltype(&specv_attention_workspace_bytes) workspace_bytes_fn;

// Other threads of Python run while one allocates or launches.
struct Released {
  PyThreadState* state = PyEval_SaveThread();
  ~Released() { PyEval_RestoreThread(state); }
};

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw python_error();
}
[[noreturn]] void refuse(const std::string& what) { raise(PyExc_ValueError, what); }
[[noreturn]] void refuse_type(const std::string& what) { raise(PyExc_TypeError, what); }

std::string name_of(at::ScalarType dtype) {
  switch (dtype) {
    case at::kInt: return "torch.int32";
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    default: return toString(dtype);
  }
}

std::string shape_of(at::IntArrayRef s) {
  std::string out = "(";
  for (size_t i = 0; i < s.size(); i++) out += (i ? ", " : "") + std::to_string(s[i]);
  return out + ")";
}

// A tensor, or nullptr for None.
const at::Tensor* given(const char* name, PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(const char* name, PyObject* o) {
  const at::Tensor* t = given(name, o);
  if (!t) refuse(std::string(name) + " must be given");
  return *t;
}

void need_like(const char* name, const at::Tensor& t, at::IntArrayRef shape, at::ScalarType dtype,
               const at::Device& dev) {
  if (t.scalar_type() != dtype || t.sizes() != shape || t.device() != dev)
    refuse(std::string(name) + " must be a " + name_of(dtype) + " tensor of shape " +
           shape_of(shape) + " on " + dev.str());
}

// A contiguous tensor of this shape, type and device, or None: its address.
template <class T>
T* need(const char* name, PyObject* o, at::IntArrayRef shape, at::ScalarType dtype,
        const at::Device& dev) {
  const at::Tensor* t = given(name, o);
  if (!t) return nullptr;
  need_like(name, *t, shape, dtype, dev);
  if (!t->is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return static_cast<T*>(t->data_ptr());
}

template <class T>
T* must(const char* name, PyObject* o, at::IntArrayRef shape, at::ScalarType dtype,
        const at::Device& dev) {
  tensor(name, o);
  return need<T>(name, o, shape, dtype, dev);
}

// Strides in elements; those of a single entry are never used.
int64_t stride(const at::Tensor& t, int i) { return t.size(i) > 1 ? t.stride(i) : 0; }

specv_rows rows_of(const char* name, const at::Tensor& t, at::IntArrayRef shape,
                   at::ScalarType dtype, const at::Device& dev) {
  need_like(name, t, shape, dtype, dev);
  if (t.stride(3) != 1 && t.size(3) > 1)
    refuse(std::string(name) + " must have a contiguous last dimension");
  return specv_rows{t.data_ptr(), stride(t, 0), stride(t, 1), stride(t, 2)};
}

int32_t small(const char* name, int64_t n) {
  if (n > INT32_MAX) refuse(std::string(name) + " is too large");
  return static_cast<int32_t>(n);
}

struct CacheOf {
  specv_cache arg;
  at::ScalarType dtype;
  at::Device dev;
  int64_t B;
};

CacheOf cache_of(PyObject* k_cache, PyObject* v_cache, PyObject* page_table, PyObject* cache_lens,
                 bool layered) {
  const at::Tensor &k = tensor("k_cache", k_cache), &v = tensor("v_cache", v_cache);
  const int dims = static_cast<int>(k.dim()), at = dims - 4;
  if (dims != 4 && !(layered && dims == 5))
    refuse(std::string("k_cache must be [pages, page_size, heads, head_dim]") +
           (layered ? " or [layers, pages, page_size, heads, head_dim]" : ""));
  if (k.scalar_type() != at::kBFloat16 && k.scalar_type() != at::kHalf)
    refuse_type(std::string("k_cache must be bfloat16 or float16, got ") + name_of(k.scalar_type()));
  bool alike = v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type() && v.device() == k.device() &&
               (k.stride(dims - 1) == 1 || k.size(dims - 1) == 1);
  for (int i = 0; alike && i < dims; i++) alike = stride(v, i) == stride(k, i);
  if (!alike)
    refuse("v_cache must have k_cache's shape, strides, type and device, and both a contiguous last "
           "dimension");
  const at::Device dev = k.device();
  const at::Tensor& table = tensor("page_table", page_table);
  if (table.dim() != 2 || table.scalar_type() != at::kInt || table.device() != dev ||
      (table.size(1) > 1 && table.stride(1) != 1))
    refuse("page_table must be an int32 tensor [B, pages of a request] on " + dev.str() +
           " with contiguous rows");
  const int64_t B = table.size(0);
  const auto* lens = must<int32_t>("cache_lens", cache_lens, {B}, at::kInt, dev);
  specv_cache c;
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.page_table = static_cast<const int32_t*>(table.data_ptr());
  c.lens = lens;
  c.layer_stride = dims == 5 ? stride(k, 0) : 0;
  c.page_stride = stride(k, at);
  c.row_stride = stride(k, at + 1);
  c.head_stride = stride(k, at + 2);
  c.layers = dims == 5 ? small("layers", k.size(0)) : 1;
  c.pages = small("pages", k.size(at));
  c.page_size = small("page_size", k.size(at + 1));
  c.heads = small("heads", k.size(at + 2));
  c.head_dim = small("head_dim", k.size(at + 3));
  c.max_pages = small("page_table", table.size(1));
  c.table_stride = B > 1 ? small("page_table", table.stride(0)) : c.max_pages;
  c.dtype = k.scalar_type() == at::kHalf ? SPECV_F16 : SPECV_BF16;
  return CacheOf{c, k.scalar_type(), dev, B};
}

// (Sizes are narrowed before this: behind it, where Python's lock is given up, nothing may
// raise.)  Whether the call is made on the current device.
bool here(const at::Device& dev) {
  if (!dev.is_cuda())
    refuse("the operators on a drafted tree take CUDA tensors, got " + dev.str());
  return dev.index() == c10::cuda::current_device();
}

specv_stream_t stream_of(const at::Device& dev) {
  return reinterpret_cast<specv_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

at::Tensor output(const char* name, PyObject* o, at::IntArrayRef shape, at::ScalarType dtype,
                  const at::Device& dev, bool rows_may_be_left) {
  const at::Tensor* t = given(name, o);
  if (t) {
    need_like(name, *t, shape, dtype, dev);
    for (int i = 0; i < t->dim(); i++)
      if (t->size(i) > 1 && t->stride(i) == 0)
        refuse(std::string(name) + " must have a place for every element");
    return *t;
  }
  const auto options = at::TensorOptions().dtype(dtype).device(dev);
  const Released released;
  return rows_may_be_left ? at::zeros(shape, options) : at::empty(shape, options);
}

at::Tensor per_request(const char* name, PyObject* o, int64_t B, const at::Device& dev) {
  const at::Tensor t = output(name, o, {B}, at::kInt, dev, false);
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t;
}

// The call, with Python's lock given up: it may not raise.
template <class Call>
PyObject* answer(Call call, const at::Tensor& first, const at::Tensor& second) {
  const specv_status status = [&] {
    const Released released;
    return call();
  }();
  if (status != SPECV_OK) return PyLong_FromLong(status);
  PyObject* a = THPVariable_Wrap(first);
  PyObject* b = THPVariable_Wrap(second);
  PyObject* pair = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return pair;
}

float number(const char* name, PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(x);
}

void count(Py_ssize_t got, Py_ssize_t wanted) {
  if (got != wanted) refuse_type("wrong number of arguments");
}

PyObject* append_nodes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 17);
  const CacheOf c = cache_of(a[3], a[4], a[5], a[6], false);
  const at::Tensor& q = tensor("q", a[0]);
  if (q.dim() != 4) refuse("q must be [B, N, q_heads, head_dim]");
  const int64_t B = q.size(0), N = q.size(1), heads = q.size(2), D = q.size(3);
  if (c.B != B || c.arg.head_dim != D)
    refuse("q is for " + std::to_string(B) + " requests and heads of " + std::to_string(D) +
           ", the cache for " + std::to_string(c.B) + " and " + std::to_string(c.arg.head_dim));
  const specv_rows q_rows = rows_of("q", q, q.sizes(), c.dtype, c.dev);
  const specv_rows k_rows = rows_of("k", tensor("k", a[1]), {B, N, c.arg.heads, D}, c.dtype, c.dev);
  const specv_rows v_rows = rows_of("v", tensor("v", a[2]), {B, N, c.arg.heads, D}, c.dtype, c.dev);
  const at::Tensor* freq = given("inv_freq", a[7]);
  const int64_t half = freq ? freq->numel() : 0;
  const auto* inv_freq = need<float>("inv_freq", a[7], {half}, at::kFloat, c.dev);
  const auto* parents = need<int32_t>("parents", a[8], {B, N}, at::kInt, c.dev);
  const auto* nodes = need<int32_t>("n_nodes", a[9], {B}, at::kInt, c.dev);
  const void* q_weight = need<void>("q_weight", a[10], {D}, c.dtype, c.dev);
  const void* k_weight = need<void>("k_weight", a[11], {D}, c.dtype, c.dev);
  const float eps = number("eps", a[12]), scale = number("rope_scale", a[14]);
  const int interleaved = PyObject_IsTrue(a[13]);
  if (interleaved < 0) throw python_error();
  const int32_t requests = small("B", B), most = small("N", N), q_heads = small("q_heads", heads);
  const int32_t rot_dim = small("inv_freq", 2 * half);
  if (!here(c.dev)) Py_RETURN_NONE;
  const at::Tensor out = output("q_out", a[15], q.sizes(), c.dtype, c.dev, nodes != nullptr);
  const specv_rows out_rows = rows_of("q_out", out, q.sizes(), c.dtype, c.dev);
  const at::Tensor status = per_request("status", a[16], B, c.dev);
  return answer([&] { return append_fn(&c.arg, &q_rows, &k_rows, &v_rows, parents, nodes, requests, most,
                          q_heads, q_weight, k_weight, eps, half ? inv_freq : nullptr, rot_dim,
                          interleaved, scale,
                          &out_rows, static_cast<int32_t*>(status.data_ptr()), stream_of(c.dev)); },
                out, status);
  END_HANDLE_TH_ERRORS
}

// A workspace for one call: it goes back to torch's allocator on return, and
// what is given it next on this stream runs behind the call.
at::Tensor new_workspace(int32_t B, int32_t N, int32_t heads, const CacheOf& c) {
  const size_t bytes = workspace_bytes_fn(B, N, heads, c.arg.heads, c.arg.head_dim);
  if (!bytes)
    refuse("unsupported attention shape B=" + std::to_string(B) + " N=" + std::to_string(N) +
           " q_heads=" + std::to_string(heads) + " kv_heads=" + std::to_string(c.arg.heads) +
           " head_dim=" + std::to_string(c.arg.head_dim));
  const Released released;
  return at::empty({static_cast<int64_t>(bytes)}, at::TensorOptions().dtype(at::kByte).device(c.dev));
}

PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 11);
  const CacheOf c = cache_of(a[1], a[2], a[3], a[4], false);
  const at::Tensor& q = tensor("q", a[0]);
  if (q.dim() != 4) refuse("q must be [B, N, q_heads, head_dim]");
  const int64_t B = q.size(0), N = q.size(1), heads = q.size(2), D = q.size(3);
  if (c.B != B || c.arg.head_dim != D || c.arg.heads < 1 || heads % c.arg.heads != 0)
    refuse("q is for " + std::to_string(B) + " requests and " + std::to_string(heads) + " heads of " +
           std::to_string(D) + ", the cache for " + std::to_string(c.B) + " and " +
           std::to_string(c.arg.heads) + " of " + std::to_string(c.arg.head_dim));
  const specv_rows q_rows = rows_of("q", q, q.sizes(), c.dtype, c.dev);
  const auto* parents = need<int32_t>("parents", a[5], {B, N}, at::kInt, c.dev);
  const auto* nodes = need<int32_t>("n_nodes", a[6], {B}, at::kInt, c.dev);
  const float scale =
      a[7] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : number("scale", a[7]);
  const int32_t requests = small("B", B), most = small("N", N), q_heads = small("q_heads", heads);
  if (!here(c.dev)) Py_RETURN_NONE;
  const at::Tensor* lent = given("workspace", a[10]);
  if (lent && (lent->device() != c.dev || lent->scalar_type() != at::kByte || !lent->is_contiguous()))
    refuse("workspace is on " + lent->device().str() + ", the cache on " + c.dev.str());
  const at::Tensor workspace =
      lent ? *lent : new_workspace(requests, most, q_heads, c);
  const at::Tensor out = output("out", a[8], q.sizes(), c.dtype, c.dev, nodes != nullptr);
  const specv_rows out_rows = rows_of("out", out, q.sizes(), c.dtype, c.dev);
  const at::Tensor status = per_request("status", a[9], B, c.dev);
  return answer([&] { return attention_fn(&c.arg, &q_rows, parents, nodes, requests, most, q_heads, scale,
                             &out_rows,
                             static_cast<int32_t*>(status.data_ptr()), workspace.data_ptr(),
                             static_cast<size_t>(workspace.numel()), stream_of(c.dev)); },
                out, status);
  END_HANDLE_TH_ERRORS
}

PyObject* keep_path(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const CacheOf c = cache_of(a[2], a[3], a[4], a[5], true);
  const at::Tensor& path = tensor("path_nodes", a[0]);
  if (path.dim() != 2) refuse("path_nodes must be [B, N]");
  const int64_t B = c.B, N = path.size(1);
  const auto* nodes = must<int32_t>("path_nodes", a[0], {B, N}, at::kInt, c.dev);
  const auto* accepted = must<int32_t>("accepted_len", a[1], {B}, at::kInt, c.dev);
  const int32_t requests = small("B", B), most = small("N", N);
  if (!here(c.dev)) Py_RETURN_NONE;
  const at::Tensor lens = per_request("new_lens", a[6], B, c.dev);
  const at::Tensor status = per_request("status", a[7], B, c.dev);
  return answer([&] { return keep_fn(&c.arg, nodes, accepted, requests, most,
                        static_cast<int32_t*>(lens.data_ptr()),
                        static_cast<int32_t*>(status.data_ptr()), stream_of(c.dev)); },
                lens, status);
  END_HANDLE_TH_ERRORS
}

PyObject* process_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 15);
  const at::Tensor& z = tensor("logits", a[0]);
  if (z.dim() != 2 && z.dim() != 3) refuse("logits must be [B, R, V] or [B, V]");
  const at::ScalarType dtype = z.scalar_type();
  if (dtype != at::kBFloat16 && dtype != at::kFloat)
    refuse_type(std::string("logits must be bfloat16 or float32, got ") + name_of(dtype));
  const at::Device dev = z.device();
  const bool three = z.dim() == 3;
  const int64_t B = z.size(0), R = three ? z.size(1) : 1, V = z.size(three ? 2 : 1);
  const at::Tensor& history = tensor("history", a[1]);
  if (history.dim() != 2 || history.scalar_type() != at::kInt || history.device() != dev ||
      history.size(0) != B || (history.size(1) > 1 && history.stride(1) != 1))
    refuse("history must be an int32 tensor [B, L] on " + dev.str() + " with contiguous rows");
  const auto* seq_lens = must<int32_t>("seq_lens", a[2], {B}, at::kInt, dev);
  const auto* prompt_lens = need<int32_t>("prompt_lens", a[3], {B}, at::kInt, dev);
  const auto* parents = need<int32_t>("parents", a[5], {B, R}, at::kInt, dev);
  const auto* tokens = need<int32_t>("tokens", a[4], {B, parents ? R : R - 1}, at::kInt, dev);
  if (R > 1 && a[4] == Py_None) refuse("tokens must be given for more than one row");
  const auto* nodes = need<int32_t>("n_nodes", a[6], {B}, at::kInt, dev);
  const auto* repetition = need<float>("repetition", a[7], {B}, at::kFloat, dev);
  const auto* frequency = need<float>("frequency", a[8], {B}, at::kFloat, dev);
  const auto* presence = need<float>("presence", a[9], {B}, at::kFloat, dev);
  const at::Tensor* names = given("bias_tokens", a[10]);
  if (!names != (a[11] == Py_None)) refuse("bias_tokens and bias_values go together");
  const int64_t biases = names ? names->size(-1) : 0;
  const auto* bias_tokens = need<int32_t>("bias_tokens", a[10], {B, biases}, at::kInt, dev);
  const auto* bias_values = need<float>("bias_values", a[11], {B, biases}, at::kFloat, dev);
  const int64_t words = (V + 31) / 32;
  const int32_t* allowed = three ? need<int32_t>("allowed", a[12], {B, R, words}, at::kInt, dev)
                                 : need<int32_t>("allowed", a[12], {B, words}, at::kInt, dev);
  auto last_is_contiguous = [&](const char* name, const at::Tensor& t) {
    if (V > 1 && t.stride(-1) != 1)
      refuse(std::string(name) + " must have a contiguous last dimension");
  };
  last_is_contiguous("logits", z);
  const int32_t requests = small("B", B), rows = small("R", R), vocab = small("V", V);
  const int32_t longest = small("L", history.size(1)), num_bias = small("biases", biases);
  if (!here(dev)) Py_RETURN_NONE;
  const at::Tensor out = output("out", a[13], z.sizes(), dtype, dev, nodes != nullptr);
  last_is_contiguous("out", out);
  const at::Tensor status = per_request("status", a[14], B, dev);
  return answer(
      [&] { return process_fn(z.data_ptr(), stride(z, 0), three ? stride(z, 1) : 0,
                 dtype == at::kFloat ? SPECV_F32 : SPECV_BF16, requests, rows, vocab,
                 R > 1 ? tokens : nullptr, parents, nodes,
                 static_cast<const int32_t*>(history.data_ptr()), stride(history, 0),
                 longest, seq_lens, prompt_lens, repetition, frequency, presence,
                 bias_tokens, bias_values, num_bias, allowed, out.data_ptr(),
                 stride(out, 0), three ? stride(out, 1) : 0, static_cast<int32_t*>(status.data_ptr()),
                 stream_of(dev)); },
      out, status);
  END_HANDLE_TH_ERRORS
}

// The addresses of the C ABI's functions: the four operators, then the size
// of the attention's workspace.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 5);
  void* at[5];
  for (int i = 0; i < 5; i++) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (!at[i]) throw python_error();
  }
  append_fn = reinterpret_cast<decltype(append_fn)>(at[0]);
  attention_fn = reinterpret_cast<decltype(attention_fn)>(at[1]);
  keep_fn = reinterpret_cast<decltype(keep_fn)>(at[2]);
  process_fn = reinterpret_cast<decltype(process_fn)>(at[3]);
  workspace_bytes_fn = reinterpret_cast<decltype(workspace_bytes_fn)>(at[4]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define SPECV_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SPECV_METHOD(bind),      SPECV_METHOD(append_nodes),
                         SPECV_METHOD(tree_attention), SPECV_METHOD(keep_path),
                         SPECV_METHOD(process_logits), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
