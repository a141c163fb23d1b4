// Python binding of the row operators (include/segtopk.h: routing, tokens
// sorted by expert and back, embedding): checks tensors, makes the results
// and calls the C entry points on the current stream. _rows.py holds the
// public functions and their documentation.
//
// It is compiled, unlike the ctypes binding of the selection, because these
// calls are made several times a layer on batches of a few tokens, where
// their kernels take 2 us: a call that goes through ctypes and makes its
// results from Python takes 9 to 11 us of a GB300's host, most of it outside
// the CUDA launch.
//
// It computes nothing and has no other way to an operator: bind() receives
// the addresses of the library's entry points.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/segtopk.h"

namespace {

#define SEGTOPK_ENTRIES(X)                                                                                       \
  X(segtopk_route)                                                                                               \
  X(segtopk_route_backward)                                                                                      \
  X(segtopk_group)                                                                                               \
  X(segtopk_group_workspace_bytes)                                                                               \
  X(segtopk_dispatch)                                                                                            \
  X(segtopk_combine)                                                                                             \
  X(segtopk_combine_backward)                                                                                    \
  X(segtopk_embedding)                                                                                           \
  X(segtopk_embedding_backward)                                                                                  \
  X(segtopk_embedding_backward_workspace_bytes)

struct Library {
#define X(NAME) decltype(&::NAME) NAME = nullptr;
  SEGTOPK_ENTRIES(X)
#undef X
} lib;
PyObject* raise_status = nullptr; // raises the package's error for a status

// ---------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------
const at::Tensor& tensor(PyObject* o, const char* name)
{
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o)
{
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred())
    throw python_error();
  return v;
}
// an argument that the C entry points take as 32 bits
int32_t integer32(PyObject* o, const char* name)
{
  const int64_t v = integer(o);
  TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, " is out of range");
  return (int32_t)v;
}
float real(PyObject* o)
{
  const double v = PyFloat_AsDouble(o);
  if (v == -1 && PyErr_Occurred())
    throw python_error();
  return (float)v;
}
int truth(PyObject* o)
{
  const int v = PyObject_IsTrue(o);
  if (v < 0)
    throw python_error();
  return v;
}
segtopk_score score_of(PyObject* o)
{
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "softmax") == 0)
      return SEGTOPK_SOFTMAX;
    if (PyUnicode_CompareWithASCIIString(o, "sigmoid") == 0)
      return SEGTOPK_SIGMOID;
  }
  TORCH_CHECK_VALUE(false, "score must be one of softmax, sigmoid");
}
at::ScalarType dtype_of(PyObject* o)
{
  TORCH_CHECK_TYPE(THPDtype_Check(o), "a dtype is wanted");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
segtopk_dtype float_type(at::ScalarType t, const char* name)
{
  switch (t) {
  case at::kHalf: return SEGTOPK_F16;
  case at::kBFloat16: return SEGTOPK_BF16;
  case at::kFloat: return SEGTOPK_F32;
  default: TORCH_CHECK_VALUE(false, name, " must be float16, bfloat16 or float32");
  }
}
int id_bytes(const at::Tensor& t, const char* name)
{
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt || t.scalar_type() == at::kLong, name, " must be int32 or int64");
  return t.scalar_type() == at::kInt ? 4 : 8;
}
void want_args(Py_ssize_t n, Py_ssize_t wanted)
{
  TORCH_CHECK_TYPE(n == wanted, "expected ", wanted, " arguments, got ", n);
}

// Whether t's memory holds other values than t has: a view whose conjugation
// or negation torch has put off.
bool put_off(const at::Tensor& t) { return t.is_conj() || t.is_neg(); }
// The values of t in memory: t, or a copy.
at::Tensor values(const at::Tensor& t) { return put_off(t) ? t.resolve_conj().resolve_neg() : t; }

// Rows of contiguous elements: t, or a copy.
at::Tensor matrix(const at::Tensor& t, const char* name)
{
  TORCH_CHECK_VALUE(t.dim() == 2, name, " must have two dimensions");
  return values(t.stride(1) == 1 ? t : t.contiguous());
}
// A contiguous tensor of this shape and type: t, or a copy.
at::Tensor dense(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type)
{
  TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == type, name, " must be ", type, " of ", shape);
  return values(t).contiguous();
}

// The device of a call: that of its first tensor, made current if it is not.
struct Place {
  at::Device device;
  c10::cuda::OptionalCUDAGuard guard;
  explicit Place(const at::Tensor& t) : device(t.device())
  {
    TORCH_CHECK_VALUE(device.is_cuda(), "tensors must be on a CUDA device");
    if (c10::cuda::current_device() != device.index())
      guard.set_index(device.index());
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
  void same(const at::Tensor& t) const
  {
    TORCH_CHECK_VALUE(t.device() == device, "tensors must be on one CUDA device");
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const
  {
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
  }
  // `given` (None: a new tensor), to write to
  at::Tensor result(PyObject* given, const char* name, at::IntArrayRef shape, at::ScalarType type) const
  {
    if (given == Py_None)
      return empty(shape, type);
    const at::Tensor& t = tensor(given, name);
    TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == type && t.is_contiguous() && !put_off(t), name,
                      " must be contiguous, ", type, " of ", shape, " and no conjugated or negated view");
    // as torch does with outputs: autograd would not see the write
    TORCH_CHECK_VALUE(!t.requires_grad() || !c10::GradMode::is_enabled(), name, " must not require a gradient");
    same(t);
    return t;
  }
};

// After a call that wrote to `given` (None: to a new tensor): whoever saved it
// for a backward pass learns that it changed. Tensors of inference mode keep
// no count and are saved by nobody.
void written(PyObject* given, const at::Tensor& t)
{
  if (given != Py_None && !t.is_inference())
    t.unsafeGetTensorImpl()->bump_version();
}

struct Groups {
  at::Tensor rows; // [tokens, k]
  const int64_t* kept;
  int64_t tokens, slots;
  int32_t k;
};
Groups groups_of(PyObject* o, const Place& place)
{
  TORCH_CHECK_VALUE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 3, "groups must come from group_by_expert");
  const at::Tensor& offsets = tensor(PyTuple_GET_ITEM(o, 0), "groups.offsets");
  const at::Tensor& rows = tensor(PyTuple_GET_ITEM(o, 1), "groups.row_of_slot");
  TORCH_CHECK_VALUE(offsets.scalar_type() == at::kLong && offsets.dim() == 1 && offsets.is_contiguous() &&
                      offsets.numel() > 0 && rows.scalar_type() == at::kInt && rows.dim() == 2 &&
                      rows.is_contiguous() && rows.size(1) <= INT32_MAX && !put_off(offsets) && !put_off(rows),
                    "groups must come from group_by_expert");
  place.same(offsets);
  place.same(rows);
  return {rows, offsets.const_data_ptr<int64_t>() + (offsets.numel() - 1), rows.size(0), rows.numel(),
          (int32_t)rows.size(1)};
}

void check(int status)
{
  if (status == SEGTOPK_SUCCESS)
    return;
  PyObject* r = PyObject_CallFunction(raise_status, "i", status);
  Py_XDECREF(r);
  if (!PyErr_Occurred())
    PyErr_SetString(PyExc_RuntimeError, "segtopk call failed");
  throw python_error();
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
template <class... T>
PyObject* tuple(T&&... t)
{
  PyObject* all = PyTuple_New(sizeof...(t));
  if (!all)
    throw python_error();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(all, i++, wrap(std::forward<T>(t))), ...);
  return all;
}

// ---------------------------------------------------------------------------
// Operators (arguments by position: _rows.py)
// ---------------------------------------------------------------------------
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 6); // logits, k, score, renormalize, scale, bias
  const at::Tensor logits = matrix(tensor(a[0], "logits"), "logits");
  const segtopk_dtype type = float_type(logits.scalar_type(), "logits");
  const int32_t k = integer32(a[1], "k");
  const segtopk_score score = score_of(a[2]);
  const int renormalize = truth(a[3]);
  const float scale = real(a[4]);
  const Place place(logits);
  const int64_t tokens = logits.size(0), experts = logits.size(1);
  TORCH_CHECK_VALUE(experts <= INT32_MAX, "too many experts");
  at::Tensor bias;
  if (a[5] != Py_None) {
    bias = dense(tensor(a[5], "bias"), "bias", {experts}, at::kFloat);
    place.same(bias);
  }
  const int64_t shape[2] = {tokens, std::max(k, 0)};
  at::Tensor ids = place.empty(shape, at::kInt), weights = place.empty(shape, at::kFloat);
  check(lib.segtopk_route(type, logits.const_data_ptr(), tokens, (int32_t)experts, logits.stride(0), k, score,
                          renormalize, scale, bias.defined() ? bias.const_data_ptr<float>() : nullptr,
                          ids.mutable_data_ptr<int32_t>(), weights.mutable_data_ptr<float>(), place.stream()));
  return tuple(std::move(ids), std::move(weights));
  END_HANDLE_TH_ERRORS
}

PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 6); // grad_weights, logits, expert_ids, score, renormalize, scale
  const at::Tensor logits = matrix(tensor(a[1], "logits"), "logits");
  const segtopk_dtype type = float_type(logits.scalar_type(), "logits");
  const at::Tensor& given = tensor(a[2], "expert_ids");
  const int64_t tokens = logits.size(0), experts = logits.size(1), k = given.dim() == 2 ? given.size(1) : -1;
  TORCH_CHECK_VALUE(k <= INT32_MAX && experts <= INT32_MAX, "too many experts");
  const at::Tensor ids = dense(given, "expert_ids", {tokens, k}, at::kInt);
  const at::Tensor grad = dense(tensor(a[0], "grad_weights"), "grad_weights", {tokens, k}, at::kFloat);
  const segtopk_score score = score_of(a[3]);
  const int renormalize = truth(a[4]);
  const float scale = real(a[5]);
  const Place place(logits);
  place.same(ids);
  place.same(grad);
  at::Tensor out = place.empty({tokens, experts}, logits.scalar_type());
  check(lib.segtopk_route_backward(type, grad.const_data_ptr<float>(), logits.const_data_ptr(), tokens,
                                   (int32_t)experts, logits.stride(0), (int32_t)k, ids.const_data_ptr<int32_t>(),
                                   score, renormalize, scale, out.mutable_data_ptr(), place.stream()));
  return wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

PyObject* group(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 2); // expert_ids, num_experts
  const at::Tensor& given = tensor(a[0], "expert_ids");
  const int bytes = id_bytes(given, "expert_ids");
  TORCH_CHECK_VALUE(given.dim() == 2, "expert_ids must have two dimensions");
  const at::Tensor ids = values(given).contiguous();
  const int32_t experts = integer32(a[1], "num_experts");
  const Place place(ids);
  const int64_t slots = ids.numel();
  at::Tensor offsets = place.empty({(int64_t)std::max(experts, 0) + 1}, at::kLong);
  at::Tensor rows = place.empty(ids.sizes(), at::kInt), slot_of_row = place.empty({slots}, at::kInt);
  const size_t need = lib.segtopk_group_workspace_bytes(slots, experts);
  at::Tensor space;
  if (need > 0)
    space = place.empty({(int64_t)need}, at::kByte);
  check(lib.segtopk_group(ids.const_data_ptr(), bytes, slots, experts, offsets.mutable_data_ptr<int64_t>(),
                          rows.mutable_data_ptr<int32_t>(), slot_of_row.mutable_data_ptr<int32_t>(),
                          need > 0 ? space.mutable_data_ptr() : nullptr, need, place.stream()));
  return tuple(std::move(offsets), std::move(rows), std::move(slot_of_row));
  END_HANDLE_TH_ERRORS
}

PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 3); // x, groups, out
  const at::Tensor x = matrix(tensor(a[0], "x"), "x");
  const Place place(x);
  const Groups g = groups_of(a[1], place);
  TORCH_CHECK_VALUE(x.size(0) == g.tokens, "x must have a row for each token of the groups");
  const int64_t width = x.size(1);
  at::Tensor out = place.result(a[2], "out", {g.slots, width}, x.scalar_type());
  check(lib.segtopk_dispatch(x.const_data_ptr(), (int32_t)x.element_size(), g.tokens, g.k, width, x.stride(0),
                             g.rows.const_data_ptr<int32_t>(), g.kept, out.mutable_data_ptr(), place.stream()));
  written(a[2], out);
  return wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 4); // rows, groups, weights or None, out
  const at::Tensor rows = matrix(tensor(a[0], "rows"), "rows");
  const segtopk_dtype type = float_type(rows.scalar_type(), "rows");
  const Place place(rows);
  const Groups g = groups_of(a[1], place);
  TORCH_CHECK_VALUE(rows.size(0) == g.slots, "rows must have a row for each slot of the groups");
  at::Tensor weights;
  if (a[2] != Py_None) {
    weights = dense(tensor(a[2], "weights"), "weights", g.rows.sizes(), at::kFloat);
    place.same(weights);
  }
  const int64_t width = rows.size(1);
  at::Tensor out = place.result(a[3], "out", {g.tokens, width}, rows.scalar_type());
  check(lib.segtopk_combine(type, rows.const_data_ptr(), g.tokens, g.k, width, rows.stride(0),
                            g.rows.const_data_ptr<int32_t>(),
                            weights.defined() ? weights.const_data_ptr<float>() : nullptr, out.mutable_data_ptr(),
                            place.stream()));
  written(a[3], out);
  return wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 4); // grad_out, rows, groups, weights
  const at::Tensor rows = matrix(tensor(a[1], "rows"), "rows");
  const segtopk_dtype type = float_type(rows.scalar_type(), "rows");
  const at::Tensor grad = matrix(tensor(a[0], "grad_out"), "grad_out");
  const Place place(rows);
  const Groups g = groups_of(a[2], place);
  const int64_t width = rows.size(1);
  TORCH_CHECK_VALUE(rows.size(0) == g.slots, "rows must have a row for each slot of the groups");
  TORCH_CHECK_VALUE(grad.size(0) == g.tokens && grad.size(1) == width && grad.scalar_type() == rows.scalar_type(),
                    "grad_out must be ", rows.scalar_type(), " of [", g.tokens, ", ", width, "]");
  const at::Tensor weights = dense(tensor(a[3], "weights"), "weights", g.rows.sizes(), at::kFloat);
  place.same(grad);
  place.same(weights);
  at::Tensor grad_rows = place.empty({g.slots, width}, rows.scalar_type());
  at::Tensor grad_weights = place.empty(g.rows.sizes(), at::kFloat);
  check(lib.segtopk_combine_backward(type, grad.const_data_ptr(), grad.stride(0), rows.const_data_ptr(),
                                     rows.stride(0), g.tokens, g.k, width, g.rows.const_data_ptr<int32_t>(), g.kept,
                                     weights.const_data_ptr<float>(), grad_rows.mutable_data_ptr(),
                                     grad_weights.mutable_data_ptr<float>(), place.stream()));
  return tuple(std::move(grad_rows), std::move(grad_weights));
  END_HANDLE_TH_ERRORS
}

PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 5); // table, tokens, scale, out_dtype or None, out
  const at::Tensor table = matrix(tensor(a[0], "table"), "table");
  const segtopk_dtype type = float_type(table.scalar_type(), "table");
  const at::Tensor& given = tensor(a[1], "tokens");
  const int bytes = id_bytes(given, "tokens");
  const at::Tensor tokens = values(given).contiguous();
  const float scale = real(a[2]);
  const Place place(table);
  place.same(tokens);
  at::ScalarType out_type = table.scalar_type();
  if (a[3] != Py_None)
    out_type = dtype_of(a[3]);
  else if (a[4] != Py_None)
    out_type = tensor(a[4], "out").scalar_type();
  const segtopk_dtype out_code = float_type(out_type, "out");
  at::DimVector shape(tokens.sizes());
  shape.push_back(table.size(1));
  at::Tensor out = place.result(a[4], "out", shape, out_type);
  check(lib.segtopk_embedding(type, table.const_data_ptr(), table.size(0), table.size(1), table.stride(0),
                              tokens.const_data_ptr(), bytes, tokens.numel(), scale, out_code,
                              out.mutable_data_ptr(), place.stream()));
  written(a[4], out);
  return wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

PyObject* embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 8); // grad_out, tokens, num_rows, scale, padding_idx or None, dtype or None, grad_table, accumulate
  const at::Tensor& given = tensor(a[0], "grad_out");
  const segtopk_dtype type = float_type(given.scalar_type(), "grad_out");
  const at::Tensor& given_tokens = tensor(a[1], "tokens");
  const int bytes = id_bytes(given_tokens, "tokens");
  TORCH_CHECK_VALUE(given.dim() >= 1 && given.sizes().slice(0, given.dim() - 1) == given_tokens.sizes(),
                    "grad_out must have a row for each token");
  const at::Tensor tokens = values(given_tokens).contiguous();
  const int64_t count = tokens.numel(), width = given.size(-1), num_rows = integer(a[2]);
  const at::Tensor grad = matrix(given.dim() == 2 ? given : given.reshape({count, width}), "grad_out");
  const float scale = real(a[3]);
  int64_t padding = -1;
  if (a[4] != Py_None) {
    padding = integer(a[4]);
    TORCH_CHECK_VALUE(-num_rows <= padding && padding < num_rows, "padding_idx must be a row of the table");
    if (padding < 0)
      padding += num_rows;
  }
  const Place place(grad);
  place.same(tokens);
  const int accumulate = truth(a[7]);
  TORCH_CHECK_VALUE(!accumulate || a[6] != Py_None, "accumulate needs grad_table");
  at::ScalarType table_type = grad.scalar_type();
  if (a[5] != Py_None)
    table_type = dtype_of(a[5]);
  else if (a[6] != Py_None)
    table_type = tensor(a[6], "grad_table").scalar_type();
  const segtopk_dtype table_code = float_type(table_type, "grad_table");
  at::Tensor out = place.result(a[6], "grad_table", {std::max<int64_t>(num_rows, 0), width}, table_type);
  const size_t need = lib.segtopk_embedding_backward_workspace_bytes(count, num_rows, width);
  at::Tensor space = place.empty({(int64_t)need}, at::kByte);
  check(lib.segtopk_embedding_backward(type, grad.const_data_ptr(), grad.stride(0), tokens.const_data_ptr(), bytes,
                                       count, num_rows, width, padding, scale, table_code, out.mutable_data_ptr(),
                                       accumulate, space.mutable_data_ptr(), need, place.stream()));
  written(a[6], out);
  return wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the entry points by name, function that raises for a status)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 2);
  Library got;
#define X(NAME)                                                                                                  \
  {                                                                                                              \
    PyObject* at = PyMapping_GetItemString(a[0], #NAME);                                                         \
    if (!at)                                                                                                     \
      throw python_error();                                                                                      \
    got.NAME = reinterpret_cast<decltype(&::NAME)>(PyLong_AsVoidPtr(at));                                        \
    Py_DECREF(at);                                                                                               \
    if (PyErr_Occurred())                                                                                        \
      throw python_error();                                                                                      \
  }
  SEGTOPK_ENTRIES(X)
#undef X
  lib = got;
  Py_INCREF(a[1]);
  Py_XSETREF(raise_status, a[1]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define FUNCTION(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FUNCTION(bind),      FUNCTION(route),    FUNCTION(route_backward),
                         FUNCTION(group),     FUNCTION(dispatch), FUNCTION(combine),
                         FUNCTION(combine_backward), FUNCTION(embedding), FUNCTION(embedding_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rows_native", nullptr, -1, methods};

} // namespace

PyMODINIT_FUNC PyInit__rows_native() { return PyModule_Create(&module); }
