// Python binding of the row operators (include/segtopk.h: routing, tokens
// sorted by expert and back, the experts' products, layer norm, embedding):
// checks tensors, makes the results and calls the C entry points on the
// current stream. _rows.py holds the
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
  X(segtopk_route_groups)                                                                                        \
  X(segtopk_route_backward)                                                                                      \
  X(segtopk_group)                                                                                               \
  X(segtopk_group_workspace_bytes)                                                                               \
  X(segtopk_dispatch)                                                                                            \
  X(segtopk_combine)                                                                                             \
  X(segtopk_combine_backward)                                                                                    \
  X(segtopk_embedding)                                                                                           \
  X(segtopk_embedding_backward)                                                                                  \
  X(segtopk_embedding_backward_workspace_bytes)                                                                  \
  X(segtopk_expert_matmul)                                                                                       \
  X(segtopk_expert_matmul_f8)                                                                                    \
  X(segtopk_expert_matmul_weights)                                                                               \
  X(segtopk_layer_norm)                                                                                          \
  X(segtopk_layer_norm_backward)                                                                                 \
  X(segtopk_layer_norm_backward_workspace_bytes)                                                                 \
  X(segtopk_quantize_rows)

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
segtopk_group_score group_score_of(PyObject* o)
{
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "best") == 0)
      return SEGTOPK_GROUP_BEST;
    if (PyUnicode_CompareWithASCIIString(o, "best_two") == 0)
      return SEGTOPK_GROUP_BEST_TWO;
  }
  TORCH_CHECK_VALUE(false, "group_score must be one of best, best_two");
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
  const int64_t* kept;    // the last of the offsets
  const int64_t* offsets;
  int64_t tokens, slots, experts;
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
  const int64_t* first = offsets.const_data_ptr<int64_t>();
  const int64_t experts = offsets.numel() - 1;
  return {rows, first + experts, first, rows.size(0), rows.numel(), experts, (int32_t)rows.size(1)};
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
  want_args(n, 9); // logits, k, score, renormalize, scale, bias, num_groups, groups_kept, group_score
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
  const int32_t groups = integer32(a[6], "num_groups");
  const int32_t kept = a[7] == Py_None ? groups : integer32(a[7], "groups_kept");
  const segtopk_group_score group_score = group_score_of(a[8]);
  if (groups != 1 || kept != 1)
    check(lib.segtopk_route_groups(type, logits.const_data_ptr(), tokens, (int32_t)experts, logits.stride(0), k, groups,
                                   kept, group_score, score, renormalize, scale,
                                   bias.defined() ? bias.const_data_ptr<float>() : nullptr,
                                   ids.mutable_data_ptr<int32_t>(), weights.mutable_data_ptr<float>(), place.stream()));
  else
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

// Rows as the tensor cores' operands are read, at least 16 bytes apart in
// steps of 16 from a 16-byte address: t, or a copy.
at::Tensor operand_rows(const at::Tensor& t, const char* name)
{
  const at::Tensor m = matrix(t, name);
  const int64_t size = m.element_size();
  const bool fits = reinterpret_cast<uintptr_t>(m.const_data_ptr()) % 16 == 0 &&
                    (m.size(0) <= 1 || (m.stride(0) >= m.size(1) && m.stride(0) * size % 16 == 0));
  return fits ? m : m.clone(at::MemoryFormat::Contiguous);
}
int64_t row_stride(const at::Tensor& m) { return m.size(0) <= 1 ? m.size(1) : m.stride(0); }

// The experts' matrices [experts, out, in], one of the last two dimensions
// contiguous: t, or a copy.
struct Matrices {
  at::Tensor t;
  int64_t expert_stride, out_stride, in_stride;
  bool turned() const { return in_stride != 1; }
};
Matrices matrices(const at::Tensor& given)
{
  TORCH_CHECK_VALUE(given.dim() == 3, "weights must have three dimensions");
  const at::Tensor t = values(given);
  auto view = [](const at::Tensor& w) {
    const int64_t n = w.size(1), k = w.size(2);
    // strides along dimensions of one element say nothing
    Matrices m{w, w.stride(0), n == 1 ? k : w.stride(1), k == 1 ? 1 : w.stride(2)};
    if (m.in_stride != 1 && k > 1 && n > 1 && w.stride(1) == 1)
      m.out_stride = 1;
    if (w.size(0) <= 1)
      m.expert_stride = n * k;
    return m;
  };
  Matrices m = view(t);
  const int64_t size = t.element_size(), n = t.size(1), k = t.size(2);
  const int64_t line = m.turned() ? m.in_stride : m.out_stride;
  const bool fits = (m.in_stride == 1 ? m.out_stride >= k : m.out_stride == 1 && m.in_stride >= n) &&
                    reinterpret_cast<uintptr_t>(t.const_data_ptr()) % 16 == 0 && line * size % 16 == 0 &&
                    m.expert_stride * size % 16 == 0 && m.expert_stride >= n * k;
  return fits ? m : view(t.clone(at::MemoryFormat::Contiguous));
}

PyObject* expert_matmul(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 7); // rows, weights, groups, row_scales or None, weight_scales or None, out_dtype or None, out
  const at::Tensor rows = operand_rows(tensor(a[0], "rows"), "rows");
  const at::ScalarType type = rows.scalar_type();
  const bool eight = type == at::kFloat8_e4m3fn;
  TORCH_CHECK_VALUE(eight || type == at::kHalf || type == at::kBFloat16,
                    "rows must be float16, bfloat16 or float8_e4m3fn");
  const at::Tensor& given = tensor(a[1], "weights");
  TORCH_CHECK_VALUE(given.scalar_type() == type && given.dim() == 3 && given.size(2) == rows.size(1), "weights must be ",
                    type, " of [experts, out, ", rows.size(1), "]");
  TORCH_CHECK_VALUE(eight == (a[3] != Py_None) && eight == (a[4] != Py_None),
                    "float8_e4m3fn rows and weights have row_scales and weight_scales, others have none");
  const Place place(rows);
  place.same(given);
  Matrices w = matrices(given);
  if (eight && w.turned())
    w = matrices(given.contiguous());
  const Groups g = groups_of(a[2], place);
  const int64_t experts = given.size(0), out_width = given.size(1), width = given.size(2);
  TORCH_CHECK_VALUE(rows.size(0) == g.slots, "rows must have a row for each slot of the groups");
  TORCH_CHECK_VALUE(experts == g.experts && experts <= INT32_MAX, "weights must have a matrix for each expert of the groups");
  at::ScalarType out_type = eight ? at::kBFloat16 : type;
  if (a[5] != Py_None)
    out_type = dtype_of(a[5]);
  else if (a[6] != Py_None)
    out_type = tensor(a[6], "out").scalar_type();
  const segtopk_dtype out_code = float_type(out_type, "out");
  at::Tensor row_scales, weight_scales;
  if (eight) {
    const int64_t blocks = (width + 127) / 128;
    row_scales = matrix(tensor(a[3], "row_scales"), "row_scales");
    TORCH_CHECK_VALUE(row_scales.scalar_type() == at::kFloat && row_scales.size(0) == g.slots &&
                        row_scales.size(1) == blocks,
                      "row_scales must be float32 of [", g.slots, ", ", blocks, "]");
    weight_scales = dense(tensor(a[4], "weight_scales"), "weight_scales", {experts, (out_width + 127) / 128, blocks},
                          at::kFloat);
    place.same(row_scales);
    place.same(weight_scales);
  }
  at::Tensor out = place.result(a[6], "out", {g.slots, out_width}, out_type);
  if (eight)
    check(lib.segtopk_expert_matmul_f8(rows.const_data_ptr(), g.slots, width, row_stride(rows),
                                       row_scales.const_data_ptr<float>(), row_scales.stride(0), w.t.const_data_ptr(),
                                       (int32_t)experts, out_width, w.expert_stride, w.out_stride,
                                       weight_scales.const_data_ptr<float>(), g.offsets, out_code,
                                       out.mutable_data_ptr(), place.stream()));
  else
    check(lib.segtopk_expert_matmul(float_type(type, "rows"), rows.const_data_ptr(), g.slots, width, row_stride(rows),
                                    w.t.const_data_ptr(), (int32_t)experts, out_width, w.expert_stride, w.out_stride,
                                    w.in_stride, g.offsets, out_code, out.mutable_data_ptr(), place.stream()));
  written(a[6], out);
  return wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

PyObject* expert_matmul_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 5); // grad_out, rows, weights, groups, dtype or None
  const at::Tensor grad = operand_rows(tensor(a[0], "grad_out"), "grad_out");
  const at::Tensor rows = operand_rows(tensor(a[1], "rows"), "rows");
  const at::Tensor& given = tensor(a[2], "weights");
  const at::ScalarType type = rows.scalar_type();
  TORCH_CHECK_VALUE(type == at::kHalf || type == at::kBFloat16, "rows must be float16 or bfloat16");
  TORCH_CHECK_VALUE(given.scalar_type() == type && given.dim() == 3 && given.size(2) == rows.size(1), "weights must be ",
                    type, " of [experts, out, ", rows.size(1), "]");
  const Place place(rows);
  place.same(given);
  place.same(grad);
  const Matrices w = matrices(given);
  const Groups g = groups_of(a[3], place);
  const int64_t experts = given.size(0), out_width = given.size(1), width = given.size(2);
  TORCH_CHECK_VALUE(rows.size(0) == g.slots, "rows must have a row for each slot of the groups");
  TORCH_CHECK_VALUE(experts == g.experts && experts <= INT32_MAX, "weights must have a matrix for each expert of the groups");
  TORCH_CHECK_VALUE(grad.scalar_type() == type && grad.size(0) == g.slots && grad.size(1) == out_width,
                    "grad_out must be ", type, " of [", g.slots, ", ", out_width, "]");
  const at::ScalarType weight_type = a[4] != Py_None ? dtype_of(a[4]) : type;
  const segtopk_dtype weight_code = float_type(weight_type, "grad_weights"), code = float_type(type, "rows");
  at::Tensor grad_rows = place.empty({g.slots, width}, type);
  check(lib.segtopk_expert_matmul(code, grad.const_data_ptr(), g.slots, out_width, row_stride(grad),
                                  w.t.const_data_ptr(), (int32_t)experts, width, w.expert_stride, w.in_stride,
                                  w.out_stride, g.offsets, code, grad_rows.mutable_data_ptr(), place.stream()));
  // in the layout of the weights
  at::Tensor grad_weights = w.turned() ? place.empty({experts, width, out_width}, weight_type)
                                       : place.empty({experts, out_width, width}, weight_type);
  const at::Tensor &outer = w.turned() ? rows : grad, &inner = w.turned() ? grad : rows;
  check(lib.segtopk_expert_matmul_weights(code, outer.const_data_ptr(), outer.size(1), row_stride(outer),
                                          inner.const_data_ptr(), inner.size(1), row_stride(inner), g.slots,
                                          (int32_t)experts, g.offsets, weight_code, grad_weights.mutable_data_ptr(),
                                          place.stream()));
  return tuple(std::move(grad_rows), w.turned() ? grad_weights.transpose(1, 2) : std::move(grad_weights));
  END_HANDLE_TH_ERRORS
}

// A row of `width` values of x's type or float32: t, or a contiguous copy.
at::Tensor norm_weight(PyObject* o, const char* name, const at::Tensor& x, const Place& place)
{
  const at::Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == x.size(1) &&
                      (t.scalar_type() == x.scalar_type() || t.scalar_type() == at::kFloat),
                    name, " must be ", x.scalar_type(), " or float32 of [", x.size(1), "]");
  place.same(t);
  return values(t).contiguous();
}

PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 5); // x, weight, bias or None, eps, out
  const at::Tensor x = matrix(tensor(a[0], "x"), "x");
  const segtopk_dtype type = float_type(x.scalar_type(), "x");
  const Place place(x);
  const at::Tensor weight = norm_weight(a[1], "weight", x, place);
  at::Tensor bias;
  if (a[2] != Py_None) {
    bias = norm_weight(a[2], "bias", x, place);
    TORCH_CHECK_VALUE(bias.scalar_type() == weight.scalar_type(), "bias must be ", weight.scalar_type(), ", as weight");
  }
  const float eps = real(a[3]);
  const int64_t rows = x.size(0), width = x.size(1);
  at::Tensor out = place.result(a[4], "out", {rows, width}, x.scalar_type());
  at::Tensor mean = place.empty({rows}, at::kFloat), rstd = place.empty({rows}, at::kFloat);
  check(lib.segtopk_layer_norm(type, x.const_data_ptr(), rows, width, x.stride(0), float_type(weight.scalar_type(), "weight"),
                               weight.const_data_ptr(), bias.defined() ? bias.const_data_ptr() : nullptr, eps,
                               out.mutable_data_ptr(), mean.mutable_data_ptr<float>(), rstd.mutable_data_ptr<float>(),
                               place.stream()));
  written(a[4], out);
  return tuple(std::move(out), std::move(mean), std::move(rstd));
  END_HANDLE_TH_ERRORS
}

PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 5); // grad_out, x, weight, mean, rstd
  const at::Tensor x = matrix(tensor(a[1], "x"), "x");
  const segtopk_dtype type = float_type(x.scalar_type(), "x");
  const at::Tensor grad = matrix(tensor(a[0], "grad_out"), "grad_out");
  TORCH_CHECK_VALUE(grad.sizes() == x.sizes() && grad.scalar_type() == x.scalar_type(), "grad_out must be ",
                    x.scalar_type(), " of ", x.sizes());
  const Place place(x);
  const at::Tensor weight = norm_weight(a[2], "weight", x, place);
  const int64_t rows = x.size(0), width = x.size(1);
  const at::Tensor mean = dense(tensor(a[3], "mean"), "mean", {rows}, at::kFloat);
  const at::Tensor rstd = dense(tensor(a[4], "rstd"), "rstd", {rows}, at::kFloat);
  place.same(grad);
  place.same(mean);
  place.same(rstd);
  at::Tensor grad_x = place.empty({rows, width}, x.scalar_type());
  at::Tensor grad_weight = place.empty({width}, weight.scalar_type()), grad_bias = place.empty({width}, weight.scalar_type());
  const size_t need = lib.segtopk_layer_norm_backward_workspace_bytes(rows, width);
  at::Tensor space = place.empty({(int64_t)need}, at::kByte);
  check(lib.segtopk_layer_norm_backward(type, grad.const_data_ptr(), grad.stride(0), x.const_data_ptr(), rows, width,
                                        x.stride(0), float_type(weight.scalar_type(), "weight"), weight.const_data_ptr(),
                                        mean.const_data_ptr<float>(), rstd.const_data_ptr<float>(),
                                        grad_x.mutable_data_ptr(), grad_weight.mutable_data_ptr(),
                                        grad_bias.mutable_data_ptr(), space.mutable_data_ptr(), need, place.stream()));
  return tuple(std::move(grad_x), std::move(grad_weight), std::move(grad_bias));
  END_HANDLE_TH_ERRORS
}

PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n)
{
  HANDLE_TH_ERRORS
  want_args(n, 1); // x
  const at::Tensor x = matrix(tensor(a[0], "x"), "x");
  const segtopk_dtype type = float_type(x.scalar_type(), "x");
  const Place place(x);
  const int64_t rows = x.size(0), width = x.size(1);
  at::Tensor out = place.empty({rows, width}, at::kFloat8_e4m3fn);
  at::Tensor scales = place.empty({rows, (width + 127) / 128}, at::kFloat);
  check(lib.segtopk_quantize_rows(type, x.const_data_ptr(), rows, width, x.stride(0), out.mutable_data_ptr(),
                                  scales.mutable_data_ptr<float>(), place.stream()));
  return tuple(std::move(out), std::move(scales));
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
                         FUNCTION(expert_matmul),    FUNCTION(expert_matmul_backward),
                         FUNCTION(layer_norm),       FUNCTION(layer_norm_backward), FUNCTION(quantize_rows),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rows_native", nullptr, -1, methods};

} // namespace

PyMODINIT_FUNC PyInit__rows_native() { return PyModule_Create(&module); }
