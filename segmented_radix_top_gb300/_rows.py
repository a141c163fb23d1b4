"""ctypes binding of the row operators of libsegtopk.so: expert routing,
tokens sorted by expert and back, token embedding, and their gradients
(argument marshalling only; include/segtopk.h has each operator's contract).

Inputs are CUDA tensors on one device. Rows may lie any distance apart (a
part of a wider tensor's columns, one row expanded to many); tensors whose
rows are not contiguous are copied first. Everything runs on the current
stream, or on `stream`, from whose memory pool results and workspaces then
come. Nothing here synchronises, so all of it can be captured in a graph.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import _binding as B

SCORE = {"softmax": 0, "sigmoid": 1}
MAX_EXPERTS = 1024    # SEGTOPK_MAX_EXPERTS
ROUTE_MAX_K = 32      # SEGTOPK_ROUTE_MAX_K
DEVICE_ERROR_INDEX = 4  # SEGTOPK_DEVICE_ERROR_INDEX

_FLOAT = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_INT_BYTES = {torch.int32: 4, torch.int64: 8}

# The current stream's handle and the current device, without building a Stream
# object or entering torch.cuda's lazy initialisation (the tensors are on the
# GPU already): the calls take about as long as the smallest kernels.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_empty = torch.empty


class ExpertGroups(NamedTuple):
    """Token slots sorted by expert (segtopk_group)."""
    offsets: torch.Tensor      # int64 [experts + 1]: expert e has the sorted rows offsets[e] to offsets[e + 1]
    row_of_slot: torch.Tensor  # int32 [tokens, k]: each slot's sorted row, -1 for none
    slot_of_row: torch.Tensor  # int32 [tokens * k]: each sorted row's slot, -1 past the last one


def declare(L) -> None:
    """Argument types of the row operators (called once per loaded library)."""
    i, i32, i64, f, vp, sz = (ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p,
                              ctypes.c_size_t)
    for name, result, args in (
            ("route", i, [i, vp, i64, i32, i64, i32, i, i, f, vp, vp, vp, vp]),
            ("route_backward", i, [i, vp, vp, i64, i32, i64, i32, vp, i, i, f, vp, vp]),
            ("group_workspace_bytes", sz, [i64, i32]),
            ("group", i, [vp, i32, i64, i32, vp, vp, vp, vp, sz, vp]),
            ("dispatch", i, [vp, i32, i64, i32, i64, i64, vp, vp, vp, vp]),
            ("combine", i, [i, vp, i64, i32, i64, i64, vp, vp, vp, vp]),
            ("combine_backward", i, [i, vp, i64, vp, i64, i64, i32, i64, vp, vp, vp, vp, vp, vp]),
            ("embedding", i, [i, vp, i64, i64, i64, vp, i32, i64, f, i, vp, vp]),
            ("embedding_backward_workspace_bytes", sz, [i64, i64, i64]),
            ("embedding_backward", i, [i, vp, i64, vp, i32, i64, i64, i64, i64, f, i, vp, i, vp, sz, vp])):
        fn = getattr(L, "segtopk_" + name)
        fn.restype, fn.argtypes = result, args


def _on_stream(call):
    """Gives an operator its `stream` argument: the call, its results and its
    workspace belong to that stream."""
    @functools.wraps(call)
    def wrapped(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return wrapped


def _run(fn, device, *args):
    """Calls a C entry point on the current stream of a tensor's device (its
    index, as Tensor.get_device gives it)."""
    if device < 0:
        raise ValueError("tensors must be on a CUDA device")
    if device == _current_device():
        rc = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(device))
    if rc:
        B._check(rc)


def _same_device(device, *tensors):
    for t in tensors:
        if t.get_device() != device:
            raise ValueError("tensors must be on one CUDA device")


def _float(t, name) -> int:
    code = _FLOAT.get(t.dtype)
    if code is None:
        raise ValueError("%s must be float16, bfloat16 or float32" % name)
    return code


def _matrix(t, name):
    """t as rows of contiguous elements (a copy where it has none)."""
    if t.dim() != 2:
        raise ValueError("%s must have two dimensions" % name)
    return t if t.stride(1) == 1 else t.contiguous()


def _dense(t, name, shape, dtype):
    """A contiguous tensor of this shape and type (t, or a copy)."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError("%s must be %s of %s" % (name, dtype, tuple(shape)))
    return t if t.is_contiguous() else t.contiguous()


def _given(out, name, shape, dtype, device):
    """Checks a tensor to write to."""
    if out.shape != shape or out.dtype != dtype or not out.is_contiguous():
        raise ValueError("%s must be contiguous, %s of %s" % (name, dtype, tuple(shape)))
    _same_device(device, out)
    return out


def _score(score) -> int:
    code = SCORE.get(score)
    if code is None:
        raise ValueError("score must be one of %s" % ", ".join(SCORE))
    return code


@_on_stream
def route(logits: torch.Tensor, k: int, *, score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
          bias=None):
    """The k best experts of each token and their weights (segtopk_route).

    logits: [tokens, experts]. score: "softmax" (over all experts) or
    "sigmoid"; renormalize divides by the sum of the k chosen scores; scale
    multiplies. bias: optional float32 [experts], added to the scores for the
    choice only. Experts with a logit of -inf are never chosen. Returns
    (expert_ids int32 [tokens, k], best first and -1 where none is left,
    weights float32 [tokens, k])."""
    L = B.load()
    how, kind = _score(score), _float(logits, "logits")
    logits = _matrix(logits, "logits")
    device, tokens, experts = logits.get_device(), *logits.shape
    at = None
    if bias is not None:
        bias = _dense(bias, "bias", (experts,), torch.float32)
        _same_device(device, bias)
        at = bias.data_ptr()
    shape, place = (tokens, max(k, 0)), logits.device
    ids = _empty(shape, dtype=torch.int32, device=place)
    weights = _empty(shape, dtype=torch.float32, device=place)
    _run(L.segtopk_route, device, kind, logits.data_ptr(), tokens, experts, logits.stride(0), k, how, bool(renormalize),
         scale, at, ids.data_ptr(), weights.data_ptr())
    return ids, weights


@_on_stream
def route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, expert_ids: torch.Tensor, *,
                   score: str = "softmax", renormalize: bool = True, scale: float = 1.0):
    """Gradient of route()'s logits from that of its weights
    (segtopk_route_backward): [tokens, experts] of the logits' type."""
    L = B.load()
    how, kind = _score(score), _float(logits, "logits")
    logits = _matrix(logits, "logits")
    device, tokens, experts = logits.get_device(), *logits.shape
    k = expert_ids.shape[-1]
    ids = _dense(expert_ids, "expert_ids", (tokens, k), torch.int32)
    grad = _dense(grad_weights, "grad_weights", (tokens, k), torch.float32)
    _same_device(device, ids, grad)
    out = _empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    _run(L.segtopk_route_backward, device, kind, grad.data_ptr(), logits.data_ptr(), tokens, experts, logits.stride(0),
         k, ids.data_ptr(), how, bool(renormalize), scale, out.data_ptr())
    return out


@_on_stream
def group_by_expert(expert_ids: torch.Tensor, num_experts: int) -> ExpertGroups:
    """Sorts the slots of expert_ids [tokens, k] (int32 or int64, negative:
    no expert) by expert, stably (segtopk_group)."""
    L = B.load()
    id_bytes = _INT_BYTES.get(expert_ids.dtype)
    if id_bytes is None or expert_ids.dim() != 2:
        raise ValueError("expert_ids must be int32 or int64 of two dimensions")
    ids = expert_ids if expert_ids.is_contiguous() else expert_ids.contiguous()
    place, slots = ids.device, ids.numel()
    offsets = _empty(max(num_experts, 0) + 1, dtype=torch.int64, device=place)
    rows = _empty(ids.shape, dtype=torch.int32, device=place)
    slot_of_row = _empty(slots, dtype=torch.int32, device=place)
    need = L.segtopk_group_workspace_bytes(slots, num_experts)
    space = _empty(need, dtype=torch.uint8, device=place) if need else None
    _run(L.segtopk_group, ids.get_device(), ids.data_ptr(), id_bytes, slots, num_experts, offsets.data_ptr(),
         rows.data_ptr(), slot_of_row.data_ptr(), space.data_ptr() if need else None, need)
    return ExpertGroups(offsets, rows, slot_of_row)


def _groups(groups, device):
    """The rows of the slots, and the address of the number of kept ones."""
    offsets, rows, _ = groups
    if offsets.dtype != torch.int64 or rows.dtype != torch.int32 or rows.dim() != 2 or offsets.dim() != 1 \
            or not (rows.is_contiguous() and offsets.is_contiguous()) or offsets.numel() < 1:
        raise ValueError("groups must come from group_by_expert")
    _same_device(device, rows, offsets)
    return rows, offsets.data_ptr() + 8 * (offsets.numel() - 1)


@_on_stream
def dispatch(x: torch.Tensor, groups: ExpertGroups, *, out=None):
    """The tokens' rows in the order of their experts (segtopk_dispatch):
    x [tokens, width] of any element type of 1 to 8 bytes; returns [tokens *
    k, width], zeros from row groups.offsets[-1] on."""
    L = B.load()
    x = _matrix(x, "x")
    device = x.get_device()
    rows, kept = _groups(groups, device)
    tokens, k = rows.shape
    count, width = x.shape
    if count != tokens:
        raise ValueError("x must have a row for each token of the groups")
    shape = (tokens * k, width)
    if out is None:
        out = _empty(shape, dtype=x.dtype, device=x.device)
    else:
        _given(out, "out", shape, x.dtype, device)
    _run(L.segtopk_dispatch, device, x.data_ptr(), x.element_size(), tokens, k, width, x.stride(0), rows.data_ptr(),
         kept, out.data_ptr())
    return out


def _combine(values, groups, weights, out):
    L = B.load()
    kind = _float(values, "rows")
    values = _matrix(values, "rows")
    device = values.get_device()
    rows, _ = _groups(groups, device)
    tokens, k = rows.shape
    count, width = values.shape
    if count != tokens * k:
        raise ValueError("rows must have a row for each slot of the groups")
    at = None
    if weights is not None:
        weights = _dense(weights, "weights", rows.shape, torch.float32)
        _same_device(device, weights)
        at = weights.data_ptr()
    if out is None:
        out = _empty((tokens, width), dtype=values.dtype, device=values.device)
    else:
        _given(out, "out", (tokens, width), values.dtype, device)
    _run(L.segtopk_combine, device, kind, values.data_ptr(), tokens, k, width, values.stride(0), rows.data_ptr(), at,
         out.data_ptr())
    return out


@_on_stream
def dispatch_backward(grad_rows: torch.Tensor, groups: ExpertGroups, *, out=None):
    """Gradient of dispatch()'s x (segtopk_combine without weights): the sum
    of each token's rows of grad_rows [tokens * k, width]."""
    return _combine(grad_rows, groups, None, out)


@_on_stream
def combine(rows: torch.Tensor, groups: ExpertGroups, weights: torch.Tensor, *, out=None):
    """The sorted rows back at their tokens, weighted and summed
    (segtopk_combine): rows [tokens * k, width], weights float32 [tokens, k];
    returns [tokens, width]."""
    if weights is None:
        raise ValueError("weights must be a tensor")
    return _combine(rows, groups, weights, out)


@_on_stream
def combine_backward(grad_out: torch.Tensor, rows: torch.Tensor, groups: ExpertGroups, weights: torch.Tensor):
    """Gradients of combine()'s rows and weights (segtopk_combine_backward):
    ([tokens * k, width] with zeros from row groups.offsets[-1] on, float32
    [tokens, k] with zeros for slots without an expert)."""
    L = B.load()
    kind = _float(rows, "rows")
    values, grad = _matrix(rows, "rows"), _matrix(grad_out, "grad_out")
    device, place = values.get_device(), values.device
    at, kept = _groups(groups, device)
    tokens, k = at.shape
    count, width = values.shape
    if count != tokens * k:
        raise ValueError("rows must have a row for each slot of the groups")
    if grad.shape != (tokens, width) or grad.dtype != values.dtype:
        raise ValueError("grad_out must be %s of %s" % (values.dtype, (tokens, width)))
    weights = _dense(weights, "weights", at.shape, torch.float32)
    _same_device(device, grad, weights)
    grad_rows = _empty((count, width), dtype=values.dtype, device=place)
    grad_weights = _empty((tokens, k), dtype=torch.float32, device=place)
    _run(L.segtopk_combine_backward, device, kind, grad.data_ptr(), grad.stride(0), values.data_ptr(), values.stride(0),
         tokens, k, width, at.data_ptr(), kept, weights.data_ptr(), grad_rows.data_ptr(), grad_weights.data_ptr())
    return grad_rows, grad_weights


def _token_ids(tokens):
    size = _INT_BYTES.get(tokens.dtype)
    if size is None:
        raise ValueError("tokens must be int32 or int64")
    return tokens if tokens.is_contiguous() else tokens.contiguous(), size


@_on_stream
def embedding(table: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0, out_dtype=None, out=None):
    """scale * table[tokens] (segtopk_embedding): table [vocab, width], tokens
    int32 or int64 of any shape; returns [*tokens.shape, width] of out_dtype
    (the table's unless given). Tokens outside the table give zeros."""
    L = B.load()
    kind = _float(table, "table")
    table = _matrix(table, "table")
    tokens, size = _token_ids(tokens)
    device, vocab, width = table.get_device(), *table.shape
    _same_device(device, tokens)
    shape = (*tokens.shape, width)
    if out is None:
        out = _empty(shape, dtype=out_dtype or table.dtype, device=table.device)
    else:
        _given(out, "out", shape, out_dtype or out.dtype, device)
    _run(L.segtopk_embedding, device, kind, table.data_ptr(), vocab, width, table.stride(0), tokens.data_ptr(), size,
         tokens.numel(), scale, _float(out, "out"), out.data_ptr())
    return out


@_on_stream
def embedding_backward(grad_out: torch.Tensor, tokens: torch.Tensor, num_rows: int, *, scale: float = 1.0,
                       padding_idx=None, dtype=None, grad_table=None, accumulate: bool = False):
    """Gradient of embedding()'s table (segtopk_embedding_backward).

    grad_out: [*tokens.shape, width]. Returns [num_rows, width] of dtype (that
    of grad_out unless given), or writes grad_table; with accumulate the
    gradient is added to grad_table, and only the rows of tokens that occur
    are touched. padding_idx (as torch's: negative ones count from the end)
    gets no gradient."""
    L = B.load()
    kind = _float(grad_out, "grad_out")
    tokens, size = _token_ids(tokens)
    if grad_out.dim() < 1 or grad_out.shape[:-1] != tokens.shape:
        raise ValueError("grad_out must have a row for each token")
    count, width = tokens.numel(), grad_out.shape[-1]
    grad = _matrix(grad_out if grad_out.dim() == 2 else grad_out.reshape(count, width), "grad_out")
    device, place = grad.get_device(), grad.device
    _same_device(device, tokens)
    if padding_idx is None:
        padding = -1
    elif -num_rows <= padding_idx < num_rows:
        padding = padding_idx % num_rows
    else:
        raise ValueError("padding_idx must be a row of the table")
    shape = (max(num_rows, 0), width)
    if grad_table is not None:
        out = _given(grad_table, "grad_table", shape, dtype or grad_table.dtype, device)
    elif accumulate:
        raise ValueError("accumulate needs grad_table")
    else:
        out = _empty(shape, dtype=dtype or grad.dtype, device=place)
    need = L.segtopk_embedding_backward_workspace_bytes(count, num_rows, width)
    space = _empty(need, dtype=torch.uint8, device=place)
    _run(L.segtopk_embedding_backward, device, kind, grad.data_ptr(), grad.stride(0), tokens.data_ptr(), size, count,
         num_rows, width, padding, scale, _float(out, "grad_table"), out.data_ptr(), bool(accumulate), space.data_ptr(),
         need)
    return out
