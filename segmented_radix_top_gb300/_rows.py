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

# the current stream's handle, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


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


def _device(first, *others) -> int:
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must be on one CUDA device")
    return index


def _run(fn, index, *args):
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc:
        B._check(rc)


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


def _like(t, name, shape, dtype):
    """Checks a tensor that is read densely, or written."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError("%s must be %s of %s" % (name, dtype, tuple(shape)))
    return t


def _output(out, name, shape, dtype, near):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=near.device)
    _like(out, name, torch.Size(shape), dtype)
    if not out.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if out.get_device() != near.get_device():
        raise ValueError("tensors must be on one CUDA device")
    return out


def _score(score) -> int:
    if score not in SCORE:
        raise ValueError("score must be one of %s" % ", ".join(SCORE))
    return SCORE[score]


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
    index = _device(logits, bias)
    tokens, experts = logits.shape
    at = None
    if bias is not None:
        bias = _like(bias, "bias", (experts,), torch.float32).contiguous()
        at = bias.data_ptr()
    ids = torch.empty((tokens, max(k, 0)), dtype=torch.int32, device=logits.device)
    weights = torch.empty((tokens, max(k, 0)), dtype=torch.float32, device=logits.device)
    _run(L.segtopk_route, index, kind, logits.data_ptr(), tokens, experts, logits.stride(0), k, how, bool(renormalize),
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
    tokens, experts = logits.shape
    k = expert_ids.shape[-1]
    ids = _like(expert_ids, "expert_ids", (tokens, k), torch.int32).contiguous()
    grad = _like(grad_weights, "grad_weights", (tokens, k), torch.float32).contiguous()
    index = _device(logits, ids, grad)
    out = torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    _run(L.segtopk_route_backward, index, kind, grad.data_ptr(), logits.data_ptr(), tokens, experts, logits.stride(0),
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
    index = _device(expert_ids)
    ids = expert_ids.contiguous()
    device, slots = ids.device, ids.numel()
    offsets = torch.empty(max(num_experts, 0) + 1, dtype=torch.int64, device=device)
    rows = torch.empty(ids.shape, dtype=torch.int32, device=device)
    slot_of_row = torch.empty(slots, dtype=torch.int32, device=device)
    need = L.segtopk_group_workspace_bytes(slots, num_experts)
    space = torch.empty(need, dtype=torch.uint8, device=device).data_ptr() if need else None
    _run(L.segtopk_group, index, ids.data_ptr(), id_bytes, slots, num_experts, offsets.data_ptr(), rows.data_ptr(),
         slot_of_row.data_ptr(), space, need)
    return ExpertGroups(offsets, rows, slot_of_row)


def _groups(groups):
    offsets, rows = groups.offsets, groups.row_of_slot
    if offsets.dtype != torch.int64 or rows.dtype != torch.int32 or rows.dim() != 2 or not rows.is_contiguous() \
            or offsets.dim() != 1 or not offsets.is_contiguous() or offsets.shape[0] < 1:
        raise ValueError("groups must come from group_by_expert")
    return rows, offsets.data_ptr() + 8 * (offsets.shape[0] - 1)


@_on_stream
def dispatch(x: torch.Tensor, groups: ExpertGroups, *, out=None):
    """The tokens' rows in the order of their experts (segtopk_dispatch):
    x [tokens, width] of any element type of 1 to 8 bytes; returns [tokens *
    k, width], zeros from row groups.offsets[-1] on."""
    L = B.load()
    x = _matrix(x, "x")
    rows, kept = _groups(groups)
    tokens, k = rows.shape
    if x.shape[0] != tokens:
        raise ValueError("x must have a row for each token of the groups")
    index = _device(x, rows, groups.offsets)
    width = x.shape[1]
    out = _output(out, "out", (tokens * k, width), x.dtype, x)
    _run(L.segtopk_dispatch, index, x.data_ptr(), x.element_size(), tokens, k, width, x.stride(0), rows.data_ptr(),
         kept, out.data_ptr())
    return out


def _combine(values, groups, weights, out):
    L = B.load()
    kind = _float(values, "rows")
    values = _matrix(values, "rows")
    rows, _ = _groups(groups)
    tokens, k = rows.shape
    if values.shape[0] != tokens * k:
        raise ValueError("rows must have a row for each slot of the groups")
    index = _device(values, rows, weights)
    at = None
    if weights is not None:
        weights = _like(weights, "weights", (tokens, k), torch.float32).contiguous()
        at = weights.data_ptr()
    width = values.shape[1]
    out = _output(out, "out", (tokens, width), values.dtype, values)
    _run(L.segtopk_combine, index, kind, values.data_ptr(), tokens, k, width, values.stride(0), rows.data_ptr(), at,
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
    at, kept = _groups(groups)
    tokens, k = at.shape
    width = values.shape[1]
    if values.shape[0] != tokens * k:
        raise ValueError("rows must have a row for each slot of the groups")
    _like(grad, "grad_out", (tokens, width), values.dtype)
    weights = _like(weights, "weights", (tokens, k), torch.float32).contiguous()
    index = _device(values, grad, at, weights, groups.offsets)
    grad_rows = torch.empty((tokens * k, width), dtype=values.dtype, device=values.device)
    grad_weights = torch.empty((tokens, k), dtype=torch.float32, device=values.device)
    _run(L.segtopk_combine_backward, index, kind, grad.data_ptr(), grad.stride(0), values.data_ptr(), values.stride(0),
         tokens, k, width, at.data_ptr(), kept, weights.data_ptr(), grad_rows.data_ptr(), grad_weights.data_ptr())
    return grad_rows, grad_weights


def _token_ids(tokens):
    size = _INT_BYTES.get(tokens.dtype)
    if size is None:
        raise ValueError("tokens must be int32 or int64")
    return tokens.contiguous(), size


@_on_stream
def embedding(table: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0, out_dtype=None, out=None):
    """scale * table[tokens] (segtopk_embedding): table [vocab, width], tokens
    int32 or int64 of any shape; returns [*tokens.shape, width] of out_dtype
    (the table's unless given). Tokens outside the table give zeros."""
    L = B.load()
    kind = _float(table, "table")
    table = _matrix(table, "table")
    tokens, size = _token_ids(tokens)
    index = _device(table, tokens)
    vocab, width = table.shape
    if out_dtype is None:
        out_dtype = table.dtype if out is None else out.dtype
    out = _output(out, "out", (*tokens.shape, width), out_dtype, table)
    _run(L.segtopk_embedding, index, kind, table.data_ptr(), vocab, width, table.stride(0), tokens.data_ptr(), size,
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
    width = grad_out.shape[-1]
    grad = _matrix(grad_out if grad_out.dim() == 2 else grad_out.reshape(tokens.numel(), width), "grad_out")
    index = _device(grad, tokens)
    if padding_idx is not None:
        if not -num_rows <= padding_idx < num_rows:
            raise ValueError("padding_idx must be a row of the table")
        padding_idx %= num_rows
    if accumulate and grad_table is None:
        raise ValueError("accumulate needs grad_table")
    if dtype is None:
        dtype = grad.dtype if grad_table is None else grad_table.dtype
    out = _output(grad_table, "grad_table", (max(num_rows, 0), width), dtype, grad)
    need = L.segtopk_embedding_backward_workspace_bytes(tokens.numel(), num_rows, width)
    space = torch.empty(need, dtype=torch.uint8, device=grad.device)
    _run(L.segtopk_embedding_backward, index, kind, grad.data_ptr(), grad.stride(0), tokens.data_ptr(), size,
         tokens.numel(), num_rows, width, -1 if padding_idx is None else padding_idx, scale, _float(out, "grad_table"),
         out.data_ptr(), bool(accumulate), space.data_ptr(), need)
    return out
