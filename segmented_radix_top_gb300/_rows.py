"""The row operators of libsegtopk.so: layer norm, expert routing, tokens sorted
by expert and back, the experts' matrix products, rows in 8 bits, token
embedding, and their gradients (include/segtopk.h has each operator's
contract).

Inputs are CUDA tensors on one device. Rows may lie any distance apart (a
part of a wider tensor's columns, one row expanded to many); tensors whose
rows are not contiguous, and views whose conjugation or negation torch has put
off (x.conj() of a complex tensor), are copied first, whole and on every call.
Everything runs on the current stream, or on `stream`, from whose memory pool
results and workspaces then come. Nothing here synchronises, so all of it can
be captured in a graph.

Gradients are functions of their own; autograd does not see these calls
(examples/sparse_layer.py wraps them for it). A given output counts as changed
for autograd; outside torch.no_grad() one that requires a gradient is refused.
Outputs must not overlap inputs.

The calls go through a compiled binding (csrc/rows_binding.cpp), which checks
the tensors and makes the results. Like the rest of the package it raises if
it is not built; there is no other implementation.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
from typing import NamedTuple

import torch

from . import _binding as B
from . import _build

MAX_EXPERTS = 1024    # SEGTOPK_MAX_EXPERTS
ROUTE_MAX_K = 32      # SEGTOPK_ROUTE_MAX_K
MAX_GROUPS = 32       # SEGTOPK_MAX_GROUPS
MAX_NORM_WIDTH = 16384  # SEGTOPK_MAX_NORM_WIDTH
DEVICE_ERROR_INDEX = 4  # SEGTOPK_DEVICE_ERROR_INDEX


class ExpertGroups(NamedTuple):
    """Token slots sorted by expert (segtopk_group)."""
    offsets: torch.Tensor      # int64 [experts + 1]: expert e has the sorted rows offsets[e] to offsets[e + 1]
    row_of_slot: torch.Tensor  # int32 [tokens, k]: each slot's sorted row, -1 for none
    slot_of_row: torch.Tensor  # int32 [tokens * k]: each sorted row's slot, -1 past the last one


def _entries():
    """Entry points: result and argument types."""
    i, i32, i64, f, vp, sz = (ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p,
                              ctypes.c_size_t)
    return {
        "segtopk_route": (i, [i, vp, i64, i32, i64, i32, i, i, f, vp, vp, vp, vp]),
        "segtopk_route_groups": (i, [i, vp, i64, i32, i64, i32, i32, i32, i, i, i, f, vp, vp, vp, vp]),
        "segtopk_route_backward": (i, [i, vp, vp, i64, i32, i64, i32, vp, i, i, f, vp, vp]),
        "segtopk_group_workspace_bytes": (sz, [i64, i32]),
        "segtopk_group": (i, [vp, i32, i64, i32, vp, vp, vp, vp, sz, vp]),
        "segtopk_dispatch": (i, [vp, i32, i64, i32, i64, i64, vp, vp, vp, vp]),
        "segtopk_combine": (i, [i, vp, i64, i32, i64, i64, vp, vp, vp, vp]),
        "segtopk_combine_backward": (i, [i, vp, i64, vp, i64, i64, i32, i64, vp, vp, vp, vp, vp, vp]),
        "segtopk_embedding": (i, [i, vp, i64, i64, i64, vp, i32, i64, f, i, vp, vp]),
        "segtopk_embedding_backward_workspace_bytes": (sz, [i64, i64, i64]),
        "segtopk_embedding_backward": (i, [i, vp, i64, vp, i32, i64, i64, i64, i64, f, i, vp, i, vp, sz, vp]),
        "segtopk_expert_matmul": (i, [i, vp, i64, i64, i64, vp, i32, i64, i64, i64, i64, vp, i, vp, vp]),
        "segtopk_expert_matmul_f8": (i, [vp, i64, i64, i64, vp, i64, vp, i32, i64, i64, i64, vp, vp, i, vp, vp]),
        "segtopk_expert_matmul_weights": (i, [i, vp, i64, i64, vp, i64, i64, i64, i32, vp, i, vp, vp]),
        "segtopk_test_expert_tile": (i, [i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]),
        "segtopk_test_free_row": (i, [i32, i32, i32, ctypes.POINTER(i64)]),
        "segtopk_layer_norm": (i, [i, vp, i64, i64, i64, i, vp, vp, f, vp, vp, vp, vp]),
        "segtopk_layer_norm_backward_workspace_bytes": (sz, [i64, i64]),
        "segtopk_layer_norm_backward": (i, [i, vp, i64, vp, i64, i64, i64, i, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "segtopk_quantize_rows": (i, [i, vp, i64, i64, i64, vp, vp, vp]),
    }


def declare(L) -> None:
    """Argument types of the entry points (once per loaded library)."""
    for name, (result, args) in _entries().items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = result, args


_native = None


def _load():
    """The compiled binding, bound to the library's entry points."""
    global _native
    if _native is None:
        L = B.load()
        path = _build.binding_path()
        if not os.path.exists(path):
            lacks = _build.binding_lacks()
            raise RuntimeError("%s is not built (%s); there is no fallback implementation"
                               % (os.path.basename(path), "not installed: " + ", ".join(lacks) if lacks else
                                  "run __graft_entry__.build()"))
        spec = importlib.util.spec_from_file_location("segmented_radix_top_gb300._rows_native", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind({name: ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in _entries()}, B._check)
        _native = module
    return _native


def _on_stream(call):
    """Gives an operator its `stream` argument: the call, its results and its
    workspace belong to that stream. The tensors that it is given are held
    for the stream, so that the memory of one dropped after the call is not
    handed out before the stream has got there. The caller orders the stream
    after what writes them."""
    @functools.wraps(call)
    def wrapped(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        with torch.cuda.stream(stream):
            result = call(*args, **kw)
        for value in (*args, *kw.values()):
            for t in value if isinstance(value, tuple) else (value,):
                if isinstance(t, torch.Tensor):
                    t.record_stream(stream)
        return result
    return wrapped


@_on_stream
def route(logits: torch.Tensor, k: int, *, score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
          bias=None, num_groups: int = 1, groups_kept=None, group_score: str = "best"):
    """The k best experts of each token and their weights (segtopk_route).

    logits: [tokens, experts]. score: "softmax" (over all experts) or
    "sigmoid"; renormalize divides by the sum of the k chosen scores; scale
    multiplies. bias: optional float32 [experts], added to the scores for the
    choice only. Experts with a logit or a bias of -inf are never chosen. Returns
    (expert_ids int32 [tokens, k], best first and -1 where none is left,
    weights float32 [tokens, k]).

    With num_groups the experts are as many groups of equal size, in order, and
    the k are chosen from the groups_kept best groups (all unless given;
    segtopk_route_groups): by group_score "best", a group's best expert, or
    "best_two", the sum of its two best ones' scores with their biases.
    route_backward() is the same for both."""
    return (_native or _load()).route(logits, k, score, renormalize, scale, bias, num_groups, groups_kept, group_score)


@_on_stream
def route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, expert_ids: torch.Tensor, *,
                   score: str = "softmax", renormalize: bool = True, scale: float = 1.0):
    """Gradient of route()'s logits from that of its weights
    (segtopk_route_backward): [tokens, experts] of the logits' type."""
    return (_native or _load()).route_backward(grad_weights, logits, expert_ids, score, renormalize, scale)


@_on_stream
def group_by_expert(expert_ids: torch.Tensor, num_experts: int) -> ExpertGroups:
    """Sorts the slots of expert_ids [tokens, k] (int32 or int64, negative:
    no expert) by expert, stably (segtopk_group)."""
    return ExpertGroups._make((_native or _load()).group(expert_ids, num_experts))


@_on_stream
def dispatch(x: torch.Tensor, groups: ExpertGroups, *, out=None):
    """The tokens' rows in the order of their experts (segtopk_dispatch):
    x [tokens, width] of any element type of 1 to 8 bytes; returns [tokens *
    k, width], zeros from row groups.offsets[-1] on."""
    return (_native or _load()).dispatch(x, groups, out)


@_on_stream
def dispatch_backward(grad_rows: torch.Tensor, groups: ExpertGroups, *, out=None):
    """Gradient of dispatch()'s x (segtopk_combine without weights): the sum
    of each token's rows of grad_rows [tokens * k, width]."""
    return (_native or _load()).combine(grad_rows, groups, None, out)


@_on_stream
def combine(rows: torch.Tensor, groups: ExpertGroups, weights: torch.Tensor, *, out=None):
    """The sorted rows back at their tokens, weighted and summed
    (segtopk_combine): rows [tokens * k, width], weights float32 [tokens, k];
    returns [tokens, width]."""
    if weights is None:
        raise ValueError("weights must be a tensor")
    return (_native or _load()).combine(rows, groups, weights, out)


@_on_stream
def combine_backward(grad_out: torch.Tensor, rows: torch.Tensor, groups: ExpertGroups, weights: torch.Tensor):
    """Gradients of combine()'s rows and weights (segtopk_combine_backward):
    ([tokens * k, width] with zeros from row groups.offsets[-1] on, float32
    [tokens, k] with zeros for slots without an expert)."""
    return (_native or _load()).combine_backward(grad_out, rows, groups, weights)


@_on_stream
def embedding(table: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0, out_dtype=None, out=None):
    """scale * table[tokens] (segtopk_embedding): table [vocab, width], tokens
    int32 or int64 of any shape; returns [*tokens.shape, width] of out_dtype
    (the table's unless given). Tokens outside the table give zeros. A table
    whose rows are not contiguous (weight.t()) is copied whole by every call."""
    return (_native or _load()).embedding(table, tokens, scale, out_dtype, out)


@_on_stream
def embedding_backward(grad_out: torch.Tensor, tokens: torch.Tensor, num_rows: int, *, scale: float = 1.0,
                       padding_idx=None, dtype=None, grad_table=None, accumulate: bool = False):
    """Gradient of embedding()'s table (segtopk_embedding_backward).

    grad_out: [*tokens.shape, width]. Returns [num_rows, width] of dtype (that
    of grad_out unless given), or writes grad_table; with accumulate the
    gradient is added to grad_table, and only the rows of tokens that occur
    are touched. padding_idx (as torch's: negative ones count from the end)
    gets no gradient."""
    return (_native or _load()).embedding_backward(grad_out, tokens, num_rows, scale, padding_idx, dtype, grad_table,
                                                   accumulate)


@_on_stream
def expert_matmul(rows: torch.Tensor, weights: torch.Tensor, groups: ExpertGroups, *, row_scales=None,
                  weight_scales=None, out_dtype=None, out=None):
    """Each expert's matrix product of its rows (segtopk_expert_matmul):
    out[r] = weights[e] @ rows[r] for the rows r of expert e; zeros for rows
    that no expert has (from groups.offsets[-1] on, and before groups.offsets[0]
    should that not be 0). The offsets stay on the device.

    rows: [tokens * k, width], in the order of dispatch(); weights: [experts,
    out, width] of the same type, float16 or bfloat16, either of the last two
    dimensions contiguous (weights.transpose(1, 2) of [experts, width, out]
    is read as it is). width, and in a transposed layout out, is a multiple
    of 8. out_dtype: that of rows unless given.

    float8_e4m3fn rows and weights (segtopk_expert_matmul_f8) have a float32
    scale for each block of 128 values: row_scales [tokens * k, blocks of
    width], as quantize_rows() gives them, and weight_scales [experts, blocks
    of out, blocks of width], one for 128 by 128 values; blocks at the end may
    be smaller. width is a multiple of 16, out is any, and the result bfloat16
    unless out_dtype is given. A frozen layer's gradient of its rows is this
    product too, with the transposed weights and scales laid out beside them.

    Tensors whose rows do not start on 16-byte boundaries are copied first, as
    are weights in another layout, by every call."""
    return (_native or _load()).expert_matmul(rows, weights, groups, row_scales, weight_scales, out_dtype, out)


@_on_stream
def expert_matmul_backward(grad_out: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor, groups: ExpertGroups, *,
                           dtype=None):
    """Gradients of expert_matmul()'s rows and weights in 16 bits
    (segtopk_expert_matmul with the weights transposed, and
    segtopk_expert_matmul_weights): ([tokens * k, width] with zeros from row
    groups.offsets[-1] on, [experts, out, width] of dtype (the weights' unless
    given) in the weights' layout, zeros for an expert without rows). width
    and out are multiples of 8."""
    return (_native or _load()).expert_matmul_backward(grad_out, rows, weights, groups, dtype)


@_on_stream
def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias=None, *, eps: float = 1e-5, out=None):
    """Layer norm of the rows of x [tokens, width] (segtopk_layer_norm):
    (x - mean) * rstd * weight + bias. weight, and bias where there is one:
    [width], both of x's type or both float32. Returns (out of x's type, mean
    and rstd float32 [tokens], for layer_norm_backward). width is at most
    MAX_NORM_WIDTH."""
    return (_native or _load()).layer_norm(x, weight, bias, eps, out)


@_on_stream
def layer_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor):
    """Gradients of layer_norm()'s x, weight and bias
    (segtopk_layer_norm_backward), the last two of weight's type: (grad_x,
    grad_weight, grad_bias). mean and rstd are those that layer_norm()
    returned."""
    return (_native or _load()).layer_norm_backward(grad_out, x, weight, mean, rstd)


@_on_stream
def quantize_rows(x: torch.Tensor):
    """The rows of x [tokens, width] in 8 bits with a scale for each block of
    128 values (segtopk_quantize_rows): (values float8_e4m3fn [tokens, width],
    scales float32 [tokens, blocks]), x being nearly values * scales. Both can
    go through dispatch() to expert_matmul()."""
    return (_native or _load()).quantize_rows(x)
