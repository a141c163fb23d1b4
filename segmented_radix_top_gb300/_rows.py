"""The row operators of libsegtopk.so: expert routing, tokens sorted by expert
and back, token embedding, and their gradients (include/segtopk.h has each
operator's contract).

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
        "segtopk_route_backward": (i, [i, vp, vp, i64, i32, i64, i32, vp, i, i, f, vp, vp]),
        "segtopk_group_workspace_bytes": (sz, [i64, i32]),
        "segtopk_group": (i, [vp, i32, i64, i32, vp, vp, vp, vp, sz, vp]),
        "segtopk_dispatch": (i, [vp, i32, i64, i32, i64, i64, vp, vp, vp, vp]),
        "segtopk_combine": (i, [i, vp, i64, i32, i64, i64, vp, vp, vp, vp]),
        "segtopk_combine_backward": (i, [i, vp, i64, vp, i64, i64, i32, i64, vp, vp, vp, vp, vp, vp]),
        "segtopk_embedding": (i, [i, vp, i64, i64, i64, vp, i32, i64, f, i, vp, vp]),
        "segtopk_embedding_backward_workspace_bytes": (sz, [i64, i64, i64]),
        "segtopk_embedding_backward": (i, [i, vp, i64, vp, i32, i64, i64, i64, i64, f, i, vp, i, vp, sz, vp]),
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
          bias=None):
    """The k best experts of each token and their weights (segtopk_route).

    logits: [tokens, experts]. score: "softmax" (over all experts) or
    "sigmoid"; renormalize divides by the sum of the k chosen scores; scale
    multiplies. bias: optional float32 [experts], added to the scores for the
    choice only. Experts with a logit or a bias of -inf are never chosen. Returns
    (expert_ids int32 [tokens, k], best first and -1 where none is left,
    weights float32 [tokens, k])."""
    return (_native or _load()).route(logits, k, score, renormalize, scale, bias)


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
