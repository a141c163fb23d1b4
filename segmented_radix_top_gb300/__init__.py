"""GB300-native segmented (batched) top-k by multi-pass radix digit selection.

The compute runs in hand-written sm_103a CUDA kernels behind the C ABI of
include/segtopk.h (libsegtopk.so); this package only marshals tensors into
that ABI (_binding.py: the selection; _rows.py: layer norm, expert routing,
tokens sorted by expert and back, the experts' products, token embedding, and
their gradients) and provides the seeded synthetic workloads (workloads.py).
"""
from ._binding import (DETERMINISM, DIRECTION, DTYPE, KEY_BYTES, MAX_K, NOALLOC_STAGING_BYTES,  # noqa: F401
                       ORDERING, TIE_BREAK, SegTopKError, batched_topk, batched_topk_host,
                       batched_topk_host_noalloc, host_workspace_bytes,
                       last_launch_count, library_path, load, load_instrumented, read_device_error,
                       read_stats, set_test_hooks, topk)
from ._rows import (DEVICE_ERROR_INDEX, MAX_EXPERTS, MAX_GROUPS, MAX_NORM_WIDTH, ROUTE_MAX_K,  # noqa: F401
                    ExpertGroups, combine, combine_backward, dispatch, dispatch_backward, embedding,
                    embedding_backward, expert_matmul, expert_matmul_backward, group_by_expert, layer_norm,
                    layer_norm_backward, quantize_rows, route, route_backward)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libsegtopk.so for sm_103a and the row operators' binding
    in-tree (nvcc, g++; no GPU needed)."""
    from . import _build
    return _build.build(force=force, verbose=verbose)
