"""Tokens sorted by expert and back against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import rows_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def ids_of(tokens, k, experts, seed, dropped=0.0, dtype=torch.int32):
    """Distinct experts per token as far as there are enough; some slots without one."""
    rng = np.random.default_rng(seed)
    if k <= experts:
        ids = np.argsort(rng.random((tokens, experts)) ** 2, axis=1)[:, :k]
    else:
        ids = rng.integers(0, experts, (tokens, k))
    ids[rng.random(ids.shape) < dropped] = -1
    return torch.from_numpy(ids.astype(np.int64)).to(dtype)


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def grouped(ids, experts):
    groups = st.group_by_expert(ids.cuda(), experts)
    offsets, rows, slots = ref.group(ids.numpy(), experts)
    assert groups.offsets.dtype == torch.int64
    assert np.array_equal(groups.offsets.cpu().numpy(), offsets)
    assert np.array_equal(groups.row_of_slot.cpu().numpy(), rows)
    assert np.array_equal(groups.slot_of_row.cpu().numpy(), slots)
    return groups, rows, slots


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,k,experts,dropped", [
    (1, 1, 1, 0), (1, 8, 64, 0), (7, 3, 5, 0.3), (100, 6, 60, 0.1), (512, 4, 8, 0), (683, 3, 64, 0.1),
    (1025, 2, 512, 0), (1500, 5, 513, 0.2), (3000, 8, 1024, 0.05), (2731, 3, 256, 1.0), (20000, 2, 3, 0.5)])
def test_group(tokens, k, experts, dropped, dtype):
    grouped(ids_of(tokens, k, experts, tokens, dropped, dtype), experts)


@pytest.mark.parametrize("slots", [4096, 4097, 8193, 16385, 32768, 32769, 99999, 131072, 131073])
@pytest.mark.parametrize("experts", [1, 100, 1024])
def test_group_sizes(slots, experts):
    # against torch's stable sort
    ids = torch.randint(-1, experts, (slots, 1), generator=torch.Generator().manual_seed(slots), dtype=torch.int32)
    groups = st.group_by_expert(ids.cuda(), experts)
    flat = ids.flatten().long()
    key = torch.where(flat < 0, experts, flat)
    order, kept = torch.argsort(key, stable=True), int((flat >= 0).sum())
    assert torch.equal(groups.slot_of_row.cpu()[:kept].long(), order[:kept])
    assert (groups.slot_of_row[kept:] == -1).all()
    rows = torch.full_like(flat, -1)
    rows[order[:kept]] = torch.arange(kept)
    assert torch.equal(groups.row_of_slot.cpu().flatten().long(), rows)
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    assert torch.equal(groups.offsets.cpu(), torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]))


def test_group_with_one_expert_for_all():
    for tokens in (33, 5000):
        grouped(torch.full((tokens, 2), 6, dtype=torch.int32), 7)


def test_group_over_more_than_the_largest_number_of_tiles():
    # 128 tiles of more than 2048 slots; sorted by torch, stably
    ids = torch.randint(-1, 200, (75001, 4), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    groups = st.group_by_expert(ids.cuda(), 200)
    flat = ids.flatten().long()
    key = torch.where(flat < 0, 200, flat)
    order = torch.argsort(key, stable=True)
    kept = int((flat >= 0).sum())
    assert int(groups.offsets[-1]) == kept
    assert torch.equal(groups.slot_of_row.cpu()[:kept].long(), order[:kept])
    assert (groups.slot_of_row[kept:] == -1).all()
    rows = torch.full_like(flat, -1)
    rows[order[:kept]] = torch.arange(kept)
    assert torch.equal(groups.row_of_slot.cpu().flatten().long(), rows)
    assert torch.equal(groups.offsets.cpu(), torch.cat([torch.zeros(1, dtype=torch.long),
                                                        torch.bincount(key, minlength=201)[:200].cumsum(0)]))


def test_ids_past_the_last_expert_count_as_none_and_set_the_error_word():
    st.read_device_error()
    ids = torch.tensor([[0, 9], [3, -2], [4, 1]], dtype=torch.int32)
    groups = st.group_by_expert(ids.cuda(), 4)
    assert st.read_device_error() == st.DEVICE_ERROR_INDEX
    assert st.read_device_error() == 0
    assert groups.offsets.tolist() == [0, 1, 2, 2, 3]
    assert groups.row_of_slot.tolist() == [[0, -1], [2, -1], [-1, 1]]
    assert groups.slot_of_row.tolist() == [0, 5, 2, -1, -1, -1]
    st.group_by_expert(torch.full((4, 2), -1, dtype=torch.int32, device="cuda"), 4)
    assert st.read_device_error() == 0


SHAPES = [(1, 1, 1, 1, 0), (1, 8, 64, 64, 0), (5, 2, 3, 7, 0.2), (33, 3, 9, 64, 0), (20, 9, 16, 136, 0.1),
          (19, 17, 40, 96, 0.1), (70, 4, 10, 1000, 0.3), (12, 2, 4, 2048, 0), (9, 6, 8, 4104, 0.2), (40, 2, 5, 33, 1.0),
          (301, 8, 30, 250, 0.05)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,experts,width,dropped", SHAPES)
def test_there_and_back(tokens, k, experts, width, dropped, dtype):
    groups, rows, slots = grouped(ids_of(tokens, k, experts, width, dropped), experts)
    kept = int(groups.offsets[-1])
    x, y, g = (randn(n, width, seed=s, dtype=dtype) for n, s in ((tokens, 1), (tokens * k, 2), (tokens, 3)))
    y[kept:] = float("nan")  # rows that belong to no slot are never read
    w = randn(tokens, k, seed=4).abs()
    X, Y, G, W = (ref.f64(t) for t in (x, y, g, w))
    assert np.array_equal(ref.f64(st.dispatch(x.cuda(), groups)), ref.dispatch(X, slots, k))

    exact, size = ref.combine(Y, rows, W)
    bound = (k + 1) * ref.U32 * size + ref.rounded(dtype, np.abs(exact))
    ref.within(st.combine(y.cuda(), groups, w.cuda()), exact, bound)

    exact, size = ref.combine(Y, rows, np.ones_like(W))
    bound = (k + 1) * ref.U32 * size + ref.rounded(dtype, np.abs(exact))
    ref.within(st.dispatch_backward(y.cuda(), groups), exact, bound)

    grad_y, grad_w = st.combine_backward(g.cuda(), y.cuda(), groups, w.cuda())
    exact_y, exact_w, size = ref.combine_backward(G, Y, rows, W)
    ref.within(grad_y, exact_y, 1.01 * ref.U32 * np.abs(exact_y) + ref.rounded(dtype, np.abs(exact_y)))
    ref.within(grad_w, exact_w, (width + 1) * ref.U32 * size)


@pytest.mark.parametrize("tokens,k,experts,width,dropped,dtype", [
    (2500, 3, 40, 2048, 0.2, torch.float32), (2433, 9, 16, 4104, 0.1, torch.bfloat16),
    (9900, 2, 8, 1000, 0, torch.float16), (40000, 1, 4, 256, 0.5, torch.bfloat16), (80000, 2, 6, 64, 0.1, torch.float32)])
def test_runs_of_many_tokens(tokens, k, experts, width, dropped, dtype):
    # enough tokens for groups of threads to take several each; the
    # definitions in 64 bits on the GPU
    groups = st.group_by_expert(ids_of(tokens, k, experts, 1, dropped).cuda(), experts)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, y = (torch.randn(n, width, generator=g, device="cuda", dtype=dtype) for n in (tokens, tokens * k))
    w = torch.rand(tokens, k, generator=g, device="cuda")
    rows, kept = groups.row_of_slot.long(), int(groups.offsets[-1])
    y[kept:] = float("nan")
    some = (rows >= 0).double()[..., None]
    at, wide = rows.clamp(min=0), w.double()[..., None] * some
    out, back = st.combine(y, groups, w), st.dispatch_backward(y, groups)
    exact, size = torch.zeros(2, tokens, width, dtype=torch.float64, device="cuda")
    exact_back, size_back = torch.zeros(2, tokens, width, dtype=torch.float64, device="cuda")
    grad_w, size_w = torch.zeros(2, tokens, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        part = torch.where(some[:, j] > 0, y[at[:, j]].double(), 0)
        exact += wide[:, j] * part
        size += wide[:, j] * part.abs()
        exact_back += part
        size_back += part.abs()
        grad_w[:, j] = (part * x.double()).sum(1)
        size_w[:, j] = (part * x.double()).abs().sum(1)

    def near(got, want, bound):
        assert bool(((got.double() - want).abs() <= bound).all())

    near(out, exact, (k + 1) * ref.U32 * size + ref.rounded(dtype, exact.abs()))
    near(back, exact_back, (k + 1) * ref.U32 * size_back + ref.rounded(dtype, exact_back.abs()))
    got_y, got_w = st.combine_backward(x, y, groups, w)
    near(got_w, grad_w, (width + 1) * ref.U32 * size_w)
    want = torch.zeros(tokens * k, width, dtype=torch.float64, device="cuda")
    slot = groups.slot_of_row[:kept].long()
    want[:kept] = w.double().reshape(-1)[slot, None] * x.double()[slot // k]
    near(got_y, want, 1.01 * ref.U32 * want.abs() + ref.rounded(dtype, want.abs()))


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int16, torch.int32, torch.float64, torch.float8_e4m3fn])
@pytest.mark.parametrize("width", [1, 5, 48, 260])
def test_dispatch_moves_any_element(dtype, width):
    groups, _, slots = grouped(ids_of(13, 3, 6, 1, 0.2), 6)
    bits = torch.randint(0, 256, (13, width * dtype.itemsize), generator=torch.Generator().manual_seed(1),
                         dtype=torch.uint8)
    got = st.dispatch(bits.cuda().view(dtype), groups).view(torch.uint8)
    assert np.array_equal(got.cpu().numpy(), ref.dispatch(bits.numpy(), slots, 3))


@pytest.mark.parametrize("left,width,extra", [(8, 64, 8), (1, 64, 7), (2, 30, 0), (0, 40, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_columns_of_wider_tensors(left, width, extra, dtype):
    tokens, k, experts = 37, 3, 8
    groups, rows, slots = grouped(ids_of(tokens, k, experts, 2, 0.1), experts)
    wide = [randn(n, left + width + extra, seed=n, dtype=dtype) for n in (tokens, tokens * k)]
    x, y = (t[:, left:left + width] for t in wide)
    gx, gy = (t.cuda()[:, left:left + width] for t in wide)
    w = randn(tokens, k, seed=5)
    assert np.array_equal(ref.f64(st.dispatch(gx, groups)), ref.dispatch(ref.f64(x), slots, k))
    exact, size = ref.combine(ref.f64(y), rows, ref.f64(w))
    ref.within(st.combine(gy, groups, w.cuda()), exact, 4 * ref.U32 * size + ref.rounded(dtype, np.abs(exact)))
    grad_y, grad_w = st.combine_backward(gx, gy, groups, w.cuda())
    exact_y, exact_w, size = ref.combine_backward(ref.f64(x), ref.f64(y), rows, ref.f64(w))
    ref.within(grad_y, exact_y, 1.01 * ref.U32 * np.abs(exact_y) + ref.rounded(dtype, np.abs(exact_y)))
    ref.within(grad_w, exact_w, (width + 1) * ref.U32 * size)


def test_expanded_and_transposed_inputs():
    groups, rows, slots = grouped(ids_of(24, 2, 4, 3), 4)
    y, w = randn(48, 16, seed=1), randn(24, 2, seed=2)
    one = randn(1, 16, seed=3)
    g = one.expand(24, 16)
    assert np.array_equal(ref.f64(st.dispatch(one.cuda().expand(24, 16), groups)), ref.dispatch(ref.f64(g), slots, 2))
    want = st.combine_backward(g.contiguous().cuda(), y.cuda(), groups, w.cuda())
    for grad in (one.cuda().expand(24, 16), g.contiguous().cuda().t().contiguous().t()):
        got = st.combine_backward(grad, y.cuda().t().contiguous().t(), groups, w.cuda().t().contiguous().t())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ones = torch.ones((), device="cuda").expand(24, 16)  # what sum().backward() sends
    assert torch.equal(st.combine_backward(ones, y.cuda(), groups, w.cuda())[0],
                       st.combine_backward(ones.contiguous(), y.cuda(), groups, w.cuda())[0])


def test_infinities_stay_where_they_are():
    ids = torch.tensor([[0, 1], [1, 2], [-1, -1]], dtype=torch.int32)
    groups, rows, _ = grouped(ids, 3)
    y = torch.ones(6, 24)
    y[int(rows[0, 1])] = float("inf")
    y[4:] = float("nan")
    out = st.combine(y.cuda(), groups, torch.tensor([[0.5, 0.5], [1, 2], [9, 9]]).cuda())
    assert torch.isinf(out[0]).all() and (out[1] == 3).all() and (out[2] == 0).all()


def test_no_tokens_and_no_width():
    groups = st.group_by_expert(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 6)
    assert groups.offsets.tolist() == [0] * 7 and groups.row_of_slot.shape == (0, 4)
    x, w = torch.zeros(0, 8, device="cuda"), torch.zeros(0, 4, device="cuda")
    assert st.dispatch(x, groups).shape == st.combine(x, groups, w).shape == (0, 8)
    assert st.combine_backward(x, x, groups, w)[1].shape == (0, 4)
    groups = st.group_by_expert(torch.zeros(3, 2, dtype=torch.int32, device="cuda"), 6)
    x, w = torch.zeros(3, 0, device="cuda"), torch.ones(3, 2, device="cuda")
    y = torch.zeros(6, 0, device="cuda")
    assert st.dispatch(x, groups).shape == (6, 0) and st.combine(y, groups, w).shape == (3, 0)
    assert (st.combine_backward(x, y, groups, w)[1] == 0).all()


def test_gradients_against_differences():
    # combine is linear in the rows and in the weights: a difference of two
    # results in 64 bits is the gradient's product with the step
    groups, rows, slots = grouped(ids_of(9, 3, 5, 6, 0.2), 5)
    kept = int(groups.offsets[-1])
    y, w, g, dy, dw = (randn(27, 8, seed=1), randn(9, 3, seed=2), randn(9, 8, seed=3), randn(27, 8, seed=4),
                       randn(9, 3, seed=5))
    Y, W, G, DY, DW = (ref.f64(t) for t in (y, w, g, dy, dw))
    grad_y, grad_w = (ref.f64(t) for t in st.combine_backward(g.cuda(), y.cuda(), groups, w.cuda()))
    grad_x = ref.f64(st.dispatch_backward(y.cuda(), groups))
    assert (grad_y[kept:] == 0).all()
    bound = 40 * ref.U32 * 27 * 8 * 4
    assert abs((grad_y * DY).sum() - (G * (ref.combine(Y + DY, rows, W)[0] - ref.combine(Y, rows, W)[0])).sum()) < bound
    assert abs((grad_w * DW).sum() - (G * (ref.combine(Y, rows, W + DW)[0] - ref.combine(Y, rows, W)[0])).sum()) < bound
    assert abs((grad_x * G).sum() - (Y * ref.dispatch(G, slots, 3)).sum()) < bound


def test_results_are_the_same_from_run_to_run():
    ids = ids_of(900, 8, 50, 1, 0.1).cuda()
    y, g, w = (randn(*s, seed=1).cuda() for s in ((7200, 136), (900, 136), (900, 8)))
    first = None
    for _ in range(5):
        groups = st.group_by_expert(ids, 50)
        got = [*groups, st.combine(y, groups, w), *st.combine_backward(g, y, groups, w), st.dispatch_backward(y, groups)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_on_another_stream_and_in_a_graph():
    ids, x, w = ids_of(700, 4, 30, 2, 0.1).cuda(), randn(700, 72, seed=1).cuda(), randn(700, 4, seed=2).cuda()

    def through(stream=None):
        groups = st.group_by_expert(ids, 30, stream=stream)
        rows = st.dispatch(x, groups, stream=stream)
        out = st.combine(rows, groups, w, stream=stream)
        return [*groups, rows, out, *st.combine_backward(out, rows, groups, w, stream=stream)]

    want = through()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = through(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = through()
    keep = ids.clone()
    ids.copy_(ids_of(700, 4, 30, 3, 0.3).cuda())
    want = through()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ids.copy_(keep)


def test_inputs_dropped_after_a_call_on_another_stream():
    # the input's memory is not given to another tensor before the call has
    # read it; a long fill keeps the stream busy meanwhile
    side = torch.cuda.Stream()
    groups = st.group_by_expert(ids_of(4000, 4, 16, 1).cuda(), 16)
    busy = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        x = torch.ones(4000, 2048, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(8):
                busy.fill_(1)
        rows = st.dispatch(x, groups, stream=side)
        del x
        torch.full((4000, 2048), 7.0, device="cuda")
        side.synchronize()
        assert (rows == 1).all()


def test_given_outputs():
    groups, rows, slots = grouped(ids_of(10, 2, 4, 1), 4)
    x, w = randn(10, 16, seed=1).cuda(), randn(10, 2, seed=2).cuda()
    out = torch.full((20, 16), 7.0, device="cuda")
    assert st.dispatch(x, groups, out=out) is out
    assert np.array_equal(ref.f64(out), ref.dispatch(ref.f64(x), slots, 2))
    back = torch.full((10, 16), 7.0, device="cuda")
    assert torch.equal(st.combine(out, groups, w, out=back), st.combine(out, groups, w))
    for bad in (torch.empty(20, 15, device="cuda"), torch.empty(20, 16), torch.empty(20, 16, device="cuda").half(),
                torch.empty(16, 20, device="cuda").t()):
        with pytest.raises(ValueError):
            st.dispatch(x, groups, out=bad)


def test_offsets_past_32_bits():
    # 70000 slots of 65536 bytes: 4.6 GB of sorted rows
    tokens, k, width = 17500, 4, 65536
    ids = ids_of(tokens, k, 16, 1)
    groups = st.group_by_expert(ids.cuda(), 16)
    x = torch.randint(0, 256, (tokens, width), dtype=torch.uint8, device="cuda")
    rows = st.dispatch(x, groups)
    at = torch.cat([torch.arange(4), torch.arange(tokens * k - 300, tokens * k)]).cuda()
    assert torch.equal(rows[at], x[groups.slot_of_row[at].long() // k])
    del rows, x
    y = torch.randn(tokens * k, width // 2, dtype=torch.bfloat16, device="cuda")
    w = torch.rand(tokens, k, device="cuda")
    out = st.combine(y, groups, w)
    t = torch.arange(tokens - 40, tokens, device="cuda")
    want = (y[groups.row_of_slot[t].long()].double() * w[t].double()[..., None]).sum(1)
    size = (y[groups.row_of_slot[t].long()].double().abs() * w[t].double()[..., None]).sum(1)
    ref.within(out[t], ref.f64(want), 5 * ref.U32 * ref.f64(size) + ref.rounded(torch.bfloat16, np.abs(ref.f64(want))))


def test_refusals():
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for experts in (0, -1, 1025):
        with pytest.raises(st.SegTopKError):
            st.group_by_expert(ids, experts)
    groups = st.group_by_expert(ids, 4)
    x = torch.zeros(4, 8, device="cuda")
    for call in (lambda: st.dispatch(torch.zeros(5, 8, device="cuda"), groups),
                 lambda: st.dispatch(x.cpu(), groups),
                 lambda: st.combine(x, groups, torch.zeros(4, 2, device="cuda")),
                 lambda: st.combine(torch.zeros(8, 8, device="cuda"), groups, torch.zeros(4, 2)),
                 lambda: st.combine(torch.zeros(8, 8, device="cuda").double(), groups, torch.zeros(4, 2, device="cuda"))):
        with pytest.raises(ValueError):
            call()
