"""The embedding gradient in each of its plans: long shares whose ends move to
row ends, a table cleared beside the sort, and odd widths of several tiles.

Gradients here are small whole numbers, so that every sum is exact in 32 bits
and a position lost, doubled or given to another row shows. They are
overlapping windows of one array (rows `step` elements apart), which makes
long batches of wide rows without their memory."""
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests.test_gpu_rows_embedding import tokens_of

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def windows(n, width, step, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.randint(-3, 4, (n * step + width,), generator=g, device="cuda").to(dtype)
    return flat.as_strided((n, width), (step, 1))


def sums(grad, tokens):
    """Distinct tokens and the sums of their rows, in 64 bits."""
    order = torch.argsort(tokens, stable=True)
    ids, counts = torch.unique_consecutive(tokens[order], return_counts=True)
    ends = counts.cumsum(0) - 1
    out = torch.empty(len(ids), grad.shape[1], dtype=torch.float64, device="cuda")
    columns = max(1, (1 << 27) // len(tokens))
    for c in range(0, grad.shape[1], columns):
        # (a sum over a long first dimension is slow: columns become rows)
        total = grad[:, c:c + columns][order].t().double().cumsum(1)[:, ends]
        out[:, c:c + columns] = torch.diff(total, dim=1, prepend=torch.zeros_like(total[:, :1])).t()
    return ids, out


def check(grad, tokens, vocab, mode, table_dtype, launches=None):
    """One gradient; where rows are written, over a table that held NaN."""
    width = grad.shape[1]
    ids, want = sums(grad, tokens)
    if mode == "add":
        table = torch.full((vocab, width), 2.0, dtype=table_dtype, device="cuda")
        want += 2.0
    else:
        table = torch.full((vocab, width), float("nan"), dtype=table_dtype, device="cuda")
    got = st.embedding_backward(grad, tokens, vocab, grad_table=table, accumulate=mode == "add")
    if launches is not None:
        assert st.last_launch_count() == launches
    assert torch.equal(got[ids], want.to(table_dtype))
    # the other rows hold one value
    other = torch.ones(vocab, dtype=torch.bool, device="cuda")
    other[ids] = False
    rest = 2.0 if mode == "add" else 0.0
    low, high = got.amin(1)[other], got.amax(1)[other]
    assert bool((low == rest).all()) and bool((high == rest).all())


# At 64 steps a share and more (a step is a position or, where all rows are
# written, a table row) ends move. That takes nine waves of shares, so 576
# steps for every group of threads that the GPU holds: 155648 threads over
# those that serve a row (a quarter of its columns in 32 bits).
LONG = [(400000, 30, 1024, torch.float32), (90000, 1000, 4096, torch.float32), (1500000, 300, 256, torch.float32),
        (6000000, 400, 64, torch.float32), (800000, 200, 257, torch.float32), (23000, 1500, 16383, torch.bfloat16),
        (100000, 3000, 8192, torch.bfloat16)]


@pytest.mark.parametrize("kind", ["uniform", "frequent"])
@pytest.mark.parametrize("mode", ["write", "add"])
@pytest.mark.parametrize("n,vocab,width,dtype", LONG)
def test_long_shares(n, vocab, width, dtype, mode, kind):
    step = 16 // dtype.itemsize if width % 8 == 0 else 3
    table_dtype = dtype if width == 8192 else torch.float32
    check(windows(n, width, step, dtype), tokens_of(kind, n, vocab).cuda(), vocab, mode, table_dtype)


@pytest.mark.parametrize("kind", ["uniform", "frequent"])
@pytest.mark.parametrize("width,table_dtype", [(65536, torch.float32), (65537, torch.bfloat16)])
def test_long_shares_beside_a_cleared_table(width, table_dtype, kind):
    # frequent: 1200 of the rows are all that occur, so that some runs are longer than a share
    n, vocab = 6000, 24000
    tokens = tokens_of(kind, n, vocab if kind == "uniform" else 1200).cuda() * (1 if kind == "uniform" else 20)
    grad = windows(n, width, 4 if width % 8 == 0 else 3, torch.float32)
    check(grad, tokens, vocab, "write", table_dtype, launches=4)


@pytest.mark.parametrize("mode", ["write", "add"])
def test_long_shares_are_the_same_from_run_to_run(mode):
    g = torch.Generator(device="cuda").manual_seed(1)
    grad = torch.randn(400000 * 4 + 1024, generator=g, device="cuda").as_strided((400000, 1024), (4, 1))
    tokens = tokens_of("frequent", 400000, 30).cuda()
    results = []
    for _ in range(4):
        table = torch.ones(30, 1024, device="cuda")
        results.append(st.embedding_backward(grad, tokens, 30, grad_table=table, accumulate=mode == "add"))
    assert all(torch.equal(results[0], r) for r in results[1:])


# at most a quarter of the rows have tokens, and at most 16384 tokens: four
# launches (the sort, the clearing beside it, the merge and the join)
CLEARED = [(0, 5, 3), (1, 5, 1), (1, 4, 16), (50, 1001, 33), (20, 333, 2051), (20, 335, 2056), (2048, 9001, 515),
           (2048, 9000, 72), (16384, 65537, 9), (16384, 70000, 16)]


@pytest.mark.parametrize("table_dtype", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,width", CLEARED)
def test_cleared_table(n, vocab, width, dtype, table_dtype):
    tokens = tokens_of("frequent", n, vocab, seed=n + 1).cuda()
    grad = windows(n, width, width, dtype)
    if n == 0:
        table = torch.full((vocab, width), float("nan"), dtype=table_dtype, device="cuda")
        assert (st.embedding_backward(grad, tokens, vocab, grad_table=table) == 0).all()
        return
    check(grad, tokens, vocab, "write", table_dtype, launches=4)


@pytest.mark.parametrize("table_dtype", DTYPES)
@pytest.mark.parametrize("vocab,width", [(1001, 33), (400, 64)])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_nothing_beside_a_cleared_table_is_written(vocab, width, shift, table_dtype):
    size = vocab * width
    memory = torch.full((size + 32,), float("nan"), dtype=table_dtype, device="cuda")
    table = memory[8 + shift:8 + shift + size].view(vocab, width)
    tokens = tokens_of("frequent", 60, vocab).cuda()
    grad = windows(60, width, width, torch.float32)
    st.embedding_backward(grad, tokens, vocab, grad_table=table)
    assert st.last_launch_count() == 4
    ids, want = sums(grad, tokens)
    assert torch.equal(table[ids], want.to(table_dtype)) and not bool(torch.isnan(table).any())
    assert bool(torch.isnan(memory[:8 + shift]).all()) and bool(torch.isnan(memory[8 + shift + size:]).all())


@pytest.mark.parametrize("vocab,width", [(20000, 40), (20001, 33)])
def test_cleared_table_on_another_stream_in_a_graph_and_again(vocab, width):
    n = 3000
    grad = torch.randn(n, width, generator=torch.Generator().manual_seed(1)).cuda()
    tokens = tokens_of("frequent", n, vocab).cuda()
    want = st.embedding_backward(grad, tokens, vocab)
    assert st.last_launch_count() == 4
    for _ in range(5):
        table = torch.full((vocab, width), float("nan"), device="cuda")
        assert torch.equal(st.embedding_backward(grad, tokens, vocab, grad_table=table), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = st.embedding_backward(grad, tokens, vocab, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # one gradient after the other into the same table, what is read of each
    # before the next is cleared
    table = torch.empty(vocab, width, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = [st.embedding_backward(grad, tokens + i, vocab, grad_table=table).clone() for i in range(3)]
    tokens.copy_(tokens_of("uniform", n, vocab - 3, seed=4).cuda())
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for i in range(3):
        assert torch.equal(kept[i], st.embedding_backward(grad, tokens + i, vocab))


@pytest.mark.parametrize("grad_dtype,table_dtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32),
                                                    (torch.float16, torch.float16)])
@pytest.mark.parametrize("mode", ["write", "add"])
@pytest.mark.parametrize("n,vocab,width", [(700, 20, 1025), (700, 900, 2047), (60, 40, 5001), (700, 60, 4104)])
def test_several_tiles_of_columns(n, vocab, width, mode, grad_dtype, table_dtype):
    tokens = tokens_of("frequent", n, vocab).cuda()
    check(windows(n, width, 7 if width % 2 else 8, grad_dtype), tokens, vocab, mode, table_dtype, launches=3)
