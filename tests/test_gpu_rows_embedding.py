"""Token embedding and its table's gradient against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import rows_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def tokens_of(kind, n, vocab, seed=1):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        t = rng.integers(0, vocab, n)
    elif kind == "frequent":  # a few tokens make up most of the text
        t = np.minimum((vocab ** rng.random(n)).astype(np.int64), vocab) - 1
    elif kind == "one":
        t = np.full(n, vocab - 1)
    elif kind == "two":
        t = np.where(rng.random(n) < 0.5, 0, vocab - 1)
    elif kind == "sorted":
        t = np.sort(rng.integers(0, vocab, n))
    else:  # some outside the table, as in a shard of a vocabulary
        t = rng.integers(-vocab, vocab, n)
    return torch.from_numpy(t)


def check_gradient(g, tokens, vocab, dtype, scale=1.0, padding=None, old=None, on_gpu=None):
    out = None if old is None else old.to(dtype).cuda()
    got = st.embedding_backward(g.cuda() if on_gpu is None else on_gpu, tokens.cuda(), vocab, scale=scale,
                                padding_idx=padding, dtype=dtype if old is None else None, grad_table=out,
                                accumulate=old is not None)
    assert got.dtype == dtype and got.shape == (vocab, g.shape[-1])
    exact, size, terms = ref.embedding_backward(ref.f64(g), tokens.numpy(), vocab, scale,
                                                -1 if padding is None else padding % vocab)
    bound = (terms + 2) * ref.U32 * size
    if old is not None:
        before = ref.f64(old.to(dtype))
        # added to what was there, in 32 bits; rows without a token are not touched
        bound = np.where(terms > 0, bound + ref.U32 * (np.abs(before) + size), 0)
        exact = exact + before
        bound = bound + np.where(terms > 0, ref.rounded(dtype, np.abs(exact)), 0)
    else:
        bound = bound + np.where(terms > 0, ref.rounded(dtype, np.abs(exact)), 0)
    ref.within(got, exact, bound)


@pytest.mark.parametrize("table_dtype", DTYPES)
@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,width", [(1, 1, 1), (3, 50, 8), (40, 1000, 64), (17, 33, 250), (9, 20, 2056)])
def test_embedding(n, vocab, width, table_dtype, out_dtype):
    table = randn(vocab, width, seed=1, dtype=table_dtype)
    tokens = tokens_of("uniform", n, vocab)
    got = st.embedding(table.cuda(), tokens.cuda(), scale=3.7, out_dtype=out_dtype)
    assert got.dtype == out_dtype
    exact = ref.embedding(ref.f64(table), tokens.numpy(), float(np.float32(3.7)))
    ref.within(got, exact, 1.01 * ref.U32 * np.abs(exact) + ref.rounded(out_dtype, np.abs(exact)))


def test_embedding_without_a_scale_copies():
    for dtype in DTYPES:
        table = randn(100, 72, seed=2, dtype=dtype).cuda()
        tokens = torch.randint(0, 100, (4, 5, 6), device="cuda")
        for t in (tokens, tokens.int(), tokens.transpose(0, 2)):
            got = st.embedding(table, t)
            assert got.shape == (*t.shape, 72) and torch.equal(got, table[t.long()])


def test_embedding_of_a_part_of_a_table():
    table = randn(60, 100, seed=3).cuda()
    for part in (table[10:30], table[:, 4:68], table[:, 3:50], table[5:].t()):
        tokens = torch.randint(0, part.shape[0], (31,), device="cuda")
        assert torch.equal(st.embedding(part, tokens), part[tokens])


def test_tokens_outside_the_table():
    st.read_device_error()
    table = randn(10, 24, seed=1)
    tokens = torch.tensor([-1, 3, -(1 << 40), 9])
    got = st.embedding(table.cuda(), tokens.cuda())
    assert np.array_equal(ref.f64(got), ref.embedding(ref.f64(table), tokens.numpy(), 1.0))
    assert st.read_device_error() == 0  # negative ones are none on purpose
    tokens = torch.tensor([10, 3, 1 << 40, (1 << 32) + 1])
    got = st.embedding(table.cuda(), tokens.cuda())
    assert np.array_equal(ref.f64(got), ref.embedding(ref.f64(table), tokens.numpy(), 1.0))
    assert st.read_device_error() == st.DEVICE_ERROR_INDEX
    g = randn(4, 24, seed=2)
    check_gradient(g, tokens, 10, torch.float32)
    assert st.read_device_error() == st.DEVICE_ERROR_INDEX
    assert st.read_device_error() == 0


@pytest.mark.parametrize("kind", ["uniform", "frequent", "one", "two", "sorted", "shard"])
@pytest.mark.parametrize("n,vocab,width", [(1, 1, 1), (1, 700, 8), (5, 3, 12), (300, 40, 64), (100, 5000, 40),
                                           (2048, 512, 33), (2049, 511, 72), (5000, 100, 8), (700, 20, 2056)])
def test_gradient(n, vocab, width, kind):
    check_gradient(randn(n, width, seed=n), tokens_of(kind, n, vocab), vocab, torch.float32, scale=0.7)


@pytest.mark.parametrize("grad_dtype", DTYPES)
@pytest.mark.parametrize("table_dtype", DTYPES)
@pytest.mark.parametrize("width", [8, 100, 515])
def test_gradient_types(grad_dtype, table_dtype, width):
    g = randn(600, width, seed=1, dtype=grad_dtype)
    tokens = tokens_of("frequent", 600, 150)
    check_gradient(g, tokens, 150, table_dtype, scale=8.0)
    check_gradient(g, tokens, 150, table_dtype, scale=8.0, old=randn(150, width, seed=2))


@pytest.mark.parametrize("kind", ["uniform", "frequent", "one", "two", "shard"])
@pytest.mark.parametrize("n,vocab,width", [(1, 700, 8), (2, 100000, 8), (9, 4, 33), (3000, 70, 40), (4100, 300000, 16)])
def test_gradient_added_to_another(n, vocab, width, kind):
    check_gradient(randn(n, width, seed=n), tokens_of(kind, n, vocab), vocab, torch.float32, scale=0.7,
                   old=randn(vocab, width, seed=9))


def test_rows_without_a_token_are_not_touched():
    table = torch.full((5000, 16), float("nan"), device="cuda")
    tokens = torch.tensor([7, 4999, 7], device="cuda")
    table[tokens] = 1.0
    st.embedding_backward(torch.ones(3, 16, device="cuda"), tokens, 5000, grad_table=table, accumulate=True)
    assert (table[7] == 3).all() and (table[4999] == 2).all()
    assert int(torch.isnan(table).all(1).sum()) == 4998


@pytest.mark.parametrize("vocab,passes", [(200, 1), (511, 1), (512, 2), (262143, 2), (262144, 3), (1 << 22, 3)])
def test_sort_passes(vocab, passes):
    # tokens that differ in each digit of the sort, the last rows among them
    t = torch.cat([torch.randint(0, vocab, (2500,), generator=torch.Generator().manual_seed(vocab)),
                   torch.tensor([0, vocab - 1, vocab - 1, 0])])
    g = randn(len(t), 8, seed=1)
    got = st.embedding_backward(g.cuda(), t.cuda(), vocab)
    some, inverse = torch.unique(t, return_inverse=True)
    exact, size, terms = ref.embedding_backward(ref.f64(g), inverse.numpy(), len(some), 1.0)
    ref.within(got[some.cuda()], exact, (terms + 2) * ref.U32 * size)
    assert int((got != 0).any(1).sum()) == len(some)


@pytest.mark.parametrize("n", [2017, 4096, 4097, 8192, 8193, 16385, 32769, 70000, 131072, 131073, 300001])
@pytest.mark.parametrize("vocab", [300, 40000, 300000])
def test_sort_sizes(n, vocab):
    # every token's positions in order: a column of ones counts them, one of
    # whole numbers below 2^24 in all adds them exactly in 32 bits
    t = tokens_of("frequent", n, vocab, seed=n).int().cuda()
    g = torch.ones(n, 4, device="cuda")
    g[:, 1] = torch.arange(n, device="cuda") % 37
    got = st.embedding_backward(g, t, vocab)
    want = torch.zeros(vocab, 4, dtype=torch.float64, device="cuda").index_add_(0, t, g.double())
    assert torch.equal(got.double(), want)


def test_padding_token():
    tokens = tokens_of("frequent", 3000, 90)
    for padding in (0, 89, -1, 45):
        check_gradient(randn(3000, 24, seed=1), tokens, 90, torch.float32, padding=padding)
        check_gradient(randn(3000, 24, seed=1), tokens, 90, torch.float32, padding=padding, old=randn(90, 24, seed=2))


def test_no_tokens():
    g, t = torch.zeros(0, 16, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    assert (st.embedding_backward(g, t, 30) == 0).all()
    old = torch.ones(30, 16, device="cuda")
    assert st.embedding_backward(g, t, 30, grad_table=old, accumulate=True) is old and (old == 1).all()
    assert st.embedding(old, t).shape == (0, 16)
    assert st.embedding(torch.zeros(4, 0, device="cuda"), t).shape == (0, 0)


def test_shapes_strides_and_broadcast_gradients():
    tokens = tokens_of("frequent", 60, 25).reshape(3, 20)
    g = randn(3, 20, 48, seed=1)
    check_gradient(g, tokens, 25, torch.float32)
    check_gradient(g, tokens, 25, torch.float32, on_gpu=g.transpose(0, 1).contiguous().cuda().transpose(0, 1))
    check_gradient(g, tokens.int(), 25, torch.float32, on_gpu=g.permute(2, 0, 1).contiguous().cuda().permute(1, 2, 0))
    wide = randn(60, 60, seed=2)
    flat = tokens.reshape(-1)
    check_gradient(wide[:, 5:53], flat, 25, torch.float32, on_gpu=wide.cuda()[:, 5:53])
    one = randn(1, 48, seed=3)
    check_gradient(one.expand(60, 48), flat, 25, torch.float32, on_gpu=one.cuda().expand(60, 48))
    ones = torch.ones(()).expand(60, 48)
    check_gradient(ones, flat, 25, torch.float32, on_gpu=torch.ones((), device="cuda").expand(60, 48))


def test_nan_and_infinities_stay_in_their_rows():
    g = torch.ones(50, 16)
    tokens = torch.arange(50) % 10
    g[3], g[14, 2] = float("nan"), float("inf")
    got = st.embedding_backward(g.cuda(), tokens.cuda(), 12)
    assert torch.isnan(got[3]).all() and torch.isinf(got[4, 2])
    got[3], got[4, 2] = 5.0, 5.0
    assert (got[:10] == 5).all() and (got[10:] == 0).all()


def test_gradient_against_differences():
    # the lookup is linear in the table
    table, step, g = randn(9, 8, seed=1), randn(9, 8, seed=2), randn(40, 8, seed=3)
    tokens = tokens_of("frequent", 40, 9)
    got = ref.f64(st.embedding_backward(g.cuda(), tokens.cuda(), 9, scale=1.5))
    T, D, G = (ref.f64(t) for t in (table, step, g))
    want = (G * (ref.embedding(T + D, tokens.numpy(), 1.5) - ref.embedding(T, tokens.numpy(), 1.5))).sum()
    assert abs((got * D).sum() - want) < 42 * ref.U32 * 1.5 * np.abs(G).sum() * np.abs(D).max()


@pytest.mark.parametrize("accumulate", [False, True])
def test_results_are_the_same_from_run_to_run(accumulate):
    g, tokens = randn(6000, 64, seed=1).cuda(), tokens_of("frequent", 6000, 300).cuda()
    old = randn(300, 64, seed=2).cuda() if accumulate else None
    first = None
    for _ in range(5):
        table = old.clone() if accumulate else None
        got = st.embedding_backward(g, tokens, 300, grad_table=table, accumulate=accumulate)
        first = got if first is None else first
        assert torch.equal(first, got)


def test_on_another_stream_and_in_a_graph():
    table, g = randn(400, 40, seed=1).cuda(), randn(3000, 40, seed=2).cuda()
    tokens = tokens_of("frequent", 3000, 400).cuda()

    def both(stream=None):
        return [st.embedding(table, tokens, scale=2.0, stream=stream),
                st.embedding_backward(g, tokens, 400, scale=2.0, stream=stream)]

    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    tokens.copy_(tokens_of("uniform", 3000, 400, seed=5).cuda())
    want = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_past_32_bits():
    # a table of 2.4e9 values, 4.8 GB in 16 bits
    vocab, width = 600000, 4000
    table = torch.empty(vocab, width, dtype=torch.bfloat16, device="cuda")
    tokens = torch.tensor([0, vocab - 1, vocab - 7, vocab // 2, vocab - 1], device="cuda")
    table[tokens] = randn(5, width, seed=1, dtype=torch.bfloat16).cuda()
    assert torch.equal(st.embedding(table, tokens), table[tokens])
    g = randn(5, width, seed=2, dtype=torch.bfloat16).cuda()
    got = st.embedding_backward(g, tokens, vocab, grad_table=table)
    assert torch.equal(got[tokens[2:4]], g[2:4]) and torch.equal(got[0], g[0])
    assert torch.equal(got[vocab - 1], (g[1].float() + g[4].float()).bfloat16())
    assert int((got != 0).any(1).sum()) == 4


def test_refusals():
    table, t = torch.zeros(4, 8, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for call in (lambda: st.embedding(table, t.cpu()), lambda: st.embedding(table, t.float()),
                 lambda: st.embedding(table.double(), t), lambda: st.embedding(table, t, out_dtype=torch.float64),
                 lambda: st.embedding_backward(table, t, 4),
                 lambda: st.embedding_backward(table[:3], t, 4, padding_idx=4),
                 lambda: st.embedding_backward(table[:3], t, 4, padding_idx=-5),
                 lambda: st.embedding_backward(table[:3], t, 4, grad_table=torch.zeros(4, 7, device="cuda")),
                 lambda: st.embedding_backward(table[:3], t, 4, grad_table=torch.zeros(8, 4, device="cuda").t())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(st.SegTopKError):
        st.embedding_backward(table[:3], t, 0)
