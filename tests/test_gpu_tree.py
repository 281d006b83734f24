"""Attention of drafted trees over the paged codes against its formula in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402
from chunkcase import FORMATS  # noqa: E402
from treecase import TreeCase, tree  # noqa: E402

pytestmark = pytest.mark.gpu

HEADS = [(2, 2), (4, 2), (6, 2), (8, 2), (5, 1), (7, 1), (8, 1)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 3, 4, 5, 9, 17, 64, 65, 200])
def test_formats(fmt, n):
    TreeCase(fmt, 8, 2, 64, [n + 400, n + 111, n], [n, max(n // 2, 1), n], seed=n).check()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 2, 3, 6, 13, 33, 64, 256])
def test_heads(heads, n):
    TreeCase(FORMATS[0], *heads, 16, [n, n + 5, n + 200], [n, n, n], seed=n).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (7, 3), (100, 4), (129, 65), (1000, 140), (1 << 30, 5)])
@pytest.mark.parametrize("n", [1, 5, 33, 150])
@pytest.mark.parametrize("heads", [(8, 2), (5, 1)])
def test_windows(window, sinks, n, heads):
    TreeCase(FORMATS[1], *heads, 48, [n, n + 1, n + 15, n + 333, n + 2000], [n] * 5, seed=n).check(window, sinks)


@pytest.mark.parametrize("context", [0, 1, 63, 64, 65, 126, 127, 128, 129, 191, 255, 300])
@pytest.mark.parametrize("n", [1, 2, 31, 63, 64, 65, 128])
def test_trees_over_block_and_word_borders(context, n):
    TreeCase(FORMATS[0], 4, 1, 16, [context + n, 40 + n], [n, 1], seed=context).check()


@pytest.mark.parametrize("heads", [(1, 1), (4, 1), (8, 1)])
@pytest.mark.parametrize("n", [3, 20, 70])
def test_any_bits(heads, n):
    """Masks that are no trees: rows without their own bit, rows without any (zero where nothing is cached), all bits,
    bits past the sequence's tokens, words to spare."""
    rng = np.random.default_rng(n)
    some = rng.random((n, n)) < 0.3
    some[0] = False
    some[n // 2] = True
    c = TreeCase(FORMATS[2], *heads, 16, [n, n + 130, n], [n, n, n], masks=[some, some.T.copy(), np.zeros((n, n), bool)], mask_words=4, junk=True)
    got = c.check()
    assert (got[0] == 0).all() and (got[2 * n:] == 0).all()


def test_positions_before_the_tree_and_far_behind_it():
    c = TreeCase(FORMATS[0], 4, 1, 16, [90, 400], [20, 33], seed=1)
    c.positions = np.random.default_rng(2).integers(-5, 700, c.T).astype(np.int32)
    c.positions[3], c.positions[40] = -(2 ** 31), 2 ** 31 - 1
    for window, sinks in ((30, 2), (350, 0), (1 << 30, 1), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)):
        c.check(window, sinks)


@pytest.mark.parametrize("n", [2, 30])
def test_ragged_batch_with_idle_sequences(n):
    rng = np.random.default_rng(n)
    news = rng.integers(0, n + 1, 37)
    news[[0, 5, 6, 36]] = 0
    c = TreeCase(FORMATS[2], 5, 1, 64, news + rng.integers(0, 900, 37), news, seed=n, spare_rows=7)
    c.check()
    c.check(200, 20)


@pytest.mark.parametrize("rows", [16, 32, 128, 256])
def test_every_tile_height_takes_every_batch(rows, monkeypatch):
    """The height is a matter of time only: a ragged batch with idle sequences, at each of them."""
    monkeypatch.setenv("VQ_TREE_ROWS", str(rows))
    TreeCase(FORMATS[1], 8, 2, 64, [70, 300, 0, 1500, 64, 129], [64, 3, 0, 40, 0, 9], seed=rows).check()


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[2], FORMATS[6]])
@pytest.mark.parametrize("n", [2, 16, 33, 90])
@pytest.mark.parametrize("window,sinks", [(0, 0), (4096, 4)])
def test_long_context_over_many_ctas(fmt, n, window, sinks):
    TreeCase(fmt, 4, 1, 256, [30011], [n], seed=n).check(window, sinks)


@pytest.mark.parametrize("n", [3, 40])
def test_scores_of_every_size(n):
    """Maxima that keep rising along the context, and scores so large that one token takes all."""
    c = TreeCase(FORMATS[0], 4, 1, 64, [1500], [n], seed=3, q_scale=20.0)
    c.check()
    c.check(scale=1e-4)
    c.check(scale=-0.05)


@pytest.mark.parametrize("n", [2, 70])
def test_bad_pages_are_skipped_and_told(n):
    c = TreeCase(FORMATS[0], 4, 2, 16, [200 + n, 300 + n], [n, n], seed=n)
    c.table[0, 3], c.table[1, 7], c.table[1, -1] = -1, 10 ** 6, -7
    c.check(expect=vq.VQ_DEV_BAD_PAGE)
    c.table[:] = -1
    got = c.check(expect=vq.VQ_DEV_BAD_PAGE)
    assert (got[:c.cu[-1]] == 0).all()


def test_sequences_out_of_their_bounds_are_left_out():
    c = TreeCase(FORMATS[0], 4, 2, 16, [50, 60, 70, 80], [5, 9, 5, 5], seed=4, max_new=8)
    lens = c.gpu()["seq_lens"]
    lens[0], lens[3] = 4, 10 ** 6  # fewer tokens than drafted ones; past the bound
    got = c.run(expect=vq.VQ_DEV_BAD_LENGTH, seq_lens=lens)
    want, tol = c.exact(seqs=[2])
    rows = slice(14, 19)
    assert (np.abs(got[rows] - want[rows]) <= tol[rows]).all()
    assert (got[:14] == 7).all() and (got[19:] == 7).all()


@pytest.mark.parametrize("n", [4, 50])
def test_a_chain_is_what_chunk_attention_computes(n):
    """Drafted tokens one after the other: the same sums in another order, each within the tolerance."""
    c = TreeCase(FORMATS[0], 8, 2, 64, [n + 700, n + 20], [n, n], masks=[np.tril(np.ones((n, n), bool))] * 2)
    a = c.gpu()
    del a["tree_masks"], a["positions"]
    for window, sinks in ((0, 0), (300, 5)):
        chunk = vq.chunk_attention(c.layout, window=window, num_sinks=sinks, **a).cpu().numpy().astype(np.float64)
        _, tol = c.exact(window, sinks)
        assert (np.abs(c.check(window, sinks) - chunk) <= 2 * tol).all()


@pytest.mark.parametrize("n", [3, 24, 60])
def test_results_do_not_vary_and_workspaces_need_no_state(n):
    c = TreeCase(FORMATS[3], 8, 2, 64, [n + 9000, n + 33], [n, n], seed=5)
    ws = vq.alloc_tree_workspace(c.layout, 2, c.T, c.max_len, c.max_new)
    first = None
    for fill in (0, 255, 127):
        ws.fill_(fill)
        got = c.run(workspace=ws)
        assert first is None or np.array_equal(first, got)
        first = got
    # a larger step's workspace does for smaller ones
    big = vq.alloc_tree_workspace(c.layout, 64, 64 * 256, 100000, 256)
    assert np.array_equal(first, c.run(workspace=big))


def test_the_smallest_call_and_empty_ones():
    TreeCase(FORMATS[0], 1, 1, 16, [1], [1]).check()
    c = TreeCase(FORMATS[0], 2, 1, 16, [5], [1])
    a = c.gpu()
    e = dict(a, q=a["q"][:0], tree_masks=a["tree_masks"][:0], positions=a["positions"][:0])
    assert vq.tree_attention(c.layout, **e).shape == (0, 2, 128)


@pytest.mark.parametrize("n", [5, 30])
def test_streams_and_graphs(n):
    c = TreeCase(FORMATS[0], 8, 2, 64, [n + 800, n + 300], [n, n], seed=6)
    want, tol = c.exact()
    a, s = c.gpu(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = vq.tree_attention(c.layout, stream=s, **a)
    s.synchronize()
    assert (np.abs(got.cpu().numpy() - want) <= tol).all()
    ws = vq.alloc_tree_workspace(c.layout, 2, c.T, c.max_len, c.max_new)
    out = torch.empty_like(got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vq.tree_attention(c.layout, out=out, workspace=ws, **a)
    # other trees and lengths within the bounds, the same graph
    d = TreeCase(FORMATS[0], 8, 2, 64, [n + 800, n + 300], [n, n], seed=7, masks=[tree(n, np.random.default_rng(i)) for i in (8, 9)])
    for name, x in d.gpu().items():
        if torch.is_tensor(x):
            a[name].copy_(x)
    a["seq_lens"][0] -= 700
    d.lens[0] -= 700
    d.positions[:n] -= 700
    ws.random_()
    g.replay()
    torch.cuda.synchronize()
    want, tol = d.exact()
    assert (np.abs(out.cpu().numpy() - want) <= tol).all()


def test_rows_that_do_not_belong_to_the_sequence_do_not_reach_it():
    """NaN queries of one sequence stay there."""
    c = TreeCase(FORMATS[0], 4, 1, 16, [100, 100], [9, 9], seed=8)
    a = c.gpu()
    a["q"][:9] = float("nan")
    got = c.run(q=a["q"])
    want, tol = c.exact(seqs=[1])
    assert np.isnan(got[:9]).all() and (np.abs(got[9:] - want[9:]) <= tol[9:]).all()


@pytest.mark.parametrize("n", [4, 12, 40])
def test_a_query_that_is_not_a_number_stays_in_its_row(n):
    c = TreeCase(FORMATS[0], 4, 1, 16, [100 + n], [n], seed=9)
    a = c.gpu()
    a["q"][1, 2, 7] = float("nan")
    a["q"][2, 1, 3] = float("inf")
    got = c.run(q=a["q"])
    want, tol = c.exact()
    fine = np.ones((n, 4), bool)
    fine[1, 2] = fine[2, 1] = False
    assert (np.abs(got - want) <= tol)[fine].all() and np.isnan(got[1, 2]).all()
