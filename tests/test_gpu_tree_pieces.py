"""Trees over many short sequences, and over short ones among long ones: a CTA's pieces of one block each, one behind the
other, in tiles of every height."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from chunkcase import FORMATS  # noqa: E402
from treecase import TreeCase  # noqa: E402

pytestmark = pytest.mark.gpu


def check(c, seqs, window=0, sinks=0):
    """The rows of some sequences against the formula, and every row written."""
    got = c.run(window, sinks).astype(np.float64)
    want, tol = c.exact(window, sinks, seqs=seqs)
    for b in seqs:
        rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
        assert (np.abs(got[rows] - want[rows]) <= tol[rows]).all(), b
    assert not (got[:int(c.cu[-1])] == 7).all(axis=(1, 2)).any()


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[2], FORMATS[6]])
@pytest.mark.parametrize("n", [1, 4, 8, 20])
def test_many_short_sequences(fmt, n):
    """128 conversations of about 100 tokens: every CTA has seven pieces of one block."""
    rng = np.random.default_rng(n)
    check(TreeCase(fmt, 32, 8, 64, n + rng.integers(0, 100, 128), [n] * 128, seed=n), [0, 1, 64, 127])


@pytest.mark.parametrize("n", [4, 8, 20])
def test_a_new_conversation_among_long_ones(n):
    """All eight heads of the short one fall to one CTA."""
    lens = [8000 + 440 * i for i in range(16)]
    check(TreeCase(FORMATS[0], 32, 8, 64, lens[:9] + [43 + n] + lens[9:], [n] * 17, seed=n), [0, 9, 16])
    check(TreeCase(FORMATS[2], 32, 8, 64, [4000] * 32 + [60], [n] * 33, seed=n), [31, 32], window=700, sinks=4)


@pytest.mark.parametrize("fmt", [FORMATS[1], FORMATS[6]])
@pytest.mark.parametrize("heads,n", [((32, 8), 1), ((8, 8), 16), ((8, 8), 32)])
def test_the_largest_batch_of_the_shortest_sequences(fmt, heads, n):
    rng = np.random.default_rng(n)
    news = rng.integers(1, n + 1, 1024)
    check(TreeCase(fmt, *heads, 16, news + rng.integers(0, 9, 1024), news, seed=n, max_new=n), [0, 1, 500, 1022, 1023])


def test_lengths_of_every_kind_in_one_batch():
    """Pieces of one block between longer ones, with idle sequences."""
    rng = np.random.default_rng(3)
    news = rng.integers(0, 9, 200)
    lens = news + np.where(rng.random(200) < 0.7, rng.integers(0, 100, 200), rng.integers(0, 6000, 200))
    c = TreeCase(FORMATS[0], 32, 8, 16, lens, news, seed=3)
    check(c, [i for i in range(0, 200, 23) if news[i]])
