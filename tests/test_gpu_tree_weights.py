"""Weights of every size: outputs are off by their own rounding, and small weights of many tokens count together."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402
from chunkcase import D, FORMATS  # noqa: E402
from treecase import TreeCase  # noqa: E402

pytestmark = pytest.mark.gpu


def row_of_ones(fmt, size):
    """A code row with code 1 in every place."""
    sub, bits = fmt
    x = np.zeros(D // sub * bits + 7, np.uint8)
    x[np.arange(D // sub) * bits] = 1
    return np.packbits(x, bitorder="little")[:size]


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[2], FORMATS[6]])
@pytest.mark.parametrize("n", [1, 4, 8, 20, 60])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("bits", [15, 21, 25, 27, 29])
def test_small_weights_reach_the_output(fmt, n, first, bits):
    """All tokens of a context have one key and one value, but its first or its last, whose weight is 2^bits of theirs.  38
    sequences share the pages, so that no context is cut into pieces with maxima of their own."""
    context, batch = 70000, 38
    c = TreeCase(fmt, 32, 8, 256, [context + n], [n], seed=n)
    c.lam[:] = 2
    c.k_pool[:], c.v_pool[:] = 0, 0
    c.ck[0], c.ck[1] = 0, 0.5
    c.cv[0], c.cv[1] = 1.5, 1.0
    at = 0 if first else context - 1
    for pool, f in ((c.k_pool, fmt[:2]), (c.v_pool, fmt[2:])):
        pool[c.table[0, at // 256], :, at % 256] = row_of_ones(f, pool.shape[-1])
    # k~ is 0 or 0.5 everywhere, so the scores are 0 and 0.5 of q~'s sum: of q lambda's first element, times root(128)
    c.q[:] = 0
    c.q[:, :, 0] = 1
    a = c.gpu()
    for name in ("q", "tree_masks", "positions", "seq_lens", "page_table"):
        a[name] = a[name].repeat(batch, *[1] * (a[name].dim() - 1))
    a["cu_new_lens"] = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * n
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = vq.tree_attention(c.layout, softmax_scale=bits * math.log(2) / (0.5 * 2 * math.sqrt(D)), status=status, **a)
    got = got.cpu().numpy().astype(np.float64).reshape(batch, n, 32, D)
    assert int(status.item()) == 0
    rest = context - 1 + c.see[0].sum(1)  # (the drafted tokens are like the context's)
    w = rest * 2.0 ** -bits
    want = (1.0 + 1.5 * w) / (1.0 + w)
    # The output's rounding; of p 2^-22 of each, and under 2^-21 of the largest 2^-31 of that; the scores' errors (2^-18 of a
    # score of `bits`, twice); the sums of values are fp32 in the tensor core, where a term is cut at 2^-23 of what the sum holds
    # already: 1 where the largest weight came first, else what the others made of it.
    sums = 2.0 ** -23 * rest * (1.0 if first else 1.5 * w)
    p = 2.0 ** -22 * (1 + 1.5 * w) + 1.5 * rest * 2.0 ** -31 * (bits >= 21)
    tol = 2.0 ** -11 * want + (p + sums) / (1 + w) + 4 * 2.0 ** -18 * bits * np.minimum(w, 1)
    off = np.abs(got - want[None, :, None, None])
    assert (off <= tol[None, :, None, None]).all(), (off.max(), tol.max())


@pytest.mark.parametrize("n", [4, 8, 20, 60])
def test_a_row_whose_maximum_rises_all_along(n):
    """Every token of 300 has a score a little above the one before it, so that the maximum lags and moves all the time."""
    c = TreeCase(FORMATS[0], 4, 1, 256, [300 + n], [n], seed=n)
    c.lam[:] = 2
    c.ck[:] = np.linspace(0, 1, 256)[:, None].astype(np.float16)
    c.k_pool[:] = 0
    for t in range(300):
        c.k_pool[c.table[0, t // 256], 0, t % 256] = min(t, 255)
    c.q[:] = 0
    c.q[:, :, 0] = 1
    for top in (10, 100, 1000):  # binary orders from the first to the last
        c.check(scale=top * math.log(2) / (2 * math.sqrt(D)))
        c.check(scale=-top * math.log(2) / (2 * math.sqrt(D)))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [3, 7, 20, 60])
def test_outputs_are_off_by_their_own_rounding(fmt, n):
    """In the 2-norm: fp16's own rounding of the exact outputs, and a tenth of it for all else."""
    c = TreeCase(fmt, 8, 2, 64, [n + 3000, n + 40, n + 700], [n, n, n], seed=n)
    got = c.run().astype(np.float64)
    want, _ = c.exact()
    rounding = np.linalg.norm(want.astype(np.float16).astype(np.float64) - want)
    assert np.linalg.norm(got - want) <= 1.1 * rounding
