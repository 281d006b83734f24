"""Centroids that no code names are not read: places that cannot be read (past a sequence's end, without a page) take none of them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402
from chunkcase import FORMATS  # noqa: E402
from treecase import TreeCase  # noqa: E402

pytestmark = pytest.mark.gpu


def named(pool, sub, bits, high):
    """Every code of the pool in the codebook's lower or upper half: its top bit cleared or set."""
    n = 128 // sub
    top = np.zeros((n, bits), np.uint8)
    top[:, -1] = 1
    row = np.packbits(top.ravel(), bitorder="little")
    row = np.concatenate([row, np.zeros(pool.shape[-1] - len(row), np.uint8)])
    pool[:] = pool | row if high else pool & ~row


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 4, 8, 20, 60])
@pytest.mark.parametrize("high", [False, True])
def test_centroids_that_no_code_names(fmt, n, high):
    c = TreeCase(fmt, 8, 2, 16, [n, n + 5, n + 70, n + 300, n], [n] * 5, seed=n)
    named(c.k_pool, *fmt[:2], high)
    named(c.v_pool, *fmt[2:], high)
    ck, cv = c.ck.copy(), c.cv.copy()
    for bad in (np.nan, np.inf):
        for cb in (c.ck, c.cv):
            cb[slice(0, len(cb) // 2) if high else slice(len(cb) // 2, None)] = bad
        a = c.gpu()
        c.ck, c.cv = ck.copy(), cv.copy()
        got = c.run(**{k: a[k] for k in ("codebook_k", "codebook_v")})
        want, tol = c.exact()
        assert (np.abs(got.astype(np.float64) - want) <= tol).all()
    c.table[3, 2] = -1
    got = c.run(expect=vq.VQ_DEV_BAD_PAGE, **{k: a[k] for k in ("codebook_k", "codebook_v")})
    want, tol = c.exact()
    assert (np.abs(got.astype(np.float64) - want) <= tol).all()
