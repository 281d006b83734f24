"""Codes of keys that lie next to borders, by roundings of their own: codes are equal to the formula's in 64 bits.

A key's smoothing factors are fp32 numbers of any size, so a head's factors set where its transformed key lies, to
fp32's last places."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from appendcase import AppendCase  # noqa: E402
from chunkcase import D, FORMATS, HADAMARD  # noqa: E402

pytestmark = pytest.mark.gpu

HEADS = 64


def keys_at(c, want, rng, token=0):
    """Keys of the case's one token and factors of its heads, so that k~ is `want` [heads][128] to about 2^-24 of its norm."""
    z = want @ HADAMARD
    x = np.sign(z) * (0.5 + rng.random(z.shape))
    x = torch.from_numpy(x).to(c.qkv.dtype)
    c.qkv[token, c.hq:c.hq + c.hkv] = x
    z = np.where(z == 0, 1, z)
    c.lam = np.abs(x.double().numpy() / z).astype(np.float32)


def case(fmt, tokens, seed, dtype=torch.float16, **kw):
    c = AppendCase(fmt, HEADS, HEADS, 16, tokens, dtype, seed=seed, **kw)
    c.positions[:] = 0
    return c


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[1], FORMATS[6]])
@pytest.mark.parametrize("other", [1, 200])
def test_small_parts_of_a_long_key(fmt, other):
    """All but one sub-vector are about halfway between two small centroids, in one group of the search or in two; what the
    key's roundings move them by grows with the whole key."""
    c = case(fmt, 1, 5)
    rng = np.random.default_rng(6)
    d = fmt[0]
    c.ck += np.where(c.ck < 0, -1, 1).astype(np.float16)  # all others are far off
    c.ck[0], c.ck[other] = 0, 0
    c.ck[0, 0], c.ck[other, 0] = 1e-4, 2e-4
    want = np.zeros((HEADS, D // d, d))
    want[..., 0] = 1.5e-4 + 4e-5 * (rng.random((HEADS, D // d)) - 0.5)
    want[:, 7] = 800 * (1 + rng.random((HEADS, d)))
    keys_at(c, want.reshape(HEADS, D), rng)
    c.check()


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[1], FORMATS[6]])
def test_parts_that_fp32_makes_zero(fmt):
    """Factors an fp32 step apart whose quotients round to one number: all but one sub-vector are zero in fp32, and nearer to
    another centroid than to that at zero in truth."""
    c = case(fmt, 1, 7)
    rng = np.random.default_rng(8)
    c.ck += np.where(c.ck < 0, -1, 1).astype(np.float16)
    c.ck[:2 * fmt[0] + 1] = 0
    for i in range(fmt[0]):  # (of different lengths: the parts' elements are whole multiples of one number, equal ones among them)
        c.ck[1 + 2 * i, i], c.ck[2 + 2 * i, i] = (34 + 2 * i) * 2.0 ** -24, -(35 + 2 * i) * 2.0 ** -24
    lam = (1.95 + 0.04 * rng.random((HEADS, 1))).astype(np.float32)
    c.lam = np.where(rng.random((HEADS, D)) < 0.5, lam, np.nextafter(lam, np.float32(2)))
    c.qkv[:, HEADS:2 * HEADS] = 255
    c.check()
