"""Codes of keys that lie next to borders, by roundings of their own: codes are equal to the formula's in 64 bits.

A key's smoothing factors are fp32 numbers of any size, so a head's factors set where its transformed key lies, to
fp32's last places."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from appendcase import AppendCase, close_calls  # noqa: E402
from chunkcase import D, FORMATS, HADAMARD  # noqa: E402

pytestmark = pytest.mark.gpu

HEADS = 64
SIGNS = np.sign(HADAMARD)


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


@pytest.mark.parametrize("x,lam,a,b", [(3.31640625, 8.648420333862305, (4.2578125, 0), (4.41796875, 0.01354217529296875)),
                                       (0.412353515625, 3.074970006942749, (1.484375, 0), (1.5478515625, 0.01157379150390625))])
def test_a_key_of_equal_channels(x, lam, a, b):
    c = case(FORMATS[1], 2, 1)
    c.lam[:] = np.float32(lam)
    c.qkv[:, HEADS:2 * HEADS] = x
    c.ck[:] = np.float16(30) + np.arange(256)[:, None]
    c.ck[4], c.ck[9] = a, b
    c.check()


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[1], FORMATS[6]])
@pytest.mark.parametrize("m", [1.0, 1.277])
@pytest.mark.parametrize("seed", range(6))
def test_keys_that_are_all_in_one_element(fmt, m, seed):
    """Rows of the transform: the roundings of the division, the last product and the attention factor are the same in all channels."""
    c = case(fmt, 3, seed, m=m)
    rng = np.random.default_rng(seed)
    border = 25
    c.ck[:] = 0
    c.ck[:, 0] = 30 + np.arange(len(c.ck)) % 64
    c.ck[:border + 1, 0] = 4 + 0.0390625 * np.arange(border + 1)
    x = (0.25 + 4 * rng.random(HEADS)).astype(np.float16)
    at = 4 + 0.0390625 * (rng.integers(0, border, HEADS) + 0.5)
    c.lam[:] = (m * x.astype(np.float64) * math.sqrt(D) / (at * (1 + 2.0 ** -24 * (6 * rng.random(HEADS) - 3)))).astype(np.float32)[:, None]
    for t, row in enumerate((0, fmt[0] * 3, D - fmt[0])):
        c.qkv[t, HEADS:2 * HEADS] = torch.from_numpy(x[:, None] * SIGNS[row].astype(np.float16))
    c.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("places", [1e-3, 1e-5, 1e-7])
def test_keys_next_to_borders(fmt, dtype, places):
    c = case(fmt, 1, 3, dtype)
    rng = np.random.default_rng(4)
    keys_at(c, close_calls(c.ck, rng, HEADS * D // fmt[0], places).reshape(HEADS, D), rng)
    c.check()


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


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[2], FORMATS[6]])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rdim", [128, 50, 2])
def test_uneven_factors_within_a_pair(fmt, interleaved, rdim):
    """A strong channel that half a turn nearly hides from its partner, whose factor is small: the angle's rounding is large
    beside what is left."""
    c = case(fmt, 4, 9, rdim=rdim, interleaved=interleaved)
    c.positions[:] = [355, 710, 355, 22]
    c.lam[:] = 1
    k = 0.05 * torch.randn(4, HEADS, D, generator=torch.Generator().manual_seed(10))
    strong, weak = 0, 1 if interleaved else rdim // 2
    c.lam[:, strong], c.lam[:, weak] = 1000, 0.01
    k[:, :, strong], k[:, :, weak] = 100, 1e-3
    c.qkv[:, HEADS:2 * HEADS] = k.half()
    c.ck = (c.ck * np.float16(0.1))
    c.check()


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[6]])
def test_many_tokens_of_uneven_factors(fmt):
    """Ordinary keys and positions with factors from 2^-6 to 2^6."""
    c = AppendCase(fmt, 4, 4, 64, 300, seed=11)
    rng = np.random.default_rng(12)
    c.lam = (2.0 ** (12 * rng.random((4, D)) - 6)).astype(np.float32)
    c.ck = c.ck * np.float16(4)
    c.check()
