"""Coding of rotated keys and values into pages against the formula in 64 bits: codes are equal, not near."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402
import oracle  # noqa: E402
from appendcase import AppendCase, close_calls  # noqa: E402
from chunkcase import D, FORMATS  # noqa: E402

pytestmark = pytest.mark.gpu


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [1, 2, 3, 17, 64, 130])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_formats(fmt, tokens, dtype):
    AppendCase(fmt, 8, 2, 64, tokens, dtype, seed=tokens).check()


@pytest.mark.parametrize("r", [2, 6, 16, 32, 64, 96, 100, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts(r, interleaved):
    AppendCase(FORMATS[0], 5, 1, 16, 90, rdim=r, interleaved=interleaved, seed=r).check()


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("base", 8.0), ("parts", 16.0), ("wavelength", 8.0)])
def test_scalings_far_out(scaling, factor):
    AppendCase(FORMATS[2], 4, 4, 48, 70, torch.bfloat16, 64, True, 500000.0, scaling, factor, 1.3, 1_000_000, seed=3).check()


@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (7, 1), (40, 8), (64, 64)])
def test_heads(heads):
    AppendCase(FORMATS[1], *heads, 16, 37, seed=heads[0]).check()


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[2], FORMATS[6]])
def test_many_tokens(fmt):
    """More vectors than the grid has warps."""
    AppendCase(fmt, 2, 2, 256, 700 if fmt[1] == 12 else 5001, seed=1).check()


def test_padding_bad_slots_and_left_out_tokens():
    c = AppendCase(FORMATS[0], 4, 2, 16, 50, seed=2)
    c.positions[[3, 40, 41]] = -1
    c.slots[[0, 7, 40]] = -1
    c.check()
    c.slots[[9, 49]] = [c.pages * c.page, 2 ** 62]
    c.check(expect=vq.VQ_DEV_BAD_SLOT)
    c.positions[:] = -1
    c.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_values_next_to_borders(fmt):
    """Values about halfway between two centroids: what fp32 cannot tell apart is told in 64 bits."""
    c = AppendCase(fmt, 2, 2, 64, 200, seed=5)
    rng = np.random.default_rng(6)
    n = 200 * 2 * D // fmt[2]
    v = np.concatenate([close_calls(c.cv, rng, n // 4, s) for s in (1e-3, 1e-4, 1e-6, 0.0)]).reshape(200, 2, D)
    c.qkv[:, 4:] = torch.from_numpy(v).half()
    c.check()


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[1], FORMATS[2], FORMATS[6]])
def test_equal_centroids_give_the_lowest_index(fmt):
    c = AppendCase(fmt, 2, 2, 64, 60, seed=7)
    rng = np.random.default_rng(8)
    for cb in (c.ck, c.cv):
        cb[rng.permutation(len(cb))[:len(cb) // 2]] = cb[3]  # half of the codebook is one centroid
    c.qkv[:30, 4:] = torch.from_numpy(np.tile(c.cv[3], D // fmt[2]))
    c.check()
    c.ck[:], c.cv[:] = c.ck[0], c.cv[0]
    _, kp, vp = c.run()
    at = c.slots
    assert not kp[at // 64, :, at % 64].any() and not vp[at // 64, :, at % 64].any()


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[1], FORMATS[6]])
@pytest.mark.parametrize("scale", [2.0 ** -14, 1.0, 2.0 ** 8])
def test_codebooks_of_every_size(fmt, scale):
    """Tiny, ordinary and large centroids and rows (fp16's range, subnormal centroids among them)."""
    c = AppendCase(fmt, 4, 2, 16, 40, seed=9)
    c.ck, c.cv = (c.ck * np.float16(scale)), (c.cv * np.float16(scale))
    c.qkv = (c.qkv.float() * scale).half()
    c.check()


def test_rows_of_zeros_and_rows_that_are_far_off():
    c = AppendCase(FORMATS[0], 4, 2, 16, 40, torch.bfloat16, seed=10)
    c.qkv[:10] = 0
    c.qkv[10:20, 4:] *= 3e4  # every score is dominated by the row
    c.qkv[20:30, 4:] *= 1e-30
    c.check()


def test_infinities_and_nan_stay_with_their_vectors():
    c = AppendCase(FORMATS[0], 4, 2, 16, 40, torch.bfloat16, seed=11)
    clean = c.run()
    c.qkv[3, 4], c.qkv[5, 6], c.qkv[7, 7, 9], c.qkv[8, 5, 100] = float("nan"), float("inf"), float("nan"), float("-inf")
    q, kp, vp = c.run()
    assert np.array_equal(q, clean[0])
    for pool, was, dirty in ((kp, clean[1], {(3, 0), (8, 1)}), (vp, clean[2], {(5, 0), (7, 1)})):
        for t in range(40):
            for h in range(2):
                s = c.slots[t]
                same = np.array_equal(pool[s // 16, h, s % 16], was[s // 16, h, s % 16])
                assert same or (t, h) in dirty


def test_against_the_two_calls():
    """Values' codes are vq_encode_kv's, keys' are those of keys that were not rounded in between."""
    c = AppendCase(FORMATS[0], 8, 2, 64, 300, seed=12)
    q, kp, vp = c.check()
    q2, k2, v2 = vq.rotary(c.config, gpu(c.positions), *c.qkv.cuda().split([8, 2, 2], 1))
    kp2, vp2 = vq.alloc_pools(c.layout, c.pages)
    kp2.fill_(0xa5), vp2.fill_(0xa5)
    vq.encode_kv(c.layout, k2, v2, gpu(c.slots), gpu(c.lam), gpu(c.ck), gpu(c.cv), kp2, vp2)
    torch.cuda.synchronize()
    assert np.array_equal(q, q2.cpu().numpy())
    assert (vp != vp2.cpu().numpy()).mean() < 1e-4  # (vq_encode_kv's may be off next to a border)
    assert (kp != kp2.cpu().numpy()).mean() < 0.02


def test_strides_of_their_own_and_without_queries():
    c = AppendCase(FORMATS[2], 4, 2, 16, 33, torch.bfloat16, seed=13)
    want = c.check()
    wide = torch.zeros(33, 9, D, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:3], wide[:, 5:7] = c.qkv[:, 4:6].cuda(), c.qkv[:, 6:].cuda()
    _, kp, vp = c.run(q=False, k=wide[:, 1:3], v=wide[:, 5:7])
    assert np.array_equal(kp, want[1]) and np.array_equal(vp, want[2])


def test_in_place_streams_and_graphs():
    c = AppendCase(FORMATS[0], 4, 2, 16, 70, seed=14)
    want = c.check()
    q = c.qkv[:, :4].contiguous().cuda()
    kp, vp = vq.alloc_pools(c.layout, c.pages)
    kp.fill_(0xa5), vp.fill_(0xa5)
    _, k, v = (x.contiguous() for x in c.qkv.cuda().split([4, 2, 2], 1))
    args = (c.layout, c.config, gpu(c.positions), gpu(c.slots), k, v, gpu(c.lam), gpu(c.ck), gpu(c.cv), kp, vp)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = vq.append_kv(*args, q=q, q_out=q, stream=s)
    s.synchronize()
    assert got is q and np.array_equal(q.cpu().numpy(), want[0])
    assert np.array_equal(kp.cpu().numpy(), want[1]) and np.array_equal(vp.cpu().numpy(), want[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vq.append_kv(*args)
    d = AppendCase(FORMATS[0], 4, 2, 16, 70, seed=15)
    d.lam, d.ck, d.cv, d.slots = c.lam, c.ck, c.cv, c.slots
    want = d.check(q=False)
    kp.fill_(0xa5), vp.fill_(0xa5)
    k.copy_(d.qkv[:, 4:6])
    v.copy_(d.qkv[:, 6:])
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(kp.cpu().numpy(), want[1]) and np.array_equal(vp.cpu().numpy(), want[2])


def test_slots_past_32_bits():
    """Pools of more than 2^32 bytes, rows at their ends."""
    layout = vq.make_layout(D, 8, 8, 4, 8, 4, 8, 256)
    pages = (1 << 32) // (8 * 256 * 32) + 3
    kp, vp = vq.alloc_pools(layout, pages)
    c = AppendCase(FORMATS[0], 8, 8, 256, 4, seed=16)
    slots = torch.tensor([0, pages * 256 - 1, (pages - 1) * 256, pages * 128], device="cuda")
    _, k, v = c.qkv.cuda().split([8, 8, 8], 1)
    vq.append_kv(layout, c.config, gpu(c.positions), slots, k, v, gpu(c.lam), gpu(c.ck), gpu(c.cv), kp, vp)
    _, _, (kc, _), (vc, _) = c.expected()
    for pool, code in ((kp, kc), (vp, vc)):
        rows = pool[slots // 256, :, slots % 256].cpu().numpy()
        assert np.array_equal(oracle.unpack(rows.reshape(-1, 1, 32), 32, 8).reshape(4, 8, 32), code)
