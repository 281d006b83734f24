"""Rotary positions against their formula in 64 bits.

Tolerance per element, before the first run: the output's rounding |y| 2^-11 (2^-25 where fp16 is
subnormal); sine and cosine off by at most 2^-23 each (the angle's fp32 conversion 2^-25 of a half
turn is pi 2^-25 rad, sincospi about 1 ulp) times the factor's and the two products' roundings:
under 2^-21 (|a| + |b|) m in all; the host's double frequencies, 4 2^-53 x (|a| + |b|) m."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402

pytestmark = pytest.mark.gpu


def frequencies(r, base, scaling, s, L, low, high):
    out = []
    if scaling == "base" and r > 2:
        base = base * s ** (r / (r - 2))
    for i in range(r // 2):
        f = base ** (-2 * i / r)
        if scaling == "linear":
            f = f / s
        elif scaling == "parts":
            at = lambda turns: r * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), r - 1)
            g = min(max((i - lo) / max(hi - lo, 1e-3), 0), 1)
            f = f * (1 - g) + f / s * g
        elif scaling == "wavelength":
            w = min(max((L * f / (2 * math.pi) - low) / (high - low), 0), 1)
            f = w * f + (1 - w) * f / s
        out.append(f)
    return np.array(out)


def plain(x, pos, f, r, interleaved, m):
    """(y, tolerance) in 64 bits; x [T][H][128]."""
    x = x.astype(np.float64)
    ang = pos.astype(np.float64)[:, None] * f
    co, si = np.cos(ang)[:, None] * m, np.sin(ang)[:, None] * m
    ia, ib = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    a, b = x[..., ia], x[..., ib]
    y, tol = x.copy(), np.zeros_like(x)
    y[..., ia], y[..., ib] = a * co - b * si, b * co + a * si
    e = (np.abs(a) + np.abs(b)) * m * (2.0 ** -21 + 4 * 2.0 ** -53 * ang[:, None])
    tol[..., ia], tol[..., ib] = e, e
    return y, tol + np.abs(y) * 2.0 ** -11 + 2.0 ** -25


def check(got, x, pos, f, r, interleaved, m=1.0):
    y, tol = plain(x, pos, f, r, interleaved, m)
    off = np.abs(got.float().cpu().numpy().astype(np.float64) - y)
    assert (off <= tol).all(), (off - tol).max()
    assert np.array_equal(got.float().cpu().numpy()[..., r:], x.astype(np.float16).astype(np.float32)[..., r:])


def inputs(T, heads, dtype, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, heads + pad, 128, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("T", [1, 3, 33, 700])
@pytest.mark.parametrize("r", [2, 6, 16, 32, 64, 96, 100, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts(T, r, interleaved):
    x = inputs(T, 7, torch.float16, T + r)
    pos = (torch.arange(T) * 91 % 5003).to(device="cuda", dtype=torch.int32)
    q, k, v = vq.rotary(vq.make_rotary(rotary_dim=r, interleaved=interleaved), pos, x[:, :5], x[:, 5:6], x[:, 6:])
    f, xs, ps = frequencies(r, 10000.0, "none", 1, 1, 1, 2), x.float().cpu().numpy(), pos.cpu().numpy()
    check(q, xs[:, :5], ps, f, r, interleaved)
    check(k, xs[:, 5:6], ps, f, r, interleaved)
    assert torch.equal(v, x[:, 6:])


@pytest.mark.parametrize("scaling,s,low,high", [("linear", 4.0, 1, 2), ("base", 8.0, 1, 2), ("parts", 16.0, 1.0, 32.0),
                                                ("wavelength", 8.0, 1.0, 4.0)])
@pytest.mark.parametrize("r,base,L", [(128, 500000.0, 8192), (64, 10000.0, 4096), (2, 10000.0, 100)])
def test_scalings_far_out(scaling, s, low, high, r, base, L):
    T, m = 257, 1.2
    pos = torch.cat([torch.arange(100), (torch.arange(T - 100) + 1) * 13000001 % (1 << 31)]).to(device="cuda", dtype=torch.int32)
    pos[-1] = (1 << 31) - 1
    x = inputs(T, 4, torch.bfloat16, 3)
    cfg = vq.make_rotary(rotary_dim=r, base=base, scaling=scaling, factor=s, original_len=L, low_turns=low, high_turns=high,
                         attention_factor=m)
    q, k, v = vq.rotary(cfg, pos, x[:, :3], x[:, 3:])
    f, xs, ps = frequencies(r, base, scaling, s, L, low, high), x.float().cpu().numpy(), pos.cpu().numpy()
    check(q, xs[:, :3], ps, f, r, False, m)
    check(k, xs[:, 3:], ps, f, r, False, m)
    assert v is None


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,hq,hkv", [(1, 32, 8), (64, 40, 8), (1000, 2, 1)])
def test_fused_projection_rows(dtype, T, hq, hkv):
    x = inputs(T, hq + 2 * hkv, dtype, 5, pad=1)  # rows with a tail that belongs to nobody
    pos = torch.randint(0, 200000, (T,), generator=torch.Generator().manual_seed(2)).to(device="cuda", dtype=torch.int32)
    parts = x.split([hq, hkv, hkv, 1], dim=1)
    q, k, v = vq.rotary(vq.make_rotary(interleaved=True, rotary_dim=96), pos, *parts[:3])
    f, xs, ps = frequencies(96, 10000.0, "none", 1, 1, 1, 2), x.float().cpu().numpy(), pos.cpu().numpy()
    check(q, xs[:, :hq], ps, f, 96, True)
    check(k, xs[:, hq:hq + hkv], ps, f, 96, True)
    assert torch.equal(v, parts[2].half())


@pytest.mark.parametrize("r,interleaved", [(128, False), (64, True), (20, False)])
def test_in_place_and_padding_rows(r, interleaved):
    T = 130
    q0, k0 = inputs(T, 8, torch.float16, 8), inputs(T, 2, torch.float16, 9)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 1000
    pos[100:] = -1
    cfg = vq.make_rotary(rotary_dim=r, interleaved=interleaved)
    q, k = q0.clone(), k0.clone()
    vq.rotary(cfg, pos, q, k, q_out=q, k_out=k)
    want = vq.rotary(cfg, pos[:100].clone(), q0[:100], k0[:100])
    assert torch.equal(q[:100], want[0]) and torch.equal(k[:100], want[1])
    assert torch.equal(q[100:], q0[100:]) and torch.equal(k[100:], k0[100:])  # left as they were


def test_infinities_stay_in_their_pair():
    x = inputs(4, 2, torch.float16, 1)
    x[1, 0, 70] = math.inf   # behind rotary_dim: passes through alone
    x[2, 1, 3] = math.nan    # pair (3, 35)
    pos = torch.tensor([5, 6, 7, 8], dtype=torch.int32, device="cuda")
    q = vq.rotary(vq.make_rotary(rotary_dim=64), pos, x)[0]
    bad = ~torch.isfinite(q)
    assert bad.nonzero().tolist() == [[1, 0, 70], [2, 1, 3], [2, 1, 35]]


def test_no_tokens_and_another_stream():
    cfg = vq.make_rotary()
    e = torch.empty(0, 4, 128, dtype=torch.float16, device="cuda")
    q, k, v = vq.rotary(cfg, torch.empty(0, dtype=torch.int32, device="cuda"), e, e, e)
    assert q.shape == (0, 4, 128)
    x, pos = inputs(50, 4, torch.float16), torch.arange(50, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q = vq.rotary(cfg, pos, x, stream=s)[0]
    s.synchronize()
    assert torch.equal(q, vq.rotary(cfg, pos, x)[0])


def test_refusals():
    cfg = vq.make_rotary()
    x, pos = inputs(8, 4, torch.float16), torch.arange(8, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        vq.rotary(cfg, pos, x.float())
    with pytest.raises(TypeError):
        vq.rotary(cfg, pos.long(), x)
    with pytest.raises(ValueError):
        vq.rotary(cfg, pos, x[:4])
    with pytest.raises(ValueError):
        vq.rotary(cfg, pos, x[:, ::2])
    with pytest.raises(ValueError):
        vq.rotary(cfg, pos)
    with pytest.raises(vq.VQError):  # an output over part of an input
        vq.rotary(cfg, pos, x[:, :2], q_out=x.view(-1)[:8 * 2 * 128].view(8, 2, 128))
    with pytest.raises(ValueError):
        vq.make_rotary(scaling="other")
