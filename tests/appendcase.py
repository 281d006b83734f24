"""Cases of the append tests: a projection's rows and the formula in 64 bits (not a test module)."""
import numpy as np
import torch

import bit_vector_quantized_gb300 as vq
import oracle
from chunkcase import D, HADAMARD
from test_gpu_rotary import frequencies, plain


class AppendCase:
    def __init__(self, fmt, hq, hkv, page, tokens, dtype=torch.float16, rdim=128, interleaved=False, base=10000.0, scaling="none", factor=1.0,
                 m=1.0, start=0, seed=0, k_scale=1.0):
        ks, kb, vs, vb = self.fmt = fmt
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.page, self.T = hq, hkv, page, tokens
        self.layout = vq.make_layout(D, hq, hkv, ks, kb, vs, vb, page)
        self.lam = (2 + rng.random((hkv, D))).astype(np.float32)
        self.lam[:, rng.permutation(D)[:4]] *= 4
        self.ck = (0.6 * rng.standard_normal((1 << kb, ks))).astype(np.float16)
        self.cv = rng.standard_normal((1 << vb, vs)).astype(np.float16)
        x = torch.randn(tokens, hq + 2 * hkv, D, generator=g)
        x[:, hq:hq + hkv] *= k_scale * torch.from_numpy(self.lam) * 0.6
        self.qkv = x.to(dtype)
        self.positions = ((start + np.arange(tokens) * 91) % (1 << 31)).astype(np.int32)
        self.pages = -(-tokens // page) + 2
        self.slots = rng.permutation(self.pages * page)[:tokens].astype(np.int64)
        self.config = vq.make_rotary(D, rdim, interleaved, base, scaling, factor, 8192, 1.0, 32.0, m)
        self.rot = (frequencies(rdim, base, scaling, factor, 8192, 1.0, 32.0), rdim, interleaved, m)

    def run(self, expect=0, q=True, **kw):
        """(q, k pool, v pool) as numpy arrays; the pools hold 0xa5 before."""
        g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        kp, vp = vq.alloc_pools(self.layout, self.pages)
        kp.fill_(0xa5)
        vp.fill_(0xa5)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        qq, k, v = self.qkv.cuda().split([self.hq, self.hkv, self.hkv], 1)
        out = torch.full((self.T, self.hq, D), 7.0, dtype=torch.float16, device="cuda")
        a = dict(positions=g(self.positions), slot_mapping=g(self.slots), k=k, v=v, lambda_=g(self.lam), codebook_k=g(self.ck), codebook_v=g(self.cv),
                 k_pool=kp, v_pool=vp, status=status)
        if q:
            a.update(q=qq, q_out=out)
        a.update(kw)
        r = vq.append_kv(self.layout, self.config, **a)
        torch.cuda.synchronize()
        assert int(status.item()) == expect
        assert r is (out if q else None)
        return (r.cpu().numpy() if q else None), kp.cpu().numpy(), vp.cpu().numpy()

    def nearest(self, x, cb):
        """(codes, gap to the next, largest score) of x [T][H][128] in 64 bits, the lowest index of equals."""
        cb = cb.astype(np.float64)
        x = x.reshape(*x.shape[:2], D // cb.shape[1], cb.shape[1])
        s = (cb * cb).sum(1) - 2 * (x @ cb.T)
        code = s.argmin(-1)
        best = np.take_along_axis(s, code[..., None], -1)
        return code, np.where(s == best, np.inf, s - best).min(-1), np.abs(s).max(-1)

    def expected(self):
        """(q, q tolerance, (K codes, whether 64 bits tell them apart), the same for V)."""
        f, r, inter, m = self.rot
        x = self.qkv.float().numpy()
        pos = np.maximum(self.positions, 0)
        q, tol = plain(x[:, :self.hq], pos, f, r, inter, m)
        k, _ = plain(x[:, self.hq:self.hq + self.hkv], pos, f, r, inter, m)
        k = (k / self.lam.astype(np.float64)) @ HADAMARD
        # Two scores in 64 bits, summed in other orders, are 2^-46 of the largest score apart at most; of keys also what
        # their angles' roundings (4 2^-53 of the angle, under 4 2^-53 of the position) make of |k~| and two centroids.
        turns = 16 * 2.0 ** -53 * float(pos.max(initial=0)) * np.linalg.norm(k, axis=-1) * np.linalg.norm(self.ck.astype(np.float64), axis=1).max()
        kc, kg, ks = self.nearest(k, self.ck)
        vc, vg, vs = self.nearest(x[:, self.hq + self.hkv:].astype(np.float64), self.cv)
        return q, tol, (kc, kg > 2.0 ** -46 * ks + turns[..., None]), (vc, vg > 2.0 ** -46 * vs)

    def check(self, expect=0, **kw):
        """Codes are equal but where 64 bits themselves cannot tell two centroids apart."""
        q, kp, vp = self.run(expect, **kw)
        want, tol, kk, vv = self.expected()
        stored = (self.positions >= 0) & (self.slots >= 0) & (self.slots < self.pages * self.page)
        if q is not None:
            live = self.positions >= 0
            assert (np.abs(q.astype(np.float64) - want) <= tol)[live].all()
            assert (q[~live] == 7.0).all()
        touched = np.zeros((self.pages, self.page), bool)
        for pool, (code, clear), cb, bits in ((kp, kk, self.ck, self.fmt[1]), (vp, vv, self.cv, self.fmt[3])):
            at = self.slots[stored]
            touched[at // self.page, at % self.page] = True
            rows = pool[at // self.page, :, at % self.page]
            n = D // cb.shape[1]
            got = oracle.unpack(rows.reshape(-1, 1, rows.shape[-1]), n, bits).reshape(rows.shape[0], rows.shape[1], n)
            off = got != code[stored]
            assert not (off & clear[stored]).any(), f"{off.sum()} of {off.size} codes differ"
            pad = oracle.pack(got.reshape(-1, 1, n), bits, rows.shape[-1]).reshape(rows.shape)
            assert np.array_equal(pad, rows)  # trailing bits are zero
            assert (pool.transpose(0, 2, 1, 3)[~touched] == 0xa5).all()
        return q, kp, vp


def close_calls(cb, rng, count, places):
    """x [count][d] about halfway between two near centroids, off by up to `places` of their distance."""
    cb = cb.astype(np.float64)
    i = rng.integers(0, len(cb), count)
    j = np.empty(count, np.int64)
    for a in range(0, count, 1024):  # (some of the codebook at a time)
        d = ((cb[i[a:a + 1024], None] - cb[None]) ** 2).sum(-1)
        d[np.arange(len(d)), i[a:a + 1024]] = np.inf
        j[a:a + 1024] = d.argmin(1)
    return (cb[i] + cb[j]) / 2 + (cb[j] - cb[i]) * (rng.random((count, 1)) - 0.5) * places
