"""Cases of the chunk-attention tests: random codes in paged pools and the formula in 64 bits (not a test module).

Tolerance of an output element, with w the row's exact softmax weights, o the exact output and
A = sum_p w_p |v_p|: the output's own rounding 2^-11 |o| + 2^-25; p rounded to fp16 once, at most
2^-11 A (and 2^-25 per token where p is subnormal next to a largest p of at least 1); the score
error d turns into at most 2 d A.  d: the query transform, the products' fp32 sums and exp2 are each
off by a few 2^-22 of the sum of the terms' magnitudes S = |q~| . |k~| * scale; together under 2^-18 S."""
import math

import numpy as np
import torch

import bit_vector_quantized_gb300 as vq
import oracle

D = 128
FORMATS = [(4, 8, 4, 8), (2, 8, 4, 8), (2, 8, 4, 9), (4, 8, 4, 9), (4, 8, 2, 8), (2, 8, 2, 8), (8, 12, 8, 12)]
HADAMARD = np.array([[(-1) ** bin(i & j).count("1") for j in range(D)] for i in range(D)]) / math.sqrt(D)


class Case:
    """A batch on the GPU; lens: tokens of each sequence with the new ones, news: new tokens."""

    def __init__(self, fmt, hq, hkv, page, lens, news, seed=0, spare_rows=0, spare_pages=2, max_new=None, q_scale=1.0):
        ks, kb, vs, vb = fmt
        rng = np.random.default_rng(seed)
        self.fmt, self.hq, self.hkv, self.page = fmt, hq, hkv, page
        self.lens, self.news = np.array(lens, np.int32), np.array(news, np.int32)
        self.layout = vq.make_layout(D, hq, hkv, ks, kb, vs, vb, page)
        need = -(-self.lens // page)
        total = int(need.sum()) + spare_pages
        phys = rng.permutation(total)
        self.table = np.full((len(lens), max(1, int(need.max(initial=0)))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = phys[at:at + n]
            at += n
        kr, vr = vq.row_bytes(self.layout)
        self.k_pool = rng.integers(0, 256, (total, hkv, page, kr), dtype=np.uint8)
        self.v_pool = rng.integers(0, 256, (total, hkv, page, vr), dtype=np.uint8)
        self.lam = (2 + rng.random((hkv, D))).astype(np.float32)
        self.lam[:, rng.permutation(D)[:4]] *= 4
        self.ck = (0.6 * rng.standard_normal((1 << kb, ks))).astype(np.float16)
        self.cv = rng.standard_normal((1 << vb, vs)).astype(np.float16)
        self.cu = np.concatenate([[0], np.cumsum(self.news)]).astype(np.int32)
        self.T = int(self.cu[-1]) + spare_rows
        self.q = (q_scale * rng.standard_normal((self.T, hq, D))).astype(np.float16)
        self.max_len, self.max_new = int(self.lens.max(initial=0)), int(self.news.max(initial=0)) if max_new is None else max_new

    def gpu(self):
        g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        return dict(q=g(self.q), lambda_=g(self.lam), codebook_k=g(self.ck), codebook_v=g(self.cv), k_pool=g(self.k_pool),
                    v_pool=g(self.v_pool), page_table=g(self.table), seq_lens=g(self.lens), max_seq_len=self.max_len,
                    cu_new_lens=g(self.cu), max_new_len=self.max_new)

    def run(self, window=0, sinks=0, scale=0.0, expect=0, fill=None, **kw):
        """fp16 [T][Hq][D] through chunk_attention; fill: what out held before."""
        a = dict(self.gpu(), **kw)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((self.T, self.hq, D), 7.0 if fill is None else fill, dtype=torch.float16, device="cuda")
        vq.chunk_attention(self.layout, window=window, num_sinks=sinks, softmax_scale=scale, status=status, out=out, **a)
        torch.cuda.synchronize()
        assert int(status.item()) == expect
        return out.cpu().numpy()

    def tokens(self, b, h):
        """(k~, v) of sequence b, KV head h in 64 bits, and which tokens have a page."""
        n = int(self.lens[b])
        t = np.arange(n)
        pg = self.table[b][t // self.page] if n else np.zeros(0, np.int32)
        ok = (pg >= 0) & (pg < self.k_pool.shape[0])
        pg = np.where(ok, pg, 0)
        ks, kb, vs, vb = self.fmt
        kc = oracle.unpack(self.k_pool[pg, h, t % self.page][:, None], D // ks, kb)[:, 0]
        vc = oracle.unpack(self.v_pool[pg, h, t % self.page][:, None], D // vs, vb)[:, 0]
        return self.ck.astype(np.float64)[kc].reshape(n, D), self.cv.astype(np.float64)[vc].reshape(n, D), ok

    def exact(self, window=0, sinks=0, scale=0.0, seqs=None):
        """(out, tolerance) in 64 bits for the rows of the sequences (0 and 0 elsewhere)."""
        scale = scale or 1 / math.sqrt(D)
        out, tol = np.zeros((self.T, self.hq, D)), np.zeros((self.T, self.hq, D))
        G = self.hq // self.hkv
        for b in range(len(self.lens)) if seqs is None else seqs:
            n, length = int(self.news[b]), int(self.lens[b])
            if n == 0:
                continue
            r0 = int(self.cu[b])
            t = (length - n + np.arange(n))[:, None]
            p = np.arange(length)[None]
            for h in range(self.hkv):
                k, v, ok = self.tokens(b, h)
                see = (p <= t) & ok[None]
                if window:
                    see &= (p > t - window) | (p < sinks)
                for j in range(h * G, (h + 1) * G):
                    qt = (self.q[r0:r0 + n, j].astype(np.float64) * self.lam[h]) @ HADAMARD
                    s = np.where(see, qt @ k.T * scale, -np.inf)
                    S = np.where(see, np.abs(qt) @ np.abs(k).T * abs(scale), 0).max(1, initial=0)
                    m = s.max(1, initial=-np.inf)
                    w = np.exp(s - np.where(np.isfinite(m), m, 0)[:, None])
                    tot = w.sum(1, keepdims=True)
                    w = np.divide(w, tot, out=np.zeros_like(w), where=tot > 0)
                    o, A = w @ v, w @ np.abs(v)
                    sub = 2.0 ** -25 * np.where(see, 1.0, 0.0) @ np.abs(v)
                    out[r0:r0 + n, j] = o
                    tol[r0:r0 + n, j] = 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + (2.0 ** -11 + 2 * 2.0 ** -18 * S[:, None]) * A + \
                        sub / np.maximum(tot, 1)
        return out, tol

    def check(self, window=0, sinks=0, scale=0.0, expect=0, **kw):
        got = self.run(window, sinks, scale, expect, **kw)
        want, tol = self.exact(window, sinks, scale)
        R = int(self.cu[-1])
        off = np.abs(got[:R].astype(np.float64) - want[:R])
        assert (off <= tol[:R]).all(), f"off by {off.max():.3e}, {np.max(off / np.maximum(tol[:R], 1e-30)):.2f} of the tolerance"
        assert (got[R:] == 7.0).all()  # rows behind the last sequence stay as they were
        return got
