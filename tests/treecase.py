"""Cases of the tree-attention tests: chunkcase's batches with masks, and the formula in 64 bits (not a test
module).  Tolerances are chunkcase's: the kernels round in the same places (scores of high and low
fp16 parts of q~, p to fp16 once, the output once)."""
import math

import numpy as np
import torch

import bit_vector_quantized_gb300 as vq
from chunkcase import D, HADAMARD, Case


def tree(n, rng):
    """bool [n][n]: ancestors of each token of a random tree, itself among them."""
    a = np.eye(n, dtype=bool)
    for i in range(1, n):
        a[i] |= a[rng.integers(0, i)]
    return a


def words(bits, count):
    """int64 [n][count] of bool [n][m]."""
    out = np.zeros((bits.shape[0], 64 * count), bool)
    out[:, :bits.shape[1]] = bits
    return np.packbits(out, axis=1, bitorder="little").view(np.int64)


class TreeCase(Case):
    """masks: bool [n][n] of each sequence (random trees where not given); junk: bits past the sequence's tokens are set."""

    def __init__(self, *args, masks=None, mask_words=None, junk=False, **kw):
        super().__init__(*args, **kw)
        rng = np.random.default_rng(self.T + 1)
        self.see = masks if masks is not None else [tree(int(n), rng) for n in self.news]
        self.words = mask_words or max(1, -(-self.max_new // 64))
        m = np.zeros((self.T, self.words), np.int64)
        self.positions = np.zeros(self.T, np.int32)
        for b, a in enumerate(self.see):
            n, r0 = len(a), int(self.cu[b])
            bits = np.zeros((n, max(64 * self.words, n)), bool)
            bits[:, :n] = a
            if junk:
                bits[:, n:] = True
            m[r0:r0 + n] = words(bits[:, :64 * self.words], self.words)
            self.positions[r0:r0 + n] = self.lens[b] - n + np.maximum(a.sum(1) - 1, 0)
        self.masks = m

    def gpu(self):
        g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        return dict(super().gpu(), tree_masks=g(self.masks), positions=g(self.positions))

    def run(self, window=0, sinks=0, scale=0.0, expect=0, fill=None, **kw):
        a = dict(self.gpu(), **kw)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((self.T, self.hq, D), 7.0 if fill is None else fill, dtype=torch.float16, device="cuda")
        vq.tree_attention(self.layout, window=window, num_sinks=sinks, softmax_scale=scale, status=status, out=out, **a)
        torch.cuda.synchronize()
        assert int(status.item()) == expect
        return out.cpu().numpy()

    def exact(self, window=0, sinks=0, scale=0.0, seqs=None):
        scale = scale or 1 / math.sqrt(D)
        out, tol = np.zeros((self.T, self.hq, D)), np.zeros((self.T, self.hq, D))
        G = self.hq // self.hkv
        for b in range(len(self.lens)) if seqs is None else seqs:
            n, length = int(self.news[b]), int(self.lens[b])
            if n == 0:
                continue
            r0, base = int(self.cu[b]), length - n
            t = np.maximum(self.positions[r0:r0 + n].astype(np.int64), base)
            at = np.concatenate([np.arange(base), t])
            for h in range(self.hkv):
                k, v, ok = self.tokens(b, h)
                see = np.concatenate([np.ones((n, base), bool), self.see[b]], 1) & ok[None]
                if window:
                    see &= (at[None] > t[:, None] - window) | (at[None] < sinks)
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
