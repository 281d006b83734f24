"""Speculative decoding as its calls are used together: pages, appended keys and values, a tree's attention, the
accepted path kept, several steps on one cache, eager and as one captured graph."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402
from appendcase import AppendCase  # noqa: E402
from chunkcase import D, FORMATS  # noqa: E402
from treecase import TreeCase, tree, words  # noqa: E402

pytestmark = pytest.mark.gpu


class Drafting:
    """Buffers of a model of `layers` layers and `batch` sequences; a call is one step."""

    def __init__(self, fmt, hq, hkv, page, batch, width, layers, tokens, most, keep, window=0, sinks=0):
        self.a = AppendCase(fmt, hq, hkv, page, 1, dtype=torch.bfloat16, base=500000.0, scaling="parts", factor=4.0, seed=1)
        self.layout, self.hq, self.hkv, self.P, self.B, self.T, self.most = self.a.layout, hq, hkv, page, batch, tokens, most
        self.window, self.sinks, self.layers, self.max_len, self.pages = window, sinks, layers, width * page, batch * width
        i32 = dict(dtype=torch.int32, device="cuda")
        self.lam, self.ck, self.cv = (torch.from_numpy(x).cuda() for x in (self.a.lam, self.a.ck, self.a.cv))
        kr, vr = vq.row_bytes(self.layout)
        shape = (layers, self.pages, hkv, page)
        self.kp, self.vp = (torch.zeros(shape + (r,), dtype=torch.uint8, device="cuda") for r in (kr, vr))
        self.table = torch.full((batch, width), -1, **i32)
        self.lens, self.nf = torch.zeros(batch, **i32), torch.tensor([self.pages], **i32)
        self.free = torch.randperm(self.pages, generator=torch.Generator().manual_seed(5)).to(**i32)
        self.new, self.status = torch.zeros(batch, **i32), torch.zeros(1, **i32)
        self.depth = torch.zeros(tokens, **i32)  # of each drafted token in its tree
        self.masks = torch.zeros(tokens, -(-most // 64), dtype=torch.int64, device="cuda")
        self.keep, self.kept = torch.zeros(batch, keep, **i32), torch.zeros(batch, **i32)
        self.qkv = torch.zeros(layers, tokens, hq + 2 * hkv, D, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros(layers, tokens, hq, D, dtype=torch.float16, device="cuda")
        self.q = torch.zeros_like(self.out)
        self.ws = vq.alloc_tree_workspace(self.layout, batch, tokens, self.max_len, most)

    def attend(self):
        r = vq.append_slots(self.lens, self.new, self.table, self.free, self.nf, self.P, self.pages, self.T, seq_lens_out=self.lens,
                            num_free_out=self.nf, status=self.status)
        self.cu = r.cu_new_lens
        # a token's position is its sequence's length before the step and its depth
        first = torch.repeat_interleave(self.lens - self.new, self.new.long(), output_size=int(self.total)) if self.total else r.positions[:0]
        self.positions = r.positions.clone()
        self.positions[:self.total] = first + self.depth[:self.total]
        for i in range(self.layers):
            q, k, v = self.qkv[i].split([self.hq, self.hkv, self.hkv], dim=1)
            vq.append_kv(self.layout, self.a.config, self.positions, r.slot_mapping, k, v, self.lam, self.ck, self.cv, self.kp[i], self.vp[i],
                         q=q, q_out=self.q[i], status=self.status)
            vq.tree_attention(self.layout, self.q[i], self.lam, self.ck, self.cv, self.kp[i], self.vp[i], self.table, self.lens, self.max_len,
                              self.cu, self.most, self.masks, self.positions, self.window, self.sinks, out=self.out[i], workspace=self.ws,
                              status=self.status)

    def accept(self):
        vq.keep_tokens(self.layout, self.lens, self.cu, self.keep, self.kept, self.table, self.kp, self.vp, self.free, self.nf,
                       seq_lens_out=self.lens, num_free_out=self.nf, status=self.status)

    def load(self, news, trees, paths, seed):
        """One step's inputs."""
        self.total = sum(news)
        g = torch.Generator().manual_seed(seed)
        self.new.copy_(torch.tensor(news, dtype=torch.int32))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g).to(torch.bfloat16))
        self.out.fill_(7.0)
        self.q.fill_(5.0)
        if self.total:
            bits = np.concatenate([words(t, self.masks.shape[1]) for t in trees if len(t)])
            self.masks[:self.total] = torch.from_numpy(bits).cuda()
            self.depth[:self.total] = torch.from_numpy(np.concatenate([t.sum(1) - 1 for t in trees]).astype(np.int32)).cuda()
        for b, path in enumerate(paths):
            self.keep[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
            self.kept[b] = len(path)


def steps(batch, most, count, seed):
    """(drafted tokens, trees, accepted paths) of some steps."""
    rng = np.random.default_rng(seed)
    for _ in range(count):
        news = rng.integers(0, most + 1, batch).tolist()
        trees = [tree(n, rng) for n in news]
        paths = [np.flatnonzero(t[rng.integers(0, n)])[:6].tolist() if n else [] for n, t in zip(news, trees)]
        yield news, trees, paths


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[2], FORMATS[6]])
@pytest.mark.parametrize("most,window,sinks", [(7, 0, 0), (40, 0, 0), (40, 25, 3), (70, 0, 0)])
def test_steps_on_one_cache(fmt, most, window, sinks):
    """Each layer's outputs against the formula over what the cache holds; codes of kept tokens against those that were appended."""
    B, page, layers = 5, 16, 2
    s = Drafting(fmt, 8, 2, page, B, 16, layers, B * most, most, 6, window, sinks)
    held = [[] for _ in range(B)]  # (K rows, V rows) of the tokens that every sequence keeps, all layers
    for k, (news, trees, paths) in enumerate(steps(B, most, 6, most)):
        s.load(news, trees, paths, 100 + k)
        s.attend()
        torch.cuda.synchronize()
        assert s.status.item() == 0
        lens, table = s.lens.cpu().numpy(), s.table.cpu().numpy()
        assert lens.tolist() == [len(h) + n for h, n in zip(held, news)]
        kp, vp = s.kp.cpu().numpy(), s.vp.cpu().numpy()

        def row(b, t):
            return kp[:, table[b, t // page], :, t % page].copy(), vp[:, table[b, t // page], :, t % page].copy()

        for b, h in enumerate(held):
            for t, was in enumerate(h):
                now = row(b, t)
                assert np.array_equal(now[0], was[0]) and np.array_equal(now[1], was[1]), (b, t)
        for i in range(layers):
            c = TreeCase(fmt, 8, 2, page, lens, news, masks=trees, max_new=most)
            c.lam, c.ck, c.cv, c.table, c.k_pool, c.v_pool = s.a.lam, s.a.ck, s.a.cv, table, kp[i], vp[i]
            R = sum(news)
            c.q, c.positions = s.q[i].cpu().numpy(), s.positions.cpu().numpy()
            want, tol = c.exact(window, sinks)
            got = s.out[i].cpu().numpy()
            assert (np.abs(got[:R].astype(np.float64) - want[:R]) <= tol[:R]).all()
            assert (got[R:] == 7.0).all() and (s.q[i, R:] == 5.0).all()
        for b, path in enumerate(paths):
            held[b] += [row(b, int(lens[b]) - news[b] + j) for j in path]
        s.accept()
        torch.cuda.synchronize()
        assert s.status.item() == 0 and s.lens.tolist() == [len(h) for h in held]
        # every page is a sequence's or free, once
        used = [p for b, n in enumerate(s.lens.tolist()) for p in s.table[b, :-(-n // page)].tolist()]
        free = s.free[:s.nf.item()].tolist()
        assert sorted(used + free) == list(range(s.pages))


def test_a_captured_step_replayed():
    """Slots, append, attention and keep in one graph, over trees and lengths that change between replays."""
    B, page, most = 4, 16, 12
    make = lambda: Drafting(FORMATS[1], 8, 2, page, B, 12, 1, B * most, most, 6)  # noqa: E731
    work = list(steps(B, most, 5, 3))

    def step(s):  # (positions by depth alone, so that no host value is in it)
        r = vq.append_slots(s.lens, s.new, s.table, s.free, s.nf, s.P, s.pages, s.T, seq_lens_out=s.lens, num_free_out=s.nf, status=s.status)
        s.cu = r.cu_new_lens
        pos = torch.where(r.positions >= 0, s.depth, -1)
        q, k, v = s.qkv[0].split([8, 2, 2], dim=1)
        vq.append_kv(s.layout, s.a.config, pos, r.slot_mapping, k, v, s.lam, s.ck, s.cv, s.kp[0], s.vp[0], q=q, q_out=s.q[0], status=s.status)
        vq.tree_attention(s.layout, s.q[0], s.lam, s.ck, s.cv, s.kp[0], s.vp[0], s.table, s.lens, s.max_len, s.cu, s.most, s.masks, out=s.out[0],
                          workspace=s.ws, status=s.status)
        s.accept()

    warm = make()
    warm.load(*work[0], 1)
    step(warm)  # the library's first calls outside a capture
    eager, held = make(), make()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held)
    for k, w in enumerate(work):
        for s in (eager, held):
            s.load(*w, 50 + k)
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert eager.status.item() == 0 and held.status.item() == 0
        for name in ("lens", "nf", "table", "free", "out", "q", "kp", "vp"):
            assert torch.equal(getattr(eager, name), getattr(held, name)), (k, name)


def test_two_calls_at_once_with_workspaces_of_their_own():
    """Two streams' attention side by side, each with its workspace: the results of one after the other."""
    cases = [TreeCase(FORMATS[0], 8, 2, 64, [n + 5000, n + 900], [n, n], seed=n) for n in (6, 40)]
    args = [c.gpu() for c in cases]
    want = [vq.tree_attention(c.layout, **a) for c, a in zip(cases, args)]
    ws = [vq.alloc_tree_workspace(c.layout, 2, c.T, c.max_len, c.max_new) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got += [vq.tree_attention(c.layout, workspace=w, stream=s, **a) for c, a, w, s in zip(cases, args, ws, streams)]
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 2])
