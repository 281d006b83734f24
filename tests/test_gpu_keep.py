"""Keeping accepted drafted tokens: pools, lengths and free pages against a plain walk."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402

pytestmark = pytest.mark.gpu

FMTS = [(4, 8, 4, 8), (2, 8, 4, 9), (8, 12, 8, 12), (1, 3, 8, 11)]


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Keep:
    def __init__(self, fmt, hkv, page, layers, lens, news, most, seed=0, free=5, room=None):
        rng = np.random.default_rng(seed)
        self.layout = vq.make_layout(128, hkv, hkv, *fmt, page)
        self.page, self.lens, self.news = page, np.array(lens, np.int32), np.array(news, np.int32)
        need = -(-self.lens // page)
        self.pages = int(need.sum()) + 3
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(1, int(need.max(initial=0)) + 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(self.news)]).astype(np.int32)
        self.keep = rng.integers(-99, 99, (len(lens), most)).astype(np.int32)
        self.kept = np.zeros(len(lens), np.int32)
        for b, n in enumerate(news):
            self.kept[b] = rng.integers(0, min(n, most) + 1)
            self.keep[b, :self.kept[b]] = np.sort(rng.permutation(n)[:self.kept[b]])
        rows = vq.row_bytes(self.layout)
        self.pools = [rng.integers(0, 256, (layers, self.pages, hkv, page, r), dtype=np.uint8) for r in rows]
        self.free = np.full(room if room is not None else free + int(need.sum()) + 4, -3, np.int32)
        self.num_free = free

    def expected(self, bad=()):
        pools, lens, free, at = [x.copy() for x in self.pools], self.lens.copy(), self.free.copy(), self.num_free
        P = self.page
        for b in range(len(lens)):
            if b in bad:
                continue
            base, k = self.lens[b] - self.news[b], self.kept[b]
            for i in range(k):
                src, dst = base + self.keep[b, i], base + i
                for x in pools:
                    x[:, self.table[b, dst // P], :, dst % P] = x[:, self.table[b, src // P], :, src % P]
            lens[b] = base + k
            for page in range(-(-self.lens[b] // P) - 1, -(-lens[b] // P) - 1, -1):
                free[at] = self.table[b, page]
                at += 1
        return pools, lens, free, at

    def run(self, in_place=False, listed=False, expect=0, **kw):
        held = [gpu(x) for x in self.pools]
        pools = [list(x) for x in held] if listed else held
        lens, nf, status = gpu(self.lens), torch.tensor([self.num_free], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        free, table, rest = gpu(self.free), gpu(self.table), [gpu(x) for x in (self.cu, self.keep, self.kept)]
        if in_place:
            kw.update(seq_lens_out=lens, num_free_out=nf)
        torch.cuda.synchronize()
        r = vq.keep_tokens(self.layout, lens, *rest, table, *pools, free, nf, status=status, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == expect and np.array_equal(table.cpu().numpy(), self.table)
        return [x.cpu().numpy() for x in held], r.seq_lens.cpu().numpy(), free.cpu().numpy(), int(r.num_free.item())

    def check(self, bad=(), **kw):
        got, want = self.run(**kw), self.expected(bad)
        for x, y in zip(got[0], want[0]):
            assert np.array_equal(x, y)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2]) and got[3] == want[3]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [16, 48, 256])
@pytest.mark.parametrize("layers", [1, 3])
def test_formats(fmt, page, layers):
    rng = np.random.default_rng(page)
    news = rng.integers(0, 70, 9)
    Keep(fmt, 2, page, layers, news + rng.integers(0, 300, 9), news, 12, seed=layers).check()


@pytest.mark.parametrize("news,most", [([256, 256, 200], 256), ([1, 1, 1], 1), ([0, 0, 0], 4), ([64, 3, 64], 64)])
@pytest.mark.parametrize("in_place,listed", [(False, False), (True, True)])
def test_lengths(news, most, in_place, listed):
    for seed in range(4):
        Keep(FMTS[0], 3, 16, 2, np.array(news) + [0, 17, 33], news, most, seed=seed).check(in_place=in_place, listed=listed)


def test_all_and_none_of_them():
    c = Keep(FMTS[0], 2, 16, 2, [100, 60, 16], [40, 60, 16], 60)
    c.kept[:] = [40, 60, 16]
    for b, n in enumerate(c.kept):
        c.keep[b, :n] = np.arange(n)
    c.check()
    c.kept[:] = 0
    c.check()


def test_many_layers_and_sequences():
    rng = np.random.default_rng(3)
    news = rng.integers(1, 20, 300)
    Keep(FMTS[1], 2, 16, 5, news + rng.integers(0, 40, 300), news, 7, seed=4).check(in_place=True)
    Keep(FMTS[0], 1, 16, 128, [30, 41], [14, 9], 9, seed=5).check()
    news = rng.integers(0, 4, 3001)
    Keep(FMTS[0], 1, 16, 1, news + rng.integers(0, 30, 3001), news, 3, seed=6).check(in_place=True)


def test_sequences_out_of_range_stay_as_they_are():
    def case():
        c = Keep(FMTS[0], 2, 16, 2, [90, 90, 90, 90, 90, 90], [40] * 6, 8, seed=7)
        c.kept[:] = 5
        c.keep[:, :5] = [0, 3, 9, 20, 39]
        return c

    for at, what in ((1, [0, 3, 3, 20, 39]), (2, [5, 3, 9, 20, 39]), (3, [0, 3, 9, 20, 40]), (4, [-1, 3, 9, 20, 39])):
        c = case()
        c.keep[at, :5] = what
        c.check(bad=(at,), expect=vq.VQ_DEV_BAD_LENGTH, in_place=True)
    c = case()
    c.kept[[0, 5]] = [-1, 9]
    c.check(bad=(0, 5), expect=vq.VQ_DEV_BAD_LENGTH)
    c = case()
    c.cu[2:] += 60  # the second sequence with more drafted tokens than tokens
    c.check(bad=(1,), expect=vq.VQ_DEV_BAD_LENGTH)
    c = case()
    c.table[2, 4] = c.pages
    c.check(bad=(2,), expect=vq.VQ_DEV_BAD_PAGE)
    c = case()
    c.table[2, 0] = -1  # a page of the context is none of its business
    c.check()


@pytest.mark.parametrize("free,room", [(5, 6), (-1, 40), (41, 40)])
def test_pages_that_do_not_fit_are_not_given_back(free, room):
    c = Keep(FMTS[0], 2, 16, 1, [90, 90], [60, 60], 3, free=free, room=room)
    roomy = object.__new__(Keep)
    roomy.__dict__.update(c.__dict__, free=np.zeros(100, np.int32), num_free=0)
    pools, lens, _, _ = roomy.expected()
    got = c.run(expect=vq.VQ_DEV_BAD_LENGTH)
    assert all(np.array_equal(x, y) for x, y in zip(got[0], pools)) and np.array_equal(got[1], lens)
    assert np.array_equal(got[2], c.free) and got[3] == free


def test_streams_and_graphs():
    c = Keep(FMTS[0], 2, 16, 2, [90, 77], [40, 33], 8, seed=8)
    c.check(stream=torch.cuda.Stream())
    d = Keep(FMTS[0], 2, 16, 2, [90, 77], [40, 33], 8, seed=9)
    pools, lens, cu, keep, kept, table, free = [gpu(x) for x in c.pools], gpu(c.lens), gpu(c.cu), gpu(c.keep), gpu(c.kept), gpu(c.table), gpu(c.free)
    nf = torch.tensor([5], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = vq.keep_tokens(c.layout, lens, cu, keep, kept, table, *pools, free, nf, seq_lens_out=lens, num_free_out=nf)
    for x, y in zip((*pools, keep, kept, table, free), (*d.pools, d.keep, d.kept, d.table, d.free)):
        x.copy_(torch.from_numpy(y))
    graph.replay()
    torch.cuda.synchronize()
    want = d.expected()
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(pools, want[0]))
    assert np.array_equal(r.seq_lens.cpu().numpy(), want[1]) and np.array_equal(free.cpu().numpy(), want[2]) and int(nf.item()) == want[3]
