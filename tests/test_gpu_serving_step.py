"""The serving step as one captured graph, replayed over changing lengths, and chunk attention's less usual shapes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402
from chunkcase import FORMATS, Case  # noqa: E402

pytestmark = pytest.mark.gpu


class Step:
    """append_slots, rotary, encode_kv and chunk_attention over buffers of their own, in place."""

    def __init__(self, case, hq, hkv, page, batch, width, pages, tokens, most, window, sinks):
        self.c, self.hq, self.hkv, self.P, self.pages, self.T, self.most = case, hq, hkv, page, pages, tokens, most
        self.window, self.sinks, self.max_len = window, sinks, width * page
        i32 = dict(dtype=torch.int32, device="cuda")
        self.lam, self.ck, self.cv = (torch.from_numpy(x).cuda() for x in (case.lam, case.ck, case.cv))
        self.kp, self.vp = vq.alloc_pools(case.layout, pages)
        self.table = torch.full((batch, width), -1, **i32)
        self.lens, self.nf = torch.zeros(batch, **i32), torch.tensor([pages], **i32)
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).to(**i32)
        self.new, self.status = torch.zeros(batch, **i32), torch.zeros(1, **i32)
        self.qkv = torch.zeros(tokens, hq + 2 * hkv, 128, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros(tokens, hq, 128, dtype=torch.float16, device="cuda")
        self.cfg = vq.make_rotary(base=500000.0, scaling="parts", factor=4.0)
        self.ws = vq.alloc_chunk_workspace(case.layout, batch, tokens, self.max_len, most)

    def __call__(self):
        r = vq.append_slots(self.lens, self.new, self.table, self.free, self.nf, self.P, self.pages, self.T,
                            seq_lens_out=self.lens, num_free_out=self.nf, status=self.status)
        self.q, k, v = vq.rotary(self.cfg, r.positions, *self.qkv.split([self.hq, self.hkv, self.hkv], dim=1))
        vq.encode_kv(self.c.layout, k, v, r.slot_mapping, self.lam, self.ck, self.cv, self.kp, self.vp, status=self.status)
        vq.chunk_attention(self.c.layout, self.q, self.lam, self.ck, self.cv, self.kp, self.vp, self.table, self.lens, self.max_len,
                           r.cu_new_lens, self.most, window=self.window, num_sinks=self.sinks, out=self.out,
                           workspace=self.ws, status=self.status)
        self.cu = r.cu_new_lens


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("most,news", [(2, ([1, 0, 2, 1], [2, 1, 1, 0], [0, 0, 0, 0], [1, 1, 1, 1], [2, 2, 2, 2])),
                                       (70, ([70, 0, 1, 33], [1, 70, 1, 0], [1, 1, 69, 1], [0, 0, 0, 0], [70, 1, 1, 70]))])
def test_a_captured_step_replayed_over_changing_lengths(most, news, window, sinks):
    hq, hkv, P, B, width, pages = 8, 2, 16, 4, 16, 64
    c = Case(FORMATS[0], hq, hkv, P, [0], [0], seed=13)
    T = max(sum(n) for n in news) + 3
    make = lambda: Step(c, hq, hkv, P, B, width, pages, T, most, window, sinks)  # noqa: E731
    make()()  # the library's first calls outside a capture
    torch.cuda.synchronize()
    eager, step = make(), make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(6)
    for new in news:
        x = torch.randn(T, hq + 2 * hkv, 128, generator=g).to(torch.bfloat16)
        for s in (eager, step):
            s.new.copy_(torch.tensor(new, dtype=torch.int32))
            s.qkv.copy_(x)
            s.out.fill_(7.0)
        eager()
        graph.replay()
        torch.cuda.synchronize()
        assert step.status.item() == 0 and eager.status.item() == 0
        for name in ("lens", "nf", "table", "out"):
            assert torch.equal(getattr(step, name), getattr(eager, name)), name
        for b, n in enumerate(step.lens.tolist()):  # (the pools' other rows were never written)
            t = torch.arange(n, device="cuda")
            pg = step.table[b, t // P].long()
            for name in ("kp", "vp"):
                assert torch.equal(getattr(step, name)[pg, :, t % P], getattr(eager, name)[pg, :, t % P]), name
        R = sum(new)
        assert (step.out[R:] == 7.0).all()
        c.table, c.k_pool, c.v_pool = step.table.cpu().numpy(), step.kp.cpu().numpy(), step.vp.cpu().numpy()
        c.lens, c.news, c.cu, c.T = step.lens.cpu().numpy(), np.array(new), step.cu.cpu().numpy(), T
        c.q = step.q.cpu().numpy()
        want, tol = c.exact(window, sinks)
        assert (np.abs(step.out.cpu().numpy().astype(np.float64) - want)[:R] <= tol[:R]).all()


@pytest.mark.parametrize("heads", [(3, 1), (6, 2), (6, 1), (7, 1)])
@pytest.mark.parametrize("n", [1, 2, 5, 19, 43, 130])
def test_head_groups_that_do_not_divide_a_tile(heads, n):
    c = Case(FORMATS[1], *heads, 48, [n, n + 77, 1500], [n, max(n // 2, 1), n], seed=n)
    c.check()
    c.check(200, 20)


@pytest.mark.parametrize("page", [112, 144, 240, 272, 400])
@pytest.mark.parametrize("n", [1, 3, 30, 90])
def test_pages_that_are_no_power_of_two(page, n):
    c = Case(FORMATS[2], 4, 1, page, [n + 2, 1000, 399], [n, n, n], seed=page)
    c.check()
    c.check(150, 130)
