"""Page tables, slot maps, positions and row offsets (append_slots) against a plain loop."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402

pytestmark = pytest.mark.gpu


def plain(lens, new, table, free, num_free, P, num_pages, max_tokens):
    """(status, outputs) of one step, sequence by sequence and token by token."""
    B, mp = table.shape
    refused = dict(table=table.copy(), lens=lens.copy(), num_free=num_free, cu=np.zeros(B + 1, np.int64),
                   slots=np.full(max_tokens, -1), pos=np.full(max_tokens, -1))
    ends = lens.astype(np.int64) + new
    if (lens < 0).any() or (new < 0).any() or (ends > mp * P).any() or not 0 <= num_free <= len(free):
        return vq.VQ_DEV_BAD_LENGTH, refused
    if new.sum() > max_tokens:
        return vq.VQ_DEV_BAD_LENGTH, refused
    out, top = table.copy(), num_free
    if sum(-(-int(e) // P) - -(-int(x) // P) for e, x in zip(ends, lens)) > num_free:
        return vq.VQ_DEV_NO_PAGES, refused
    slots, pos = [], []
    for b in range(B):
        for lp in range(-(-int(lens[b]) // P), -(-int(ends[b]) // P)):
            top -= 1
            out[b, lp] = free[top]
        for t in range(int(lens[b]), int(ends[b])):
            if not 0 <= out[b, t // P] < num_pages:
                return vq.VQ_DEV_BAD_PAGE, refused
            slots.append(int(out[b, t // P]) * P + t % P)
            pos.append(t)
    pad = [-1] * (max_tokens - len(slots))
    return vq.VQ_DEV_OK, dict(table=out, lens=ends, num_free=top, cu=np.concatenate([[0], np.cumsum(new)]),
                              slots=np.array(slots + pad, np.int64), pos=np.array(pos + pad, np.int64))


def call(lens, new, table, free, num_free, P, num_pages, max_tokens, in_place=False, stream=None):
    g = lambda x, d=torch.int32: torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=d)  # noqa: E731
    t, sl, nf = g(table), g(lens), g(np.array([num_free]))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(seq_lens_out=sl, num_free_out=nf) if in_place else {}
    args = (g(new), t, g(free), nf)
    torch.cuda.synchronize()
    r = vq.append_slots(sl, *args, P, num_pages, max_tokens, status=status, stream=stream, **kw)
    torch.cuda.synchronize()
    return int(status.item()), dict(table=t.cpu().numpy(), lens=r.seq_lens.cpu().numpy(),
                                    num_free=int(r.num_free.item()), cu=r.cu_new_lens.cpu().numpy(),
                                    slots=r.slot_mapping.cpu().numpy(), pos=r.positions.cpu().numpy())


def make(B, P, lens, new, spare=3, room=0, seed=0):
    """A consistent state: every sequence owns the pages of its cached tokens."""
    rng = np.random.default_rng(seed)
    lens, new = np.array(lens, np.int32), np.array(new, np.int32)
    have = -(-lens // P)
    need = -(-(lens.astype(np.int64) + new) // P)
    total = int(need.sum()) + spare
    pages = rng.permutation(total).astype(np.int32)
    table = np.full((B, max(1, int(need.max(initial=0))) + room), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = pages[at:at + have[b]]
        at += have[b]
    return lens, new, table, pages[at:].copy(), len(pages) - at, P, total


def same(got, want):
    for k in want:
        assert np.array_equal(got[k], want[k]), k


CASES = [
    (1, 16, [0], [1]), (1, 16, [0], [0]), (1, 16, [15], [1]), (1, 16, [16], [1]), (1, 16, [0], [16]),
    (1, 48, [47], [50]), (3, 64, [5, 0, 64], [0, 130, 0]), (5, 256, [255, 256, 257, 0, 1], [1, 1, 1, 1, 255]),
    (2, 16, [0, 0], [2500, 1]), (1, 16, [7], [20000]),
]


@pytest.mark.parametrize("B,P,lens,new", CASES)
@pytest.mark.parametrize("pad", [0, 1, 5])
def test_small(B, P, lens, new, pad):
    a = make(B, P, lens, new, room=pad)
    st, want = plain(*a, int(sum(new)) + pad)
    assert st == vq.VQ_DEV_OK
    got_st, got = call(*a, int(sum(new)) + pad, in_place=pad == 1)
    assert got_st == st
    same(got, want)


@pytest.mark.parametrize("B,P,hi,n", [(300, 64, 3000, 1), (513, 16, 100, 40), (1024, 48, 50, 3), (16384, 16, 40, 2),
                                      (40, 256, 9000, 3000)])
def test_batches(B, P, hi, n):
    rng = np.random.default_rng(B)
    a = make(B, P, rng.integers(0, hi, B), rng.integers(0, n + 1, B), seed=B)
    T = int(a[1].sum()) + 3
    st, want = plain(*a, T)
    for in_place in (False, True):
        got_st, got = call(*a, T, in_place=in_place)
        assert got_st == st == vq.VQ_DEV_OK
        same(got, want)


def test_no_sequences():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    free = torch.arange(4, dtype=torch.int32, device="cuda")
    r = vq.append_slots(e, e, torch.empty((0, 3), dtype=torch.int32, device="cuda"), free,
                        torch.tensor([4], dtype=torch.int32, device="cuda"), 16, 4, 7, status=status)
    assert r.cu_new_lens.tolist() == [0] and r.num_free.tolist() == [4]
    assert r.slot_mapping.tolist() == [-1] * 7 and r.positions.tolist() == [-1] * 7 and status.item() == 0


@pytest.mark.parametrize("what", ["few pages", "tokens", "negative length", "negative new", "table full", "num_free",
                                  "free page", "old page"])
@pytest.mark.parametrize("in_place", [False, True])
def test_refused_steps_change_nothing(what, in_place):
    lens, new, table, free, nf, P, pages = make(4, 16, [20, 0, 33, 16], [40, 17, 0, 1], spare=0)
    T = int(new.sum())
    if what == "few pages":
        nf -= 1
    elif what == "tokens":
        T -= 1
    elif what == "negative length":
        lens[2] = -1
    elif what == "negative new":
        new[2] = -5
    elif what == "table full":
        new[3] = 16 * table.shape[1]
        T = 1000
    elif what == "num_free":
        nf = len(free) + 1
    elif what == "free page":
        free[1] = pages
    elif what == "old page":
        table[0, 1] = -1
    st, want = plain(lens, new, table, free, nf, P, pages, T)
    assert st != vq.VQ_DEV_OK
    got_st, got = call(lens, new, table, free, nf, P, pages, T, in_place=in_place)
    assert got_st == st
    same(got, want)


@pytest.mark.parametrize("faults", [("page", "length"), ("page", "tokens"), ("page", "few"), ("page", "few", "length"),
                                    ("few", "num_free")])
def test_of_several_faults_the_same_is_reported(faults):
    """The old page's fault is met first, by the thread that meets the others too (two sequences per thread)."""
    B, P = 1024, 16
    lens, new, table, free, nf, P, pages = make(B, P, [5] * B, [20] * B, spare=0)
    T = int(new.sum())
    for f in faults:
        if f == "page":
            table[0, 0] = pages
        elif f == "length":
            lens[1] = -1
        elif f == "tokens":
            T -= 1
        elif f == "few":
            nf -= 1
        elif f == "num_free":
            nf = len(free) + 1
    st, want = plain(lens, new, table, free, nf, P, pages, T)
    for _ in range(5):
        got_st, got = call(lens, new, table, free, nf, P, pages, T)
        assert got_st == st
        same(got, want)


def test_sums_past_32_bits_are_refused():
    B = 8
    lens, new = np.zeros(B, np.int32), np.full(B, (1 << 31) - 1, np.int32)
    table = np.full((B, 1 << 10), -1, np.int32)
    got_st, got = call(lens, new, table, np.arange(4, dtype=np.int32), 4, 1 << 21, 4, 8)
    assert got_st == vq.VQ_DEV_BAD_LENGTH
    assert got["num_free"] == 4 and (got["slots"] == -1).all() and (got["cu"] == 0).all() and (got["table"] == -1).all()


def test_slots_past_32_bits():
    """Page numbers whose slots do not fit 32 bits."""
    P, pages = 1 << 16, 1 << 20
    free = np.array([7, pages - 1], np.int32)
    lens, new, table = np.array([0], np.int32), np.array([5], np.int32), np.full((1, 2), -1, np.int32)
    st, got = call(lens, new, table, free, 2, P, pages, 5)
    assert st == 0 and got["slots"].tolist() == [(pages - 1) * P + i for i in range(5)]


def test_replayed_steps():
    """Two graphs of in-place steps, replayed in turn: lengths and free pages carry over."""
    P, B, steps = 16, 5, 40
    free = torch.randperm(200, generator=torch.Generator().manual_seed(1)).to(device="cuda", dtype=torch.int32)
    state = []
    for n in ([1, 0, 3, 1, 2], [0, 7, 1, 1, 0]):
        state.append(torch.tensor(n, dtype=torch.int32, device="cuda"))
    table = torch.full((B, 40), -1, dtype=torch.int32, device="cuda")
    lens, nf = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.tensor([200], dtype=torch.int32, device="cuda")
    outs, graphs = [], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for n in state:  # the library's first call outside a capture
            vq.append_slots(lens.clone(), n, table.clone(), free, nf, P, 200, 10)
    torch.cuda.synchronize()
    for n in state:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(vq.append_slots(lens, n, table, free, nf, P, 200, 10, seq_lens_out=lens, num_free_out=nf))
        graphs.append(g)
    h = (np.zeros(B, np.int32), np.full((B, 40), -1, np.int32), 200)
    for i in range(steps):
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        st, want = plain(h[0], state[i % 2].cpu().numpy(), h[1], free.cpu().numpy(), h[2], P, 200, 10)
        assert st == 0
        assert np.array_equal(lens.cpu().numpy(), want["lens"]) and int(nf.item()) == want["num_free"]
        assert np.array_equal(table.cpu().numpy(), want["table"])
        assert np.array_equal(outs[i % 2].slot_mapping.cpu().numpy(), want["slots"])
        h = (want["lens"].astype(np.int32), want["table"], want["num_free"])


def test_another_stream():
    a = make(3, 64, [5, 0, 64], [0, 130, 0])
    st, want = plain(*a, 140)
    got_st, got = call(*a, 140, stream=torch.cuda.Stream())
    assert got_st == st
    same(got, want)
