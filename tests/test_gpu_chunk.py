"""Chunk attention over the paged codes, with and without window and sinks, against its formula in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402
from chunkcase import FORMATS, Case  # noqa: E402

pytestmark = pytest.mark.gpu

WINDOWS = [(0, 0), (1, 0), (7, 3), (16, 0), (100, 4), (129, 65), (1 << 30, 5)]
HEADS = [(2, 2), (4, 2), (8, 2), (5, 1), (8, 1)]  # 1, 2, 4, 5 and 8 query heads per KV head


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 2, 9, 70, 300])
def test_formats(fmt, n):
    Case(fmt, 8, 2, 64, [400, 311], [n, n // 2], seed=n).check()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 2, 3, 17, 64, 130])
def test_heads(heads, n):
    Case(FORMATS[0], *heads, 16, [n, n + 5, n + 200], [n, n, n], seed=n).check()


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("n", [1, 5, 33, 150])
@pytest.mark.parametrize("heads", [(8, 2), (5, 1)])
def test_windows(window, sinks, n, heads):
    c = Case(FORMATS[1], *heads, 48, [n, n + 1, n + 15, n + 333, 2000], [n] * 5, seed=n)
    c.check(window, sinks)


@pytest.mark.parametrize("length", [0, 1, 2, 15, 16, 17, 31, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("n", [1, 16, 129])
def test_short_sequences_and_rows_before_the_first_token(length, n):
    """More new rows than tokens: rows before token 0 see nothing and are zero."""
    got = Case(FORMATS[0], 8, 2, 16, [length, 40], [n, 1], seed=length).check(5 if length % 2 else 0, 2 if length % 2 else 0)
    if n > length:
        assert (got[:n - length] == 0).all()


@pytest.mark.parametrize("n", [1, 40])
def test_ragged_batch_with_idle_sequences(n):
    rng = np.random.default_rng(n)
    news = rng.integers(0, n + 1, 37)
    news[[0, 5, 6, 36]] = 0
    lens = news + rng.integers(0, 900, 37)
    Case(FORMATS[2], 5, 1, 64, lens, news, seed=n, spare_rows=7).check()
    Case(FORMATS[2], 5, 1, 64, lens, news, seed=n, spare_rows=7).check(200, 20)


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[2], FORMATS[6]])
@pytest.mark.parametrize("n", [1, 4, 33])
@pytest.mark.parametrize("window,sinks", [(0, 0), (4096, 4)])
def test_long_context_over_many_ctas(fmt, n, window, sinks):
    Case(fmt, 4, 1, 256, [30011], [n], seed=n).check(window, sinks)


def test_chunk_of_a_long_prompt():
    Case(FORMATS[0], 4, 1, 256, [2500, 700], [600, 700], seed=3).check()
    Case(FORMATS[0], 4, 1, 256, [2500, 700], [600, 700], seed=3).check(300, 33)


@pytest.mark.parametrize("n", [1, 2, 4, 20, 50])
def test_pools_past_32_bits(n):
    """The same codes on the last pages of pools of more than 2^32 bytes: the same bits."""
    c = Case(FORMATS[0], 8, 2, 64, [700, 130], [n, n], seed=11)
    want = c.check()
    pages = (1 << 32) // (c.hkv * c.page * c.k_pool.shape[3]) + 1000
    at = pages - c.k_pool.shape[0]
    pools = {}
    for name, small in (("k_pool", c.k_pool), ("v_pool", c.v_pool)):
        big = torch.empty((pages,) + small.shape[1:], dtype=torch.uint8, device="cuda")
        big[at:] = torch.from_numpy(small).cuda()
        assert big[:at].numel() > 1 << 32
        pools[name] = big
    table = torch.from_numpy(np.where(c.table >= 0, c.table + at, -1).astype(np.int32)).cuda()
    assert np.array_equal(c.run(page_table=table, **pools), want)


@pytest.mark.parametrize("n", [1, 2, 4, 20, 50])
def test_the_largest_batch(n):
    rng = np.random.default_rng(n)
    news = np.where(rng.random(1024) < 0.5, 0, rng.integers(1, n + 1, 1024))
    news[[0, 1023]] = n
    Case(FORMATS[0], 4, 1, 16, news + rng.integers(0, 60, 1024), news, seed=n).check()


@pytest.mark.parametrize("n", [1, 100])
def test_large_scores_and_scale(n):
    Case(FORMATS[0], 8, 2, 64, [500, 100], [n, n], seed=5, q_scale=6.0).check()
    Case(FORMATS[0], 8, 2, 64, [500, 100], [n, n], seed=5).check(scale=0.5)
    Case(FORMATS[0], 8, 2, 64, [500, 100], [n, n], seed=5).check(scale=-0.03)


@pytest.mark.parametrize("n", [1, 3, 90])
def test_pages_out_of_range_are_not_seen(n):
    c = Case(FORMATS[0], 8, 2, 16, [100, 160, 20], [n if n < 100 else 90, n, min(n, 20)], seed=1)
    c.table[0, 3] = -1
    c.table[1, 0] = c.k_pool.shape[0]
    c.table[2, :] = -7
    got = c.check(expect=vq.VQ_DEV_BAD_PAGE)
    assert (got[c.cu[2]:c.cu[3]] == 0).all()


@pytest.mark.parametrize("n", [1, 80])
def test_sequences_outside_their_bounds_are_left_out(n):
    c = Case(FORMATS[0], 8, 2, 64, [200, 210, 220, 230], [n, n, n, n], seed=2)
    want = c.run()
    for what in ("length", "negative", "rows"):
        d = c.gpu()
        bad = 1
        if what == "length":
            d["seq_lens"][1] = c.max_len + 1
        elif what == "negative":
            d["seq_lens"][1] = -1
        else:
            bad = 3
            d["cu_new_lens"][4] = c.T + 1
        got = c.run(expect=vq.VQ_DEV_BAD_LENGTH, seq_lens=d["seq_lens"], cu_new_lens=d["cu_new_lens"], max_new_len=n + 1)
        keep = np.arange(c.T) // n != bad
        tol = c.exact()[1]
        assert (got[~keep] == 7.0).all()
        assert (np.abs(got[keep].astype(np.float64) - want[keep]) <= 2 * tol[keep]).all()


@pytest.mark.parametrize("n", [1, 4, 60])
def test_a_row_of_nan_or_infinity_stays_alone(n):
    c = Case(FORMATS[0], 8, 2, 64, [300, 310], [n, n], seed=4)
    want = c.run()
    c.q[0, 3, 5] = np.nan
    c.q[-1, 0, 100] = np.inf
    got = c.run()
    touched = np.zeros((c.T, c.hq), bool)
    touched[0, 3] = touched[-1, 0] = True
    assert np.isnan(got[touched]).all()
    assert np.array_equal(got[~touched], want[~touched])


def test_one_row_per_sequence_without_offsets_and_decode_attention():
    c = Case(FORMATS[1], 8, 2, 64, [1000, 1, 77, 0], [1, 1, 1, 1], seed=6)
    got = c.check()
    assert np.array_equal(c.run(cu_new_lens=None), got)
    a = c.gpu()
    dec = vq.decode_attention(c.layout, a["q"], a["lambda_"], a["codebook_k"], a["codebook_v"], a["k_pool"], a["v_pool"],
                              a["page_table"], a["seq_lens"], c.max_len).cpu().numpy().astype(np.float64)
    want, tol = c.exact()
    assert (np.abs(dec - want) <= tol).all() and (np.abs(dec - got) <= 2 * tol).all()


@pytest.mark.parametrize("n,window", [(1, 0), (5, 300), (200, 0)])
def test_same_bits_again_and_in_a_larger_workspace(n, window):
    c = Case(FORMATS[0], 8, 2, 64, [5000, 900, 40], [n, n, min(n, 40)], seed=8)
    first = c.run(window, 0)
    big = vq.alloc_chunk_workspace(c.layout, 64, 100000, 1 << 20, 4096)
    big.fill_(0xff)  # (NaN partials)
    for _ in range(3):
        assert np.array_equal(first, c.run(window, 0, workspace=big))


@pytest.mark.parametrize("n", [1, 48])
def test_replayed_graph_follows_lengths_and_two_streams(n):
    c = Case(FORMATS[0], 8, 2, 64, [600, 900], [n, n], seed=9)
    a = c.gpu()
    ws = [vq.alloc_chunk_workspace(c.layout, 2, c.T, 900, n) for _ in range(2)]
    vq.chunk_attention(c.layout, workspace=ws[0], **a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = vq.chunk_attention(c.layout, workspace=ws[0], **a)
    for lens in ([600, 900], [n, 500], [333, n + 1]):
        c.lens[:] = lens
        a["seq_lens"].copy_(torch.from_numpy(c.lens))
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        graph.replay()
        other = vq.chunk_attention(c.layout, workspace=ws[1], stream=s, **a)
        torch.cuda.synchronize()
        want, tol = c.exact()
        for x in (out, other):
            assert (np.abs(x.cpu().numpy().astype(np.float64) - want) <= tol).all()


def test_a_serving_step_end_to_end():
    """append_slots, rotary, encode_kv and chunk_attention together, three steps of a mixed batch,
    against dequantised keys and a plain softmax in 64 bits."""
    from test_gpu_rotary import frequencies, plain as turned
    fmt, hq, hkv, P, B, pages = (4, 8, 4, 8), 8, 2, 16, 3, 64
    c = Case(fmt, hq, hkv, P, [0], [0], seed=11)  # codebooks, lambda, layout
    g = torch.Generator().manual_seed(4)
    dev = lambda x, d=None: torch.as_tensor(x, dtype=d).cuda()  # noqa: E731
    lam, ck, cv = dev(c.lam), dev(c.ck), dev(c.cv)
    kp, vp = vq.alloc_pools(c.layout, pages)
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    lens, nf = torch.zeros(B, dtype=torch.int32, device="cuda"), dev([pages], torch.int32)
    free = dev(torch.randperm(pages, generator=g).to(torch.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cfg = vq.make_rotary(base=500000.0)
    f = frequencies(128, 500000.0, "none", 1, 1, 1, 2)
    for step, new in enumerate(([40, 0, 7], [1, 33, 1], [1, 1, 19])):
        T = sum(new) + 3
        qkv = torch.randn(T, hq + 2 * hkv, 128, generator=g).to(torch.bfloat16).cuda()
        r = vq.append_slots(lens, dev(new, torch.int32), table, free, nf, P, pages, T, seq_lens_out=lens, num_free_out=nf, status=status)
        q, k, v = vq.rotary(cfg, r.positions, *qkv.split([hq, hkv, hkv], dim=1))
        vq.encode_kv(c.layout, k, v, r.slot_mapping, lam, ck, cv, kp, vp, status=status)
        out = vq.chunk_attention(c.layout, q, lam, ck, cv, kp, vp, table, lens, 12 * P, r.cu_new_lens, max(new), status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        c.table, c.k_pool, c.v_pool = table.cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy()
        c.lens, c.news, c.cu, c.T = lens.cpu().numpy(), np.array(new), r.cu_new_lens.cpu().numpy(), T
        c.q = q.cpu().numpy()
        pos = r.positions.cpu().numpy()
        y, tol = turned(qkv[:, :hq].float().cpu().numpy(), pos, f, 128, False, 1.0)
        live = pos >= 0
        assert (np.abs(c.q.astype(np.float64) - y)[live] <= tol[live]).all()
        want, tol = c.exact()
        assert (np.abs(out.cpu().numpy().astype(np.float64) - want)[live] <= tol[live]).all()
        # the codes of the new tokens are those of the turned keys: nearest centroids of every sub-vector
        x = k.cpu().numpy().astype(np.float64)[live]
        for h in range(hkv):
            from chunkcase import HADAMARD
            xt = (x[:, h] / c.lam[h]) @ HADAMARD
            d2 = ((xt.reshape(len(xt), -1, 1, 4) - c.ck.astype(np.float64)) ** 2).sum(-1)
            rows = []
            for b in range(B):
                n, L = new[b], int(c.lens[b])
                for t in range(L - n, L):
                    rows.append(c.k_pool[c.table[b, t // P], h, t % P])
            got = np.take_along_axis(d2, np.array(rows).astype(np.int64)[:, :, None], 2)[:, :, 0]
            assert (got <= d2.min(2) * (1 + 1e-4) + 1e-5).all()
