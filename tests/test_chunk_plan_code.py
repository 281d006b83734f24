"""The plan of chunk attention as the kernels have it (CPU): csrc/vq_chunk_plan.cuh compiled for the host, its
pieces against the definition, up to lengths of 2^30, batches of 1024 and sums past 32 bits."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from bit_vector_quantized_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    try:
        nvcc = build._nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    lib = str(tmp_path_factory.mktemp("plan") / "chunk_plan_host.so")
    subprocess.check_call([nvcc, *build.ARCH, "-O1", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-o", lib,
                           os.path.join(HERE, "chunk_plan_host.cu")])
    fn = ctypes.CDLL(lib).chunk_plan_pieces
    P = ctypes.c_void_p
    fn.restype = ctypes.c_longlong
    fn.argtypes = [ctypes.c_int] * 8 + [P, P] + [ctypes.c_int] * 4 + [P, ctypes.c_longlong]

    def pieces(c):
        lens = np.array([s[0] for s in c["seqs"]], np.int32)
        cu = np.concatenate([[0], np.cumsum([s[1] for s in c["seqs"]])]).astype(np.int32)
        cap = 1 << 16
        while True:
            out = np.empty((cap, 11), np.int32)
            n = fn(c["block"], c["tile_tok"], c["gap"], 512, c["window"], c["sinks"], c["hkv"], len(lens), lens.ctypes.data,
                   cu.ctypes.data, max(1, int(lens.max())), int(np.diff(cu).max()), int(cu[-1]), c["workers"],
                   out.ctypes.data, cap)
            if n <= cap:
                return out[:n]
            cap = n

    return pieces


def shape(rows, G):
    """(block, tokens per tile, a tile's fixed cost) of the kernels' heights."""
    tok = 2 * (128 // G) if rows == 256 else max(1, rows // G)
    return dict(block=16 if rows <= 16 else 128, tile_tok=tok, gap=256 if rows <= 16 else 640)


def check(c, rows):
    """Every block that a tile's rows see is taken once, in order, none past the sequence's end; slots are
    shared by nobody, and a cut tile's record names the workers that have its pieces."""
    CW, window, sinks = c["block"], c["window"], c["sinks"]
    slots, records, tiles = set(), {}, {}
    for me, b, h, t, b0, b1, slot, last, sink, lo, count in rows.tolist():
        tiles.setdefault((b, h, t), []).append((b0, b1, me, slot, sink, lo, count))
        if slot >= 0:
            assert slot not in slots and slot < 2 * c["workers"]
            slots.add(slot)
            if slot % 2:
                assert me not in records
                records[me] = ((b, h, t), last)
    for b, (length, n) in enumerate(c["seqs"]):
        for t in range(-(-n // c["tile_tok"])):
            first = length - n + t * c["tile_tok"]
            end = max(min(length - n + min((t + 1) * c["tile_tok"], n), length), 0)  # tokens that the tile's last row sees
            for h in range(c["hkv"]):
                got = tiles.pop((b, h, t))
                _, _, _, _, sink, lo, count = got[0]
                assert all(g[4:] == got[0][4:] for g in got)
                assert got[0][0] == 0 and got[-1][1] == count and all(x[1] == y[0] for x, y in zip(got, got[1:]))
                # the keys: blocks 0 .. sink - 1 and lo .. lo + count - sink - 1
                if end == 0:
                    assert count == 0
                else:
                    seen = max(first - window + 1, 0) if window else 0  # first token inside the window of its first row
                    assert 0 <= sink <= lo or count == sink
                    assert lo * CW <= seen or lo == sink
                    assert lo + count - sink == max(-(-end // CW), lo if count == sink else 0)
                    if window:
                        assert sink * CW >= min(sinks, seen) or lo <= sink
                    else:
                        assert sink == 0 and lo == 0
                if len(got) == 1:
                    assert got[0][3] == -1
                else:
                    w = got[0][2]
                    assert records[w] == ((b, h, t), got[-1][2])
                    assert [(x[2], x[3]) for x in got] == [(w, 2 * w + 1)] + [(w + i, 2 * (w + i)) for i in range(1, len(got))]
    assert not tiles


@pytest.mark.parametrize("seed", range(120))
def test_random_batches(plan, seed):
    rng = random.Random(seed)
    G, rows = rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), rng.choice([4, 8, 16, 128, 256])
    window = rng.choice([0, 0, rng.randint(1, 3000), 1 << 30])
    seqs = []
    for _ in range(rng.randint(1, 12)):
        n = rng.choice([0, 0, 1, rng.randint(1, 600)])
        seqs.append((rng.choice([0, n, rng.randint(0, 9000), n + rng.randint(0, 4000)]) if n else 0, n))
    c = dict(shape(rows, G), window=window, sinks=rng.choice([0, 4, 100, 5000]) if window else 0, hkv=rng.choice([1, 2, 8]),
             workers=rng.choice([1, 3, 76, 152, 608]), seqs=seqs)
    check(c, plan(c))


@pytest.mark.parametrize("rows,workers", [(8, 608), (16, 152), (128, 152), (256, 76)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (4096, 4), (1 << 30, 1 << 30), (1, 0)])
def test_lengths_up_to_2_30(plan, rows, workers, window, sinks):
    top = 1 << 30
    for seqs in ([(top, 1)], [(top, 300), (top - 1, 1), (0, 0), (17, 5)], [(top, 2)] * 9):
        c = dict(shape(rows, 4), window=window, sinks=sinks, hkv=8, workers=workers, seqs=seqs)
        check(c, plan(c))


@pytest.mark.parametrize("rows,workers", [(8, 608), (256, 76)])
def test_batches_of_1024(plan, rows, workers):
    rng = random.Random(rows)
    for top in (60, 1 << 20, 1 << 30):
        seqs = [(0, 0) if rng.random() < 0.3 else (rng.randint(1, top), rng.randint(1, 9)) for _ in range(1024)]
        seqs[0], seqs[-1] = (0, 0), (top, 9)
        c = dict(shape(rows, 4), window=0, sinks=0, hkv=8, workers=workers, seqs=seqs)
        check(c, plan(c))
