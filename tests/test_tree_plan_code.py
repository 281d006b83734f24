"""The plan of tree attention as the kernels have it (CPU): csrc/vq_chunk_plan.cuh compiled for the host with kTree, its
pieces against the definition."""
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
    lib = str(tmp_path_factory.mktemp("plan") / "tree_plan_host.so")
    subprocess.check_call([nvcc, *build.ARCH, "-O1", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-o", lib,
                           os.path.join(HERE, "tree_plan_host.cu")])
    fn = ctypes.CDLL(lib).tree_plan_pieces
    P = ctypes.c_void_p
    fn.restype = ctypes.c_longlong
    fn.argtypes = [ctypes.c_int] * 7 + [P, P] + [ctypes.c_int] * 4 + [P, ctypes.c_longlong]

    def pieces(c):
        lens = np.array([s[0] for s in c["seqs"]], np.int32)
        cu = np.concatenate([[0], np.cumsum([s[1] for s in c["seqs"]])]).astype(np.int32)
        cap = 1 << 16
        while True:
            out = np.empty((cap, 11), np.int32)
            n = fn(c["tile_tok"], 640, 512, c["window"], c["sinks"], c["hkv"], len(lens), lens.ctypes.data, cu.ctypes.data,
                   c.get("max_len", max(1, int(lens.max()))), 256, int(cu[-1]), c["workers"], out.ctypes.data, cap)
            if n <= cap:
                return out[:n]
            cap = n

    return pieces


def check(c, rows):
    """Every tile's blocks are taken once, in order, and hold every token that one of its rows may see; a cut tile's pieces have
    slots of their own, and its first worker's record names the last."""
    W, S = c["window"], c["sinks"]
    tiles, slots = {}, set()
    for me, b, h, t, b0, b1, slot, last, sink, lo, count in rows.tolist():
        tiles.setdefault((b, h, t), []).append((me, b0, b1, slot, last, sink, lo, count))
        if slot >= 0:
            assert slot not in slots and slot < 2 * c["workers"]
            slots.add(slot)
    want = {(b, h, t) for b, (length, n) in enumerate(c["seqs"]) if n <= length <= c.get("max_len", 1 << 30)
            for h in range(c["hkv"]) for t in range(-(-n // c["tile_tok"]))}
    assert set(tiles) == want
    for (b, h, t), p in tiles.items():
        length, n = c["seqs"][b]
        base = length - n
        me, _, _, slot, last, sink, lo, count = p[0]
        assert [x[0] for x in p] == list(range(me, me + len(p)))
        assert p[0][1] == 0 and p[-1][2] == count and all(x[2] == y[1] for x, y in zip(p, p[1:]))
        if len(p) == 1:
            assert slot == -1
        else:
            assert slot == 2 * me + 1 and last == p[-1][0] and all(x[3] == 2 * x[0] for x in p[1:])
        first = max(base - W + 1, 0) if W else 0
        blocks = list(range(sink)) + list(range(lo, lo + count - sink))
        assert len(set(blocks)) == count and (not blocks or blocks[-1] * 128 < length)
        seen = set(blocks)
        assert all(i in seen for i in range(first // 128, -(-length // 128)))
        assert all(i in seen for i in range(-(-min(S, first) // 128) if W else 0))


@pytest.mark.parametrize("seed", range(60))
def test_drawn_batches(plan, seed):
    rng = random.Random(seed)
    window = rng.choice([0, 0, 1, 100, 1000, 1 << 30, 2 ** 31 - 1])
    seqs = []
    for _ in range(rng.choice([1, 2, 7, 48, 300])):
        n = rng.choice([0, 1, 5, 64, 256, rng.randint(1, 256)])
        seqs.append((n + rng.choice([0, 1, 127, 128, rng.randint(0, 40000)]), n))
    c = dict(seqs=seqs, window=window, sinks=rng.choice([0, 1, 4, 130, 2 ** 31 - 1]) if window else 0, hkv=rng.choice([1, 2, 8]),
             tile_tok=rng.choice([2, 4, 8, 16, 25, 32, 50, 64, 128, 256]), workers=rng.choice([1, 3, 76, 152]))
    check(c, plan(c))


def test_sequences_that_are_left_out(plan):
    c = dict(seqs=[(5, 9), (100, 9), (30000, 9), (0, 0), (9, 9)], max_len=20000, window=0, sinks=0, hkv=2, tile_tok=4, workers=152)
    check(c, plan(c))


def test_far_lengths(plan):
    c = dict(seqs=[(1 << 30, 256), (1 << 30, 3), (300, 200)], window=4096, sinks=68, hkv=8, tile_tok=32, workers=152)
    check(c, plan(c))
