"""The tcgen05 attention kernels' rings of pieces (CPU): their warps as programs that wait for one another in the kernels'
order, over the plan's pieces and drawn ones.  A ring with too few slots makes them wait in a circle."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from bit_vector_quantized_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    try:
        nvcc = build._nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    lib = str(tmp_path_factory.mktemp("ring") / "piece_ring_host.so")
    subprocess.check_call([nvcc, *build.ARCH, "-O1", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-o", lib,
                           os.path.join(HERE, "piece_ring_host.cu")])
    lib = ctypes.CDLL(lib)
    P = ctypes.c_void_p
    lib.ring_blocks.restype = ctypes.c_longlong
    lib.ring_blocks.argtypes = [ctypes.c_int] * 4 + [P, P] + [ctypes.c_int] * 2 + [P, ctypes.c_longlong]
    return lib


class Cta:
    """What the warps of one CTA have done: pieces handed out and taken, blocks stored, scored, summed."""

    def __init__(self, pieces):
        self.first = np.concatenate([[0], np.cumsum(pieces)]).tolist()  # first block of each piece
        self.total = self.first[-1]
        self.out = 0           # pieces handed out (the last one says that there are no more)
        self.taken = {}        # warp -> pieces taken
        self.k, self.v, self.mask, self.p = set(), set(), set(), set()
        self.q = 0             # pieces whose Q~ is there


def planner(c, slots):
    for i in range(len(c.first)):  # the pieces, then the end
        while i >= slots and min(c.taken.values()) <= i - slots:
            yield
        c.out += 1


def take(c, who):
    while c.out <= c.taken[who]:
        yield
    c.taken[who] += 1


def ahead_of(c, who, block):
    """Pieces until the one that holds `block`, or the end."""
    while c.taken[who] < len(c.first) and c.first[c.taken[who]] <= block:
        yield from take(c, who)


def prefetch(c):
    for _ in c.first:
        yield from take(c, "prefetch")


def soft(c, s):
    for i in range(len(c.first) - 1):
        yield from take(c, "soft")
        c.q += 1
        end = c.first[i + 1]
        for b in range(c.first[i], end):
            while not (b in s["scores"] and b in c.mask):
                yield
            if b > c.first[i]:  # the maxima may have moved: the block before it is summed up
                while not ((b + 1 in s["scores"] and b + 1 in c.mask) if b + 1 < end else b - 1 in s["values"]):
                    yield
            c.p.add(b)
        while end - 1 not in s["values"]:
            yield
    yield from take(c, "soft")


def tree_codes(c, s, is_k, half):
    """vq_tree.cu: every other block; the page two blocks of its own ahead, and the arrival comes after that look."""
    who = ("k" if is_k else "v") + str(half)
    blk = half
    yield from ahead_of(c, who, blk)
    yield from ahead_of(c, who, blk + 2)
    while blk < c.total:
        if not is_k:
            c.mask.add(blk)
        while blk >= (4 if is_k else 2) and blk - (4 if is_k else 2) not in s["scores" if is_k else "values"]:
            yield
        yield from ahead_of(c, who, blk + 4)
        (c.k if is_k else c.v).add(blk)
        blk += 2
    if is_k:
        while blk >= 4 and blk - 4 < c.total and blk - 4 not in s["scores"]:
            yield
        c.k.add(blk)


def wide_codes(c, s, is_k, stages):
    """vq_chunk_wide.cu: every block; the page two blocks ahead, before the block is stored."""
    who = "k" if is_k else "v"
    yield from ahead_of(c, who, 0)
    yield from ahead_of(c, who, 1)
    for blk in range(c.total + (2 if is_k else 0)):
        if blk < c.total:
            yield from ahead_of(c, who, blk + 2)
            if not is_k:
                c.mask.add(blk)
        while blk >= stages and blk - stages not in s["scores" if is_k else "values"]:
            yield
        (c.k if is_k else c.v).add(blk)


def issuer(ctas, s):
    """One thread issues for the CTA, or for both of a pair."""
    c = ctas[0]
    for i in range(len(c.first) - 1):
        yield from take(c, "issue")
        while not all(x.q > i for x in ctas):
            yield
        if i == 0:
            while not all({0, 1} <= x.k for x in ctas):
                yield
        b0, b1 = c.first[i], c.first[i + 1]
        s["scores"].update(range(b0, min(b0 + 2, b1)))
        for b in range(b0, b1):
            while not all(b in x.p and b in x.v and b + 2 in x.k for x in ctas):
                yield
            s["values"].add(b)
            if b + 2 < b1:
                s["scores"].add(b + 2)
    yield from take(c, "issue")


def passer(c):
    """The second CTA of a pair: its tiles are passed on, a block at a time."""
    for i in range(len(c.first) - 1):
        yield from take(c, "issue")
        for b in range(c.first[i], c.first[i + 1]):
            while not (b in c.v and b + 2 in c.k):
                yield
    yield from take(c, "issue")


def ends(kind, slots, pieces):
    """Whether all the warps come to their end.  kind: tree, one or pair (of vq_chunk_wide.cu)."""
    s = dict(scores=set(), values=set())
    ctas = [Cta(pieces) for _ in range(2 if kind == "pair" else 1)]
    warps = [issuer(ctas, s)]
    for c in ctas:
        warps += [planner(c, slots), soft(c, s), prefetch(c)]
        c.taken = dict(soft=0, prefetch=0, issue=0)
        if kind == "tree":
            c.taken.update(k0=0, k1=0, v0=0, v1=0)
            warps += [tree_codes(c, s, k, h) for k in (True, False) for h in (0, 1)]
        else:
            c.taken.update(k=0, v=0)
            warps += [wide_codes(c, s, True, 3 if kind == "pair" else 2), wide_codes(c, s, False, 3 if kind == "pair" else 1)]
        if c is not ctas[0]:
            warps.append(passer(c))
    live = list(warps)
    state = None
    while live:
        was = [(sum(c.taken.values()), c.out, c.q, len(c.k), len(c.v), len(c.mask), len(c.p)) for c in ctas], len(s["scores"]), len(s["values"])
        if was == state:
            return False
        state = was
        rest = []
        for w in live:
            try:
                next(w)
                rest.append(w)
            except StopIteration:
                pass
        if len(rest) < len(live):
            state = None
        live = rest
    return True


def blocks_of_workers(host, rng_gap, seqs, hkv, tile_tok, workers):
    """Blocks of each worker's pieces (those without any are not handed out)."""
    lens = np.array([x for x, _ in seqs], np.int32)
    cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])]).astype(np.int32)
    cap = 1 << 18
    out = np.empty((cap, 2), np.int32)
    n = host.ring_blocks(tile_tok, rng_gap, hkv, len(seqs), lens.ctypes.data, cu.ctypes.data, workers, int(lens.max()), out.ctypes.data, cap)
    assert n <= cap
    lists = {}
    for me, blocks in out[:n].tolist():
        if blocks > 0:
            lists.setdefault(me, []).append(blocks)
    return lists.values()


KINDS = ("tree", "one", "pair")


@pytest.mark.parametrize("kind", KINDS)
def test_pieces_of_few_blocks(host, kind):
    slots = host.ring_slots(kind == "tree")
    for n in range(1, 24):
        assert ends(kind, slots, [1] * n), n
    rng = random.Random(1)
    for _ in range(300):
        pieces = [rng.choice([1, 1, 1, 2, 3, rng.randint(1, 9)]) for _ in range(rng.randint(1, 20))]
        assert ends(kind, slots, pieces), pieces
    for before in range(1, 6):  # one-block pieces between longer ones
        for ones in range(1, 10):
            assert ends(kind, slots, [before] + [1] * ones + [7, 1, 1]), (before, ones)


@pytest.mark.parametrize("kind", KINDS)
def test_a_slot_less_is_too_few(host, kind):
    """The bound is the kernels' own, and the programs above show a ring that is too small."""
    assert not ends(kind, host.ring_slots(kind == "tree") - 1, [1] * 12)


SHORT_AMONG_LONG = [
    ([(8000 + 440 * i, 8) for i in range(16)] + [(47, 4)], 8, 8),
    ([(4000, 4)] * 32 + [(60, 4)], 8, 8),
    ([(100, 4)] * 128, 8, 8),
    ([(20 + i % 100, 1 + i % 8) for i in range(512)], 8, 8),
    ([(9, 1)] * 1024, 8, 4),
]


@pytest.mark.parametrize("seqs,hkv,tile_tok", SHORT_AMONG_LONG)
@pytest.mark.parametrize("gap", [256, 640])
def test_short_sequences_among_long_ones(host, seqs, hkv, tile_tok, gap):
    for kind in KINDS:
        for pieces in blocks_of_workers(host, gap, seqs, hkv, tile_tok, 76 if kind == "pair" else 152):
            assert ends(kind, host.ring_slots(kind == "tree"), pieces), pieces


@pytest.mark.parametrize("seed", range(12))
def test_drawn_batches(host, seed):
    rng = random.Random(seed)
    seqs = []
    for _ in range(rng.choice([2, 30, 200, 900])):
        n = rng.randint(0, 8)
        seqs.append((n + rng.choice([0, 1, rng.randint(0, 120), rng.randint(0, 120), rng.randint(0, 20000)]), n))
    seqs.append((5, 1))
    lists = {tuple(x) for x in blocks_of_workers(host, rng.choice([256, 640]), seqs, rng.choice([1, 2, 8]), rng.choice([2, 4, 8]), 152)}
    for pieces in lists:
        for kind in KINDS:
            assert ends(kind, host.ring_slots(kind == "tree"), pieces), pieces
