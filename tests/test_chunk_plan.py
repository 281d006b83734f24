"""How chunk attention divides its tiles over the grid (CPU): the arithmetic of csrc/vq_chunk_common.cuh,
restated.  Every block of every tile is taken exactly once, in order; slots are not shared; a cut tile's
record names the workers that hold its pieces."""
import random

import pytest

import bit_vector_quantized_gb300 as vq


class Plan:
    def __init__(self, tile_tok, block, gap, min_range, window, sinks, hkv, workers, seqs):
        self.__dict__.update(locals())

    def length(self, s, j):  # of tiles 0 .. j - 1 of one (sequence, KV head); s: (tokens, new tokens)
        limit, n = s
        base, cap = max(limit - n, 0), limit
        if self.window > 0:
            cap = min(limit, self.window + self.sinks + self.tile_tok)
        rise = min((cap - base) // self.tile_tok if cap > base else 0, j)
        return j * self.gap + rise * base + self.tile_tok * (rise * (rise + 1) // 2) + (j - rise) * cap

    def tiles(self, s):
        return -(-s[1] // self.tile_tok)

    def keys(self, s, t):  # blocks of tile t
        limit, n = s
        base, i0 = limit - n, t * self.tile_tok
        i1 = min(i0 + self.tile_tok, n)
        hi, lo, sink = max(min(base + i1, limit), 0), 0, 0
        if self.window > 0:
            lo = min(max(base + i0 - self.window + 1, 0), hi)
            sink = -(-min(self.sinks, lo) // self.block)
        first = max(lo // self.block, sink)
        return sink + max(-(-hi // self.block) - first, 0) if hi > 0 else 0

    def pieces(self, me, pre):
        """(sequence, KV head, tile, first block, end block, slot, last worker) of a worker's range."""
        total = pre[-1]
        W = max(-(-total // self.workers), self.min_range, int((32 * (total // (self.hkv * len(self.seqs)))) ** 0.5))
        x = min(W * me, total)
        x1 = min(x + W, total)
        if x >= x1:
            return
        b = max(i for i in range(len(self.seqs)) if pre[i] <= x)
        s = self.seqs[b]
        per_head = self.length(s, self.tiles(s))
        h = (x - pre[b]) // per_head
        off = x - pre[b] - h * per_head
        t = max(i for i in range(self.tiles(s)) if self.length(s, i) <= off)
        tile_x = pre[b] + h * per_head + self.length(s, t)
        while x < x1:
            w = self.length(s, t + 1) - self.length(s, t)
            o0 = x - tile_x
            o1 = min(w, o0 + x1 - x)
            count = self.keys(s, t)
            yield (b, h, t, 0 if o0 == 0 else o0 * count // w, count if o1 == w else o1 * count // w,
                   2 * me if o0 > 0 else 2 * me + 1 if o1 < w else -1, (tile_x + w - 1) // W)
            x += o1 - o0
            if o1 == w:
                tile_x += w
                t += 1
                if t == self.tiles(s):
                    t, h = 0, h + 1
                    if h == self.hkv:
                        h = 0
                        if x < x1:
                            b += 1
                            while self.seqs[b][1] == 0:
                                b += 1
                            s = self.seqs[b]


@pytest.mark.parametrize("seed", range(200))
def test_tiles_are_divided_without_gap_or_overlap(seed):
    rng = random.Random(seed)
    G, rows = rng.choice([1, 2, 4, 5, 8]), rng.choice([4, 8, 16, 128, 256])
    tile_tok = max(1, 2 * (128 // G) if rows == 256 else rows // G)
    window = rng.choice([0, 0, rng.randint(1, 3000), 1 << 30])
    seqs = []
    for _ in range(rng.randint(1, 12)):
        n = rng.choice([0, 0, 1, rng.randint(1, 600)])
        seqs.append((rng.choice([0, n, rng.randint(0, 9000), n + rng.randint(0, 4000)]) if n else 0, n))
    p = Plan(tile_tok, 16 if rows <= 16 else 128, rng.choice([256, 640]), 512, window, rng.choice([0, 4, 100]) if window else 0,
             rng.choice([1, 2, 8]), rng.choice([1, 3, 76, 152, 608]), seqs)
    pre = [0]
    for s in seqs:
        pre.append(pre[-1] + p.hkv * p.length(s, p.tiles(s)))
    taken, slots, records = {}, set(), {}
    for me in range(p.workers):
        for b, h, t, b0, b1, slot, last in p.pieces(me, pre):
            taken.setdefault((b, h, t), []).append((b0, b1, me, slot))
            if slot >= 0:
                assert slot not in slots and slot < 2 * p.workers
                slots.add(slot)
                if slot % 2:
                    assert me not in records
                    records[me] = ((b, h, t), last)
    for b, s in enumerate(seqs):
        for h in range(p.hkv):
            for t in range(p.tiles(s)):
                got = taken.pop((b, h, t))
                assert got[0][0] == 0 and got[-1][1] == p.keys(s, t)
                assert all(x[1] == y[0] for x, y in zip(got, got[1:]))
                if len(got) == 1:
                    assert got[0][3] == -1
                else:
                    first = got[0][2]
                    assert records[first] == ((b, h, t), got[-1][2])
                    assert [(x[2], x[3]) for x in got] == [(first, 2 * first + 1)] + [(first + i, 2 * (first + i)) for i in range(1, len(got))]
    assert not taken


@pytest.mark.parametrize("fmt", [(4, 8, 4, 8), (2, 8, 4, 9), (8, 12, 8, 12)])
@pytest.mark.parametrize("group", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("sms", [1, 2, 151, 152])
def test_a_workspace_of_larger_bounds_serves_smaller_ones(fmt, group, sms):
    layout = vq.make_layout(128, 2 * group, 2, *fmt, 64)
    sizes = [vq.vq_chunk_workspace_bytes(layout, 4, 4 * n, 1 << 20, n, sms) for n in range(1, 600)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[0] > 0
