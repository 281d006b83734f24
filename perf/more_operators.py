"""Operators of speculative decoding over the quantized KV cache: plain forms, calls and cases.

Operators (``op`` of a case):

* ``append``  keys turned by their positions, coded and stored in the paged pools, values coded and
              stored beside them, queries turned, straight from a projection's rows;
* ``tree``    attention of a tree of drafted tokens over the paged codes: each row sees the context
              and, of the drafted tokens, those that its bits name (its ancestors and itself);
* ``keep``    the accepted drafted tokens moved together in the pools of all layers, and the pages
              that the others leave empty given back.

With ``own`` false ``run`` computes them with elementary torch operations, with ``own`` true it
calls this package.
"""
import math

import numpy as np
import torch

own = False

D = 128
ORIGINAL = 8192  # positions that the rotary frequencies were made for
DEV = "cuda"


# ------------------------------------------------------------------ cases ---

def _tree(name, batch, hq, hkv, fmt, page, ctx, new, window=0, sinks=0):
    return dict(name=name, op="tree", batch=batch, hq=hq, hkv=hkv, ks=fmt[0], kb=fmt[1], vs=fmt[2], vb=fmt[3],
                page=page, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0], new_hi=new[1], window=window, sinks=sinks)


def _append(name, tokens, hq, hkv, fmt, page, dtype, rdim, interleaved, scaling, factor, far):
    return dict(name=name, op="append", tokens=tokens, hq=hq, hkv=hkv, ks=fmt[0], kb=fmt[1], vs=fmt[2], vb=fmt[3], page=page,
                dtype=dtype, rdim=rdim, interleaved=interleaved, scaling=scaling, factor=factor, far=far)


def _keep(name, batch, layers, hkv, fmt, page, ctx, new, most):
    return dict(name=name, op="keep", batch=batch, layers=layers, hkv=hkv, ks=fmt[0], kb=fmt[1], vs=fmt[2], vb=fmt[3],
                page=page, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0], new_hi=new[1], most=most)


def listed():
    return [
        # one long conversation, a full tree of drafted tokens, the Llama layer shape
        _tree("tree of 64 in 32K", 1, 32, 8, (4, 8, 4, 8), 256, (32700, 32700), (64, 64)),
        # the same tree for every sequence of a batch, the 40-head layer with 9-bit V codes
        _tree("tree of 26 batch 16", 16, 40, 8, (2, 8, 4, 9), 256, (8000, 16384), (26, 26)),
        # trees cut to size by their confidence, ragged, small permuted pages, new conversations among them
        _tree("trees of 1 to 61 paged 64", 24, 32, 8, (2, 8, 4, 8), 64, (0, 9001), (1, 61)),
        # a few candidates each at 1.5 bit
        _tree("tree of 7 at 1.5 bit", 48, 32, 8, (8, 12, 8, 12), 256, (3000, 6000), (7, 7)),
        # large trees in a model with a sliding window and sinks that end inside a page
        _tree("trees of 250 window 4096", 4, 32, 8, (4, 8, 4, 8), 256, (9001, 20011), (180, 250), 4096, 68),
        # the smallest call: a token and its two candidates in one short conversation
        _tree("tree of 3 in 333", 1, 8, 2, (2, 8, 4, 8), 64, (333, 333), (3, 3)),
        # one decode step of a batch
        _append("append 64 tokens", 64, 32, 8, (2, 8, 4, 8), 64, "fp16", 128, False, "none", 1.0, 131072),
        # a prompt chunk out of a bf16 projection, half of the head turned, interleaved pairs, 9-bit V codes
        _append("append 4099 bf16", 4099, 40, 8, (2, 8, 4, 9), 256, "bf16", 64, True, "linear", 4.0, 32768),
        # a long prompt chunk, frequencies scaled by parts for far positions
        _append("append 8192 far", 8192, 32, 8, (4, 8, 4, 8), 256, "fp16", 128, False, "parts", 16.0, 1000000),
        # drafted tokens of a batch at 1.5 bit
        _append("append 333 at 1.5 bit", 333, 32, 8, (8, 12, 8, 12), 256, "bf16", 128, False, "wavelength", 8.0, 131072),
        # one conversation's accepted path, all layers
        _keep("keep up to 6 of 64", 1, 32, 8, (4, 8, 4, 8), 256, (700, 700), (64, 64), 6),
        # a batch's accepted paths, small pages
        _keep("keep batch 48 paged 16", 48, 32, 8, (2, 8, 4, 9), 16, (0, 400), (1, 61), 9),
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


_FORMATS = [(4, 8, 4, 8), (2, 8, 4, 8), (2, 8, 4, 9), (4, 8, 4, 9), (4, 8, 2, 8), (8, 12, 8, 12)]


def draw(rng):
    most = max(work(c)["flops"] for c in listed() if c["op"] == "tree")
    op = rng.choice(["tree", "tree", "tree", "append", "append", "keep"])
    fmt = rng.choice(_FORMATS)
    if op == "append":
        hkv = rng.choice([1, 2, 8])
        c = _append("", _log(rng, 1, 8000), hkv * rng.choice([1, 4, 5]), hkv, fmt, rng.choice([16, 48, 64, 256]), rng.choice(["fp16", "bf16"]),
                    rng.choice([128, 96, 64, 32, 2]), rng.random() < 0.5, rng.choice(["none", "linear", "base", "parts", "wavelength"]),
                    rng.choice([2.0, 8.0, 13.5]), _log(rng, 8192, 2000000))
        # (scores of a large codebook: no more of them than the largest listed case has)
        while c["tokens"] * hkv * _codebooks(c) > 8192 * 8 * 65536:
            c["tokens"] = c["tokens"] * 2 // 3
    elif op == "keep":
        lo, n, layers = _log(rng, 1, 400), _log(rng, 1, 64), _log(rng, 1, 32)
        c = _keep("", _log(rng, 1, 48), layers, rng.choice([1, 2, 8]), fmt, rng.choice([16, 48, 64, 256]), (lo - 1, lo + _log(rng, 1, 200)),
                  (rng.randint(1, n), n), rng.randint(1, n))
    else:
        hkv, g = rng.choice([(8, 4), (8, 5), (2, 4), (1, 2), (4, 8), (4, 1), (1, 7)])
        lo, n = _log(rng, 1, 24000), _log(rng, 1, 250)
        window, sinks = (_log(rng, 1, 8192), rng.choice([0, 1, 4, 65, 500])) if rng.random() < 0.3 else (0, 0)
        c = _tree("", _log(rng, 1, 48), hkv * g, hkv, fmt, rng.choice([16, 48, 64, 256]), (lo - 1, lo + _log(rng, 1, 8000)),
                  (rng.randint(1, n), n), window, sinks)
        # the plain form holds all scores: the padded batch is kept below the largest listed case
        while c["batch"] * (c["ctx_hi"] + c["new_hi"]) * c["new_hi"] * c["hq"] * 512 > most or c["batch"] * (c["ctx_hi"] + c["new_hi"]) * c["hkv"] > 2_200_000:
            if c["batch"] > 1:
                c["batch"] = c["batch"] * 2 // 3
            else:
                c["new_hi"] = max(1, c["new_hi"] * 2 // 3)
                c["new_lo"] = min(c["new_lo"], c["new_hi"])
    del c["name"]
    return c


def _spread(lo, hi, n, mul):
    """n whole numbers over [lo, hi], both ends among them where n > 1, in a mixed order."""
    if n == 1:
        return np.array([hi], dtype=np.int64)
    x = lo + (np.arange(n, dtype=np.int64) * (hi - lo)) // (n - 1)
    step = next(s for s in range(mul, mul + n + 2) if math.gcd(s, n) == 1)
    return x[(np.arange(n) * step + n // 2) % n]


def _lens(c):
    """(tokens of each sequence before its drafted ones, drafted tokens)."""
    return _spread(c["ctx_lo"], c["ctx_hi"], c["batch"], 7), _spread(c["new_lo"], c["new_hi"], c["batch"], 5)


def _row(sub, bits):
    return (D // sub * bits + 31) // 32 * 4


def _codebooks(c):
    """Products that the nearest centroids of one token-head's key and value take."""
    return D * ((1 << c["kb"]) + (1 << c["vb"]))


def work(case):
    c = case
    rows = _row(c["ks"], c["kb"]) + _row(c["vs"], c["vb"])
    if c["op"] == "append":
        q, kv = c["tokens"] * c["hq"] * D, c["tokens"] * c["hkv"]
        return {"bytes": 4 * q + kv * (4 * D + rows) + 12 * c["tokens"],
                "flops": 2 * kv * _codebooks(c) + 8 * kv * D + 3 * c["tokens"] * (c["hq"] + c["hkv"]) * c["rdim"]}
    old, new = _lens(c)
    if c["op"] == "keep":
        moved = np.minimum(np.log(new), c["most"] - 1)  # a path of the drawn trees, about; its root stays where it is
        return {"bytes": int(2 * moved.sum() * c["layers"] * c["hkv"] * rows + 4 * c["batch"] * c["most"] + 20 * c["batch"]), "flops": int(moved.sum()) + c["batch"]}
    pairs, seen = 0, 0
    w, s = c["window"], c["sinks"]
    for o, n in zip(old.tolist(), new.tolist()):
        first = max(0, o - w + 1) if w else 0
        ctx = o - first + min(first, s)
        pairs += n * ctx + n * max(1, int(math.log2(n + 1)))  # (the context, and a path of the tree)
        seen += ctx + n
    n = int(new.sum())
    tables = 2 * ((1 << c["kb"]) * c["ks"] + (1 << c["vb"]) * c["vs"]) + 4 * c["hkv"] * D
    return {"bytes": seen * c["hkv"] * rows + 4 * n * c["hq"] * D + 8 * n * -(-c["new_hi"] // 64) + tables,
            "flops": 4 * D * c["hq"] * pairs}


# ----------------------------------------------------------------- inputs ---

def _pages(c, g):
    """Page tables of all sequences with room for their drafted tokens, physical pages in a drawn order."""
    old, new = _lens(c)
    need = -(-(old + new) // c["page"])
    total = int(need.sum())
    table = torch.full((c["batch"], max(1, int(need.max()))), -1, dtype=torch.int32, device=DEV)
    col = torch.arange(table.shape[1], device=DEV)
    table[col[None] < torch.from_numpy(need).to(DEV)[:, None]] = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    return table, total


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x.astype(np.int32))).to(DEV)


def _trees(new, rng):
    """Parents of each sequence's drafted tokens: token 0 is the root, the others hang on a token before them, early ones first."""
    return [np.concatenate([[-1], np.floor(rng.random(n - 1) ** 1.5 * np.arange(1, n)).astype(np.int64)])[:n] for n in new.tolist()]


def _ancestors(parents):
    """bool [n][n]: which drafted tokens are on the way from token i to the root, itself among them."""
    n = len(parents)
    a = np.eye(n, dtype=bool)
    for i in range(n):
        if parents[i] >= 0:
            a[i] |= a[parents[i]]
    return a


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * scale

    def pool(row, *shape):
        return torch.randint(0, 256, (*shape, c["hkv"], c["page"], row), generator=g, device=DEV, dtype=torch.uint8)

    # keys with a few strong channels: smoothing factors near 2, near 9 for those channels; the
    # smoothed and transformed keys, and with them their centroids, are near N(0, 0.6^2)
    lam = 2.0 + 0.1 * normal(c["hkv"], D).abs()
    strong = torch.randperm(D, generator=g, device=DEV)[:4]
    lam[:, strong] *= 4.5
    s = dict(case=c, lam=lam, ck=normal(1 << c["kb"], c["ks"], scale=0.6).half(), cv=normal(1 << c["vb"], c["vs"]).half())
    if own:  # what a program makes once
        import bit_vector_quantized_gb300 as vq
        s["layout"] = vq.make_layout(D, c.get("hq", c["hkv"]), c["hkv"], c["ks"], c["kb"], c["vs"], c["vb"], c["page"])
    if c["op"] == "append":
        dt = torch.float16 if c["dtype"] == "fp16" else torch.bfloat16
        x = normal(c["tokens"], c["hq"] + 2 * c["hkv"], D)  # a fused projection's output
        x[:, c["hq"]:c["hq"] + c["hkv"]] *= 1.2
        x[:, c["hq"]:c["hq"] + c["hkv"], strong] *= 4.5
        start = torch.randint(0, c["far"] - min(c["far"], c["tokens"]) + 1, (1,), generator=g, device=DEV)
        pos = (start + torch.arange(c["tokens"], device=DEV) % c["far"]).to(torch.int32)
        pages = -(-c["tokens"] // c["page"]) + 1
        order = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(c["tokens"], device=DEV) + int(rng.integers(0, c["page"]))  # the first page is partly full
        s |= dict(qkv=x.to(dt), positions=pos, slots=order[t // c["page"]] * c["page"] + t % c["page"],
                  k_pool=pool(_row(c["ks"], c["kb"]), pages), v_pool=pool(_row(c["vs"], c["vb"]), pages))
        if own:
            s["rotary"] = vq.make_rotary(D, c["rdim"], c["interleaved"], 500000.0, c["scaling"], c["factor"], ORIGINAL, 1.0,
                                         32.0 if c["scaling"] == "parts" else 4.0, _attention_factor(c))
        return s
    old, new = _lens(c)
    table, total = _pages(c, g)
    s |= dict(page_table=table, seq_lens=_i32(old + new), cu=_i32(np.concatenate([[0], np.cumsum(new)])), max_new_len=int(new.max()))
    kr, vr = _row(c["ks"], c["kb"]), _row(c["vs"], c["vb"])
    trees = [_ancestors(p) for p in _trees(new, rng)]
    if c["op"] == "keep":
        keep, kept = np.full((c["batch"], c["most"]), -1), np.zeros(c["batch"])
        for b, a in enumerate(trees):  # an accepted path from the root to some token, cut to the most that are kept
            path = np.flatnonzero(a[rng.integers(0, len(a))])[:c["most"]]
            keep[b, :len(path)], kept[b] = path, len(path)
        free = torch.randperm(total + 37, generator=g, device=DEV).to(torch.int32)
        s |= dict(keep=_i32(keep), kept=_i32(kept), k_pool=pool(kr, c["layers"], total), v_pool=pool(vr, c["layers"], total),
                  free_pages=free, num_free=torch.tensor([37], dtype=torch.int32, device=DEV))
        return s
    words = -(-s["max_new_len"] // 64)
    bits = [np.packbits(np.pad(a, ((0, 0), (0, 64 * words - len(a)))), axis=1, bitorder="little").view(np.int64) for a in trees]
    s |= dict(k_pool=pool(kr, total), v_pool=pool(vr, total), q=normal(int(new.sum()), c["hq"], D).half(), max_seq_len=int((old + new).max()),
              masks=torch.from_numpy(np.concatenate(bits)).to(DEV),
              positions=_i32(np.concatenate([o + a.sum(1) - 1 for o, a in zip(old, trees)])))
    if own:  # the workspace of the program's largest step
        s["workspace"] = vq.alloc_tree_workspace(s["layout"], c["batch"], len(s["q"]), s["max_seq_len"], s["max_new_len"])
    return s


# ------------------------------------------------------------ plain forms ---

def _codes(rows, count, bits):
    """int64 codes of packed rows [..., row bytes]: code i is bits [i b, (i + 1) b) of the stream."""
    if bits == 8:
        return rows[..., :count].long()
    at = torch.arange(count, device=rows.device) * bits
    x = torch.nn.functional.pad(rows, (0, 2)).int()
    x = x[..., at // 8] | x[..., at // 8 + 1] << 8 | x[..., at // 8 + 2] << 16
    return ((x >> (at % 8)) & ((1 << bits) - 1)).long()


def _packed(codes, bits, row):
    """Packed rows [..., row bytes] of int64 codes."""
    x = (codes[..., None] >> torch.arange(bits, device=DEV)) & 1
    x = torch.nn.functional.pad(x.flatten(-2), (0, 8 * row - x.shape[-1] * x.shape[-2]))
    return (x.unflatten(-1, (row, 8)) << torch.arange(8, device=DEV)).sum(-1).to(torch.uint8)


def _hadamard(dtype):
    i = torch.arange(D, device=DEV)
    x = i[:, None] & i[None]
    x = x ^ x >> 4
    x = x ^ x >> 2
    x = x ^ x >> 1
    return (1 - 2 * (x & 1)).to(dtype) / math.sqrt(D)


def _plain_tree(s):
    c = s["case"]
    B, hkv, G, P = c["batch"], c["hkv"], c["hq"] // c["hkv"], c["page"]
    L, N = s["max_seq_len"], s["max_new_len"]
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    base = s["seq_lens"].long() - new
    p = torch.arange(L, device=DEV)
    page = s["page_table"][:, (p // P).clamp(max=s["page_table"].shape[1] - 1)].long().clamp(min=0)

    def read(pool, cb, sub, bits):
        x = cb.float()[_codes(pool[page, :, (p % P)[None].expand(B, L)], D // sub, bits)]
        return x.reshape(B, L, hkv, D).transpose(1, 2)  # [B][Hkv][L][D]

    i = torch.arange(N, device=DEV)
    row = (s["cu"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    qt = (s["q"].float().reshape(-1, hkv, G, D) * s["lam"][:, None]) @ _hadamard(torch.float32)
    qt = qt[row].permute(0, 2, 1, 3, 4).reshape(B, hkv, N * G, D)
    x = qt @ read(s["k_pool"], s["ck"], c["ks"], c["kb"]).transpose(2, 3)
    x = x.mul_(1 / math.sqrt(D)).view(B, hkv, N, G, L)
    j = p - base[:, None]  # place among the drafted tokens [B][L]
    at = j.clamp(0, N - 1)
    words = s["masks"][row]  # [B][N][words]
    bit = words.gather(2, (at // 64)[:, None].expand(B, N, L)) >> (at % 64)[:, None] & 1
    see = (j < 0)[:, None] | (bit == 1) & (j < new[:, None])[:, None]
    if c["window"]:
        where = s["positions"].long()[row]  # [B][N]
        its = torch.where(j < 0, p, where.gather(1, at))  # positions of the tokens
        see &= (its[:, None] > where[..., None] - c["window"]) | (its < c["sinks"])[:, None]
    x = x.masked_fill_(~see[:, None, :, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    o = x.view(B, hkv, N * G, L) @ read(s["v_pool"], s["cv"], c["vs"], c["vb"])
    o = o.view(B, hkv, N, G, D) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(B, N, c["hq"], D)
    return o[i[None] < new[:, None]].half()


def _attention_factor(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "parts" else 1.0


def _frequencies(c):
    """Angle per position of each pair, in 64 bits."""
    r, s, base = c["rdim"], c["factor"], 500000.0
    if c["scaling"] == "base" and r > 2:
        base *= s ** (r / (r - 2))
    i = torch.arange(r // 2, device=DEV, dtype=torch.float64)
    f = base ** (-2 * i / r)
    if c["scaling"] == "linear":
        f = f / s
    elif c["scaling"] == "parts":  # pairs of more than 32 turns keep their frequency, of less than one are divided
        lo = max(0, math.floor(r * math.log(ORIGINAL / (32 * 2 * math.pi)) / (2 * math.log(base))))
        hi = min(r - 1, math.ceil(r * math.log(ORIGINAL / (1 * 2 * math.pi)) / (2 * math.log(base))))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / s * ramp
    elif c["scaling"] == "wavelength":  # by turns within the original length: 4 and more kept, 1 and less divided
        t = ((ORIGINAL * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = (1 - t) * f / s + t * f
    return f


def _plain_append(s):
    """Queries in 32 bits; keys and values in 64, because the nearest centroid is next to a border for some of them."""
    c = s["case"]
    r, hq, hkv, P = c["rdim"], c["hq"], c["hkv"], c["page"]
    angle = s["positions"].double()[:, None] * _frequencies(c)
    m = _attention_factor(c)
    co, si = (angle.cos() * m)[:, None], (angle.sin() * m)[:, None]

    def turned(x):
        qk, rest, co_, si_ = x[..., :r], x[..., r:], co.to(x.dtype), si.to(x.dtype)
        a, b = (qk[..., 0::2], qk[..., 1::2]) if c["interleaved"] else (qk[..., :r // 2], qk[..., r // 2:])
        y = (a * co_ - b * si_, b * co_ + a * si_)
        return torch.cat([torch.stack(y, -1).flatten(-2) if c["interleaved"] else torch.cat(y, -1), rest], -1)

    def store(x, cb, sub, bits, pool):
        cb = cb.double()
        x = x.unflatten(-1, (D // sub, sub))
        codes = ((cb * cb).sum(-1) - 2 * (x @ cb.T)).argmin(-1)
        pool[s["slots"] // P, :, s["slots"] % P] = _packed(codes, bits, pool.shape[-1])

    q, k, v = s["qkv"].split([hq, hkv, hkv], 1)
    store((turned(k.double()) / s["lam"].double()) @ _hadamard(torch.float64), s["ck"], c["ks"], c["kb"], s["k_pool"])
    store(v.double(), s["cv"], c["vs"], c["vb"], s["v_pool"])
    return dict(q=turned(q.float()).half(), k_pool=s["k_pool"], v_pool=s["v_pool"])


def _plain_keep(s):
    P, table = s["case"]["page"], s["page_table"].long()
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    base, end, kept = s["seq_lens"].long() - new, s["seq_lens"].long(), s["kept"].long()
    i = torch.arange(s["keep"].shape[1], device=DEV)
    some = i < kept[:, None]
    to, at = (base[:, None] + i)[some], (base[:, None] + s["keep"])[some]
    b = torch.arange(len(base), device=DEV)[:, None].expand(some.shape)[some]
    for pool in (s["k_pool"], s["v_pool"]):
        pool[:, table[b, to // P], :, to % P] = pool[:, table[b, at // P], :, at % P]
    # the pages that are left empty: sequences in order, of each the last one first
    have, need = (end + P - 1) // P, (base + kept + P - 1) // P
    pages = torch.arange(table.shape[1] - 1, -1, -1, device=DEV)
    gone = table.flip(1)[(pages >= need[:, None]) & (pages < have[:, None])]
    n = torch.arange(len(s["free_pages"]), device=DEV) - s["num_free"]
    s["free_pages"].copy_(torch.where((n >= 0) & (n < len(gone)), torch.nn.functional.pad(gone, (0, 1))[n.clamp(0, len(gone))], s["free_pages"]))
    return dict(k_pool=s["k_pool"], v_pool=s["v_pool"], seq_lens=(base + kept).int(), num_free=(s["num_free"] + len(gone)).int(),
                free_pages=s["free_pages"])


# -------------------------------------------------------------------- run ---

def _own(s):
    import bit_vector_quantized_gb300 as vq
    c = s["case"]
    if c["op"] == "append":
        q, k, v = s["qkv"].split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        q = vq.append_kv(s["layout"], s["rotary"], s["positions"], s["slots"], k, v, s["lam"], s["ck"], s["cv"], s["k_pool"], s["v_pool"], q=q)
        return dict(q=q, k_pool=s["k_pool"], v_pool=s["v_pool"])
    if c["op"] == "keep":
        r = vq.keep_tokens(s["layout"], s["seq_lens"], s["cu"], s["keep"], s["kept"], s["page_table"], s["k_pool"], s["v_pool"],
                           s["free_pages"], s["num_free"])
        return dict(k_pool=s["k_pool"], v_pool=s["v_pool"], seq_lens=r.seq_lens, num_free=r.num_free, free_pages=s["free_pages"])
    return vq.tree_attention(s["layout"], s["q"], s["lam"], s["ck"], s["cv"], s["k_pool"], s["v_pool"], s["page_table"], s["seq_lens"],
                             s["max_seq_len"], s["cu"], s["max_new_len"], s["masks"], positions=s["positions"], window=c["window"],
                             num_sinks=c["sinks"], workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"tree": _plain_tree, "append": _plain_append, "keep": _plain_keep}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact ---

def _exact_tree(s):
    """Per sequence and KV head, keys read back into their own space, everything in 64 bits."""
    c = s["case"]
    G, P = c["hq"] // c["hkv"], c["page"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    cu, lens = s["cu"].tolist(), s["seq_lens"].tolist()
    H = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    while H.shape[0] < D:
        H = torch.cat([torch.cat([H, H], 1), torch.cat([H, -H], 1)], 0)
    H = H / D ** 0.5

    def tokens(pool, cb, bits, pages, h, n):
        rows = pool[pages, h].reshape(-1, pool.shape[-1])[:n].long()
        bit = (rows[:, :, None] >> torch.arange(8, device=DEV)) & 1
        bit = bit.reshape(n, -1)[:, :D // cb.shape[1] * bits].reshape(n, -1, bits)
        return cb.double()[(bit << torch.arange(bits, device=DEV)).sum(-1)].reshape(n, D)

    for b in range(c["batch"]):
        n, length = cu[b + 1] - cu[b], lens[b]
        if n == 0:
            continue
        pages = s["page_table"][b, :-(-length // P)].long()
        tree = (s["masks"][cu[b]:cu[b + 1], :, None] >> torch.arange(64, device=DEV) & 1).bool().flatten(1)[:, :n]
        see = torch.cat([torch.ones(n, length - n, dtype=torch.bool, device=DEV), tree], 1)
        at = s["positions"][cu[b]:cu[b + 1]].long()
        of = torch.cat([torch.arange(length - n, device=DEV), at])
        if c["window"]:
            see &= (at[:, None] - of[None] < c["window"]) | (of[None] < c["sinks"])
        for h in range(c["hkv"]):
            k = tokens(s["k_pool"], s["ck"], c["kb"], pages, h, length) @ H * s["lam"][h].double()
            v = tokens(s["v_pool"], s["cv"], c["vb"], pages, h, length)
            for j in range(h * G, (h + 1) * G):
                w = s["q"][cu[b]:cu[b + 1], j].double() @ k.T / D ** 0.5
                out[cu[b]:cu[b + 1], j] = torch.softmax(torch.where(see, w, -math.inf), 1) @ v
    return out


def _exact_turned(s):
    """The queries' pairs as complex numbers, turned by an angle that is reduced before its sine and cosine."""
    c = s["case"]
    r, h = c["rdim"], c["hq"]
    k = np.arange(r // 2, dtype=np.float64)
    base, sc = 500000.0, c["factor"]
    if c["scaling"] == "base" and r > 2:
        base = base * sc ** (r / (r - 2.0))
    f = np.exp(-np.log(base) * 2 * k / r)
    keep = np.ones_like(f)  # 1: kept, 0: divided by the factor
    if c["scaling"] == "linear":
        keep[:] = 0
    elif c["scaling"] == "parts":
        at = lambda turns: r * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), r - 1)
        keep = 1 - np.clip((k - lo) / max(hi - lo, 1e-3), 0, 1)
    elif c["scaling"] == "wavelength":
        keep = np.clip((ORIGINAL * f / (2 * np.pi) - 1) / 3, 0, 1)
    f = torch.from_numpy(f * keep + f / sc * (1 - keep)).to(DEV)
    angle = torch.remainder(s["positions"].double()[:, None] * f, 2 * math.pi)
    turn = torch.polar(torch.full_like(angle, _attention_factor(c)), angle)[:, None]
    q = s["qkv"][:, :h].double()
    if c["interleaved"]:
        q[..., :r] = torch.view_as_real(torch.view_as_complex(q[..., :r].reshape(-1, h, r // 2, 2)) * turn).flatten(-2)
    else:
        z = torch.complex(q[..., :r // 2].contiguous(), q[..., r // 2:r].contiguous()) * turn
        q[..., :r] = torch.cat([z.real, z.imag], -1)
    return q


def exact(case, seed):
    """(Codes and pages are whole numbers: None in their places.)"""
    if case["op"] == "keep":
        return None
    s = prepare(case, seed)
    return _exact_tree(s) if case["op"] == "tree" else dict(q=_exact_turned(s), k_pool=None, v_pool=None)
