"""The serving-step operators around the quantized KV cache: plain forms, calls and cases.

Operators (``op`` of a case):

* ``chunk``   attention of each sequence's newest tokens over its paged codes, causal, optionally
              with a sliding window and first tokens that stay visible;
* ``slots``   page tables, slot map, positions and row offsets from request lengths;
* ``rotary``  rotary positions of q and k out of a fused projection, v carried along.

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

def _chunk(name, batch, hq, hkv, fmt, page, ctx, new, window=0, sinks=0):
    return dict(name=name, op="chunk", batch=batch, hq=hq, hkv=hkv, ks=fmt[0], kb=fmt[1], vs=fmt[2], vb=fmt[3],
                page=page, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0], new_hi=new[1], window=window, sinks=sinks)


def _slots(name, batch, page, ctx, new):
    return dict(name=name, op="slots", batch=batch, page=page, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0], new_hi=new[1])


def _rotary(name, tokens, hq, hkv, dtype, rdim, interleaved, scaling, factor, far):
    return dict(name=name, op="rotary", tokens=tokens, hq=hq, hkv=hkv, dtype=dtype, rdim=rdim, interleaved=interleaved,
                scaling=scaling, factor=factor, far=far)


def listed():
    return [
        # one step of a chunked prompt deep in a 32K context, the Llama layer shape
        _chunk("chunk 2048 in 32K", 1, 32, 8, (4, 8, 4, 8), 256, (30720, 30720), (2048, 2048)),
        # a batch that mixes prompt chunks and single tokens, ragged, small permuted pages
        _chunk("mixed chunks paged 64", 16, 32, 8, (2, 8, 4, 8), 64, (4096, 8192), (1, 509)),
        # checking a few drafted tokens of each sequence, the 40-head layer with 9-bit V codes
        _chunk("5 drafted tokens batch 16", 16, 40, 8, (2, 8, 4, 9), 256, (8000, 16384), (5, 5)),
        # a whole prompt from an empty cache, 1.5-bit codes
        _chunk("prompt of 2049 at 1.5 bit", 1, 32, 8, (8, 12, 8, 12), 256, (0, 0), (2049, 2049)),
        # single tokens of many long sequences, window of 4096 and four sinks
        _chunk("window 4096 batch 64", 64, 40, 8, (2, 8, 4, 9), 256, (9001, 16384), (1, 1), 4096, 4),
        # prompt chunks with a short window and sinks that end inside a page
        _chunk("window 1024 chunks of 1000", 4, 32, 8, (4, 8, 4, 8), 256, (5000, 20011), (777, 1000), 1024, 68),
        # the smallest call: one token of one short conversation
        _chunk("one token window 256", 1, 8, 2, (2, 8, 4, 8), 64, (333, 333), (1, 1), 256, 4),
        # one new token for each sequence of a large decode batch
        _slots("slots 256 decode tokens", 256, 64, (1, 8192), (1, 1)),
        # a step that admits long prompts beside decode tokens
        _slots("slots 120K prompt tokens", 48, 256, (0, 5000), (1, 5001)),
        # one decode step's q, k, v
        _rotary("rotary 64 tokens", 64, 32, 8, "fp16", 128, False, "none", 1.0, 131072),
        # a prompt chunk out of a bf16 projection, half of the head rotated, interleaved pairs
        _rotary("rotary 4099 bf16", 4099, 40, 8, "bf16", 64, True, "linear", 4.0, 32768),
        # a long prompt, frequencies scaled by parts for far positions
        _rotary("rotary 32768 far", 32768, 32, 8, "fp16", 128, False, "parts", 16.0, 1000000),
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    most = max(work(c)["flops"] for c in listed() if c["op"] == "chunk")
    op = rng.choice(["chunk", "chunk", "chunk", "slots", "rotary"])
    if op == "slots":
        lo, new = _log(rng, 1, 4096), _log(rng, 1, 4096)
        c = _slots("", _log(rng, 1, 300), rng.choice([16, 48, 64, 256]), (lo - 1, lo + _log(rng, 1, 4000)), (rng.choice([0, 1]), new))
        while c["batch"] * (c["new_hi"] + 1) > 240000:
            c["new_hi"] = c["new_hi"] * 2 // 3
    elif op == "rotary":
        hkv = rng.choice([1, 2, 8])
        c = _rotary("", _log(rng, 1, 30000), hkv * rng.choice([1, 4, 5]), hkv, rng.choice(["fp16", "bf16"]),
                    rng.choice([128, 96, 64, 32, 2]), rng.random() < 0.5, rng.choice(["none", "linear", "base", "parts", "wavelength"]),
                    rng.choice([2.0, 8.0, 13.5]), _log(rng, 4096, 2000000))
    else:
        hkv, g = rng.choice([(8, 4), (8, 5), (2, 4), (1, 2), (4, 8), (4, 1)])
        fmt = rng.choice([(4, 8, 4, 8), (2, 8, 4, 8), (2, 8, 4, 9), (4, 8, 2, 8), (8, 12, 8, 12)])
        lo, n = _log(rng, 1, 24000), _log(rng, 1, 2048)
        window, sinks = (_log(rng, 1, 8192), rng.choice([0, 1, 4, 65, 500])) if rng.random() < 0.5 else (0, 0)
        c = _chunk("", _log(rng, 1, 48), hkv * g, hkv, fmt, rng.choice([16, 48, 64, 256]), (lo - 1, lo + _log(rng, 1, 8000)),
                   (rng.randint(1, n), n), window, sinks)
        # the plain form holds all scores: the padded batch is kept below the largest listed case
        while c["batch"] * (c["ctx_hi"] + c["new_hi"]) * c["new_hi"] * c["hq"] * 512 > most or c["batch"] * (c["ctx_hi"] + c["new_hi"]) * c["hkv"] > 4_500_000:
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
    """(tokens cached before the step, new tokens) of each sequence."""
    return _spread(c["ctx_lo"], c["ctx_hi"], c["batch"], 7), _spread(c["new_lo"], c["new_hi"], c["batch"], 5)


def _row(sub, bits):
    return (D // sub * bits + 31) // 32 * 4


def work(case):
    if case["op"] == "rotary":
        n = case["tokens"] * D * (case["hq"] + 2 * case["hkv"])
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 3 * case["tokens"] * (case["hq"] + case["hkv"]) * case["rdim"]}
    old, new = _lens(case)
    if case["op"] == "slots":
        taken = -(-(old + new) // case["page"]) - -(-old // case["page"])
        touched = np.where(new > 0, (old + new - 1) // case["page"] - old // case["page"] + 1, 0)
        return {"bytes": int(12 * new.sum() + 8 * taken.sum() + 4 * (touched - taken).clip(0).sum() + 16 * case["batch"]),
                "flops": int(4 * new.sum())}
    pairs, seen = 0, 0
    w, s = case["window"], case["sinks"]
    for o, n in zip(old.tolist(), new.tolist()):
        t = np.arange(o, o + n, dtype=np.int64)
        lo = np.zeros_like(t) if w == 0 else np.maximum(t - w + 1, 0)
        pairs += int((t + 1 - lo + np.minimum(lo, s)).sum())
        if n:
            seen += o + n - int(lo[0]) + min(int(lo[0]), s)
    rows = int(new.sum()) * case["hq"]
    tables = 2 * ((1 << case["kb"]) * case["ks"] + (1 << case["vb"]) * case["vs"]) + 4 * case["hkv"] * D
    return {"bytes": seen * case["hkv"] * (_row(case["ks"], case["kb"]) + _row(case["vs"], case["vb"])) + 4 * rows * D + tables,
            "flops": 4 * D * case["hq"] * pairs}


# ----------------------------------------------------------------- inputs ---

def _pages(c, g):
    """Page tables of all sequences with room for their new tokens, physical pages in a drawn order."""
    old, new = _lens(c)
    need = -(-(old + new) // c["page"])
    total = int(need.sum())
    table = torch.full((c["batch"], max(1, int(need.max()))), -1, dtype=torch.int32, device=DEV)
    col = torch.arange(table.shape[1], device=DEV)
    table[col[None] < torch.from_numpy(need).to(DEV)[:, None]] = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    return table, total


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x.astype(np.int32))).to(DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * scale

    if c["op"] == "rotary":
        dt = torch.float16 if c["dtype"] == "fp16" else torch.bfloat16
        qkv = normal(c["tokens"], c["hq"] + 2 * c["hkv"], D).to(dt)  # a fused projection's output
        start = torch.randint(0, c["far"] - min(c["far"], c["tokens"]) + 1, (1,), generator=g, device=DEV)
        pos = (start + torch.arange(c["tokens"], device=DEV) % c["far"]).to(torch.int32)
        s = dict(case=c, qkv=qkv, positions=pos)
        if own:  # what a program makes once: the frequencies
            import bit_vector_quantized_gb300 as vq
            s["rotary"] = vq.make_rotary(D, c["rdim"], c["interleaved"], 500000.0, c["scaling"], c["factor"], ORIGINAL, 1.0,
                                         32.0 if c["scaling"] == "parts" else 4.0, _attention_factor(c))
        return s
    old, new = _lens(c)
    table, total = _pages(c, g)
    if c["op"] == "slots":
        have = torch.from_numpy(-(-old // c["page"])).to(DEV)
        mine = torch.arange(table.shape[1], device=DEV)[None] < have[:, None]
        free = table[(table >= 0) & ~mine]
        free = torch.cat([torch.arange(total, total + 37, device=DEV, dtype=torch.int32), free])
        free = free[torch.randperm(len(free), generator=g, device=DEV)]
        table[~mine] = -1
        return dict(case=c, seq_lens=_i32(old), new_lens=_i32(new), page_table=table, free_pages=free, num_pages=total + 37,
                    num_free=torch.tensor([len(free)], dtype=torch.int32, device=DEV), max_tokens=int(new.sum()) + 5)
    # keys with a few strong channels: smoothing factors near 2, near 9 for those channels; the
    # smoothed and transformed keys, and with them their centroids, are near N(0, 0.6^2)
    lam = 2.0 + 0.1 * normal(c["hkv"], D).abs()
    lam[:, torch.randperm(D, generator=g, device=DEV)[:4]] *= 4.5
    pool = lambda row: torch.randint(0, 256, (total, c["hkv"], c["page"], row), generator=g, device=DEV, dtype=torch.uint8)  # noqa: E731
    tokens = int(new.sum())
    s = dict(case=c, page_table=table, lam=lam,
             ck=normal(1 << c["kb"], c["ks"], scale=0.6).half(), cv=normal(1 << c["vb"], c["vs"]).half(),
             k_pool=pool(_row(c["ks"], c["kb"])), v_pool=pool(_row(c["vs"], c["vb"])),
             q=normal(tokens, c["hq"], D).half(), seq_lens=_i32(old + new), cu=_i32(np.concatenate([[0], np.cumsum(new)])),
             max_seq_len=int((old + new).max()), max_new_len=int(new.max()))
    if own:  # what a program makes once: the layout and the workspace of its largest step
        import bit_vector_quantized_gb300 as vq
        s["layout"] = vq.make_layout(D, c["hq"], c["hkv"], c["ks"], c["kb"], c["vs"], c["vb"], c["page"])
        s["workspace"] = vq.alloc_chunk_workspace(s["layout"], c["batch"], tokens, s["max_seq_len"], s["max_new_len"])
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


def _hadamard(dtype):
    i = torch.arange(D, device=DEV)
    x = i[:, None] & i[None]
    x = x ^ x >> 4
    x = x ^ x >> 2
    x = x ^ x >> 1
    return (1 - 2 * (x & 1)).to(dtype) / math.sqrt(D)


def _plain_chunk(s):
    c = s["case"]
    B, hkv, G, P = c["batch"], c["hkv"], c["hq"] // c["hkv"], c["page"]
    L, N = s["max_seq_len"], s["max_new_len"]
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    p = torch.arange(L, device=DEV)
    page = s["page_table"][:, p // P].long().clamp(min=0)

    def read(pool, cb, sub, bits):
        x = cb.float()[_codes(pool[page, :, (p % P)[None].expand(B, L)], D // sub, bits)]
        return x.reshape(B, L, hkv, D).transpose(1, 2)  # [B][Hkv][L][D]

    i = torch.arange(N, device=DEV)
    row = (s["cu"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    qt = (s["q"].float().reshape(-1, hkv, G, D) * s["lam"][:, None]) @ _hadamard(torch.float32)
    qt = qt[row].permute(0, 2, 1, 3, 4).reshape(B, hkv, N * G, D)
    x = qt @ read(s["k_pool"], s["ck"], c["ks"], c["kb"]).transpose(2, 3)
    x = x.mul_(1 / math.sqrt(D)).view(B, hkv, N, G, L)
    t = (s["seq_lens"].long() - new)[:, None] + i  # positions of the new tokens [B][N]
    hidden = p > t[..., None]
    if c["window"]:
        hidden |= (p <= t[..., None] - c["window"]) & (p >= c["sinks"])
    x = x.masked_fill_(hidden[:, None, :, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    o = x.view(B, hkv, N * G, L) @ read(s["v_pool"], s["cv"], c["vs"], c["vb"])
    o = o.view(B, hkv, N, G, D) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(B, N, c["hq"], D)
    return o[i[None] < new[:, None]].half()


def _plain_slots(s):
    P, table = s["case"]["page"], s["page_table"]
    old, new, T = s["seq_lens"].long(), s["new_lens"].long(), s["max_tokens"]
    have, need = (old + P - 1) // P, (old + new + P - 1) // P
    take = need - have
    first = take.cumsum(0) - take
    col = torch.arange(table.shape[1], device=DEV)
    j = col[None] - have[:, None]
    at = s["num_free"].long() - 1 - (first[:, None] + j)
    table.copy_(torch.where((j >= 0) & (j < take[:, None]), s["free_pages"][at.clamp(0, len(s["free_pages"]) - 1)], table))
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    tok = torch.arange(T, device=DEV)
    b = (torch.searchsorted(cu, tok, right=True) - 1).clamp(max=len(old) - 1)
    pos = old[b] + tok - cu[b]
    real = tok < cu[-1]
    pos = torch.where(real, pos, 0)
    slot = table[b, pos // P].long() * P + pos % P
    return dict(page_table=table, seq_lens=(old + new).int(), num_free=(s["num_free"] - take.sum()).int(), cu_new_lens=cu.int(),
                slots=torch.where(real, slot, -1), positions=torch.where(real, pos, -1).int())


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


def _plain_rotary(s):
    c = s["case"]
    r, hq, hkv = c["rdim"], c["hq"], c["hkv"]
    angle = s["positions"].double()[:, None] * _frequencies(c)
    m = _attention_factor(c)
    co, si = (angle.cos() * m).float()[:, None], (angle.sin() * m).float()[:, None]
    x = s["qkv"].float()
    qk, rest = x[:, :hq + hkv, :r], x[:, :hq + hkv, r:]
    a, b = (qk[..., 0::2], qk[..., 1::2]) if c["interleaved"] else (qk[..., :r // 2], qk[..., r // 2:])
    y = (a * co - b * si, b * co + a * si)
    y = torch.stack(y, -1).flatten(-2) if c["interleaved"] else torch.cat(y, -1)
    y = torch.cat([y, rest], -1).half()
    return y[:, :hq].contiguous(), y[:, hq:].contiguous(), x[:, hq + hkv:].half()


# -------------------------------------------------------------------- run ---

def _own(s):
    import bit_vector_quantized_gb300 as vq
    c = s["case"]
    if c["op"] == "rotary":
        q, k, v = s["qkv"].split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        return vq.rotary(s["rotary"], s["positions"], q, k, v)
    if c["op"] == "slots":
        r = vq.append_slots(s["seq_lens"], s["new_lens"], s["page_table"], s["free_pages"], s["num_free"], c["page"],
                            s["num_pages"], s["max_tokens"])
        return dict(page_table=s["page_table"], seq_lens=r.seq_lens, num_free=r.num_free, cu_new_lens=r.cu_new_lens,
                    slots=r.slot_mapping, positions=r.positions)
    return vq.chunk_attention(s["layout"], s["q"], s["lam"], s["ck"], s["cv"], s["k_pool"], s["v_pool"], s["page_table"],
                              s["seq_lens"], s["max_seq_len"], s["cu"], s["max_new_len"], window=c["window"],
                              num_sinks=c["sinks"], workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"chunk": _plain_chunk, "slots": _plain_slots, "rotary": _plain_rotary}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact ---

def _exact_chunk(s):
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
        t = torch.arange(length - n, length, device=DEV)[:, None]
        p = torch.arange(length, device=DEV)[None]
        see = p <= t
        if c["window"]:
            see &= (t - p < c["window"]) | (p < c["sinks"])
        for h in range(c["hkv"]):
            k = tokens(s["k_pool"], s["ck"], c["kb"], pages, h, length) @ H * s["lam"][h].double()
            v = tokens(s["v_pool"], s["cv"], c["vb"], pages, h, length)
            for j in range(h * G, (h + 1) * G):
                w = s["q"][cu[b]:cu[b + 1], j].double() @ k.T / D ** 0.5
                out[cu[b]:cu[b + 1], j] = torch.softmax(torch.where(see, w, -math.inf), 1) @ v
    return out


def _exact_rotary(s):
    """Pairs as complex numbers, turned by an angle that is reduced before its sine and cosine."""
    c = s["case"]
    r, h = c["rdim"], c["hq"] + c["hkv"]
    x = s["qkv"].double()
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
    qk = x[:, :h].clone()
    if c["interleaved"]:
        qk[..., :r] = torch.view_as_real(torch.view_as_complex(qk[..., :r].reshape(-1, h, r // 2, 2)) * turn).flatten(-2)
    else:
        z = torch.complex(qk[..., :r // 2].contiguous(), qk[..., r // 2:r].contiguous()) * turn
        qk[..., :r] = torch.cat([z.real, z.imag], -1)
    return qk[:, :c["hq"]], qk[:, c["hq"]:], x[:, h:]


def exact(case, seed):
    if case["op"] == "slots":
        return None
    s = prepare(case, seed)
    return _exact_rotary(s) if case["op"] == "rotary" else _exact_chunk(s)
