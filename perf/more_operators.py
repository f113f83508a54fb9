"""New tokens on their way into the cache, and caches held in 4 bits: the cases
they are measured on, their plain forms, and the calls a user makes.

Three operators on the library's cache descriptor (contiguous slices or block
pools, one row count per slice):

  append   the keys and values of a chunk of new tokens (views of a fused
           projection's output) go behind the rows of their slices, keys and
           queries rotated at the tokens' positions on the way (one position, or
           several axes that share the bands between them); a 4-bit cache's rows
           are then read back, as the values they stand for;
  decode   one new token per sequence attends the rows of a 4-bit cache
           (optionally the first n_sink rows and the newest `window`), optionally
           adding every row's weight to its accumulated mass;
  prefill  a chunk of new tokens (the newest rows of a 4-bit cache) attends
           causally, optionally windowed with sinks.

A row of a 4-bit cache is d / 2 bytes of codes and four pairs (scale, minimum) in
fp16, one for each quarter of its elements: element e of quarter j is minimum_j +
scale_j * code_e. With min and max of a quarter (magnitudes above 30656 count as
that), minimum = fp16(min), scale = fp16(max(0, max - minimum) / 15), code =
(x - minimum) / scale to the nearest whole number (ties to even), within 0 .. 15.

Row counts, chunk lengths and block tables' sizes follow from the case alone;
every value (queries, keys, values, masses, which block holds what) comes from
the seed. Keys and queries are drawn as per-head centres of norm 8 plus unit
noise, rotated at their positions where a cache holds them already.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "q4": torch.bfloat16}
THETA = 1e6
NEG = float("-inf")
MOST = 30656.0  # largest magnitude of a 4-bit row


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _append(name, n_seq, heads, group, d, dtype, rows, n_new, ragged=False, block=0, half=False, axes=""):
    return {"name": name, "op": "append", "n_seq": n_seq, "heads": heads, "group": group, "d": d, "dtype": dtype, "rows": rows, "n_new": n_new,
            "ragged": ragged, "block": block, "half": half, "axes": axes}


def _decode(name, n_seq, heads, group, d, rows, ragged=False, block=0, n_sink=0, window=0, mass=False):
    return {"name": name, "op": "decode", "n_seq": n_seq, "heads": heads, "group": group, "d": d, "dtype": "q4", "rows": rows, "ragged": ragged,
            "block": block, "n_sink": n_sink, "window": window, "mass": mass}


def _prefill(name, n_seq, heads, group, d, rows, n_new, ragged=False, block=0, n_sink=0, window=0):
    return {"name": name, "op": "prefill", "n_seq": n_seq, "heads": heads, "group": group, "d": d, "dtype": "q4", "rows": rows, "n_new": n_new,
            "ragged": ragged, "block": block, "n_sink": n_sink, "window": window}


def listed():
    return [
        # the tiny configuration's cache, fp32: one token, the shortest call
        _append("append tiny fp32", 1, 2, 1, 64, "fp32", 512, 1),
        # one token of each of 16 sequences whose heads were compressed to different lengths, in an engine's block pool
        _append("append decode paged", 16, 8, 4, 128, "bf16", 4096, 1, ragged=True, block=64),
        # a whole prompt of the layer shape, the rotation in halves
        _append("append prompt", 1, 8, 4, 128, "bf16", 0, 8192, half=True),
        # video frames between text in a padded batch: three axes, each with a run of the bands
        _append("append video", 4, 8, 4, 128, "bf16", 513, 2048, ragged=True, block=16, half=True, axes="sections"),
        # a prompt into a 4-bit cache in a block pool
        _append("append prompt q4", 1, 8, 4, 128, "q4", 0, 8192, block=64),
        # image patches behind short caches in 4 bits: the bands take turns at two axes
        _append("append image q4", 16, 8, 1, 64, "q4", 97, 577, ragged=True, axes="turns"),
        # one layer of the Qwen3-8B-shaped model, one user, a cache between two evictions
        _decode("decode layer q4", 1, 8, 4, 128, 2113),
        # one layer of the 16-sequence stack before its first eviction, in an engine's block pool
        _decode("decode stack paged q4", 16, 8, 4, 128, 32768, block=64),
        # the large batch of periodically compressed caches, heads of different lengths, weights accumulated for the next eviction
        _decode("decode periodic mass q4", 64, 8, 1, 64, 2176, ragged=True, mass=True),
        # a follow-up question of odd length on a compressed cache
        _prefill("prefill follow-up q4", 1, 8, 4, 128, 2176, 131),
        # the second part of a long prompt
        _prefill("prefill part q4", 1, 8, 4, 128, 8192, 4096),
        # a padded batch of prompts with sinks and a window, block pool, the periodic model's head size
        _prefill("prefill sinks batch q4", 8, 8, 2, 64, 4096, 4096, ragged=True, block=64, n_sink=4, window=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "prefill"])
    d = rng.choice([64, 128])
    block = rng.choice([0, 0, 16, 64, 256])
    n_sink, window = (rng.choice([0, 1, 4, 130]), _log(rng, 16, 8192)) if rng.random() < 0.4 else (0, 0)
    ragged = rng.random() < 0.5
    heads, group = rng.choice([1, 2, 8]), rng.choice([1, 2, 3, 4, 7, 8])
    if op == "append":
        dtype = rng.choice(["bf16", "bf16", "fp32", "q4", "q4"])
        n_new = _log(rng, 1, 8192)
        rows = _log(rng, 1, 4096) - 1
        n_seq = max(1, min(_log(rng, 1, 64), 8192 * 48 // (n_new * heads * (group + 2)), 16 * 8 * 4096 // (heads * (rows + n_new))))
        c = _append("", n_seq, heads, group, d, dtype, rows, n_new, ragged, block, rng.random() < 0.5, rng.choice(["", "", "sections", "turns"]))
        most = work(listed()[2])["bytes"]
        while work(c)["bytes"] > most:  # (a single token of one sequence is far below)
            key = max(("n_seq", "n_new", "rows"), key=lambda x: c[x] if x != "n_seq" else 64 * (c[x] - 1))
            c[key] = c[key] * 2 // 3
    elif op == "decode":
        rows = _log(rng, 16, 32768)
        n_seq = max(1, min(_log(rng, 1, 64), 15 * 8 * 32768 // (heads * rows)))
        c = _decode("", n_seq, heads, group, d, rows, ragged, block, n_sink, window, rng.random() < 0.5)
    else:
        n_new = _log(rng, 1, 6000)
        rows = max(n_new, _log(rng, 64, 16384))
        most = 8192 * 8192 * 32 // 4
        n_seq = max(1, min(_log(rng, 1, 16), most // (heads * group * n_new * rows)))
        while heads * group * n_new * rows > most:
            n_new = (n_new + 1) // 2
        c = _prefill("", n_seq, heads, group, d, rows, n_new, ragged, block, n_sink, window)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# sizes that follow from the case
# --------------------------------------------------------------------------
def _cap(c):
    """Rows a slice can hold: room for a round of 128 more (and for the chunk), in whole blocks."""
    unit = max(c["block"], 16)
    return (c["rows"] + (c["n_new"] if c["op"] == "append" else 0) + 128 + unit - 1) // unit * unit


def _lengths(c):
    """Cached rows of every (sequence, head) before an append, or with the new ones: equal, or spread."""
    B, H, n = c["n_seq"], c["heads"], c["rows"]
    if not c["ragged"]:
        return [[n] * H for _ in range(B)]
    if c["op"] == "prefill":
        return [[max(1, n - (577 * b) % (n // 2 + 1))] * H for b in range(B)]
    # heads differ: each was compressed to its own rows
    spread = [(0 if B * H > 8 and (b, h) == (B // 2, 0) else max(min(n, 1), n - (577 * (b * H + h) + 131 * b) % (n // 2 + 1))) for b in range(B) for h in range(H)]
    return [spread[b * H:(b + 1) * H] for b in range(B)]


def _news(c):
    """New tokens of every sequence of a chunk."""
    n_new, B = c["n_new"], c["n_seq"]
    short = [n_new - (311 * b) % (n_new // 2 + 1) if c["ragged"] else n_new for b in range(B)]
    if c["op"] == "append":
        return short
    return [max(1, min(x, row[0])) for x, row in zip(short, _lengths(c))]


def _band_axis(c):
    """Which axis of the positions rotates each band, or None for one position."""
    F = c["d"] // 2
    if c["axes"] == "sections":  # time, height, width: a quarter and two times three eighths
        return [0] * (F // 4) + [1] * (3 * F // 8) + [2] * (3 * F // 8)
    if c["axes"] == "turns":  # height, width
        return [f % 2 for f in range(F)]
    return None


def _visible(r, n_sink, window):
    """How many rows the query at row r sees."""
    if r < 0:
        return 0
    if window == 0 or r + 1 <= window:
        return r + 1
    lo = r + 1 - window
    return window + min(n_sink, lo)


def _row_bytes(c):
    return c["d"] // 2 + 16 if c["dtype"] == "q4" else c["d"] * (2 if c["dtype"] == "bf16" else 4)


def work(c):
    d, H, G, lens, rb = c["d"], c["heads"], c["group"], _lengths(c), _row_bytes(c)
    e = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "append":
        new = sum(_news(c))
        axes = max(_band_axis(c) or [0]) + 1
        tokens = new * ((2 * H + 2 * H * G) * d * e + H * (2 * rb + 4) + 4 * axes)  # rows in and out, positions
        back = 0
        if c["dtype"] == "q4":  # all rows, read back
            back = sum(n + x for row, x in zip(lens, _news(c)) for n in row) * (2 * rb + 2 * d * 2)
        return {"bytes": tokens + back, "flops": 3 * d * H * (G + 1) * new}
    if c["op"] == "decode":
        seen = sum(_visible(n - 1, c["n_sink"], c["window"]) for row in lens for n in row)
        io = c["n_seq"] * H * G * (2 * d * 2 + 4)
        return {"bytes": seen * (2 * rb + (8 if c["mass"] else 0)) + io, "flops": 4 * d * G * seen}
    pairs, rows = 0, 0
    for row, new in zip(lens, _news(c)):
        n = row[0]
        pairs += H * G * sum(_visible(r, c["n_sink"], c["window"]) for r in range(n - new, n))
        first = max(0, n - new + 1 - c["window"]) if c["window"] else 0
        rows += H * (n - first + min(first, c["n_sink"]))
    q = sum(_news(c)) * H * G
    return {"bytes": rows * 2 * rb + q * (2 * d * 2 + 4), "flops": 4 * d * pairs}


# --------------------------------------------------------------------------
# rows in 4 bits
# --------------------------------------------------------------------------
def _half(x):
    """fp64 to the nearest fp16 value (ties to even), rounded once; |x| < 65504."""
    e = torch.frexp(x)[1].long() - 1
    step = ((torch.clamp(e, min=-14) - 10 + 1023) << 52).view(torch.float64)
    return torch.round(x / step) * step


def _place(codes, d):
    """Codes of a row's elements [..., d] in the order of the row's nibbles. A row is read by four lanes, each with a
    run of its chunks, so a lane's codes of all four quarters are next to each other."""
    if d == 128:  # (quarter, lane, code) -> (lane, quarter, code)
        return codes.unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-3)
    # (half, quarter of it, lane, pair, code) -> (lane, half, pair, quarter of it, code)
    return codes.unflatten(-1, (2, 2, 4, 2, 2)).movedim(-3, -5).transpose(-3, -2).flatten(-5)


def _unplace(nibbles, d):
    if d == 128:
        return nibbles.unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-3)
    return nibbles.unflatten(-1, (4, 2, 2, 2, 2)).transpose(-3, -2).movedim(-5, -3).flatten(-5)


def _pack(x):
    """Rows [..., d] as a 4-bit cache holds them, uint8 [..., d / 2 + 16], in x's precision (fp64: to the letter)."""
    d = x.shape[-1]
    g = x.clamp(-MOST, MOST).unflatten(-1, (4, d // 4))
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    exact64 = x.dtype == torch.float64
    low = _half(low) if exact64 else low.half().to(x.dtype)
    scale = (high - low).clamp(min=0) / 15
    scale = _half(scale) if exact64 else scale.half().to(x.dtype)
    c = torch.round((g - low) / torch.where(scale > 0, scale, 1.0)).clamp(0, 15)
    c = torch.where(scale > 0, c, 0.0).to(torch.uint8).flatten(-2)
    n = _place(c, d)
    pairs = torch.cat((scale, low), -1).half().flatten(-2).contiguous()  # [..., 4 * (scale, minimum)]
    return torch.cat((n[..., 0::2] | (n[..., 1::2] << 4), pairs.view(torch.uint8)), -1)


def _values(rows, dtype=torch.float32):
    """What 4-bit rows stand for."""
    d = (rows.shape[-1] - 16) * 2
    codes, pairs = rows[..., :d // 2], rows[..., d // 2:].contiguous().view(torch.float16).to(dtype)
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    c = _unplace(n, d).to(dtype).unflatten(-1, (4, d // 4))
    return (pairs[..., 1::2, None] + pairs[..., 0::2, None] * c).flatten(-2)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _rotate(x, pos, half=False, band_axis=None, dtype=torch.float64):
    """x [..., n, d] at positions pos [n] (or [n, axes]), computed in `dtype` from fp64 angles."""
    d = x.shape[-1]
    F = d // 2
    f = torch.arange(F, dtype=torch.float64, device=x.device)
    at = pos.double()[:, None] if pos.dim() == 1 else pos.double()[:, torch.tensor(band_axis or [0] * F, device=x.device)]
    ang = at * THETA ** (-2.0 * f / d)
    cs, sn = torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)
    x = x.to(dtype)
    a, b = (x[..., :F], x[..., F:]) if half else (x[..., 0::2], x[..., 1::2])
    u, v = a * cs - b * sn, a * sn + b * cs
    return torch.cat((u, v), dim=-1) if half else torch.stack((u, v), dim=-1).flatten(-2)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _centres(g, *shape):
    x = _normal(g, *shape)
    return x * (8.0 / x.norm(dim=-1, keepdim=True))


def _store(c, table, rows):
    """Rows [n_seq, 1, heads, cap, width] as the cache holds them: the slices themselves, or a pool with its table."""
    if table is None:
        return rows.contiguous()
    B, L, H, cap, w = rows.shape
    bs = c["block"]
    per = cap // bs
    pool = torch.zeros(B * per + 2, L, H, bs, w, dtype=rows.dtype, device="cuda")
    pool[table.view(-1).long()] = rows.view(B, L, H, per, bs, w).permute(0, 3, 1, 2, 4, 5).reshape(B * per, L, H, bs, w)
    return pool


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, B, H, G, d, cap = DTYPES[c["dtype"]], c["n_seq"], c["heads"], c["group"], c["d"], _cap(c)
    q4 = c["dtype"] == "q4"
    half = c.get("half", False)
    mu, mu_q = _centres(g, H, 1, d), _centres(g, H, G, d)
    pos = torch.arange(cap, device="cuda")
    k, v = (torch.empty(B, 1, H, cap, d // 2 + 16 if q4 else d, dtype=torch.uint8 if q4 else dt, device="cuda") for _ in range(2))
    for b in range(B):
        kb, vb = _rotate(mu + _normal(g, H, cap, d), pos, half, dtype=torch.float32), _normal(g, H, cap, d)
        k[b, 0], v[b, 0] = (_pack(kb), _pack(vb)) if q4 else (kb.to(dt), vb.to(dt))
    table = None
    if c["block"]:
        per = cap // c["block"]
        table = torch.randperm(B * per + 2, generator=g, device="cuda")[:B * per].view(B, per).to(torch.int32)
    k, v = _store(c, table, k), _store(c, table, v)
    lens = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")  # [B, H]
    st = {"case": dict(c), "k": k, "v": v, "table": table, "cap": cap, "n_valid": lens.flatten().contiguous()}
    if c["op"] == "append":
        n_q, Hq = max(_news(c)), H * G
        x = torch.empty(B, n_q, (Hq + 2 * H) * d, dtype=dt, device="cuda")  # the fused projection's output
        for b in range(B):
            x[b, :, :Hq * d] = (mu_q.view(1, H, G, d) + _normal(g, n_q, H, G, d)).view(n_q, Hq * d).to(dt)
            x[b, :, Hq * d:(Hq + H) * d] = (mu.view(1, H, d) + _normal(g, n_q, H, d)).view(n_q, H * d).to(dt)
            x[b, :, (Hq + H) * d:] = _normal(g, n_q, H * d).to(dt)
        i = torch.arange(n_q, device="cuda")
        first = (torch.randint(0, 30000, (B, 1), generator=g, device="cuda") if c["rows"] else torch.zeros(B, 1, dtype=torch.long, device="cuda"))
        axes = _band_axis(c)
        if axes is None:
            at = (first + i)[..., None]
        else:  # seven tokens of text, then frames of 16 x 24 patches
            j = (i - 7).clamp(min=0)
            t, y, z = (torch.where(i < 7, i, 7 + u) for u in (j // 384, j // 24 % 16, j % 24))
            at = first[..., None] + torch.stack((t, y, z) if max(axes) == 2 else (y, z), -1)
        st.update(x=x, positions=at.to(torch.int32).contiguous(), rows=st["n_valid"].clone(), band_axis=axes,
                  news=torch.tensor(_news(c), dtype=torch.int32, device="cuda"), pos=torch.zeros(B * H, cap, dtype=torch.int32, device="cuda"),
                  q_out=torch.zeros(B, n_q, Hq, d, dtype=dt, device="cuda"))
        if q4:
            st["k_read"], st["v_read"] = (torch.zeros(B, H, cap, d, dtype=dt, device="cuda") for _ in range(2))
        return st
    # a program keeps one scratch buffer for its calls
    st["scratch"] = torch.empty((64 << 20) + 4 * B * H * cap * max(G, d + 1), dtype=torch.uint8, device="cuda")
    if c["op"] == "decode":
        q = mu_q + _normal(g, B, H, G, d)
        st["q"] = torch.stack([_rotate(q[b].reshape(H * G, 1, d), lens[b, :1] - 1, dtype=torch.float32)[:, 0] for b in range(B)]).to(dt)
        st["out"] = torch.zeros_like(st["q"])  # [B, Hq, d]
        st["lse"] = torch.zeros(B, H * G, device="cuda")
        if c["mass"]:
            st["mass"] = torch.rand(B * H, cap, generator=g, device="cuda")  # what earlier tokens gave
        return st
    n_q = max(_news(c))
    news = torch.tensor(_news(c), dtype=torch.int32, device="cuda")
    q = torch.empty(B, n_q, H * G, d, dtype=dt, device="cuda")
    for b in range(B):
        r = torch.arange(n_q, device="cuda") + (lens[b, 0] - news[b])
        q[b] = _rotate((mu_q + _normal(g, n_q, H, G, d)).view(n_q, H * G, d).transpose(0, 1), r, dtype=torch.float32).transpose(0, 1).to(dt)
    st.update(q=q, n_new=news, out=torch.zeros_like(q), lse=torch.zeros(B, n_q, H * G, device="cuda"))
    return st


def _rows(st, pool, n):
    """The cache's first n rows in order: [n_seq, heads, n, width] of its one layer."""
    if st["table"] is None:
        return pool[:, 0, :, :n]
    B, per = st["table"].shape
    t = pool[st["table"].long()][:, :, 0]  # [B, per, H, bs, width]
    return t.permute(0, 2, 1, 3, 4).reshape(B, t.shape[2], -1, t.shape[4])[:, :, :n]


def _split(st):
    """Queries, keys and values of the new tokens, [n_seq, n_q, heads, d] views of the projection's output."""
    c, x = st["case"], st["x"]
    H, Hq, d = c["heads"], c["heads"] * c["group"], c["d"]
    q, k, v = x.split((Hq * d, H * d, H * d), dim=-1)
    return q.unflatten(-1, (Hq, d)), k.unflatten(-1, (H, d)), v.unflatten(-1, (H, d))


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _plain_append(st):
    c = st["case"]
    B, H, q4 = c["n_seq"], c["heads"], c["dtype"] == "q4"
    q, k, v = _split(st)
    real = torch.float64 if q4 else torch.float32  # (which code is nearest is decided at a border)
    st["n_valid"].copy_(st["rows"])
    base = st["n_valid"].view(B, H)
    for b, n in enumerate(_news(c)):
        at = st["positions"][b, :n]
        st["q_out"][b, :n] = _rotate(q[b, :n].transpose(0, 1), at, c["half"], st["band_axis"], torch.float32).transpose(0, 1).to(q.dtype)
        kb = _rotate(k[b, :n].transpose(0, 1), at, c["half"], st["band_axis"], real)  # [H, n, d]
        vb = v[b, :n].transpose(0, 1).to(real)
        kb, vb = (_pack(kb), _pack(vb)) if q4 else (kb.to(k.dtype), vb.to(v.dtype))
        r = base[b, :, None].long() + torch.arange(n, device="cuda")  # [H, n]
        h = torch.arange(H, device="cuda")[:, None]
        if st["table"] is None:
            st["k"][b, 0, h, r], st["v"][b, 0, h, r] = kb, vb
        else:
            blk = st["table"][b].long()[r // c["block"]]
            st["k"][blk, 0, h, r % c["block"]], st["v"][blk, 0, h, r % c["block"]] = kb, vb
        st["pos"].view(B, H, -1)[b].scatter_(1, r, at[:, 0].expand(H, n))
    st["n_valid"] += st["news"][:, None].expand(B, H).flatten()
    if q4:
        seen = (torch.arange(st["cap"], device="cuda") < st["n_valid"].view(B, H, 1))[..., None]
        for pool, out in (("k", "k_read"), ("v", "v_read")):
            x = _values(_rows(st, st[pool], st["cap"])).to(torch.bfloat16)
            torch.where(seen, x, st[out], out=st[out])
    return _appended(st)


def _appended(st):
    out = {"q": st["q_out"], "n_valid": st["n_valid"], "pos": st["pos"]}
    if st["case"]["dtype"] == "q4":
        return {**out, "k": st["k_read"], "v": st["v_read"]}
    return {**out, "k": st["k"], "v": st["v"]}


def _softmax(s, seen):
    """Weights, and log of their sum, over the visible entries; nothing visible: zeros and -inf."""
    s = torch.where(seen, s, NEG)
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == NEG, 0.0, m)
    p = torch.exp(s - m0)
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l > 0, l, 1.0), (m0 + torch.log(l)).squeeze(-1)


def _plain_decode(st):
    c = st["case"]
    B, H, G, d = c["n_seq"], c["heads"], c["group"], c["d"]
    k, v = (_values(_rows(st, st[x], c["rows"])) for x in ("k", "v"))
    n = st["n_valid"].view(B, H, 1)
    j = torch.arange(c["rows"], device="cuda")
    seen = j < n
    if c["window"]:
        seen &= (j < c["n_sink"]) | (j >= n - c["window"])
    p, lse = _softmax(st["q"].view(B, H, G, d).float() @ k.transpose(-1, -2) * d ** -0.5, seen[:, :, None])
    out = {"out": (p @ v).to(st["q"].dtype).view(B, H * G, d), "lse": lse.view(B, H * G)}
    if c["mass"]:
        st["mass"][:, :c["rows"]] += p.sum(2).view(B * H, -1)
        out["mass"] = st["mass"]
    return out


def _plain_prefill(st):
    c = st["case"]
    B, H, G, d = c["n_seq"], c["heads"], c["group"], c["d"]
    k, v = (_values(_rows(st, st[x], c["rows"])) for x in ("k", "v"))
    n_q = st["q"].shape[1]
    base = st["n_valid"].view(B, H) - st["n_new"][:, None]
    r = base[:, :, None, None] + torch.arange(n_q, device="cuda")[:, None]
    j = torch.arange(c["rows"], device="cuda")
    seen = j <= r  # [B, H, n_q, rows]
    if c["window"]:
        seen &= (j < c["n_sink"]) | (j > r - c["window"])
    q = st["q"].view(B, n_q, H, G, d).permute(0, 2, 3, 1, 4).float()  # [B, H, G, n_q, d]
    p, lse = _softmax(q @ k[:, :, None].transpose(-1, -2) * d ** -0.5, seen[:, :, None])
    o = (p @ v[:, :, None]).permute(0, 3, 1, 2, 4).reshape(B, n_q, H * G, d).to(st["q"].dtype)
    live = (torch.arange(n_q, device="cuda") < st["n_new"][:, None])[:, :, None]
    lse = lse.permute(0, 3, 1, 2).reshape(B, n_q, H * G)
    return {"out": torch.where(live[..., None], o, st["out"]), "lse": torch.where(live, lse, st["lse"])}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _own(st):
    import kv_cache_compression_tri_gb300 as tri
    c = st["case"]
    if st["table"] is None:
        kv = tri.KVCache(st["k"], st["v"], st["n_valid"], st.get("pos"), None, post_rope=True)
    else:
        kv = tri.PagedKVCache(st["k"], st["v"], st["table"], st["n_valid"], st.get("pos"), None, post_rope=True)
    if c["op"] == "append":
        q, k, v = _split(st)
        st["n_valid"].copy_(st["rows"])  # the rows a step starts from
        tri.append(kv, 0, k, v, st["positions"], THETA, q=q, q_out=st["q_out"], n_new=st["news"], band_axis=st["band_axis"],
                   style=tri.ROPE_HALF if c["half"] else tri.ROPE_INTERLEAVED)
        if c["dtype"] == "q4":
            tri.read_rows(kv, 0, st["k_read"], st["v_read"])
        return _appended(st)
    if c["op"] == "decode":
        tri.attn_decode(kv, 0, st["q"], st["out"], n_sink=c["n_sink"], window=c["window"], lse=st["lse"], mass=st.get("mass"), workspace=st["scratch"])
        out = {"out": st["out"], "lse": st["lse"]}
        if c["mass"]:
            out["mass"] = st["mass"]
        return out
    if "chunk_scratch" not in st:  # (a size that the library tells; kept like the other)
        st["chunk_scratch"] = torch.empty(tri.attn_prefill_workspace_bytes(kv), dtype=torch.uint8, device="cuda")
    tri.attn_prefill(kv, 0, st["q"], st["out"], n_new=st["n_new"], n_sink=c["n_sink"], window=c["window"], lse=st["lse"], workspace=st["chunk_scratch"])
    return {"out": st["out"], "lse": st["lse"]}


def run(st):
    if own:
        return _own(st)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}[st["case"]["op"]](st)


# --------------------------------------------------------------------------
# the definitions in 64 bits, slice by slice
# --------------------------------------------------------------------------
def _code_row(d):
    """Where the nibble of each element is: (byte, shift)."""
    where = []
    for e in range(d):
        j, i = divmod(e, d // 4)
        t, s = divmod(i, d // 16)
        nib = (4 * t + j) * 8 + s if d == 128 else (2 * t + j // 2) * 8 + 4 * (s // 2) + 2 * (j % 2) + s % 2
        where.append((nib // 2, 4 * (nib % 2)))
    return where


def _numbers64(rows):
    """Values of 4-bit rows, numpy [..., d / 2 + 16] to fp64 [..., d]."""
    d = (rows.shape[-1] - 16) * 2
    pairs = np.ascontiguousarray(rows[..., d // 2:]).view(np.float16).astype(np.float64)
    byte, shift = (np.array(x) for x in zip(*_code_row(d)))
    codes = (rows[..., byte] >> shift.astype(np.uint8)) & 15
    quarter = np.arange(d) * 4 // d
    return pairs[..., 2 * quarter + 1] + pairs[..., 2 * quarter] * codes


def _rounded64(x):
    """fp64 rows [..., d], numpy: the values that their 4-bit rows stand for."""
    d = x.shape[-1]
    out = np.empty_like(x)
    for a in range(0, d, d // 4):
        part = np.clip(x[..., a:a + d // 4], -MOST, MOST)
        low = part.min(-1, keepdims=True).astype(np.float16).astype(np.float64)  # (numpy rounds once)
        scale = (np.maximum(part.max(-1, keepdims=True) - low, 0) / 15).astype(np.float16).astype(np.float64)
        code = np.rint(np.divide(part - low, scale, out=np.zeros_like(part), where=scale > 0))
        out[..., a:a + d // 4] = low + scale * np.clip(code, 0, 15)
    return out


def _slice(st, pool, b, h):
    """Rows of a slice, in order, on the host: numpy."""
    if st["table"] is None:
        return pool[b, 0, h].cpu().numpy()
    return torch.cat([pool[i, 0, h] for i in st["table"][b].tolist()]).cpu().numpy()


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(st)
    B, H, G, d, lens = c["n_seq"], c["heads"], c["group"], c["d"], _lengths(c)
    scale = 1.0 / math.sqrt(d)
    q = st["q"].double().view(B, -1, H * G, d)
    news = [1] * B if c["op"] == "decode" else _news(c)
    n_q = q.shape[1]
    out = torch.zeros(B, n_q, H * G, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, n_q, H * G, dtype=torch.float64, device="cuda")
    mass = st["mass"].double() if "mass" in st else None
    for b in range(B):
        for h in range(H):
            n, new = lens[b][h], news[b]
            k, v = (torch.from_numpy(_numbers64(_slice(st, st[x], b, h)[:n])).cuda() for x in ("k", "v"))
            for gq in range(h * G, (h + 1) * G):
                if n == 0:
                    lse[b, :, gq] = NEG
                    continue
                x = scale * (q[b, :new, gq] @ k.T)  # [new, n]
                row = torch.arange(n - new, n, device="cuda").unsqueeze(1)
                col = torch.arange(n, device="cuda").unsqueeze(0)
                hidden = col > row
                if c["window"] > 0:
                    hidden = hidden | ((col <= row - c["window"]) & (col >= c["n_sink"]))
                x = x.masked_fill(hidden, NEG)
                z = torch.logsumexp(x, dim=1)
                w = torch.exp(x - z[:, None])
                out[b, :new, gq] = w @ v
                lse[b, :new, gq] = z
                if mass is not None:
                    mass[b * H + h, :n] += w.sum(0)
    r = {"out": out, "lse": lse} if c["op"] == "prefill" else {"out": out[:, 0], "lse": lse[:, 0]}
    if mass is not None:
        r["mass"] = mass
    return r


def _exact_append(st):
    c = st["case"]
    B, H, d, q4 = c["n_seq"], c["heads"], c["d"], c["dtype"] == "q4"
    F = d // 2
    q, k, v = _split(st)
    axis = st["band_axis"] or [0] * F
    q_out = st["q_out"].double()
    k_out, v_out = (st[x].double() for x in (("k_read", "v_read") if q4 else ("k", "v")))
    omega = torch.tensor([THETA ** (-2.0 * f / d) for f in range(F)], dtype=torch.float64, device="cuda")
    pair = (lambda x: (x[..., :F], x[..., F:])) if c["half"] else (lambda x: (x[..., ::2], x[..., 1::2]))

    def turned(x, at):  # [n, heads, d] as complex numbers times e^{i omega p}
        re, im = pair(x.double())
        p = torch.stack([at[:, a] for a in axis], -1).double()
        z = torch.complex(re, im) * torch.exp(1j * (p * omega))[:, None]
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for part, to in zip((z.real, z.imag), pair(y)):
            to.copy_(part)
        return y

    for b, n in enumerate(_news(c)):
        at = st["positions"][b, :n]
        q_out[b, :n] = turned(q[b, :n], at)
        kb, vb = turned(k[b, :n], at), v[b, :n].double()
        for h in range(H):
            r0 = int(st["rows"][b * H + h])
            for pool, out, new in (("k", k_out, kb), ("v", v_out, vb)):
                if q4:
                    out[b, h, :r0] = torch.from_numpy(_numbers64(_slice(st, st[pool], b, h)[:r0])).cuda()
                    out[b, h, r0:r0 + n] = torch.from_numpy(_rounded64(new[:, h].cpu().numpy())).cuda()
                elif st["table"] is None:
                    out[b, 0, h, r0:r0 + n] = new[:, h]
                else:
                    bs, i = c["block"], 0
                    while i < n:  # block by block
                        blk, off = int(st["table"][b, (r0 + i) // bs]), (r0 + i) % bs
                        m = min(bs - off, n - i)
                        out[blk, 0, h, off:off + m] = new[i:i + m, h]
                        i += m
    return {"q": q_out, "n_valid": None, "pos": None, "k": k_out, "v": v_out}
