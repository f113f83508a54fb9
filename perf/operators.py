"""Attention over the compressed cache and eviction by attention weight: the
cases they are measured on, their plain forms, and the calls a user makes.

Four operators on the library's cache descriptor (contiguous slices or block
pools, one row count per slice):

  decode   one new token per sequence attends its cached rows (optionally the
           first n_sink rows and the newest `window`), optionally adding every
           row's weight to its accumulated mass;
  prefill  a chunk of new tokens (the newest rows of the cache) attends
           causally, optionally windowed with sinks;
  mass     the weights a chunk of queries gives each cached row, summed into
           the row's accumulated mass;
  evict    the rows with the largest accumulated mass are kept under a
           protected prompt and recent window, and K, V, positions and masses
           are compacted.

Row counts, chunk lengths and block tables' sizes follow from the case alone;
every value (queries, keys, values, masses, which block holds what) comes from
the seed. Keys and queries are drawn as per-head centres of norm 8 plus unit
noise, rotated at their positions, as an engine caches them.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
THETA = 1e6
NEG = float("-inf")


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _decode(name, n_seq, heads, group, d, dtype, rows, ragged=False, block=0, n_sink=0, window=0, mass=False):
    return {"name": name, "op": "decode", "n_seq": n_seq, "heads": heads, "group": group, "d": d, "dtype": dtype, "rows": rows,
            "ragged": ragged, "block": block, "n_sink": n_sink, "window": window, "mass": mass}


def _chunk(name, op, n_seq, heads, group, d, dtype, rows, n_new, ragged=False, block=0, n_sink=0, window=0):
    return {"name": name, "op": op, "n_seq": n_seq, "heads": heads, "group": group, "d": d, "dtype": dtype, "rows": rows, "n_new": n_new,
            "ragged": ragged, "block": block, "n_sink": n_sink, "window": window}


def _evict(name, n_seq, layers, heads, d, dtype, rows, budget, n_prompt, n_recent, block=0):
    return {"name": name, "op": "evict", "n_seq": n_seq, "layers": layers, "heads": heads, "d": d, "dtype": dtype, "rows": rows, "budget": budget,
            "n_prompt": n_prompt, "n_recent": n_recent, "block": block}


def listed():
    return [
        # the tiny configuration's cache, fp32: the shortest call
        _decode("decode tiny fp32", 1, 2, 1, 64, "fp32", 512),
        # one layer of the Qwen3-8B-shaped model, one user, a cache between two evictions
        _decode("decode layer", 1, 8, 4, 128, "bf16", 2113),
        # one layer of the 16-sequence stack before its first eviction, in an engine's block pool
        _decode("decode stack paged", 16, 8, 4, 128, "bf16", 32768, block=64),
        # the large batch of periodically compressed caches, heads of different lengths, weights accumulated for the next eviction
        _decode("decode periodic mass", 64, 8, 1, 64, "bf16", 2176, ragged=True, mass=True),
        # long streams that attend four first rows and a window, their weights accumulated
        _decode("decode sinks mass", 16, 8, 4, 128, "bf16", 32768, ragged=True, block=16, n_sink=4, window=4000, mass=True),
        # a follow-up question of odd length on a compressed cache
        _chunk("prefill follow-up", "prefill", 1, 8, 4, 128, "bf16", 2176, 131),
        # a whole prompt of the layer shape
        _chunk("prefill prompt", "prefill", 1, 8, 4, 128, "bf16", 8192, 8192),
        # a padded batch of prompts with sinks and a window, block pool, the periodic model's head size
        _chunk("prefill sinks batch", "prefill", 8, 8, 2, 64, "bf16", 4096, 4096, ragged=True, block=64, n_sink=4, window=1000),
        # the weights a whole prompt gives its rows
        _chunk("mass prompt", "mass", 1, 8, 4, 128, "bf16", 4096, 4096),
        # the last 32 queries of 16 long prompts judge every cached row
        _chunk("mass observe", "mass", 16, 8, 4, 128, "bf16", 32768, 32, ragged=True, block=64),
        # one sequence of the stack after a round of 128 tokens
        _evict("evict round", 1, 36, 8, 128, "bf16", 2176, 2048, 256, 128),
        # four sequences of the stack at 32768 rows, in a block pool
        _evict("evict stack paged", 4, 36, 8, 128, "bf16", 32768, 4096, 512, 128, block=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "mass", "evict"])
    d = rng.choice([64, 128])
    block = rng.choice([0, 0, 16, 64, 256])
    n_sink, window = (rng.choice([0, 1, 4, 130]), _log(rng, 16, 8192)) if rng.random() < 0.4 else (0, 0)
    ragged = rng.random() < 0.5
    heads, group = rng.choice([1, 2, 8]), rng.choice([1, 2, 3, 4, 7, 8])
    if op == "decode":
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        rows = _log(rng, 16, 32768)
        n_seq = max(1, min(_log(rng, 1, 64), 16 * 8 * 32768 // (heads * rows * (2 if dtype == "fp32" else 1))))
        c = _decode("", n_seq, heads, group, d, dtype, rows, ragged, block, n_sink, window, rng.random() < 0.5)
    elif op in ("prefill", "mass"):
        n_new = _log(rng, 1, 6000)
        rows = max(n_new, _log(rng, 64, 16384))
        most = 8192 * 8192 * 32 // 4
        n_seq = max(1, min(_log(rng, 1, 16), most // (heads * group * n_new * rows)))
        while heads * group * n_new * rows > most:
            n_new = (n_new + 1) // 2
        c = _chunk("", op, n_seq, heads, group, d, "bf16", rows, n_new, ragged, block, n_sink, window)
    else:
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        rows = _log(rng, 300, 32768)
        budget = max(64, int(rows * rng.uniform(0.05, 0.97)))
        n_prompt, n_recent = rng.randrange(0, budget // 2), rng.randrange(0, budget // 4)
        layers = rng.choice([1, 2, 24, 36])
        c = _evict("", _log(rng, 1, 16), layers, heads, d, dtype, rows, budget, n_prompt, n_recent, block)
        most = work(listed()[-1])["bytes"]
        while work(c)["bytes"] > most:
            key = "n_seq" if c["n_seq"] > 1 else "layers"
            c[key] = c[key] * 2 // 3
    del c["name"]
    return c


# --------------------------------------------------------------------------
# sizes that follow from the case
# --------------------------------------------------------------------------
def _cap(c):
    """Rows a slice can hold: room for a round of 128 more, in whole blocks."""
    unit = max(c["block"], 16)
    return (c["rows"] + 128 + unit - 1) // unit * unit


def _lengths(c):
    """Cached rows of every (sequence, head): equal, or spread from none to all."""
    B, H, n = c["n_seq"], c["heads"], c["rows"]
    if not c["ragged"]:
        return [[n] * H for _ in range(B)]
    if c["op"] == "decode":  # heads differ: each was compressed to its own rows
        spread = [(0 if B * H > 8 and (b, h) == (B // 2, 0) else max(1, n - (577 * (b * H + h) + 131 * b) % (n // 2 + 1))) for b in range(B) for h in range(H)]
        return [spread[b * H:(b + 1) * H] for b in range(B)]
    return [[max(1, n - (577 * b) % (n // 2 + 1))] * H for b in range(B)]


def _news(c):
    """New tokens of every sequence of a chunk."""
    n = [row[0] for row in _lengths(c)]
    if not c["ragged"]:
        return [min(c["n_new"], x) for x in n]
    return [max(1, min(x, c["n_new"] - (311 * b) % (c["n_new"] // 2 + 1))) for b, x in enumerate(n)]


def _visible(r, n_sink, window):
    """How many rows the query at row r sees."""
    if r < 0:
        return 0
    if window == 0 or r + 1 <= window:
        return r + 1
    lo = r + 1 - window
    return window + min(n_sink, lo)


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    d, H = c["d"], c["heads"]
    if c["op"] == "evict":
        S = c["n_seq"] * c["layers"] * H
        moved = c["budget"] - c["n_prompt"] if c["rows"] > c["budget"] else 0
        return {"bytes": S * (4 * c["rows"] + moved * (2 * 2 * d * e + 4 + 8) + 4 * c["budget"]), "flops": 0}
    G, lens = c["group"], _lengths(c)
    if c["op"] == "decode":
        seen = sum(_visible(n - 1, c["n_sink"], c["window"]) for row in lens for n in row)
        io = c["n_seq"] * H * G * (2 * d * e + 4)
        return {"bytes": seen * (2 * d * e + (8 if c["mass"] else 0)) + io, "flops": 4 * d * G * seen}
    pairs, rows = 0, 0
    for row, new in zip(lens, _news(c)):
        n = row[0]
        pairs += H * G * sum(_visible(r, c["n_sink"], c["window"]) for r in range(n - new, n))
        first = max(0, n - new + 1 - c["window"]) if c["window"] else 0
        rows += H * (n - first + min(first, c["n_sink"]))
    q = sum(_news(c)) * H * G
    if c["op"] == "prefill":
        return {"bytes": rows * 2 * d * e + q * (2 * d * e + 4), "flops": 4 * d * pairs}
    return {"bytes": rows * (d * e + 8) + q * (d * e + 4), "flops": 2 * d * pairs}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _rotate(x, pos):
    """x [..., n, d] at positions pos [n], coordinate pairs (2f, 2f + 1)."""
    d = x.shape[-1]
    f = torch.arange(d // 2, dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None] * THETA ** (-2.0 * f / d)
    cs, sn = torch.cos(ang).float(), torch.sin(ang).float()
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cs - b * sn, a * sn + b * cs), dim=-1).flatten(-2)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _centres(g, *shape):
    x = _normal(g, *shape)
    return x * (8.0 / x.norm(dim=-1, keepdim=True))


def _store(c, g, rows):
    """Rows [n_seq, layers, heads, cap, d] as the cache holds them: the slices themselves, or a pool with its table."""
    if not c["block"]:
        return rows.contiguous(), None
    B, L, H, cap, d = rows.shape
    bs = c["block"]
    per = cap // bs
    table = torch.randperm(B * per + 2, generator=g, device="cuda")[:B * per].view(B, per)
    pool = torch.zeros(B * per + 2, L, H, bs, d, dtype=rows.dtype, device="cuda")
    pool[table.view(-1)] = rows.view(B, L, H, per, bs, d).permute(0, 3, 1, 2, 4, 5).reshape(B * per, L, H, bs, d)
    return pool, table.to(torch.int32)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, B, H, d, cap = DTYPES[c["dtype"]], c["n_seq"], c["heads"], c["d"], _cap(c)
    L = c.get("layers", 1)
    k, v = (torch.empty(B, L, H, cap, d, dtype=dt, device="cuda") for _ in range(2))
    pos = torch.arange(cap, device="cuda")
    mu = _centres(g, L, H, 1, d)
    for b in range(B):
        for l in range(L):
            k[b, l] = _rotate(mu[l] + _normal(g, H, cap, d), pos).to(dt)
            v[b, l] = _normal(g, H, cap, d).to(dt)
    at = g.get_state()
    k, table = _store(c, g, k)
    g.set_state(at)  # V's blocks are K's
    v, _ = _store(c, g, v)
    st = {"case": dict(c), "k": k, "v": v, "table": table, "cap": cap}
    if c["op"] == "evict":
        S = B * L * H
        # heavy tailed, as accumulated weights are; the newest rows have gathered little, some nothing at all
        mass = torch.exp(2.0 * _normal(g, S, cap)) * torch.rand(S, cap, generator=g, device="cuda")
        mass *= torch.rand(S, cap, generator=g, device="cuda") > 0.02
        st["mass"], st["mass_out"] = mass, torch.zeros_like(mass)
        st["rows"] = torch.full((S,), c["rows"], dtype=torch.int32, device="cuda")
        st["n_valid"] = st["rows"].clone()
        st["pos"] = torch.arange(cap, dtype=torch.int32, device="cuda").expand(S, cap).contiguous()
        st["pos_out"] = torch.zeros_like(st["pos"])
        st["keep"] = torch.zeros(S, c["budget"], dtype=torch.int32, device="cuda")
        return st
    G = c["group"]
    lens = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")  # [B, H]
    st["n_valid"] = lens.flatten().contiguous()
    mu_q = _centres(g, H, G, d)
    # a program keeps one scratch buffer for its calls
    st["scratch"] = torch.empty((64 << 20) + 4 * B * H * G * cap, dtype=torch.uint8, device="cuda")
    if c["op"] == "decode":
        q = mu_q + _normal(g, B, H, G, d)
        st["q"] = torch.stack([_rotate(q[b].reshape(H * G, 1, d), lens[b, :1] - 1)[:, 0] for b in range(B)]).to(dt)  # [B, Hq, d]
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(B, H * G, device="cuda")
        if c["mass"]:
            st["mass"] = torch.rand(B * H, cap, generator=g, device="cuda")  # what earlier tokens gave
        return st
    n_q = max(_news(c))
    news = torch.tensor(_news(c), dtype=torch.int32, device="cuda")
    q = torch.empty(B, n_q, H * G, d, dtype=dt, device="cuda")
    for b in range(B):
        r = torch.arange(n_q, device="cuda") + (lens[b, 0] - news[b])
        q[b] = _rotate((mu_q + _normal(g, n_q, H, G, d)).view(n_q, H * G, d).transpose(0, 1), r).transpose(0, 1).to(dt)
    st.update(q=q, n_new=news)
    if c["op"] == "prefill":
        st["out"] = torch.zeros_like(q)
        st["lse"] = torch.zeros(B, n_q, H * G, device="cuda")
        return st
    st["mass"] = torch.rand(B * H, cap, generator=g, device="cuda")
    st["lse"] = torch.zeros(B, n_q, H * G, device="cuda")  # as the prompt's own attention returned it
    kl = _rows(st, k)
    for b in range(B):
        for h in range(H):
            s, seen = _logits(st, kl, q, b, h)
            x = torch.logsumexp(torch.where(seen, s, NEG), dim=-1)  # [n_q, G]
            st["lse"][b, :, h * G:(h + 1) * G] = torch.where((torch.arange(n_q, device="cuda") < news[b])[:, None], x, 0.0)
    return st


def _rows(st, pool):
    """The cache's rows in order: [n_seq, heads, rows, d] of its one layer."""
    n = st["case"]["rows"]
    if st["table"] is None:
        return pool[:, 0, :, :n]
    B, per = st["table"].shape
    t = pool[st["table"].long()][:, :, 0]  # [B, per, H, bs, d]
    return t.permute(0, 2, 1, 3, 4).reshape(B, t.shape[2], -1, t.shape[4])[:, :, :n]


def _logits(st, kl, q, b, h):
    """One head's fp32 logits [n_q, G, n] and which of them are visible."""
    c = st["case"]
    G, n, n_q = c["group"], kl.shape[2], q.shape[1]
    s = (q[b, :, h * G:(h + 1) * G].float().reshape(n_q * G, -1) @ kl[b, h].float().T).view(n_q, G, n) * c["d"] ** -0.5
    r = torch.arange(n_q, device="cuda") + (st["n_valid"].view(c["n_seq"], -1)[b, h] - st["n_new"][b])
    j = torch.arange(n, device="cuda")
    seen = j[None] <= r[:, None]
    if c["window"]:
        seen &= (j < c["n_sink"])[None] | (j[None] > r[:, None] - c["window"])
    return s, seen[:, None]


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _softmax(s, seen):
    """Weights, and log of their sum, over the visible entries; nothing visible: zeros and -inf."""
    s = torch.where(seen, s, NEG)
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == NEG, 0.0, m)
    p = torch.exp(s - m0)
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l > 0, l, 1.0), (m0 + torch.log(l)).squeeze(-1)


def _seen_chunk(st, n):
    """[n_seq, heads, n_q, n]: which rows each new token sees."""
    c = st["case"]
    n_q = st["q"].shape[1]
    base = st["n_valid"].view(c["n_seq"], c["heads"]) - st["n_new"][:, None]
    r = base[:, :, None, None] + torch.arange(n_q, device="cuda")[:, None]
    j = torch.arange(n, device="cuda")
    seen = j <= r
    if c["window"]:
        seen &= (j < c["n_sink"]) | (j > r - c["window"])
    return seen


def _plain_decode(st):
    c = st["case"]
    B, H, G, d = c["n_seq"], c["heads"], c["group"], c["d"]
    k, v = _rows(st, st["k"]).float(), _rows(st, st["v"]).float()
    n = st["n_valid"].view(B, H, 1)
    j = torch.arange(k.shape[2], device="cuda")
    seen = j < n
    if c["window"]:
        seen &= (j < c["n_sink"]) | (j >= n - c["window"])
    p, lse = _softmax(st["q"].view(B, H, G, d).float() @ k.transpose(-1, -2) * d ** -0.5, seen[:, :, None])
    out = {"out": (p @ v).to(st["q"].dtype).view(B, H * G, d), "lse": lse.view(B, H * G)}
    if c["mass"]:
        st["mass"][:, :k.shape[2]] += p.sum(2).view(B * H, -1)
        out["mass"] = st["mass"]
    return out


def _plain_prefill(st):
    c = st["case"]
    B, H, G, d = c["n_seq"], c["heads"], c["group"], c["d"]
    k, v = _rows(st, st["k"]).float(), _rows(st, st["v"]).float()
    n_q = st["q"].shape[1]
    q = st["q"].view(B, n_q, H, G, d).permute(0, 2, 3, 1, 4).float()  # [B, H, G, n_q, d]
    p, lse = _softmax(q @ k[:, :, None].transpose(-1, -2) * d ** -0.5, _seen_chunk(st, k.shape[2])[:, :, None])
    o = (p @ v[:, :, None]).permute(0, 3, 1, 2, 4).reshape(B, n_q, H * G, d).to(st["q"].dtype)
    live = (torch.arange(n_q, device="cuda") < st["n_new"][:, None])[:, :, None]
    lse = lse.permute(0, 3, 1, 2).reshape(B, n_q, H * G)
    return {"out": torch.where(live[..., None], o, st["out"]), "lse": torch.where(live, lse, st["lse"])}


def _plain_mass(st):
    c = st["case"]
    B, H, G, d = c["n_seq"], c["heads"], c["group"], c["d"]
    k = _rows(st, st["k"]).float()
    n_q = st["q"].shape[1]
    q = st["q"].view(B, n_q, H, G, d).permute(0, 2, 3, 1, 4).float()
    s = q @ k[:, :, None].transpose(-1, -2) * d ** -0.5 - st["lse"].view(B, n_q, H, G).permute(0, 2, 3, 1)[..., None]
    live = torch.arange(n_q, device="cuda") < st["n_new"][:, None]
    p = torch.where(_seen_chunk(st, k.shape[2])[:, :, None] & live[:, None, None, :, None], torch.exp(s), 0.0)
    st["mass"][:, :k.shape[2]] += p.sum((2, 3)).view(B * H, -1)
    return {"mass": st["mass"]}


def _plain_evict(st):
    c = st["case"]
    S, n, P, W, budget = st["mass"].shape[0], c["rows"], c["n_prompt"], c["n_recent"], c["budget"]
    st["n_valid"].copy_(st["rows"])
    if n > budget:
        cand = st["mass"][:, P:n - W]
        best = torch.sort(cand, dim=1, descending=True, stable=True).indices[:, :budget - P - W] + P
        ends = [torch.arange(a, b, device="cuda").expand(S, -1) for a, b in ((0, P), (n - W, n))]
        keep = torch.cat([ends[0], torch.sort(best, dim=1).values, ends[1]], dim=1)
    else:
        keep = torch.arange(n, device="cuda").expand(S, n)
    kept = keep.shape[1]
    st["keep"].fill_(-1)
    st["keep"][:, :kept] = keep
    for name in ("k", "v"):
        _move(st, st[name], keep)
    st["pos_out"][:, :kept] = st["pos"].gather(1, keep)
    st["mass_out"][:, :kept] = st["mass"].gather(1, keep)
    st["mass_out"][:, kept:n] = 0
    st["n_valid"].fill_(kept)
    return _evicted(st)


def _move(st, pool, keep):
    """Row keep[s, j] to row j of every slice, in place."""
    if st["table"] is None:
        B, L, H, cap, d = pool.shape
        rows = pool.view(B * L * H, cap, d)
        rows[:, :keep.shape[1]] = rows.gather(1, keep[..., None].expand(-1, -1, d))
        return
    nb, L, H, bs, d = pool.shape
    B = st["table"].shape[0]
    flat = pool.view(nb * L * H * bs, d)
    lh = torch.arange(L * H, device="cuda").repeat(B)[:, None]
    seq = torch.arange(B, device="cuda").repeat_interleave(L * H)[:, None]

    def place(r):
        return (st["table"].long()[seq, r // bs] * (L * H) + lh) * bs + r % bs

    flat[place(torch.arange(keep.shape[1], device="cuda").expand_as(keep))] = flat[place(keep)]


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _cache(st):
    import kv_cache_compression_tri_gb300 as tri
    pos, pos_out = st.get("pos"), st.get("pos_out")
    if st["table"] is None:
        return tri.KVCache(st["k"], st["v"], st["n_valid"], pos, pos_out, post_rope=True)
    return tri.PagedKVCache(st["k"], st["v"], st["table"], st["n_valid"], pos, pos_out, post_rope=True)


def _own(st):
    import kv_cache_compression_tri_gb300 as tri
    c = st["case"]
    kv = _cache(st)
    if c["op"] == "decode":
        tri.attn_decode(kv, 0, st["q"], st["out"], n_sink=c["n_sink"], window=c["window"], lse=st["lse"], mass=st.get("mass"), workspace=st["scratch"])
        out = {"out": st["out"], "lse": st["lse"]}
        if c["mass"]:
            out["mass"] = st["mass"]
        return out
    if c["op"] == "prefill":
        tri.attn_prefill(kv, 0, st["q"], st["out"], n_new=st["n_new"], n_sink=c["n_sink"], window=c["window"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if c["op"] == "mass":
        tri.attn_mass(kv, 0, st["q"], st["lse"], st["mass"], n_new=st["n_new"], n_sink=c["n_sink"], window=c["window"])
        return {"mass": st["mass"]}
    st["n_valid"].copy_(st["rows"])  # the rows a round starts from
    tri.mass_evict(kv, st["mass"], st["mass_out"], c["n_prompt"], c["n_recent"], c["budget"], st["keep"])
    return _evicted(st)


def _evicted(st):
    kept = min(st["case"]["rows"], st["case"]["budget"])
    return {"keep": st["keep"], "n_valid": st["n_valid"], "pos": st["pos_out"][:, :kept], "mass": st["mass_out"], "k": st["k"], "v": st["v"]}


def run(st):
    if own:
        return _own(st)
    return {"decode": _plain_decode, "prefill": _plain_prefill, "mass": _plain_mass, "evict": _plain_evict}[st["case"]["op"]](st)


# --------------------------------------------------------------------------
# the definitions in 64 bits, slice by slice
# --------------------------------------------------------------------------
def _slice64(st, pool, b, l, h):
    if st["table"] is None:
        return pool[b, l, h].double()
    return torch.cat([pool[i, l, h] for i in st["table"][b].tolist()]).double()


def exact(c, seed):
    st = prepare(c, seed)
    B, H, d = c["n_seq"], c["heads"], c["d"]
    if c["op"] == "evict":
        return _exact_evict(st)
    G, lens = c["group"], _lengths(c)
    scale = 1.0 / math.sqrt(d)
    if c["op"] == "decode":
        q = st["q"].double().view(B, 1, H * G, d)
        news = [1] * B
    else:
        q, news = st["q"].double(), _news(c)
    n_q = q.shape[1]
    out = torch.zeros(B, n_q, H * G, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, n_q, H * G, dtype=torch.float64, device="cuda")
    mass = st["mass"].double() if "mass" in st else None
    for b in range(B):
        for h in range(H):
            n, new = lens[b][h], news[b]
            k, v = _slice64(st, st["k"], b, 0, h)[:n], _slice64(st, st["v"], b, 0, h)[:n]
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
                if c["op"] == "mass":
                    mass[b * H + h, :n] += torch.exp(x - st["lse"][b, :new, gq].double()[:, None]).sum(0)
                    continue
                z = torch.logsumexp(x, dim=1)
                w = torch.exp(x - z[:, None])
                out[b, :new, gq] = w @ v
                lse[b, :new, gq] = z
                if mass is not None:
                    mass[b * H + h, :n] += w.sum(0)
    if c["op"] == "mass":
        return {"mass": mass}
    r = {"out": out, "lse": lse} if c["op"] == "prefill" else {"out": out[:, 0], "lse": lse[:, 0]}
    if mass is not None:
        r["mass"] = mass
    return r


def _exact_evict(st):
    c = st["case"]
    n, P, W, budget = c["rows"], c["n_prompt"], c["n_recent"], c["budget"]
    B, L, H = c["n_seq"], c["layers"], c["heads"]
    kept = min(n, budget)
    new = {"k": st["k"].double(), "v": st["v"].double()}
    mass_out = torch.zeros_like(st["mass_out"], dtype=torch.float64)
    pos = torch.zeros(B * L * H, kept, dtype=torch.int32, device="cuda")
    for s in range(B * L * H):
        m = st["mass"][s, :n].double()
        # order by (protected first, mass descending, slot ascending); the first `kept` survive
        rank = m.clone()
        rank[:P] = float("inf")
        rank[n - W:] = float("inf")
        order = torch.argsort(-rank, stable=True)[:kept]
        alive = torch.zeros(n, dtype=torch.bool, device="cuda")
        alive[order] = True
        rows = alive.nonzero().flatten()
        b, l, h = s // (L * H), s // H % L, s % H
        for name in ("k", "v"):
            got = _slice64(st, st[name], b, l, h)[rows]
            if st["table"] is None:
                new[name][b, l, h, :kept] = got
                continue
            size = st[name].shape[3]
            for i, block in enumerate(st["table"][b, :-(-kept // size)].tolist()):
                part = got[i * size:(i + 1) * size]
                new[name][block, l, h, :len(part)] = part
        pos[s] = st["pos"][s][rows]
        mass_out[s, :kept] = m[rows]
    return {"keep": None, "n_valid": None, "pos": pos, "mass": mass_out, **new}
