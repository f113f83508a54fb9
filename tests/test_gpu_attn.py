"""Attention over the cache (tri_attn_decode, tri_attn_prefill, tri_attn_mass)
and eviction by accumulated weight (tri_mass_evict) against the definitions in
64 bits (attn_oracle.py).

Tolerances, for one query with weights w over rows j (sum w = 1), A = sum w_j |v_j|
per element and X = max_j |x_j|-sized bounds:
  logits   x = scale * q.k summed in fp32 over d products of bf16 (exact
           products) or fp32 values; each of the at most d + 8 additions and the
           scaling err by at most 2^-23 of the running magnitude (truncation
           included), so |dx| <= (d + 10) 2^-23 * scale * sum_i |q_i k_i| =: ex,
           largest over the visible rows.
  weights  w = 2^(x' - m) with ex2 good to 2^-22 relative and x' - m rounded
           (|x'| <= 2^k costs |x| 2^-23 more): relative error ew = 2 ex +
           2^-20 + 2^-22 max|x|; the sum's error adds the same again at most.
  out      |d out| <= A * (2 ew + p) + o |out|, where p = 2^-8 (half a step of
           bf16) for the prefill of a bf16 cache, whose weights are rounded for
           the product with V, p = 2^-16 for the decode of one (weights as a
           bf16 pair), 0 for fp32, and o = half a step of the output's type;
           fp32 sums over n rows add n 2^-24 A at most.
  lse      |d lse| <= ex + ew + 2^-22 max(1, |lse|)
  mass     |d mass| <= (2 ew + n_terms 2^-24 + 2^-23) * mass
Eviction moves rows: equal bytes.
"""
import numpy as np
import pytest
import torch

import kv_cache_compression_tri_gb300 as tri
from attn_oracle import attend, evict
from gpu_helpers import f64

pytestmark = pytest.mark.gpu

NAN = float("nan")
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tri.load_library()


class Case:
    """A cache of given row counts [n_seq][H] (same for every layer) whose rows
    past the count hold NaN, contiguous (with guard rows after each slice) or
    paged, and its logical rows on the host."""

    def __init__(self, lens, d, dtype, L=2, block=0, n_cap=None, seed=0, big=1.0):
        lens = np.asarray(lens, dtype=np.int64)
        B, H = lens.shape
        g = torch.Generator(device="cuda").manual_seed(seed)
        n_cap = n_cap or int(max(lens.max(), 1)) + 5
        if block:
            n_cap = (n_cap + block - 1) // block * block
        k = torch.randn(B, L, H, n_cap, d, generator=g, device="cuda") * big
        v = torch.randn(B, L, H, n_cap, d, generator=g, device="cuda")
        for b in range(B):
            for h in range(H):
                k[b, :, h, lens[b, h]:] = NAN
                v[b, :, h, lens[b, h]:] = NAN
        k, v = k.to(dtype), v.to(dtype)
        self.kr, self.vr = f64(k), f64(v)
        self.lens, self.B, self.H, self.L, self.d, self.n_cap, self.dtype, self.g = lens, B, H, L, d, n_cap, dtype, g
        S = B * L * H
        nv = torch.tensor(np.repeat(lens[:, None, :], L, 1).reshape(-1), dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pos = torch.arange(n_cap, dtype=torch.int32, device="cuda").expand(S, n_cap).contiguous()
        pos_out = torch.full((S, n_cap), -7, dtype=torch.int32, device="cuda")
        if block:
            per = n_cap // block
            t = torch.randperm(B * per + 3, generator=g, device="cuda")[: B * per].view(B, per)
            kp = torch.full((B * per + 3, L, H, block, d), NAN, dtype=dtype, device="cuda")
            vp = kp.clone()
            for pool, x in ((kp, k), (vp, v)):
                pool[t.view(-1)] = x.view(B, L, H, per, block, d).permute(0, 3, 1, 2, 4, 5).reshape(B * per, L, H, block, d)
            table = t.to(torch.int32).contiguous()
            self.kv = tri.PagedKVCache(kp, vp, table, nv, pos, pos_out, self.status, post_rope=True)
        else:
            wide = [torch.full((B, L, H, n_cap + 3, d), NAN, dtype=dtype, device="cuda") for _ in range(2)]
            for w, x in zip(wide, (k, v)):
                w[:, :, :, :n_cap] = x
            self.kv = tri.KVCache(wide[0][:, :, :, :n_cap], wide[1][:, :, :, :n_cap], nv, pos, pos_out, self.status, post_rope=True)

    def rows(self, b, layer, h):
        n = self.lens[b, h]
        return self.kr[b, layer, h, :n], self.vr[b, layer, h, :n]

    def slice(self, b, layer, h):
        return (b * self.L + layer) * self.H + h

    def ok(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0


def _bounds(q, k, v, r, scale, w, o, lse, n_sink, window, dtype, p):
    """The tolerances of one query: out [d], lse."""
    seen = w > 0
    if not seen.any():
        return np.zeros_like(o), 0.0, 0.0
    ks, vs = k[seen], v[seen]
    d = len(q)
    ex = (d + 10) * 2.0 ** -23 * scale * (np.abs(ks) @ np.abs(q)).max()
    x = scale * (ks @ q)
    ew = 2 * ex + 2.0 ** -20 + 2.0 ** -22 * np.abs(x).max()
    A = w[seen] @ np.abs(vs)
    return A * (2 * ew + p + len(vs) * 2.0 ** -24) + HALF[dtype] * np.abs(o) + 1e-30, ex + ew + 2.0 ** -22 * max(1.0, abs(lse)), ew


def check_decode(c, G, layer=1, n_sink=0, window=0, with_mass=False, n_new=None, scale=None, seed=1, stream=None, qscale=1.0):
    B, H, d = c.B, c.H, c.d
    g = torch.Generator(device="cuda").manual_seed(seed)
    big = (torch.randn(B, 3, H * G, d, generator=g, device="cuda") * qscale).to(c.dtype)
    q = big[:, 1]  # a view with a sequence stride of its own
    out = torch.full((B, H * G, d), 9.0, dtype=c.dtype, device="cuda")
    lse = torch.full((B, H * G), 9.0, device="cuda")
    mass0 = torch.rand(B * c.L * H, c.n_cap, generator=g, device="cuda")
    mass = mass0.clone() if with_mass else None
    nn = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device="cuda")
    need = tri.attn_decode_workspace_bytes(c.kv, G, with_mass)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    tri.attn_decode(c.kv, layer, q, out, n_new=nn, scale=scale, n_sink=n_sink, window=window, lse=lse, mass=mass, workspace=ws[:need])
    c.ok()
    assert bool((ws[need:] == 0xA5).all())
    sc = d ** -0.5 if scale is None else scale
    got_o, got_l, qn = f64(out), f64(lse), f64(q)
    got_m, ref_m = (f64(mass), f64(mass0)) if with_mass else (None, None)
    tol_m = np.zeros_like(ref_m) if with_mass else None
    p = 2.0 ** -16 if c.dtype == torch.bfloat16 else 0.0
    for b in range(B):
        for h in range(H):
            k, v = c.rows(b, layer, h)
            for gq in range(G):
                hq = h * G + gq
                if n_new is not None and n_new[b] == 0:
                    assert (got_o[b, hq] == 9.0).all() and got_l[b, hq] == 9.0
                    continue
                r = len(k) - 1
                o, l, w = attend(qn[b, hq], k, v, r, sc, n_sink, window)
                to, tl, ew = _bounds(qn[b, hq], k, v, r, sc, w, o, l, n_sink, window, c.dtype, p)
                assert np.all(np.abs(got_o[b, hq] - o) <= to), (b, hq, np.abs(got_o[b, hq] - o).max())
                assert got_l[b, hq] == l or abs(got_l[b, hq] - l) <= tl, (b, hq, got_l[b, hq], l)
                if with_mass:
                    s = c.slice(b, layer, h)
                    ref_m[s, :len(k)] += w
                    tol_m[s, :len(k)] += (2 * ew + (G + 2) * 2.0 ** -23) * w
    if with_mass:
        assert np.all(np.abs(got_m - ref_m) <= tol_m + 2.0 ** -23 * ref_m * (tol_m > 0))
    return out, lse, mass


LENS = {
    "ragged": [[0, 1, 17], [63, 64, 65], [200, 2, 333]],
    "short": [[1, 1], [2, 3]],
    "long": [[1111, 4099]],
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [0, 16, 64])
def test_decode_ragged(dtype, d, block):
    check_decode(Case(LENS["ragged"], d, dtype, block=block), 4, with_mass=True)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_groups(group, dtype):
    check_decode(Case([[37, 130]], 128 if group % 2 else 64, dtype), group, layer=0, with_mass=group != 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", ["short", "long"])
def test_decode_lengths(dtype, lens):
    check_decode(Case(LENS[lens], 128, dtype), 2)
    check_decode(Case(LENS[lens], 64, dtype, block=32), 8, with_mass=True)


@pytest.mark.parametrize("n_sink,window", [(0, 1), (0, 7), (4, 1), (4, 60), (4, 64), (130, 65), (1000, 3), (3, 1 << 30), (1 << 30, 5), (0, 4096)])
@pytest.mark.parametrize("block", [0, 16])
def test_decode_sinks_and_window(n_sink, window, block):
    check_decode(Case([[0, 1, 64], [65, 333, 1000]], 128, torch.bfloat16, block=block), 4, n_sink=n_sink, window=window, with_mass=True)
    check_decode(Case([[5, 600]], 64, torch.float32, block=block), 1, n_sink=n_sink, window=window, with_mass=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_sequences_left_out_and_scale(dtype):
    check_decode(Case([[40, 9], [11, 70], [0, 5]], 64, dtype), 3, n_new=[0, 1, 1], scale=0.37, with_mass=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_peaked_weights(dtype):
    # logits of several hundred: one row takes all, the others underflow
    check_decode(Case([[300, 129]], 128, dtype, big=4.0), 4, qscale=8.0, with_mass=True)


def test_decode_rows_out_of_sight_may_be_anything():
    c = Case([[300, 299]], 128, torch.bfloat16)
    c.kv.k[:, :, :, 4:200] = NAN
    c.kv.v[:, :, :, 4:200] = float("inf")
    check_decode(c, 4, n_sink=4, window=90, with_mass=True)


def check_prefill(c, G, n_new, n_q=None, layer=1, n_sink=0, window=0, seed=2, scale=None, mass_last=None, qscale=1.0):
    """attn_prefill, then attn_mass with the same queries (or the last mass_last tokens of them)."""
    B, H, d = c.B, c.H, c.d
    n_q = n_q or max(n_new)
    g = torch.Generator(device="cuda").manual_seed(seed)
    fused = (torch.randn(B, n_q, (G + 2) * H, d, generator=g, device="cuda") * qscale).to(c.dtype)
    q = fused[:, :, : G * H]  # queries inside a fused projection's rows
    out = torch.full((B, n_q, H * G, d), 9.0, dtype=c.dtype, device="cuda")
    lse = torch.full((B, n_q, H * G), 9.0, device="cuda")
    nn = torch.tensor(n_new, dtype=torch.int32, device="cuda")
    tri.attn_prefill(c.kv, layer, q, out, n_new=nn, scale=scale, n_sink=n_sink, window=window, lse=lse)
    c.ok()
    mass0 = torch.rand(B * c.L * H, c.n_cap, generator=g, device="cuda")
    mass = mass0.clone()
    if mass_last is None:
        tri.attn_mass(c.kv, layer, q, lse, mass, n_new=nn, scale=scale, n_sink=n_sink, window=window)
        first = [0] * B
    else:
        assert all(x == n_q for x in n_new)
        tri.attn_mass(c.kv, layer, q[:, -mass_last:], lse[:, -mass_last:], mass, scale=scale, n_sink=n_sink, window=window)
        first = [n_q - mass_last] * B
    c.ok()
    sc = d ** -0.5 if scale is None else scale
    got_o, got_l, qn, got_m, ref_m = f64(out), f64(lse), f64(q), f64(mass), f64(mass0)
    tol_m = np.zeros_like(ref_m)
    p = 2.0 ** -8 if c.dtype == torch.bfloat16 else 0.0
    for b in range(B):
        assert (got_o[b, n_new[b]:] == 9.0).all() and (got_l[b, n_new[b]:] == 9.0).all()
        for h in range(H):
            k, v = c.rows(b, layer, h)
            s = c.slice(b, layer, h)
            for i in range(n_new[b]):
                r = len(k) - n_new[b] + i
                for gq in range(G):
                    hq = h * G + gq
                    o, l, w = attend(qn[b, i, hq], k, v, r, sc, n_sink, window)
                    to, tl, ew = _bounds(qn[b, i, hq], k, v, r, sc, w, o, l, n_sink, window, c.dtype, p)
                    assert np.all(np.abs(got_o[b, i, hq] - o) <= to), (b, i, hq, np.abs(got_o[b, i, hq] - o).max())
                    assert got_l[b, i, hq] == l or abs(got_l[b, i, hq] - l) <= tl, (b, i, hq)
                    if i >= first[b] and l > -np.inf:
                        ref_m[s, :len(k)] += w
                        # the weight is taken under the rounded lse it was given
                        tol_m[s, :len(k)] += (2 * ew + tl + (G * n_new[b] + 2) * 2.0 ** -24) * w
    assert np.all(np.abs(got_m - ref_m) <= tol_m + 2.0 ** -23 * ref_m * (tol_m > 0))
    return out, lse, mass


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [0, 16, 128])
def test_prefill_ragged(dtype, d, block):
    c = Case([[65, 65], [1, 2], [200, 333], [0, 40]], d, dtype, block=block)
    check_prefill(c, 4, [65, 1, 70, 40], n_q=75)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8])
def test_prefill_groups(group):
    check_prefill(Case([[150, 131]], 64 if group % 2 else 128, torch.bfloat16), group, [131])


@pytest.mark.parametrize("n_sink,window", [(0, 1), (0, 33), (4, 1), (4, 60), (5, 128), (130, 65), (1000, 3), (3, 1 << 30), (1 << 30, 5)])
@pytest.mark.parametrize("block", [0, 64])
def test_prefill_sinks_and_window(n_sink, window, block):
    c = Case([[300, 460]], 128, torch.bfloat16, L=1, block=block)
    check_prefill(c, 2, [290], layer=0, n_sink=n_sink, window=window)


@pytest.mark.parametrize("n_new", [1, 2, 31, 32, 33, 127, 128, 129, 257])
def test_prefill_lengths(n_new):
    check_prefill(Case([[n_new + 3], [n_new]], 128, torch.bfloat16, L=1), 4, [n_new, n_new], layer=0)
    check_prefill(Case([[n_new + 300]], 64, torch.bfloat16, L=1, block=32), 1, [n_new], layer=0)


def test_prefill_queries_before_the_first_row():
    # a head that holds fewer rows than there are new tokens: the early queries see nothing
    out, lse, _ = check_prefill(Case([[5, 40]], 64, torch.bfloat16, L=1), 2, [30], layer=0)
    assert bool((out[0, :25, :2] == 0).all()) and bool((lse[0, :25, :2] == float("-inf")).all())


def test_mass_of_an_observation_window():
    check_prefill(Case([[333, 200], [200, 260]], 128, torch.bfloat16, L=1), 4, [150, 150], layer=0, mass_last=32)
    check_prefill(Case([[333, 200], [200, 260]], 64, torch.float32, L=1, block=16), 1, [50, 50], layer=0, mass_last=7)


def test_prefill_peaked_weights():
    check_prefill(Case([[400]], 128, torch.bfloat16, L=1, big=4.0), 2, [140], layer=0, qscale=8.0)


def test_prefill_long_rows_sampled():
    # a long past: many tiles, the running maximum moving
    check_prefill(Case([[4500]], 128, torch.bfloat16, L=1), 4, [40], layer=0)
    check_prefill(Case([[4500]], 64, torch.bfloat16, L=1, block=256), 2, [40], layer=0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("in_place", [False, True])
def test_mass_evict(dtype, block, in_place):
    lens = [[0, 1, 90], [91, 200, 999], [100, 333, 1000]]
    c = Case(lens, 64, dtype, L=2, block=block)
    P, W, budget = 10, 20, 90
    S = c.B * c.L * c.H
    mass0 = torch.rand(S, c.n_cap, generator=c.g, device="cuda")
    mass0 *= torch.rand(S, c.n_cap, generator=c.g, device="cuda") > 0.4  # many equal (zero) masses
    mass = mass0.clone()
    mass_out = mass if in_place else torch.full_like(mass, 5.0)
    if in_place:
        c.kv.pos_out = c.kv.pos
    keep = torch.zeros(S, budget, dtype=torch.int32, device="cuda")
    tri.mass_evict(c.kv, mass, mass_out, P, W, budget, keep)
    c.ok()
    m0, got, gk, nv, po = mass0.cpu().numpy(), mass_out.cpu().numpy(), keep.cpu().numpy(), c.kv.n_valid.cpu().numpy(), c.kv.pos_out.cpu().numpy()
    bs = block
    for b in range(c.B):
        for l in range(c.L):
            for h in range(c.H):
                s, n = c.slice(b, l, h), int(c.lens[b, h])
                ref = evict(m0[s], n, P, W, budget)
                nk = len(ref)
                assert np.array_equal(gk[s], np.concatenate([ref, -np.ones(budget - nk, dtype=np.int64)]))
                assert nv[s] == nk
                assert np.array_equal(po[s, :nk], ref)
                assert np.array_equal(got[s, :nk], m0[s, ref])
                assert np.all(got[s, nk:n] == 0)
                assert np.array_equal(got[s, n:], m0[s, n:] if in_place else np.full_like(m0[s, n:], 5.0))
                for pool, ref_rows in ((c.kv.k, c.kr), (c.kv.v, c.vr)):
                    if bs:
                        t = c.kv.block_table[b].cpu().numpy()
                        rows = np.concatenate([f64(pool[int(i), l, h]) for i in t])
                    else:
                        rows = f64(pool[b, l, h])
                    assert np.array_equal(rows[:nk], ref_rows[b, l, h, ref])
                    assert np.array_equal(rows[nk:], ref_rows[b, l, h, nk:], equal_nan=True)


@pytest.mark.parametrize("block", [0, 16])
def test_serving_run(block):
    """Prompt, masses, tokens, eviction, tokens: each step against the definitions on the cache as it then is."""
    c = Case([[150, 150], [90, 90]], 64, torch.bfloat16, L=2, block=block, n_cap=208)
    G, layer = 4, 1
    S = c.B * c.L * c.H
    _, _, _ = check_prefill(c, G, [150, 90], layer=layer)
    mass = torch.zeros(S, c.n_cap, device="cuda")
    q = torch.randn(c.B, 32, c.H * G, c.d, generator=c.g, device="cuda").to(c.dtype)
    o, l = torch.empty_like(q), torch.empty(c.B, 32, c.H * G, device="cuda")
    for lay in range(c.L):
        tri.attn_prefill(c.kv, lay, q, o, lse=l)
        tri.attn_mass(c.kv, lay, q, l, mass)
    # every query gives each head's rows weights that sum to 1
    total = f64(mass).sum(1)
    assert np.allclose(total, 32 * G, rtol=1e-5)
    for step in range(3):
        qt = torch.randn(c.B, c.H * G, c.d, generator=c.g, device="cuda").to(c.dtype)
        ot = torch.empty_like(qt)
        for lay in range(c.L):
            tri.attn_decode(c.kv, lay, qt, ot, mass=mass)
    c.ok()
    assert np.allclose(f64(mass).sum(1), 35 * G, rtol=1e-5)
    budget, P, W = 64, 4, 16
    keep = torch.zeros(S, budget, dtype=torch.int32, device="cuda")
    m0 = mass.cpu().numpy().copy()
    tri.mass_evict(c.kv, mass, mass, P, W, budget, keep)
    c.ok()
    old = c.lens.copy()
    kr, vr = np.full_like(c.kr, np.nan), np.full_like(c.vr, np.nan)
    for b in range(c.B):
        for lay in range(c.L):
            for h in range(c.H):
                s = c.slice(b, lay, h)
                ref = evict(m0[s], int(old[b, h]), P, W, budget)
                assert np.array_equal(keep[s].cpu().numpy(), ref)
                kr[b, lay, h, :budget] = c.kr[b, lay, h, ref]
                vr[b, lay, h, :budget] = c.vr[b, lay, h, ref]
    c.kr, c.vr, c.lens = kr, vr, np.full_like(c.lens, budget)
    check_decode(c, G, layer=layer, with_mass=True)
    check_decode(c, G, layer=0, n_sink=4, window=20, with_mass=True)
    check_prefill(c, G, [16, 5], layer=layer)


def test_prefill_sequences_left_out_and_scale():
    check_prefill(Case([[50, 60], [33, 200], [0, 4]], 128, torch.bfloat16), 3, [0, 33, 4], n_q=40, scale=0.2)
    check_prefill(Case([[50, 60], [33, 200], [0, 4]], 64, torch.float32), 2, [20, 0, 4], n_q=30, scale=0.2)


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_many_tiles(d):
    """More query tiles than the GPU has SMs for in one go: the kernel with several CTAs' worth of work per SM (few queries
    go through another), sampled against the definition."""
    B, H, G, n_new, n = 8, 8, 2, 300, 700
    c = Case([[n] * H] * B, d, torch.bfloat16, L=1)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(B, n_new, H * G, d, generator=g, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(B, n_new, H * G, device="cuda")
    for n_sink, window in ((0, 0), (4, 150)):
        tri.attn_prefill(c.kv, 0, q, out, n_sink=n_sink, window=window, lse=lse)
        mass0 = torch.rand(B * H, c.n_cap, generator=g, device="cuda")
        mass = mass0.clone()
        tri.attn_mass(c.kv, 0, q, lse, mass, n_sink=n_sink, window=window)
        c.ok()
        qn, on, ln, mn = f64(q), f64(out), f64(lse), f64(mass) - f64(mass0)
        for b, h in ((0, 0), (3, 5), (7, 7)):
            k, v = c.rows(b, 0, h)
            total = np.zeros(n)
            for i in range(n_new):
                for gq in range(G):
                    r, hq = n - n_new + i, h * G + gq
                    o, l, w = attend(qn[b, i, hq], k, v, r, d ** -0.5, n_sink, window)
                    to, tl, _ = _bounds(qn[b, i, hq], k, v, r, d ** -0.5, w, o, l, n_sink, window, torch.bfloat16, 2.0 ** -8)
                    assert np.all(np.abs(on[b, i, hq] - o) <= to) and abs(ln[b, i, hq] - l) <= tl
                    total += w
            # (mass0 < 1 is added in fp32: half a step of the sum, and the weights' own error, see check_prefill)
            assert np.all(np.abs(mn[b * H + h, :n] - total) <= 1e-4 * total + 2.0 ** -23 * (total + 1))


@pytest.mark.parametrize("n_q", [64, 65, 130])
def test_mass_of_more_queries_than_stay_resident(n_q):
    # group 4: 32 tokens to a query tile; two tiles stay in shared memory, more stream past the rows
    check_prefill(Case([[n_q + 40, 300]], 128, torch.bfloat16, L=1, block=16), 4, [n_q], layer=0)
    check_prefill(Case([[n_q + 200, n_q + 1]], 64, torch.bfloat16, L=1), 4, [n_q], layer=0, n_sink=3, window=50)


@pytest.mark.parametrize("layout", ["blh", "lbh"])
def test_pool_layouts(layout):
    """A pool whose layers are outermost (a view with other strides) gives the same bits."""
    c = Case([[70, 33], [100, 129]], 128, torch.bfloat16, L=3, block=32)
    if layout == "lbh":
        for name in ("k", "v"):
            x = getattr(c.kv, name)
            setattr(c.kv, name, x.permute(1, 0, 2, 3, 4).contiguous().permute(1, 0, 2, 3, 4))
    check_decode(c, 4, layer=2, with_mass=True)
    check_prefill(c, 2, [33, 40], layer=2)


def test_queries_broadcast_over_sequences():
    c = Case([[70, 33], [100, 129], [5, 6]], 64, torch.bfloat16)
    one = torch.randn(1, 5, 6, 64, device="cuda").to(torch.bfloat16)
    out, ref = torch.zeros(3, 5, 6, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 5, 6, 64, dtype=torch.bfloat16, device="cuda")
    lse, lse_ref = torch.zeros(3, 5, 6, device="cuda"), torch.zeros(3, 5, 6, device="cuda")
    m, m_ref = torch.zeros(12, c.n_cap, device="cuda"), torch.zeros(12, c.n_cap, device="cuda")
    q = one.expand(3, 5, 6, 64)
    tri.attn_prefill(c.kv, 0, q, out, lse=lse)
    tri.attn_prefill(c.kv, 0, q.contiguous(), ref, lse=lse_ref)
    tri.attn_mass(c.kv, 0, q, lse, m)
    tri.attn_mass(c.kv, 0, q.contiguous(), lse, m_ref)
    c.ok()
    assert torch.equal(out, ref) and torch.equal(lse, lse_ref) and torch.equal(m, m_ref)
    d, d_ref = torch.zeros(3, 6, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 6, 64, dtype=torch.bfloat16, device="cuda")
    tri.attn_decode(c.kv, 0, q[:, 0], d)
    tri.attn_decode(c.kv, 0, q[:, 0].contiguous(), d_ref)
    c.ok()
    assert torch.equal(d, d_ref)


@pytest.mark.parametrize("lens", [[[900, 1500], [40, 2000]], [[30000, 20001]]])
def test_captured_calls_follow_the_cache(lens):
    """A captured step replayed after the cache grew equals the eager calls, bit for bit, on a stream of its own."""
    c = Case(lens, 128, torch.bfloat16, L=1, n_cap=max(map(max, lens)) + 40)
    G, B = 4, len(lens)
    S = B * 2
    c.kv.k.nan_to_num_(0.5)
    c.kv.v.nan_to_num_(0.25)
    q = torch.randn(B, 9, 8, 128, device="cuda").to(torch.bfloat16)
    nn = torch.full((B,), 9, dtype=torch.int32, device="cuda")
    ws = torch.empty(tri.attn_decode_workspace_bytes(c.kv, G, True), dtype=torch.uint8, device="cuda")

    def bufs():
        return (torch.zeros(B, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, 9, 8, 128, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(B, 9, 8, device="cuda"), torch.zeros(S, c.n_cap, device="cuda"))

    def step(d, o, l, m):
        tri.attn_prefill(c.kv, 0, q, o, n_new=nn, lse=l, n_sink=4, window=500)
        tri.attn_mass(c.kv, 0, q, l, m, n_new=nn, n_sink=4, window=500)
        tri.attn_decode(c.kv, 0, q[:, 0], d, mass=m, workspace=ws)

    captured, eager = bufs(), bufs()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(*bufs())
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(*captured)
    torch.cuda.synchronize()
    for b in captured:
        b.zero_()
    for grow in (0, 7, 20):
        c.kv.n_valid += grow
        nn.fill_(9 - grow // 7)
        graph.replay()
        torch.cuda.synchronize()
        step(*eager)
        torch.cuda.synchronize()
        for x, y in zip(captured, eager):
            assert torch.equal(x, y)
    assert int(c.status.item()) == 0


def test_two_streams_at_once():
    """Calls on two streams, each with its workspace, do not disturb each other."""
    cases = [Case([[3000, 4000]] * 4, 128, torch.bfloat16, L=1, seed=i) for i in range(2)]
    for c in cases:
        c.kv.k.nan_to_num_(0.5)
        c.kv.v.nan_to_num_(0.25)
    q = torch.randn(4, 40, 8, 128, device="cuda").to(torch.bfloat16)

    def run(c, stream, ws):
        o, l = torch.zeros(4, 40, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 40, 8, device="cuda")
        m, d = torch.zeros(8, c.n_cap, device="cuda"), torch.zeros(4, 8, 128, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        return (o, l, m, d), lambda: (tri.attn_prefill(c.kv, 0, q, o, lse=l, stream=stream), tri.attn_mass(c.kv, 0, q, l, m, stream=stream),
                                      tri.attn_decode(c.kv, 0, q[:, 3], d, mass=m, workspace=ws, stream=stream))

    ref = []
    for c in cases:
        bufs, go = run(c, torch.cuda.current_stream(), None)
        go()
        torch.cuda.synchronize()
        ref.append(bufs)
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [torch.empty(tri.attn_decode_workspace_bytes(c.kv, 4, True), dtype=torch.uint8, device="cuda") for c in cases]
    for _ in range(3):
        got = [run(c, s, w) for c, s, w in zip(cases, streams, ws)]
        for _, go in got:
            go()
        torch.cuda.synchronize()
        for (bufs, _), want in zip(got, ref):
            for x, y in zip(bufs, want):
                assert torch.equal(x, y)


def test_calls_repeat_bit_for_bit():
    c = Case([[3000, 129], [64, 5000]], 64, torch.bfloat16, L=1, block=64)
    q = torch.randn(2, 70, 6, 64, device="cuda").to(torch.bfloat16)
    first = None
    for _ in range(3):
        o, l = torch.zeros_like(q), torch.zeros(2, 70, 6, device="cuda")
        m, d = torch.zeros(4, c.n_cap, device="cuda"), torch.zeros(2, 6, 64, dtype=torch.bfloat16, device="cuda")
        tri.attn_prefill(c.kv, 0, q, o, lse=l, n_new=torch.tensor([70, 64], dtype=torch.int32, device="cuda"))
        tri.attn_mass(c.kv, 0, q, l, m, n_new=torch.tensor([70, 64], dtype=torch.int32, device="cuda"))
        tri.attn_decode(c.kv, 0, q[:, 0], d, mass=m)
        c.ok()
        got = (o, l, m, d)
        first = first or got
        for x, y in zip(got, first):
            assert torch.equal(x, y)


def test_neighbours_are_left_alone():
    """Guard bytes around every output and after the workspace, rows and slices of other layers."""
    c = Case([[130, 40], [64, 100]], 128, torch.bfloat16, L=2)
    def guarded(*shape, dtype):
        n = int(np.prod(shape)) * torch.tensor([], dtype=dtype).element_size()
        buf = torch.full((256 + n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[256:256 + n].view(dtype).view(shape)
    q = torch.randn(2, 33, 8, 128, device="cuda").to(torch.bfloat16)
    ob, o = guarded(2, 33, 8, 128, dtype=torch.bfloat16)
    lb, l = guarded(2, 33, 8, dtype=torch.float32)
    mb, m = guarded(8, c.n_cap, dtype=torch.float32)
    db, d = guarded(2, 8, 128, dtype=torch.bfloat16)
    m.zero_()
    k0, v0, nv0 = c.kv.k.clone(), c.kv.v.clone(), c.kv.n_valid.clone()
    tri.attn_prefill(c.kv, 1, q, o, lse=l)
    tri.attn_mass(c.kv, 1, q, l, m)
    tri.attn_decode(c.kv, 1, q[:, 0], d, mass=m)
    c.ok()
    for buf in (ob, lb, mb, db):
        assert bool((buf[:256] == 0xA5).all()) and bool((buf[-256:] == 0xA5).all())
    mm = m.view(2, 2, 2, -1)
    assert bool((mm[:, 0] == 0).all())  # layer 0's slices
    for b in range(2):
        for h in range(2):
            assert bool((mm[b, 1, h, int(c.lens[b, h]):] == 0).all())
    assert torch.equal(c.kv.k.view(torch.int16), k0.view(torch.int16)) and torch.equal(c.kv.v.view(torch.int16), v0.view(torch.int16))
    assert torch.equal(c.kv.n_valid, nv0)


def test_faults_are_reported_and_skipped():
    def fresh(**kw):
        return Case([[40, 50], [30, 60]], 64, torch.bfloat16, L=1, **kw)

    def run(c, n_new=None, n_q=1):
        q = torch.randn(2, n_q, 4, 64, device="cuda").to(torch.bfloat16)
        res = []
        o, l = torch.full((2, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, 4), 9.0, device="cuda")
        m = torch.zeros(4, c.n_cap, device="cuda")
        tri.attn_decode(c.kv, 0, q[:, 0], o, lse=l, mass=m, n_new=n_new)
        torch.cuda.synchronize()
        res.append((int(c.status.item()), o.float().cpu(), m.cpu()))
        c.status.zero_()
        op, lp = torch.full((2, n_q, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, n_q, 4), 1.0, device="cuda")
        tri.attn_prefill(c.kv, 0, q, op, lse=lp, n_new=n_new)
        torch.cuda.synchronize()
        res.append((int(c.status.item()), op.float().cpu()[:, 0], None))
        c.status.zero_()
        m2 = torch.zeros(4, c.n_cap, device="cuda")
        tri.attn_mass(c.kv, 0, q, torch.ones(2, n_q, 4, device="cuda"), m2, n_new=n_new)
        torch.cuda.synchronize()
        res.append((int(c.status.item()), None, m2.cpu()))
        c.status.zero_()
        return res

    c = fresh()
    c.kv.n_valid[1] = c.n_cap + 1  # sequence 0, head 1
    for st, o, m in run(c):
        assert st == tri.DEV_NVALID_OVER_CAP
        if o is not None:
            assert bool((o[0, 2:] == 9.0).all()) and bool((o[0, :2] != 9.0).all()) and bool((o[1] != 9.0).all())
        if m is not None:
            assert bool((m[1] == 0).all()) and bool((m[0, :40] > 0).all())
    c = fresh(block=16)
    c.kv.block_table[1, 2] = 1 << 20  # rows 32..47 of sequence 1: head 0 holds 30 rows, head 1 60
    for st, o, m in run(c):
        assert st == tri.DEV_BAD_BLOCK
        if o is not None:
            assert bool((o[1, 2:] == 9.0).all()) and bool((o[1, :2] != 9.0).all()) and bool((o[0] != 9.0).all())
    c = fresh()
    for st, o, m in run(c, n_new=torch.tensor([1, 2], dtype=torch.int32, device="cuda")):
        assert st == tri.DEV_BAD_QUERY
        if o is not None:
            assert bool((o[1] == 9.0).all()) and bool((o[0] != 9.0).all())


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_tiles_that_see_nothing(d):
    """Whole query tiles before the first cached row, in the kernel for many queries and the one for few."""
    for B, H, n_new in ((10, 8, 300), (1, 1, 300)):
        c = Case([[0] * H] * (B - 1) + [[7] * H], d, torch.bfloat16, L=1)
        q = torch.randn(B, n_new, H * 2, d, device="cuda").to(torch.bfloat16)
        out, lse = torch.full_like(q, 9.0), torch.zeros(B, n_new, H * 2, device="cuda")
        tri.attn_prefill(c.kv, 0, q, out, lse=lse)
        c.ok()
        assert bool((out[:-1] == 0).all()) and bool((lse[:-1] == float("-inf")).all())
        assert bool((out[-1, :-7] == 0).all()) and bool((lse[-1, :-7] == float("-inf")).all())
        assert bool((out[-1, -7:].float().abs().amax(-1) > 0).all()) and bool(torch.isfinite(lse[-1, -7:]).all())


@pytest.mark.parametrize("B,L,H,n,budget", [(2, 1, 8, 5000, 4300), (2, 1, 8, 5000, 700), (10, 2, 8, 700, 600), (1, 1, 1, 9000, 8999)])
@pytest.mark.parametrize("block", [0, 32])
@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.float32)])
def test_mass_evict_moves_what_select_compact_moves(B, L, H, n, budget, block, d, dtype):
    """Few and many slices (they take different tiles) and rows over many tiles, against tri_select_compact bit for bit."""
    res = []
    for own in (False, True):
        c = Case([[n - 3 * h for h in range(H)]] * B, d, dtype, L=L, block=block, seed=3)
        S = B * L * H
        mass = torch.exp(2 * torch.randn(S, c.n_cap, generator=c.g, device="cuda"))
        keep = torch.zeros(S, budget, dtype=torch.int32, device="cuda")
        if own:
            out = torch.full_like(mass, 5.0)
            tri.mass_evict(c.kv, mass, out, 20, 30, budget, keep)
            c.ok()
            k = keep.clamp(min=0).long()
            kept, old = (keep >= 0).sum(1, keepdim=True), torch.tensor([n - 3 * h for h in range(H)] * (B * L), device="cuda")[:, None]
            j = torch.arange(c.n_cap, device="cuda")[None]
            want = torch.where(j < old, 0.0, 5.0)
            want = torch.where(j < kept, torch.nn.functional.pad(mass.gather(1, k), (0, c.n_cap - budget)), want)
            assert torch.equal(out, want)
        else:
            tri.select_compact(mass, c.kv, 20, 30, budget, keep)
            c.ok()
        bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
        res.append((keep, c.kv.n_valid.clone(), c.kv.pos_out.clone(), c.kv.k.view(bits).clone(), c.kv.v.view(bits).clone()))
    for x, y in zip(*res):
        assert torch.equal(x, y)
