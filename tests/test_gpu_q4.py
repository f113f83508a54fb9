"""Caches in 4 bits: attention over them (tri_attn_decode, tri_attn_prefill_q4), rows
read back (tri_read_rows), and the compactions, against the definitions in 64 bits.

Tolerances, for one query with weights w over rows j, c codes, s scales, m minima:
  logits   x = scale * sum over quarters of (s (q.c) + m sum q). q in fp16 is exact to 2^-35 of
           its largest element, products with codes are exact, each of at most d / 4 + 8 additions
           and the scalings err by at most 2^-23 of the running magnitude (truncation
           included); the quarters' sums of q go in to 2^-22. With
           B = sum_e |q_e| (s c_e + |m|), the largest over the visible rows,
           |dx| <= (d / 4 + 16) 2^-23 scale B =: ex.
  weights  as for bf16 caches: ew = 2 ex + 2^-20 + 2^-22 max|x|.
  out      weights rounded to fp16, then their product with the scale: p = 2^-10 of
           A = sum w (s c + |m|) at most, and where they are subnormal 2^-25 of 2^4 (the largest weight):
           n 2^-29 (15 + max (s c + |m|)). fp32 sums n 2^-24 A. Result rounded to bf16.
  lse, mass  as for bf16 caches.
For a chunk K is a bf16 pair, 2^-16 of a value (half a step of half a step) in every product, V and the
weights are fp16, 2^-11 each: ex = (d + 10) 2^-23 scale sum |q k| + 2^-16 scale sum |q k|, p = 2^-10 of
A = sum w |v|, and for the subnormal ones of weights up to 2^6 and more, and of V: n 2^-31 max |v| + 2^-25.
"""
import numpy as np
import pytest
import torch

import kv_cache_compression_tri_gb300 as tri
from attn_oracle import attend, evict
from gpu_helpers import f64
from q4_oracle import values
from test_gpu_append import Cache, close, host
from q4_oracle import pack, rotate

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tri.load_library()


class Case(Cache):
    """A 4-bit cache of random codes, scales and minima; rows past the counts have NaN scales and minima."""

    def __init__(self, lens, d, cap=None, L=2, block=0, seed=0, big=0.4):
        lens = np.asarray(lens)
        cap = cap or int(max(lens.max(), 1)) + 5
        if block:
            cap = (cap + block - 1) // block * block
        super().__init__(lens, d, torch.uint8, cap, L, block, seed)
        for p in self.pools:
            pairs = torch.rand(*p.shape[:4], 4, 2, generator=self.g, device="cuda") * big + big / 8
            pairs[..., 1] = -pairs[..., 1] * 7.5 + torch.randn(pairs.shape[:-1], generator=self.g, device="cuda") * big
            p[..., d // 2:] = pairs.half().view(*p.shape[:4], 8).view(torch.uint8)
        nan = torch.full((4, 2), NAN, device="cuda").half().view(8).view(torch.uint8)
        for b in range(self.B):
            for h in range(self.H):
                for layer in range(L):
                    for r in range(int(lens[b, h]), cap):
                        for p in self.pools:
                            p[self.place(b, layer, h, r)][d // 2:] = nan
        self.h = [host(p) for p in self.pools]

    def slice_rows(self, b, layer, h):
        """Bytes of the slice's rows, K and V."""
        return [self.rows(x, b, layer, h, 0, int(self.lens[b, h])) for x in self.h]

    def ok(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0


def sizes(rows):
    """scale * code + |minimum| of every element."""
    d = (rows.shape[-1] - 16) * 2
    m = np.ascontiguousarray(rows[..., d // 2:]).view(np.float16).astype(np.float64)[..., 1::2]
    m = np.repeat(m, d // 4, -1)
    return (values(rows) - m) + np.abs(m)


def check_decode(c, G, layer=1, n_sink=0, window=0, with_mass=False, n_new=None, scale=None, seed=1, qscale=1.0, repeat=False):
    B, H, d = c.B, c.H, c.d
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn(B, 3, H * G, d, generator=g, device="cuda") * qscale).bfloat16()[:, 1]
    out = torch.full((B, H * G, d), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H * G), 9.0, device="cuda")
    mass0 = torch.rand(B * c.L * H, c.cap, generator=g, device="cuda")
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
    for b in range(B):
        for h in range(H):
            kb, vb = c.slice_rows(b, layer, h)
            k, v = values(kb), values(vb)
            n = len(kb)
            for gq in range(G):
                hq = h * G + gq
                if n_new is not None and n_new[b] == 0:
                    assert (got_o[b, hq] == 9.0).all() and got_l[b, hq] == 9.0
                    continue
                o, l, w = attend(qn[b, hq], k, v, n - 1, sc, n_sink, window) if n else (np.zeros(d), -np.inf, np.zeros(0))
                seen = w > 0
                if not seen.any():
                    assert (got_o[b, hq] == 0).all() and got_l[b, hq] == -np.inf
                    continue
                ex = (d / 4 + 16) * 2.0 ** -23 * sc * (sizes(kb[seen]) @ np.abs(qn[b, hq])).max()
                x = sc * (k[seen] @ qn[b, hq])
                ew = 2 * ex + 2.0 ** -20 + 2.0 ** -22 * np.abs(x).max()
                sv = sizes(vb[seen])
                A = w[seen] @ sv
                tol = A * (2 * ew + 2.0 ** -10 + n * 2.0 ** -24) + n * 2.0 ** -29 * (15 + sv.max()) + 2.0 ** -8 * np.abs(o)
                assert (np.abs(got_o[b, hq] - o) <= tol).all(), (b, hq, float((np.abs(got_o[b, hq] - o) / tol).max()))
                assert abs(got_l[b, hq] - l) <= ex + ew + 2.0 ** -22 * max(1.0, abs(l))
                if with_mass:
                    s = (b * c.L + layer) * H + h
                    ref_m[s, :n] += w
                    tol_m[s, :n] += w * (2 * ew + 2.0 ** -22)
    if with_mass:
        untouched = tol_m == 0
        assert np.array_equal(got_m[untouched], ref_m[untouched])
        assert (np.abs(got_m - ref_m) <= tol_m + 2.0 ** -23 * ref_m).all()
    return out, lse, mass


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [0, 16, 64])
def test_decode_ragged(d, block):
    check_decode(Case([[0, 1, 31], [32, 33, 200]], d, block=block), 4, with_mass=True)


@pytest.mark.parametrize("group", range(1, 9))
def test_decode_groups(group):
    check_decode(Case([[70, 5]], 128 if group % 2 else 64), group, with_mass=group > 4)


@pytest.mark.parametrize("lens", [[[1]], [[2]], [[15]], [[16]], [[17]], [[64]], [[65]], [[1000]], [[2113] * 8], [[3000, 2]] * 3])
def test_decode_lengths(lens):
    check_decode(Case(lens, 128, L=1), 2, layer=0, with_mass=True)


@pytest.mark.parametrize("n_sink,window,block", [(0, 1, 0), (4, 30, 16), (40, 100, 16), (4, 100, 64), (130, 64, 0), (0, 199, 0), (3, 4000, 0), (7, 33, 32)])
def test_decode_sinks_and_window(n_sink, window, block):
    check_decode(Case([[150, 201], [3, 64]], 64, block=block), 3, n_sink=n_sink, window=window, with_mass=True)


def test_decode_sequences_left_out_and_scale():
    check_decode(Case([[33, 20], [40, 8]], 128), 2, n_new=[0, 1], scale=0.3, with_mass=True)


@pytest.mark.parametrize("qscale", [1e-30, 1e-3, 30.0])
def test_decode_sizes_of_queries(qscale):
    check_decode(Case([[300, 40]], 128, L=1), 4, layer=0, qscale=qscale)


@pytest.mark.parametrize("big", [1e-3, 200.0])
def test_decode_sizes_of_values(big):
    check_decode(Case([[300, 40]], 64, L=1, big=big), 4, layer=0, scale=0.02 if big > 1 else None)


def test_decode_zero_query():
    check_decode(Case([[300, 40]], 64, L=1), 2, layer=0, qscale=0.0)


def test_decode_long_rows_sampled():
    # many runs per slice, joined by the second kernel; offsets of a pool past 2^31 bytes
    check_decode(Case([[8192]], 128, L=1, block=256), 1, layer=0, with_mass=True)


def test_offsets_past_32_bits():
    # a pool of which every block but the last ones lies past 2^31 bytes; slices too
    nb, block = 30000, 256
    k = torch.zeros(nb, 1, 4, block, 80, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    small = Case([[600, 500, 1, 300]], 128, L=1, block=block)
    per = small.table.shape[1]
    table = torch.arange(nb - per, nb, dtype=torch.int32, device="cuda").view(1, per)
    for big, pool in ((k, small.pools[0]), (v, small.pools[1])):
        big[nb - per:] = pool[small.table[0].long()]
    q = torch.randn(1, 16, 128, device="cuda").bfloat16()
    outs = []
    for kv in (small.kv, tri.PagedKVCache(k, v, table, small.kv.n_valid, None, None, small.status, post_rope=True)):
        out, rows = torch.zeros_like(q), torch.zeros(1, 4, small.cap, 128, dtype=torch.bfloat16, device="cuda")
        chunks = []
        tri.attn_decode(kv, 0, q, out)
        tri.read_rows(kv, 0, rows, None)
        for n in (2, 20):  # read, and written out
            chunks.append(torch.zeros(1, n, 16, 128, dtype=torch.bfloat16, device="cuda"))
            tri.attn_prefill(kv, 0, q.view(1, 1, 16, 128).expand(1, n, 16, 128).contiguous(), chunks[-1])
        outs.append((out, rows, *chunks))
    small.ok()
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("order", [(0, 1, 2), (2, 0, 1), (1, 2, 0)])
@pytest.mark.parametrize("pad", [0, 1, 3])
def test_pools_in_any_order(order, pad):
    """Blocks, layers and heads in any order in memory, with rows of 16 bytes between."""
    c = Case([[70, 33], [5, 64]], 64, block=16)
    nb, L, H, bs, w = c.pools[0].shape
    dims = (nb, L, H)
    views = []
    for p in c.pools:
        flat = torch.full([dims[i] for i in order] + [bs * w + 16 * pad], 0xFF, dtype=torch.uint8, device="cuda")
        rows = flat[..., :bs * w].view(*[dims[i] for i in order], bs, w) if pad == 0 else flat[..., :bs * w].unflatten(-1, (bs, w))
        view = rows.permute(*[order.index(i) for i in range(3)], 3, 4)
        view.copy_(p)
        views.append(view)
    kv = tri.PagedKVCache(*views, c.kv.block_table, c.kv.n_valid, None, None, c.status, post_rope=True)
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    tri.attn_decode(c.kv, 1, q, a)
    tri.attn_decode(kv, 1, q, b)
    c.ok()
    assert torch.equal(a, b)


@pytest.mark.parametrize("n_slices,rows", [(38, 65536), (19, 131072), (20, 65600), (60, 33000), (304, 8192), (400, 4096)])
def test_runs_stay_within_the_workspace(n_slices, rows):
    k = torch.randint(0, 256, (1, 1, n_slices, rows, 48), dtype=torch.uint8, device="cuda")
    k[..., 32:] = torch.tensor([0.125, -1.0] * 4).half().view(torch.uint8).cuda()
    nv = torch.full((n_slices,), rows, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = tri.KVCache(k, k, nv, None, None, status, post_rope=True)
    q = torch.zeros(1, n_slices, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    need = tri.attn_decode_workspace_bytes(kv, 1)
    ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    tri.attn_decode(kv, 0, q, out, workspace=ws[:need])
    assert int(status) == 0 and bool((ws[need:] == 0xA5).all())
    # equal weights: the mean of the rows. Weights are exact; 32-bit sums and the result's rounding
    rows_out = torch.zeros(1, n_slices, rows, 64, dtype=torch.bfloat16, device="cuda")
    tri.read_rows(kv, 0, None, rows_out)  # (codes / 8 - 1: exact in bf16)
    want = rows_out.double().mean(2)
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + rows * 2.0 ** -24 * 2).all())


def test_bad_row_counts():
    c = Case([[40, 39], [60, 50]], 64)
    c.kv.n_valid[4] = c.cap + 1  # sequence 1, layer 0, head 0
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    out = torch.full((2, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    tri.attn_decode(c.kv, 0, q, out)
    assert int(c.status) == 1 and bool((out[1, :2] == 9).all()) and bool((out[1, 2:] != 9).any()) and bool((out[0] != 9).any())
    c.status.zero_()
    for n in (3, 41):
        chunk, x = torch.full((2, n, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda"), torch.randn(2, n, 4, 64, device="cuda").bfloat16()
        tri.attn_prefill(c.kv, 0, x, chunk)
        assert int(c.status) == 1 and bool((chunk[1, :, :2] == 9).all()) and bool((chunk[0] != 9).any())
        c.status.zero_()


def test_decode_repeats_bit_for_bit():
    c = Case([[700, 40], [2, 333]], 128, block=16)
    a, b = check_decode(c, 4, with_mass=True), check_decode(c, 4, with_mass=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("what", [-1, 1 << 20])
def test_decode_blocks_out_of_sight(block, what):
    c = Case([[400, 390]], 64, block=block)
    w = 400 - 2 * block
    for e in range(1, (390 - w) // block):  # blocks with no row in either run
        c.kv.block_table[0, e] = what
    check_decode(c, 2, n_sink=3, window=w, with_mass=True)


@pytest.mark.parametrize("n", [200, 3000])
def test_decode_reports_a_bad_block(n):
    c = Case([[n, 9], [20, 30]], 64, L=1, block=16)
    c.kv.block_table[0, n // 32] = -1
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    out = torch.full((2, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    mass = torch.zeros(4, c.cap, device="cuda")
    tri.attn_decode(c.kv, 0, q, out, mass=mass)
    assert int(c.status) == 6
    assert bool((out[0, :2] == 9).all()) and bool((out[0, 2:] != 9).any()) and bool((out[1] != 9).any())
    assert not bool(mass[0].any()) and bool(mass[1].any())


def bf16(x):
    return torch.from_numpy(x).float().bfloat16().double().numpy()


def test_read_rows():
    for d, block in ((64, 0), (128, 16), (64, 32), (128, 0)):
        c = Case([[0, 1, 70], [33, 64, 65]], d, block=block)
        k, v = (torch.full((2, 3, c.cap, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        tri.read_rows(c.kv, 1, k, v)
        c.ok()
        for b in range(2):
            for h in range(3):
                n = int(c.lens[b, h])
                for got, rows in zip((k, v), c.slice_rows(b, 1, h)):
                    # (minimum + scale * code is rounded to fp32 first: fp16 pairs and 4-bit codes, exact in fp64)
                    assert np.array_equal(f64(got[b, h, :n]), bf16(values(rows)))
                    assert bool((got[b, h, n:] == 9).all())
        v2 = torch.full_like(v, 9.0)
        tri.read_rows(c.kv, 1, None, v2)
        assert torch.equal(v, v2)


def test_read_rows_leaves_out_faults():
    c = Case([[40, 70], [33, 64]], 64, L=1, block=16)
    c.kv.n_valid[1] = c.cap + 1
    c.kv.block_table[1, 1] = -5
    k = torch.full((2, 2, c.cap, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    tri.read_rows(c.kv, 0, k, None)
    assert int(c.status) in (1, 6)
    assert bool((k[0, 1] == 9).all()) and bool((k[1, :, 16:32] == 9).all())
    assert np.array_equal(f64(k[1, 1, 32:64]), bf16(values(c.slice_rows(1, 0, 1)[0]))[32:64])


def check_prefill(c, G, n_q, layer=1, n_new=None, n_sink=0, window=0, seed=1, expect=0, left_out=()):
    B, H, d = c.B, c.H, c.d
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(B, n_q, H * G, d, generator=g, device="cuda").bfloat16()
    out = torch.full((B, n_q, H * G, d), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, n_q, H * G), 9.0, device="cuda")
    nn = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device="cuda")
    need = tri.attn_prefill_workspace_bytes(c.kv)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # (NaN wherever it is read as bf16)
    tri.attn_prefill(c.kv, layer, q, out, n_new=nn, n_sink=n_sink, window=window, lse=lse, workspace=ws[:need])
    torch.cuda.synchronize()
    assert int(c.status) == expect
    assert bool((ws[need:] == 0xFF).all())
    sc = d ** -0.5
    got_o, got_l, qn = f64(out), f64(lse), f64(q)
    for b in range(B):
        new = n_q if n_new is None else n_new[b]
        if b in left_out:
            assert (got_o[b] == 9).all() and (got_l[b] == 9).all()
            continue
        assert (got_o[b, new:] == 9).all() and (got_l[b, new:] == 9).all()
        for h in range(H):
            kb, vb = c.slice_rows(b, layer, h)
            k, v = values(kb), values(vb)
            n = len(k)
            few = -(-n_q // (8 // G)) <= 8  # passes of the decode kernel
            for i in range(new):
                for hq in range(h * G, (h + 1) * G):
                    o, l, w = attend(qn[b, i, hq], k, v, n - new + i, sc, n_sink, window) if n else (np.zeros(d), -np.inf, np.zeros(0))
                    seen = w > 0
                    if not seen.any():
                        assert (got_o[b, i, hq] == 0).all() and got_l[b, i, hq] == -np.inf
                        continue
                    if few:  # the decode's: codes, scales and minima apart
                        ex = (d / 4 + 16) * 2.0 ** -23 * sc * (sizes(kb[seen]) @ np.abs(qn[b, i, hq])).max()
                        sv = sizes(vb[seen])
                        small = n * 2.0 ** -29 * (15 + sv.max())
                    else:
                        ex = ((d + 10) * 2.0 ** -23 + 2.0 ** -16) * sc * (np.abs(k[seen]) @ np.abs(qn[b, i, hq])).max()
                        sv = np.abs(v[seen])
                        small = n * 2.0 ** -31 * sv.max() + 2.0 ** -25
                    x = sc * (k[seen] @ qn[b, i, hq])
                    ew = 2 * ex + 2.0 ** -20 + 2.0 ** -22 * np.abs(x).max()
                    tol = (w[seen] @ sv) * (2 * ew + 2.0 ** -10 + n * 2.0 ** -24) + small + 2.0 ** -8 * np.abs(o)
                    assert (np.abs(got_o[b, i, hq] - o) <= tol).all()
                    assert abs(got_l[b, i, hq] - l) <= ex + ew + 2.0 ** -22 * max(1.0, abs(l))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [0, 16, 64])
def test_prefill_ragged(d, block):
    check_prefill(Case([[40, 1, 131], [64, 33, 200]], d, block=block), 3, 33, n_new=[33, 20])  # 17 passes: written out


@pytest.mark.parametrize("n_sink,window", [(0, 1), (4, 30), (40, 100), (130, 64), (3, 4000)])
def test_prefill_sinks_and_window(n_sink, window):
    check_prefill(Case([[450, 301]], 64, block=16), 2, 40, n_sink=n_sink, window=window)  # 10


def test_prefill_queries_before_the_first_row():
    check_prefill(Case([[3, 0], [9, 12]], 128), 2, 7, n_new=[7, 0])
    check_prefill(Case([[3, 0], [9, 12]], 128), 2, 37, n_new=[37, 0])


# Few tokens read the 4-bit rows themselves, with the decode's tolerances: a weight's two roundings are of its products with
# scale * code and with the minimum, so they count on s c + |m|, which is more than |v| where the two nearly cancel.
@pytest.mark.parametrize("n_q,group", [(1, 8), (2, 4), (2, 3), (3, 2), (5, 1), (8, 1), (3, 4), (5, 3), (16, 4), (8, 5), (33, 1), (64, 1)])
@pytest.mark.parametrize("block,n_sink,window", [(0, 0, 0), (64, 0, 0), (16, 3, 20), (32, 40, 64)])
def test_prefill_of_few_tokens(n_q, group, block, n_sink, window):
    c = Case([[0, 1, 70], [33, 200, 64], [5, 129, 3]], 64 if n_q % 2 else 128, block=block)
    check_prefill(c, group, n_q, n_new=[n_q, max(n_q - 1, 1), n_q // 2], n_sink=n_sink, window=window)


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_of_few_tokens_over_many_rows(d):
    check_prefill(Case([[5000, 4990]], d, L=1), 2, 3, layer=0)
    check_prefill(Case([[5000, 4990]], d, L=1, block=64), 4, 2, layer=0, n_sink=7, window=3000)
    check_prefill(Case([[3] * 3] * 100, d, L=1, cap=64), 1, 5, layer=0)  # (tokens before the first row)
    check_prefill(Case([[5000, 4990]], d, L=1, block=64), 4, 7, layer=0, n_sink=7, window=3000)
    check_prefill(Case([[3, 20] * 2] * 9, d, L=1, cap=64), 8, 6, layer=0, n_new=[6, 0, 1, 2, 3, 4, 5, 6, 6])


def test_prefill_of_few_tokens_with_faults():
    c = Case([[400, 390], [60, 50]], 64, block=16)
    for e in range(2, 10):  # rows 32 .. 159
        c.kv.block_table[0, e] = -1
    check_prefill(c, 2, 3, n_sink=5, window=100)
    c.kv.block_table[0, 20] = 1 << 20
    check_prefill(c, 2, 3, n_sink=5, window=100, expect=6, left_out=(0,))
    check_prefill(Case([[40, 39], [60, 50]], 64), 2, 3, n_new=[4, 3], expect=7, left_out=(0,))


@pytest.mark.parametrize("n_q", [20, 41])  # read, and written out
@pytest.mark.parametrize("what", [-1, 1 << 20])
def test_prefill_blocks_out_of_sight_and_bad_ones(what, n_q):
    c = Case([[400, 390], [60, 50]], 64, block=16)
    for e in range(2, 10):  # rows 32 .. 159
        c.kv.block_table[0, e] = what
    check_prefill(c, 2, n_q, n_sink=5, window=100)  # (the first rows that a window sees: 250 and on)
    c.kv.block_table[0, 20] = what
    check_prefill(c, 2, n_q, n_sink=5, window=100, expect=6, left_out=(0,))


def test_prefill_of_few_tokens_leaves_out_those_that_need_a_bad_block():
    outs = []
    for bad in (False, True):
        c = Case([[400, 399, 350]], 64, block=16)
        q = torch.randn(1, 20, 6, 64, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
        out, lse = torch.full_like(q, 9.0), torch.full((1, 20, 6), 9.0, device="cuda")
        if bad:
            c.kv.block_table[0, 17] = -1  # rows 272 .. 287: seen from rows up to 386
        tri.attn_prefill(c.kv, 0, q, out, n_sink=5, window=100, lse=lse)
        outs += [out[0].view(20, 3, 2, 64), lse[0].view(20, 3, 2)]
    assert int(c.status) == 6
    for want, got in zip(outs[:2], outs[2:]):
        assert bool((got[:8, 0] == 9).all()) and bool((got[:8, 1] == 9).all())  # tokens 0 .. 6 and 0 .. 7, by fours
        assert torch.equal(got[8:, :2], want[8:, :2]) and bool((got[:, 2] == 9).all())


@pytest.mark.parametrize("n_q", [20, 41])
def test_prefill_bad_counts(n_q):
    c = Case([[40, 39], [60, 50]], 64)
    check_prefill(c, 2, n_q, n_new=[n_q + 1, n_q], expect=7, left_out=(0,))


@pytest.mark.parametrize("n_q", [5, 41])
def test_captured_attention_follows_the_cache(n_q):
    c = Case([[100, 90]], 128, block=16)
    q = torch.randn(1, n_q, 4, 128, device="cuda").bfloat16()
    out, lse = torch.zeros_like(q), torch.zeros(1, n_q, 4, device="cuda")
    dout = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(tri.attn_prefill_workspace_bytes(c.kv), dtype=torch.uint8, device="cuda")
    dws = torch.empty(tri.attn_decode_workspace_bytes(c.kv, 2), dtype=torch.uint8, device="cuda")

    def run():
        tri.attn_prefill(c.kv, 1, q, out, lse=lse, workspace=ws)
        tri.attn_decode(c.kv, 1, q[:, 4], dout, workspace=dws)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    c.kv.n_valid.copy_(torch.tensor([0, 0, 61, 50], dtype=torch.int32))
    graph.replay()
    got = out.clone(), dout.clone()
    run()
    assert torch.equal(out, got[0]) and torch.equal(dout, got[1])
    c.ok()


def test_two_streams_at_once():
    cs = [Case([[700, 650]], 128, block=16, seed=s) for s in range(2)]
    qs = [torch.randn(1, 4, 128, device="cuda").bfloat16() for _ in range(2)]
    want = []
    for c, q in zip(cs, qs):
        o = torch.zeros_like(q)
        tri.attn_decode(c.kv, 0, q, o)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(q) for q in qs]
    for _ in range(20):
        for c, q, o, s in zip(cs, qs, outs, streams):
            s.wait_stream(torch.cuda.current_stream())
            tri.attn_decode(c.kv, 0, q, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("block", [0, 16, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("call", ["compact", "select", "random", "mass"])
def test_compactions_move_4_bit_rows(block, d, call):
    B, L, H, n, budget, P, W = 2, 2, 2, 300, 120, 10, 7
    c = Case([[n] * H] * B, d, L=L, block=block)
    S = B * L * H
    pos_out = torch.full((S, c.cap), -7, dtype=torch.int32, device="cuda")
    c.pos.copy_(torch.arange(c.cap, device="cuda").expand(S, -1) * 3)
    c.kv.pos_out = pos_out
    score = torch.rand(S, c.cap, generator=c.g, device="cuda")
    keep = torch.full((S, budget), -9, dtype=torch.int32, device="cuda")
    mass_out = torch.full_like(score, 5.0)
    if call == "compact":
        tri.select_topk(score, c.kv, P, W, budget, keep)
        tri.compact_kv(c.kv, keep, budget)
    elif call == "select":
        tri.select_compact(score, c.kv, P, W, budget, keep)
    elif call == "random":
        tri.rand_evict_compact(c.kv, 5, 1, P, W, budget, keep)
    else:
        tri.mass_evict(c.kv, score, mass_out, P, W, budget, keep)
    c.ok()
    after = [host(p) for p in c.pools]
    kept, sc = keep.cpu().numpy(), f64(score)
    for b in range(B):
        for layer in range(L):
            for h in range(H):
                s = (b * L + layer) * H + h
                if call != "random":
                    assert np.array_equal(kept[s], evict(sc[s], n, P, W, budget))
                for was, now in zip(c.h, after):
                    old = c.rows(was, b, layer, h, 0, n)
                    assert np.array_equal(c.rows(now, b, layer, h, 0, budget), old[kept[s]])
                    assert np.array_equal(c.rows(now, b, layer, h, budget, n), old[budget:])
                assert np.array_equal(pos_out[s, :budget].cpu().numpy(), 3 * kept[s])
                if call == "mass":
                    assert np.array_equal(f64(mass_out[s, :budget]), sc[s, kept[s]]) and not bool(mass_out[s, budget:n].any())
    assert bool((c.kv.n_valid == budget).all())
    if not block:  # the guard rows between slices
        assert all(np.array_equal(x[:, :, :, c.cap:], y[:, :, :, c.cap:]) for x, y in zip(c.h, after))


def test_eviction_of_many_slices_in_4_bits():
    S, cap, budget = 200, 1024, 640
    k, v = (torch.randint(0, 256, (1, 25, 8, cap, 80), dtype=torch.uint8, device="cuda") for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    nv = torch.full((S,), 1000, dtype=torch.int32, device="cuda")
    pos_out = torch.zeros(S, cap, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = tri.KVCache(k, v, nv, None, pos_out, status, post_rope=True)
    mass = torch.rand(S, cap, device="cuda")
    keep = torch.zeros(S, budget, dtype=torch.int32, device="cuda")
    tri.mass_evict(kv, mass, torch.zeros_like(mass), 16, 32, budget, keep)
    assert int(status) == 0
    idx = keep.long().view(1, 25, 8, budget, 1).expand(-1, -1, -1, -1, 80)
    for now, was in ((k, k0), (v, v0)):
        assert torch.equal(now[:, :, :, :budget], was.gather(3, idx)) and torch.equal(now[:, :, :, budget:], was[:, :, :, budget:])


@pytest.mark.parametrize("block", [0, 16])
def test_serving_run(block):
    """A prompt, tokens, an eviction and more tokens, on a cache in 4 bits that only tri_append fills."""
    H, G, d, theta, n0 = 2, 2, 64, 1e4, 37
    c = Cache([[0] * H], d, torch.uint8, 128, L=1, block=block)
    c.kv.pos_out = torch.zeros_like(c.pos)
    g = torch.Generator(device="cuda").manual_seed(9)
    mass = torch.zeros(H, c.cap, device="cuda")
    rows = [[], []]  # (K bytes, V bytes) of each head's rows

    def step(n, at):
        q = torch.randn(1, n, H * G, d, generator=g, device="cuda").bfloat16()
        k, v = (torch.randn(1, n, H, d, generator=g, device="cuda").bfloat16() for _ in range(2))
        p = torch.arange(at, at + n, dtype=torch.int32, device="cuda").view(1, n)
        qr = tri.append(c.kv, 0, k, v, p, theta, q=q)
        for h in range(H):
            for i in range(n):
                rows[h].append((pack(rotate(f64(k[0, i, h]), [at + i], theta)), pack(f64(v[0, i, h]))))
        for i in range(n):
            x = f64(q[0, i, 0])
            close(f64(qr[0, i, 0]), rotate(x, [at + i], theta), x, False, torch.bfloat16)
        return qr

    def sync_case():
        c.h = [host(p) for p in c.pools]
        c.lens = np.array([[len(r) for r in rows]])
        for h in range(H):
            for x, part in zip(c.h, (0, 1)):
                assert np.array_equal(c.rows(x, 0, 0, h, 0, len(rows[h])), np.stack([r[part] for r in rows[h]]))

    def attention(qr, n):
        out = torch.zeros_like(qr)
        if n > 1:
            tri.attn_prefill(c.kv, 0, qr, out)
        else:
            tri.attn_decode(c.kv, 0, qr[:, 0], out[:, 0], mass=mass)
        for h in range(H):
            m = len(rows[h])
            k, v = (values(np.stack([r[part] for r in rows[h]])) for part in (0, 1))
            for i in range(n):
                o, _, w = attend(f64(qr[0, i, h * G]), k, v, m - n + i, d ** -0.5)
                # half a step of the result, 2^-10 of sum w |v| (weights and V in fp16), and K's 2^-16 in a logit, in both cases
                x = 2.0 ** -15 * d ** -0.5 * (np.abs(k) @ np.abs(f64(qr[0, i, h * G]))).max()
                A = w @ np.abs(v) if n > 1 else w @ sizes(np.stack([r[1] for r in rows[h]]))
                assert (np.abs(f64(out[0, i, h * G]) - o) <= (2 * x + 2.0 ** -9) * A + 2.0 ** -8 * np.abs(o) + 2.0 ** -20).all()

    at = 0
    qr = step(n0, at)
    sync_case()
    attention(qr, n0)
    at += n0
    for _ in range(5):
        qr = step(1, at)
        attention(qr, 1)
        at += 1
    sync_case()
    budget = 24
    keep = torch.zeros(H, budget, dtype=torch.int32, device="cuda")
    tri.mass_evict(c.kv, mass, mass, 4, 6, budget, keep)
    for h in range(H):
        rows[h][:] = [rows[h][j] for j in keep[h].tolist()]
    c.kv.pos, c.kv.pos_out = c.kv.pos_out, c.kv.pos
    sync_case()
    assert c.kv.pos[0, budget - 1] == at - 1  # the newest row's position
    if block:
        used = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert tri.paged_blocks_used(c.kv, used).item() == 2
    for n in (1, 9):
        qr = step(n, at)
        attention(qr, n)
        at += n
    sync_case()
    assert c.kv.pos[1, len(rows[1]) - 1] == at - 1
    torch.cuda.synchronize()
    assert int(c.status) == 0
