"""Attention over 4-bit caches (tri_attn_decode, and chunks of few tokens) at sizes of V and of the
logits where numbers of few bits could lose it: small V under a row that dominates, scales of very
different sizes, logits of 2^17 with the largest scales.

Tolerances as in test_gpu_q4.py: A = sum w (s c + |m|); 2^-10 of A for the weights' two roundings to fp16, 2 ew of it for
the logits, n 2^-24 of it for fp32 sums, half a step of the result. Without that file's term for fp16's subnormal
numbers: what falls among them is below 2^-35 of the largest weight times the largest s c + |m| (of 2^-11 and more: 2^k
is at most 2^15), n 2^-35 of that in all.
"""
import numpy as np
import pytest
import torch

import kv_cache_compression_tri_gb300 as tri
from attn_oracle import attend
from gpu_helpers import f64
from q4_oracle import pack, values
from test_gpu_q4 import Case, sizes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tri.load_library()


class Values(Case):
    """A cache of one sequence and layer whose rows are packed from numbers: k, v [H][n, d]."""

    def __init__(self, k, v, d, block=0):
        super().__init__([[len(x) for x in k]], d, L=1, block=block)
        for pool, x in zip(self.pools, (k, v)):
            for h in range(self.H):
                for r, row in enumerate(x[h]):
                    pool[self.place(0, 0, h, r)] = torch.from_numpy(pack(row)).cuda()
        self.h = [p.cpu().numpy() for p in self.pools]


def check(c, q, sc, n_q):
    """q [n_q, Hq, d] fp64, of bf16 numbers."""
    H, G, d = c.H, q.shape[1] // c.H, c.d
    qt = torch.from_numpy(q).bfloat16().cuda()[None]
    assert np.array_equal(f64(qt)[0], q)
    out = torch.full(qt.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(qt.shape[:3], 9.0, device="cuda")
    if n_q:
        tri.attn_prefill(c.kv, 0, qt, out, scale=sc, lse=lse)
    else:
        tri.attn_decode(c.kv, 0, qt[:, 0], out[:, 0], scale=sc, lse=lse[:, 0])
    c.ok()
    got, got_l, worst = f64(out)[0], f64(lse)[0], 0.0
    assert np.isfinite(got).all()
    for i in range(len(q)):
        for hq in range(H * G):
            kb, vb = c.slice_rows(0, 0, hq // G)
            n = len(kb)
            o, l, w = attend(q[i, hq], values(kb), values(vb), n - len(q) + i, sc)
            seen = w > 0
            ex = (d / 4 + 16) * 2.0 ** -23 * sc * (sizes(kb[seen]) @ np.abs(q[i, hq])).max()
            ew = 2 * ex + 2.0 ** -20 + 2.0 ** -22 * np.abs(sc * (values(kb[seen]) @ q[i, hq])).max()
            sv = sizes(vb[seen])
            A = w[seen] @ sv
            tol = A * (min(2 * ew, 2) + 2.0 ** -10 + n * 2.0 ** -24) + n * 2.0 ** -35 * sv.max() + 2.0 ** -8 * np.abs(o)
            worst = max(worst, float((np.abs(got[i, hq] - o) / np.maximum(tol, 1e-300)).max()))
            assert abs(got_l[i, hq] - l) <= ex + ew + 2.0 ** -22 * max(1.0, abs(l))
    assert worst <= 1, worst


def queries(rng, n_q, heads, d):
    return f64(torch.from_numpy(rng.normal(size=(max(n_q, 1), heads, d))).bfloat16())


def dominated(rng, q, lens, gap, small):
    """K with a first row `gap` above the rest in the logit of every query of the slice (which are one vector), V with a
    first row `small` times the others; scale d^-1/2."""
    H, d = len(lens), q.shape[-1]
    k = [rng.normal(size=(n, d)) for n in lens]
    v = [rng.normal(size=(n, d)) for n in lens]
    for h in range(H):
        u = q[0, h * (q.shape[1] // H)]
        k[h][0] = u * gap * d ** 0.5 / (u @ u)
        v[h][0] *= small
    return k, v


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q", [0, 3])  # one new token; a chunk
@pytest.mark.parametrize("size,gap,small", [(1e-2, 14, 1e-2), (1e-3, 14, 1e-3), (1e-4, 12, 1.0), (1e-4, 12, 1e-3), (1.0, 20, 1e-3), (1e-4, 0, 1.0),
                                            (300.0, 14, 1e-2)])
def test_a_row_that_dominates(d, n_q, size, gap, small):
    rng = np.random.default_rng(int(gap) + d)
    lens, G = [64, 700], 2
    q = queries(rng, 1, 2, d)[:, [0, 0, 1, 1]]
    q = np.repeat(q, max(n_q, 1), 0)
    k, v = dominated(rng, q, lens, gap, small)
    check(Values(k, [x * size for x in v], d, block=16 if n_q else 0), q, d ** -0.5, n_q)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q", [0, 2])
@pytest.mark.parametrize("order", [1, -1])
def test_scales_that_grow_and_shrink(d, n_q, order):
    # V from 2^-12 to 2^7 along the rows, or the other way round; logits that make up for it, so that every size counts
    rng = np.random.default_rng(d)
    n, H = 600, 2
    q = queries(rng, 1, H, d)
    q = np.repeat(q, max(n_q, 1), 0)
    e = np.linspace(-12, 7, n)[::order]
    k, v = [], []
    for h in range(H):
        u = q[0, h]
        x = rng.normal(size=(n, d)) * 0.3
        k.append(x + np.outer(-e * np.log(2.0) * d ** 0.5 / (u @ u), u))
        v.append(rng.normal(size=(n, d)) * 2.0 ** e[:, None])
    check(Values(k, v, d), q, d ** -0.5, n_q)


@pytest.mark.parametrize("n_q", [0, 3])
def test_zero_and_missing_scales(n_q):
    # constant quarters (scale 0), and rows of zeros between others
    rng = np.random.default_rng(3)
    d, n = 64, 200
    q = queries(rng, n_q, 2, d)
    k = [rng.normal(size=(n, d)) for _ in range(2)]
    v = [np.repeat(rng.normal(size=(n, 4)), d // 4, 1), np.where(np.arange(n)[:, None] % 3 == 0, 0.0, 1e-5 * rng.normal(size=(n, d)))]
    check(Values(k, v, d), q, d ** -0.5, n_q)
    check(Values(k, [v[0], 0 * v[1]], d), q, d ** -0.5, n_q)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q", [0, 1])
def test_large_logits_with_the_largest_scales(d, n_q):
    # logits of about 2^17, whose rounding moves a weight's exponent by 2^-7 and more; all rows are alike, so the result is their V
    rng = np.random.default_rng(d)
    H, n = 8, 40
    q = queries(rng, 1, H, d)
    k = [np.repeat(u[None] * 2.0 ** 17 / (u @ u), n, 0) for u in q[0]]
    v = [np.repeat((np.where(rng.random(d) < 0.5, 1.0, -1.0) * 3e4)[None], n, 0) for _ in range(H)]
    for x in v:  # both ends in every quarter
        x[:, ::d // 4], x[:, 1::d // 4] = 30656.0, -30656.0
    check(Values(k, v, d), q, 1.0, n_q)
