"""Appending new tokens with rotation (tri_append) against the definition in 64
bits (q4_oracle.py): contiguous and paged caches, every type, one and several axes.

Tolerances. A rotated element x c - y s errs in fp32 by at most 2^-21 max(|x|, |y|): cosine
and sine by 2^-23 each (the phase to 2^-32 turns, sincospi to one step, one
first-order step), three roundings. It is then rounded once to the cache's type: half a
step, eps / 2 of its size. V is copied, and 4-bit rows are decided as in 64 bits:
equal bytes (the two 64-bit angles differ by 2^-36 turns at the tests' positions).
"""
import numpy as np
import pytest
import torch

import kv_cache_compression_tri_gb300 as tri
from gpu_helpers import f64
from q4_oracle import pack, rotate, values

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
THETA = 1e4
Q4 = torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tri.load_library()


class Cache:
    """A cache with `lens` [B][H] rows in every layer and random bytes everywhere, contiguous (slices three
    rows apart) or paged, and the host's copy of its rows in order."""

    def __init__(self, lens, d, dtype, cap, L=2, block=0, seed=0, post=True):
        lens = np.asarray(lens)
        B, H = lens.shape
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.H, self.L, self.d, self.cap, self.dtype, self.block, self.lens = B, H, L, d, cap, dtype, block, lens
        w = tri.q4_row_bytes(d) if dtype == Q4 else d
        S = B * L * H
        shape = (B * (cap // block) + 3, L, H, block, w) if block else (B, L, H, cap + 3, w)

        def fill():
            if dtype == Q4:
                return torch.randint(0, 256, shape, generator=self.g, device="cuda", dtype=torch.uint8)
            return torch.randn(shape, generator=self.g, device="cuda").to(dtype)

        self.pools = fill(), fill()
        nv = torch.tensor(np.repeat(lens[:, None, :], L, 1).reshape(-1), dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.pos = torch.full((S, cap), -7, dtype=torch.int32, device="cuda")
        if block:
            t = torch.randperm(shape[0], generator=self.g, device="cuda")[: B * (cap // block)].view(B, -1)
            self.table = t.to(torch.int32).contiguous()
            self.kv = tri.PagedKVCache(*self.pools, self.table.clone(), nv, self.pos, None, self.status, post_rope=post)
        else:
            self.kv = tri.KVCache(*(p[:, :, :, :cap] for p in self.pools), nv, self.pos, None, self.status, post_rope=post)

    def place(self, b, layer, h, r):
        """Index of row r of a slice in a pool."""
        if not self.block:
            return b, layer, h, r
        return int(self.table[b, r // self.block]), layer, h, r % self.block

    def rows(self, x, b, layer, h, r0, r1):
        return np.stack([x[self.place(b, layer, h, r)] for r in range(r0, r1)]) if r1 > r0 else x[:0, 0, 0, 0]


def host(t):
    return t.cpu().numpy() if t.dtype == Q4 else f64(t)


def tokens(c, n_q, group, seed=3, scale=1.0):
    """q, k, v as views of a fused projection's output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, Hq, d = c.H, c.H * group, c.d
    dt = torch.bfloat16 if c.dtype == Q4 else c.dtype
    x = (torch.randn(c.B, n_q, (Hq + 2 * H) * d + 16, generator=g, device="cuda") * scale).to(dt)
    q, k, v, _ = x.split((Hq * d, H * d, H * d, 16), dim=-1)
    return q.unflatten(-1, (Hq, d)), k.unflatten(-1, (H, d)), v.unflatten(-1, (H, d))


def rotated(x, at, half, axes):
    return rotate(x, at, THETA, half, axes)


def close(got, want, x, half, dtype):
    """got against the exact rotation `want` of x [d]."""
    d = x.shape[-1]
    big = np.abs(x)
    pair = np.maximum(big, np.roll(big, d // 2) if half else big.reshape(-1, 2)[:, ::-1].reshape(-1))
    tol = 2.0 ** -21 * pair + HALF[dtype] * np.abs(want)
    tol = tol + HALF[dtype] * tol + 1e-37
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


def check(c, n_q, group, layer=1, n_new=None, half=False, axes=None, positions=None, in_place=False, post=True, seed=3, scale=1.0, skipped=()):
    """One call against the definition; `skipped`: (sequence, head) whose rows stay."""
    q, k, v = tokens(c, n_q, group, seed, scale)
    n_axes = max(axes) + 1 if axes else 1
    if positions is None:
        positions = torch.randint(0, 100000, (c.B, n_q, n_axes), generator=c.g, device="cuda", dtype=torch.int32)
    if n_axes == 1:
        positions = positions.view(c.B, n_q)
    before = [host(p) for p in c.pools]
    nv0, pos0 = c.kv.n_valid.cpu().numpy(), c.pos.cpu().numpy()
    q0, kh, vh, ph = f64(q), f64(k), f64(v), positions.cpu().numpy().reshape(c.B, n_q, n_axes)
    out = q if in_place else torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    nn = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device="cuda")
    style = tri.ROPE_HALF if half else tri.ROPE_INTERLEAVED
    got_q = tri.append(c.kv, layer, k, v, positions, THETA, q=q, q_out=out, n_new=nn, band_axis=axes, style=style)
    assert got_q is out
    torch.cuda.synchronize()
    after, got_q = [host(p) for p in c.pools], f64(out)
    want_nv, want_pos = nv0.copy(), pos0.copy()
    same = [np.ones(p.shape[:4], dtype=bool) for p in before]
    for b in range(c.B):
        n = n_q if n_new is None else n_new[b]
        for i in range(n_q):
            for h in range(c.H * group):
                if i >= n:
                    assert np.array_equal(got_q[b, i, h], q0[b, i, h] if in_place else np.full(c.d, 5.0))
                else:
                    close(got_q[b, i, h], rotated(q0[b, i, h], ph[b, i], half, axes), q0[b, i, h], half, q.dtype)
        for h in range(c.H):
            if (b, h) in skipped:
                continue
            s = (b * c.L + layer) * c.H + h
            for i in range(n):
                at = c.place(b, layer, h, nv0[s] + i)
                turned = rotated(kh[b, i, h], ph[b, i], half, axes) if post else kh[b, i, h]
                if c.dtype == Q4:
                    assert np.array_equal(after[0][at], pack(turned)), (b, h, i)
                    assert np.array_equal(after[1][at], pack(vh[b, i, h])), (b, h, i)
                else:
                    if post:
                        close(after[0][at], turned, kh[b, i, h], half, c.dtype)
                    else:
                        assert np.array_equal(after[0][at], turned)
                    assert np.array_equal(after[1][at], vh[b, i, h])
                same[0][at] = same[1][at] = False
                want_pos[s, nv0[s] + i] = ph[b, i, 0]
            want_nv[s] += n
    for x, y, m in zip(before, after, same):
        assert np.array_equal(x[m], y[m], equal_nan=x.dtype != np.uint8)  # all other rows
    assert np.array_equal(c.kv.n_valid.cpu().numpy(), want_nv)
    if not skipped:
        assert np.array_equal(c.pos.cpu().numpy(), want_pos)
    return after


TYPES = [torch.bfloat16, torch.float32, Q4]
SECTIONS = lambda d: [0] * (d // 8) + [1] * (3 * d // 16) + [2] * (3 * d // 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("half", [False, True])
def test_append(dtype, d, block, half):
    c = Cache([[0, 5, 17], [30, 1, 16]], d, dtype, 64, block=block)
    check(c, 13, 2, n_new=[13, 4], half=half)
    assert int(c.status) == 0


@pytest.mark.parametrize("n_q", [1, 2, 3, 8, 9, 40])
@pytest.mark.parametrize("heads,group", [(1, 8), (3, 7), (8, 4), (9, 1)])
def test_lengths_and_heads(n_q, heads, group):
    c = Cache([[(7 * h) % 20 for h in range(heads)]] * 2, 64, Q4 if (n_q + heads) % 2 else torch.bfloat16, 64, block=(0, 32)[heads % 2])
    check(c, n_q, group, n_new=[n_q, n_q // 2])
    assert int(c.status) == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["sections", "turns", "four"])
@pytest.mark.parametrize("half", [False, True])
def test_several_axes(dtype, kind, half):
    d = 128 if kind == "sections" else 64
    axes = {"sections": SECTIONS(d), "turns": [f % 2 for f in range(d // 2)], "four": [(3 * f) % 4 for f in range(d // 2)]}[kind]
    check(Cache([[3, 0]], d, dtype, 48, block=16), 11, 2, half=half, axes=axes)


@pytest.mark.parametrize("dtype", TYPES)
def test_more_heads_than_a_cta_takes(dtype):
    c = Cache([[(5 * h) % 23 for h in range(20)]], 64 if dtype == torch.float32 else 128, dtype, 64)
    check(c, 3, 2)
    check(c, 1, 2, seed=4)
    assert int(c.status) == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_in_place_queries(dtype):
    check(Cache([[3, 0]], 64, dtype, 48), 5, 2, half=True, in_place=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_keys_before_the_rotation_are_copied(dtype):
    check(Cache([[3, 0]], 64, dtype, 48, post=False), 5, 2, post=False)


def test_far_and_negative_positions():
    # at 2^31 the oracle's own fp64 angle errs by 2^-23 turns (2^31 2^-53 radians): eight times the kernel's error there
    c = Cache([[0]], 64, torch.bfloat16, 48)
    at = torch.tensor([[[2 ** 31 - 1], [2 ** 30 + 7], [-5], [0], [2 ** 24 + 1]]], dtype=torch.int32, device="cuda")
    check(c, 5, 1, positions=at)
    turned = check(Cache([[0]], 64, torch.float32, 48), 2, 1, positions=at[:, 2:4])[0]
    assert np.isfinite(turned).all()


@pytest.mark.parametrize("scale", [1e-4, 3e-2, 1e3, 1e5])
def test_magnitudes_in_4_bits(scale):
    check(Cache([[3, 0]], 128, Q4, 48), 6, 1, scale=scale)


def test_many_rows_in_4_bits_are_decided_as_in_64_bits():
    # enough quarters (16384 of keys) that fp32 arithmetic alone would miss some
    c = Cache([[0] * 4], 128, Q4, 512, L=1, block=64)
    check(c, 512, 1, layer=0, half=True)
    c = Cache([[0] * 4], 64, Q4, 512, L=1)
    check(c, 512, 1, layer=0)


def test_odd_values_in_4_bits():
    c = Cache([[1, 2]], 128, Q4, 48)
    q, k, v = tokens(c, 4, 1)
    inf, nan = float("inf"), float("nan")
    v[0, 0, 0, 3], v[0, 1, 0, 40], v[0, 2, 1, 100] = nan, inf, -inf
    v[0, 3, 0] = 2.5
    v[0, 3, 1] = 0.0
    k[0, 0, 1, 5] = nan  # (its pair and, through the rotation, its partner)
    k[0, 1, 1] = 0.0
    positions = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    tri.append(c.kv, 1, k, v, positions, THETA)
    torch.cuda.synchronize()
    after = [host(p) for p in c.pools]
    for h in range(2):
        for i in range(4):
            at = c.place(0, 1, h, int(c.lens[0, h]) + i)
            for x, src, turn in ((after[0], k, True), (after[1], v, False)):
                row = f64(src[0, i, h])
                row = rotated(row, [i], False, None) if turn else row
                got, want = values(x[at]), values(pack(row))
                assert np.array_equal(got, want, equal_nan=True), (h, i, turn)
    got = values(after[1][c.place(0, 1, 0, 4)])
    assert (got == 2.5).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, Q4])
@pytest.mark.parametrize("n_q", [2, 20])
def test_faults_keep_the_slice(dtype, n_q):
    # no room, a bad count, a bad count of new tokens, a bad block
    c = Cache([[3, 48 - n_q + 1], [3, 5]], 64, dtype, 48)
    check(c, n_q, 1, skipped=((0, 1),))
    assert int(c.status) == 1
    c = Cache([[3, 2], [3, 5]], 64, dtype, 48)
    c.kv.n_valid[(1 * 2 + 1) * 2] = 49
    before = c.kv.n_valid.clone()
    q, k, v = tokens(c, n_q, 1)
    at = torch.zeros(2, n_q, dtype=torch.int32, device="cuda")
    tri.append(c.kv, 1, k, v, at, THETA)
    before[2:4] += n_q
    before[7] += n_q
    assert int(c.status) == 1 and torch.equal(c.kv.n_valid, before)
    for bad in (-1, n_q + 1):
        c = Cache([[3, 2], [3, 5]], 64, dtype, 48)
        n0 = c.kv.n_valid.clone()
        pools = [p.clone() for p in c.pools]
        tri.append(c.kv, 0, k, v, at, THETA, n_new=torch.tensor([bad, 0], dtype=torch.int32, device="cuda"))
        assert int(c.status) == 7 and torch.equal(c.kv.n_valid, n0)
        assert all(torch.equal(a, b) for a, b in zip(pools, c.pools))
    for entry in (-1, 1 << 20):
        c = Cache([[14, 31 - n_q], [3, 5]], 64, dtype, 64, block=16)
        c.kv.block_table[0, 0 if n_q == 20 else 1] = entry  # (head 1 of 20 tokens: rows 11 .. 30)
        n0 = c.kv.n_valid.clone()
        valid = {h: c.rows(host(c.pools[1]), 1, 0, h, 0, int(c.lens[1, h])) for h in range(2)}
        tri.append(c.kv, 0, k, v, at, THETA)
        n0[4:6] += n_q  # sequence 1, layer 0
        skip = torch.tensor([True, True] if n_q == 20 else [n_q + 14 > 16, True])
        n0[0:2] += torch.where(skip, 0, n_q).int().cuda()
        assert int(c.status) == 6
        assert torch.equal(c.kv.n_valid, n0)
        for h in range(2):
            assert np.array_equal(c.rows(host(c.pools[1]), 1, 0, h, 0, int(c.lens[1, h])), valid[h])


def test_a_full_slice_and_no_new_tokens():
    c = Cache([[48, 28]], 64, torch.bfloat16, 48)
    check(c, 20, 1, skipped=((0, 0),))
    c = Cache([[48, 28]], 64, torch.bfloat16, 48)
    check(c, 20, 1, n_new=[0])
    assert int(c.status) == 0


def test_captured_appends_follow_the_counts():
    for n_q in (1, 12):  # one launch, and two
        c = Cache([[0, 2]], 64, torch.bfloat16, 64)
        q, k, v = tokens(c, n_q, 2)
        at = torch.arange(n_q, dtype=torch.int32, device="cuda").view(1, n_q)
        out = torch.zeros(q.shape, dtype=q.dtype, device="cuda")
        run = lambda: tri.append(c.kv, 1, k, v, at, THETA, q=q, q_out=out)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for step in range(1, 4):
            at += 100
            graph.replay()
            torch.cuda.synchronize()
            assert c.kv.n_valid.tolist() == [0, 2, (step + 1) * n_q, 2 + (step + 1) * n_q]
            for h in range(2):
                rows = c.rows(f64(c.pools[0]), 0, 1, h, c.lens[0, h] + step * n_q, c.lens[0, h] + (step + 1) * n_q)
                for i in range(n_q):
                    x = f64(k[0, i, h])
                    close(rows[i], rotate(x, [i + 100 * step], THETA), x, False, torch.bfloat16)
        assert int(c.status) == 0


def test_another_stream_and_a_new_result():
    c = Cache([[0, 2]], 64, torch.bfloat16, 64)
    q, k, v = tokens(c, 3, 2)
    at = torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = tri.append(c.kv, 1, k, v, at, THETA, q=q, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert out.shape == q.shape and out.is_contiguous()
    for i in range(3):
        x = f64(q[0, i, 1])
        close(f64(out[0, i, 1]), rotate(x, [i], THETA), x, False, torch.bfloat16)


def test_the_binding_refuses():
    c = Cache([[0, 2]], 64, torch.bfloat16, 64)
    q, k, v = tokens(c, 3, 2)
    at = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    bad = [
        (k.float(), v, at, {}), (k, v[:, :2], at, {}), (k[:, :, :1], v, at, {}), (k, v, at.long(), {}), (k, v, at[:, :2], {}),
        (k, v, at, dict(q=q[:, :, :3])), (k, v, at, dict(q=q.float())), (k, v, at, dict(q_out=torch.empty_like(q))),
        (k, v, at, dict(n_new=torch.zeros(2, dtype=torch.int32, device="cuda"))), (k, v, at, dict(band_axis=[0] * 31)),
        (k.transpose(2, 3).contiguous().transpose(2, 3), v, at, {}),
    ]
    for kk, vv, p, kw in bad:
        with pytest.raises(AssertionError):
            tri.append(c.kv, 0, kk, vv, p, THETA, **kw)
    with pytest.raises(tri.TriError):
        tri.append(c.kv, 0, k, v, at, 0.5)
    with pytest.raises(tri.TriError):
        tri.append(c.kv, 0, k, v, at, THETA, band_axis=[1] * 32)


def test_offsets_past_32_bits():
    # slices and tokens more than 2^31 elements from the first
    n_cap = 1 << 21
    k = torch.zeros(9, 1, 1, n_cap, 128, dtype=torch.bfloat16, device="cuda")
    nv = torch.full((9,), n_cap - 1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    v = torch.zeros_like(k)
    kv = tri.KVCache(k, v, nv, None, None, status, post_rope=True)
    x = torch.randn(9, 1, 1, 128, device="cuda").bfloat16()
    tri.append(kv, 0, x, x, torch.full((9, 1), 11, dtype=torch.int32, device="cuda"), THETA)
    assert int(status) == 0 and nv.tolist() == [n_cap] * 9
    for b in (0, 8):
        close(f64(k[b, 0, 0, -1]), rotate(f64(x[b, 0, 0]), [11], THETA), f64(x[b, 0, 0]), False, torch.bfloat16)
        assert torch.equal(v[b, 0, 0, -1], x[b, 0, 0]) and not bool(v[b, 0, 0, -2].any())
