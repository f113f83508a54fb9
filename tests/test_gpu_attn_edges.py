"""Attention at its edges: table entries of rows out of sight, windows in both
types, queries before the first row, faults, memory orders of pools and
queries, workspaces. Definitions and tolerances are test_gpu_attn.py's; where a
call may not change its result at all, its bits are compared."""
import numpy as np
import pytest
import torch

import kv_cache_compression_tri_gb300 as tri
from attn_oracle import visible
from test_gpu_attn import Case, check_decode, check_prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tri.load_library()


def hide(c, n_new, n_sink, window, what):
    """Point every table entry whose rows no query of its sequence sees at a block of the pool that holds NaN
    (what = "nan") or nowhere (a number). Returns how many there were."""
    table = c.kv.block_table
    bs = c.kv.k.shape[3]
    if what == "nan":
        what = min(set(range(c.kv.k.shape[0])) - set(table.flatten().tolist()))
        assert bool(c.kv.k[what].isnan().all()) and bool(c.kv.v[what].isnan().all())
    new, count = table.clone(), 0
    for b in range(c.B):
        seen = np.zeros(c.n_cap, dtype=bool)
        for h in range(c.H):
            n = int(c.lens[b, h])
            for r in range(n - n_new[b], n):
                seen |= visible(r, c.n_cap, n_sink, window)
        for i in range(table.shape[1]):
            if not seen[i * bs:(i + 1) * bs].any():
                new[b, i] = what
                count += 1
    c.kv.block_table = new
    return count


def chunk_bufs(c, G, n_q, seed=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(c.B, n_q, c.H * G, c.d, generator=g, device="cuda").to(c.dtype)
    return q, torch.full_like(q, 9.0), torch.full((c.B, n_q, c.H * G), 9.0, device="cuda")


# (row counts, new tokens, sinks, window): few queries and many, edges inside a tile of rows, heads of different lengths
HIDDEN = [
    ([[314, 314]], [64], 4, 90),
    ([[700, 333], [512, 640]], [70, 1], 4, 90),
    ([[700, 333], [512, 640]], [70, 1], 0, 17),
    ([[900, 1100]], [200], 130, 65),
    ([[1500] * 4] * 5, [300] * 5, 4, 200),
]


@pytest.mark.parametrize("lens,n_new,n_sink,window", HIDDEN)
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["nan", -1, 1 << 20])
def test_prefill_fp32_blocks_out_of_sight(lens, n_new, n_sink, window, block, d, what):
    c = Case(lens, d, torch.float32, L=1, block=block)
    nn = torch.tensor(n_new, dtype=torch.int32, device="cuda")
    res = []
    for hidden in (False, True):
        if hidden:
            assert hide(c, n_new, n_sink, window, what) > 0
        q, out, lse = chunk_bufs(c, 2, max(n_new))
        tri.attn_prefill(c.kv, 0, q, out, n_new=nn, n_sink=n_sink, window=window, lse=lse)
        c.ok()
        res.append((out, lse))
    for x, y in zip(*res):
        assert torch.equal(x, y)


@pytest.mark.parametrize("lens,n_new,n_sink,window", HIDDEN)
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what", ["nan", -1, 1 << 20])
def test_mass_blocks_out_of_sight(lens, n_new, n_sink, window, block, dtype, what):
    c = Case(lens, 128, dtype, L=1, block=block)
    nn = torch.tensor(n_new, dtype=torch.int32, device="cuda")
    q, out, lse = chunk_bufs(c, 2, max(n_new))
    tri.attn_prefill(c.kv, 0, q, out, n_new=nn, n_sink=n_sink, window=window, lse=lse)
    res = []
    for hidden in (False, True):
        if hidden:
            assert hide(c, n_new, n_sink, window, what) > 0
        mass = torch.zeros(c.B * c.H, c.n_cap, device="cuda")
        tri.attn_mass(c.kv, 0, q, lse, mass, n_new=nn, n_sink=n_sink, window=window)
        c.ok()
        res.append(mass)
    assert torch.equal(*res)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_new", [5, 200])
def test_mass_of_a_slice_with_a_bad_block_stays(dtype, n_new):
    """A bad entry for rows that a query sees leaves the masses of the whole slice as they were, and no other's."""
    c = Case([[300, 400], [330, 310]], 128, dtype, L=1, block=32)
    q, out, lse = chunk_bufs(c, 2, n_new)
    tri.attn_prefill(c.kv, 0, q, out, lse=lse)
    good = torch.zeros(4, c.n_cap, device="cuda")
    tri.attn_mass(c.kv, 0, q, lse, good, n_sink=4, window=100)
    c.ok()
    c.kv.block_table[0, 11] = -1  # rows 352 .. 383 of sequence 0: its head 0 holds 300 rows, head 1 400
    mass = torch.zeros_like(good)
    tri.attn_mass(c.kv, 0, q, lse, mass, n_sink=4, window=100)
    torch.cuda.synchronize()
    assert int(c.status.item()) == tri.DEV_BAD_BLOCK
    assert bool((mass[1] == 0).all())
    for s in (0, 2, 3):
        assert torch.equal(mass[s], good[s]) and bool((mass[s] > 0).any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_sink,window", [(0, 1), (0, 6), (2, 3), (0, 1 << 30), (4, (1 << 31) - 1), ((1 << 31) - 1, (1 << 31) - 1),
                                           ((1 << 31) - 1, 4)])
def test_windows_and_queries_before_the_first_row(dtype, n_sink, window):
    """Heads that hold fewer rows than there are new tokens, under every size of window."""
    check_prefill(Case([[5, 40], [0, 30]], 64, dtype, L=1), 2, [30, 30], layer=0, n_sink=n_sink, window=window)
    check_prefill(Case([[3, 160]], 128, dtype, L=1, block=16), 4, [150], layer=0, n_sink=n_sink, window=window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [76, 77, 78, 1 << 30, (1 << 31) - 1])
def test_windows_about_the_capacity(dtype, window):
    """77 rows fit a slice: a window of as many or more is none."""
    c = Case([[77, 70]], 64, dtype, L=1, n_cap=77)
    check_decode(c, 3, layer=0, n_sink=1, window=window, with_mass=True)
    check_prefill(c, 3, [60], layer=0, n_sink=1, window=window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,n_cap", [(150, 160), (1500, 1504), (12000, 12000)])
def test_decode_reports_a_bad_block_wherever_it_is(dtype, n, n_cap):
    """Every run, every warp and the first and last tile of a slice may be the one that meets the bad entry: the slice
    is left out and reported, sequence by sequence, and the others are not touched by it."""
    B = 6
    c = Case([[n, n - 20]] * B, 64, dtype, L=1, block=16, n_cap=n_cap)
    q = torch.randn(B, 4, 64, generator=c.g, device="cuda").to(dtype)

    def run():
        out, lse = torch.full_like(q, 9.0), torch.full((B, 4), 9.0, device="cuda")
        mass = torch.zeros(2 * B, c.n_cap, device="cuda")
        c.status.zero_()
        tri.attn_decode(c.kv, 0, q, out, lse=lse, mass=mass)
        torch.cuda.synchronize()
        return int(c.status.item()), out, lse, mass

    st, *good = run()
    assert st == 0
    table = c.kv.block_table.clone()
    last = (n - 21) // 16  # head 1's last block
    for i in sorted({*range(0, min(last, 24) + 1), last - 1, last, *range(0, last, max(1, last // 20))}):
        b = i % B
        c.kv.block_table = table.clone()
        c.kv.block_table[b, i] = -1 if i % 2 else c.kv.k.shape[0]
        st, *got = run()
        assert st == tri.DEV_BAD_BLOCK, i
        for x, y in zip(got, good):
            x, y = x.view(B, -1), y.view(B, -1)
            assert torch.equal(x[torch.arange(B) != b], y[torch.arange(B) != b])
            assert bool((x[b] == (0.0 if x.shape[1] == 2 * c.n_cap else 9.0)).all()), i


@pytest.mark.parametrize("lens,n_new,n_sink,window", HIDDEN)
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["nan", -1, 1 << 20])
def test_prefill_bf16_blocks_out_of_sight(lens, n_new, n_sink, window, block, d, what):
    c = Case(lens, d, torch.bfloat16, L=1, block=block)
    nn = torch.tensor(n_new, dtype=torch.int32, device="cuda")
    res = []
    for hidden in (False, True):
        if hidden:
            assert hide(c, n_new, n_sink, window, what) > 0
        q, out, lse = chunk_bufs(c, 2, max(n_new))
        tri.attn_prefill(c.kv, 0, q, out, n_new=nn, n_sink=n_sink, window=window, lse=lse)
        c.ok()
        res.append((out, lse))
    for x, y in zip(*res):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [1, 80])  # few query tiles, and more than the GPU has room for at once
@pytest.mark.parametrize("n_sink,window", [(0, 0), (4, 50)])
def test_prefill_leaves_out_the_tiles_that_see_a_bad_block(dtype, d, heads, n_sink, window):
    G, n_new, n, bs = 4, 128, 300, 16
    per = (128 if dtype == torch.bfloat16 else 64) // G
    c = Case([[n] * heads], d, dtype, L=1, block=bs)
    q = torch.randn(1, n_new, heads * G, d, generator=c.g, device="cuda").to(dtype)

    def run():
        c.status.zero_()
        out, lse = torch.full_like(q, 9.0), torch.full((1, n_new, heads * G), 9.0, device="cuda")
        tri.attn_prefill(c.kv, 0, q, out, n_sink=n_sink, window=window, lse=lse)
        torch.cuda.synchronize()
        return int(c.status.item()), out, lse

    st, good, good_lse = run()
    assert st == 0
    table = c.kv.block_table.clone()
    for i in range((n + bs - 1) // bs):
        c.kv.block_table = table.clone()
        c.kv.block_table[0, i] = -1 if i % 2 else 1 << 20
        hit = np.zeros(n_new, dtype=bool)
        for t0 in range(0, n_new, per):
            hit[t0:t0 + per] = any(visible(n - n_new + t, n, n_sink, window)[i * bs:(i + 1) * bs].any() for t in range(t0, t0 + per))
        for _ in range(3):
            st, out, lse = run()
            assert st == (tri.DEV_BAD_BLOCK if hit.any() else 0), i
            h = torch.from_numpy(hit).cuda()
            assert bool((out[:, h] == 9.0).all()) and bool((lse[:, h] == 9.0).all()), i
            assert torch.equal(out[:, ~h], good[:, ~h]) and torch.equal(lse[:, ~h], good_lse[:, ~h]), i


def strided(x, order, pad):
    """x in memory with its dimensions in `order`, `pad` elements of NaN after each slice of the second innermost dimension
    outwards (so strides grow by pad), as a view of x's shape."""
    dims = [x.shape[i] for i in order]
    strides, step = [0] * 5, 1
    for k in reversed(range(5)):
        strides[order[k]] = step
        step *= dims[k]
        if k == 3:
            step += pad
    buf = torch.full((step,), float("nan"), dtype=x.dtype, device=x.device)
    view = buf.as_strided(x.shape, strides)
    view.copy_(x)
    return view


def same_results(c, G, n_new, change, **kw):
    """Decode, prompt attention and masses of layer 0 before and after `change` laid the cache or the queries out anew."""
    res = []
    g = torch.Generator(device="cuda").manual_seed(4)
    q0 = torch.randn(c.B, n_new, c.H * G, c.d, generator=g, device="cuda").to(c.dtype)
    nn = torch.tensor([n_new - 3 * b for b in range(c.B)], dtype=torch.int32, device="cuda")
    for again in (False, True):
        q = change(q0) if again else q0
        out, lse = torch.full_like(q0, 9.0), torch.full((c.B, n_new, c.H * G), 9.0, device="cuda")
        mass = torch.zeros(c.B * c.L * c.H, c.n_cap, device="cuda")
        dec = torch.full((c.B, c.H * G, c.d), 9.0, dtype=c.dtype, device="cuda")
        tri.attn_prefill(c.kv, 0, q, out, n_new=nn, lse=lse, **kw)
        tri.attn_mass(c.kv, 0, q, lse, mass, n_new=nn, **kw)
        tri.attn_decode(c.kv, 0, q[:, 0], dec, mass=mass, **kw)
        c.ok()
        assert bool((mass.sum(1) > 0).any())
        res.append((out, lse, mass, dec))
    for x, y in zip(*res):
        assert torch.equal(x, y)


# blocks, layers, heads, rows, elements: heads outermost, blocks innermost, layers outermost, and blocks that do not follow
# each other at whole slices or whole rows
@pytest.mark.parametrize("order", [(0, 1, 2, 3, 4), (2, 0, 1, 3, 4), (2, 1, 0, 3, 4), (1, 0, 2, 3, 4), (1, 2, 0, 3, 4)])
@pytest.mark.parametrize("pad", ["none", "row", "16 bytes"])
@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.bfloat16), (64, torch.float32)])
def test_pools_in_any_order(order, pad, d, dtype):
    for lens, G, n_new, block in (([[300, 270]] * 3, 4, 60, 16), ([[250] * 8] * 4, 3, 240, 256)):
        c = Case(lens, d, dtype, L=2, block=block)

        def change(q):
            n = {"none": 0, "row": d, "16 bytes": 16 // q.element_size()}[pad]
            c.kv.k, c.kv.v = strided(c.kv.k, order, n), strided(c.kv.v, order, n)
            return q

        same_results(c, G, n_new, change, n_sink=4, window=120)


@pytest.mark.parametrize("pad", ["row", "16 bytes"])
@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.bfloat16), (64, torch.float32)])
def test_slices_at_any_stride(pad, d, dtype):
    for lens, G, n_new in (([[300, 270]] * 3, 4, 60), ([[250] * 8] * 4, 3, 240)):
        c = Case(lens, d, dtype, L=2)

        def change(q):
            n = {"row": d, "16 bytes": 16 // q.element_size()}[pad]
            c.kv.k, c.kv.v = strided(c.kv.k, (0, 1, 2, 3, 4), n), strided(c.kv.v, (0, 1, 2, 3, 4), n)
            return q

        same_results(c, G, n_new, change)


# strides between sequences and tokens in units of a token's heads, and elements more
QUERIES = [
    (lambda B, T: (1, B), 0, 0),  # sequences inside tokens
    (lambda B, T: (2, 2 * B), 0, 0),
    (lambda B, T: (T, 1), 64, 0),  # sequences that are not whole tokens apart
    (lambda B, T: (T, 1), 8, 0),
    (lambda B, T: (2 * T, 2), 0, 8),  # tokens that are not whole rows apart
    (lambda B, T: (1, B + 1), 8, 8),
    (lambda B, T: (5, 1), 0, 0),  # sequences that share tokens
]


@pytest.mark.parametrize("case", range(len(QUERIES)))
@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.bfloat16), (64, torch.float32)])
def test_queries_at_any_stride(case, d, dtype):
    units, seq_more, token_more = QUERIES[case]
    for lens, G, n_new in (([[300, 270]] * 3, 4, 60), ([[250] * 8] * 4, 3, 240), ([[70, 80]] * 3, 2, 10)):
        c = Case(lens, d, dtype, L=1)

        def change(q):
            B, T, Hq, _ = q.shape
            us, ut = units(B, T)
            ss, st = us * Hq * d + seq_more, ut * Hq * d + token_more
            if (us, ut) == (2 * T, 2):
                ss = us * (Hq * d + token_more) + seq_more
            buf = torch.full(((B - 1) * ss + (T - 1) * st + Hq * d,), float("nan"), dtype=q.dtype, device="cuda")
            view = buf.as_strided(q.shape, (ss, st, d, 1))
            if case == len(QUERIES) - 1:
                buf.copy_(torch.randn(buf.shape, generator=c.g, device="cuda"))
            else:
                view.copy_(q)
            return view

        if case == len(QUERIES) - 1:
            same_queries(c, G, n_new, change(torch.empty(c.B, n_new, c.H * G, d, dtype=dtype, device="cuda")))
        else:
            same_results(c, G, n_new, change)
            same_results(c, G, n_new, change, n_sink=4, window=50)


def same_queries(c, G, n_new, q):
    """Queries in memory of any kind give what their copy gives."""
    res = []
    for x in (q.contiguous(), q):
        out, lse = torch.empty(x.shape, dtype=x.dtype, device="cuda"), torch.empty(x.shape[:3], device="cuda")
        mass = torch.zeros(c.B * c.L * c.H, c.n_cap, device="cuda")
        dec = torch.empty(c.B, c.H * G, c.d, dtype=c.dtype, device="cuda")
        tri.attn_prefill(c.kv, 0, x, out, lse=lse)
        tri.attn_mass(c.kv, 0, x, lse, mass)
        tri.attn_decode(c.kv, 0, x[:, 0], dec, mass=mass)
        c.ok()
        res.append((out, lse, mass, dec))
    for x, y in zip(*res):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
def test_one_query_of_each_sequence(d):
    """One token per sequence, sequences at any stride, through the calls for chunks."""
    c = Case([[300, 270], [5, 0], [129, 128]], d, torch.bfloat16, L=1)
    for more in (0, 8, 6 * d):
        buf = torch.randn(3 * (6 * d + more), generator=c.g, device="cuda").to(torch.bfloat16)
        same_queries(c, 3, 1, buf.as_strided((3, 1, 6, d), (6 * d + more, 6 * d, d, 1)))


def test_default_workspaces_are_the_streams_own():
    """A call on a stream other than the current one, with no workspace given: its scratch may not be memory that the
    current stream's pending work still writes."""
    c = Case([[30000, 20001]], 128, torch.bfloat16, L=1)
    q = torch.randn(1, 8, 128, generator=c.g, device="cuda").to(torch.bfloat16)
    want, want_m = torch.empty_like(q), torch.zeros(2, c.n_cap, device="cuda")
    tri.attn_decode(c.kv, 0, q, want, mass=want_m)
    need = tri.attn_decode_workspace_bytes(c.kv, 4, True)
    side, busy = torch.cuda.Stream(), torch.randn(8192, 8192, device="cuda").to(torch.bfloat16)
    product = torch.empty_like(busy)
    outs = [(torch.empty_like(q), torch.zeros(2, c.n_cap, device="cuda")) for _ in range(20)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")  # the workspace's size, in use on the current stream ...
    for _ in range(40):  # (the host is ahead of the GPU from here on)
        torch.mm(busy, busy, out=product)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2000):
        scratch.fill_(255)
    del scratch  # ... and still to be written when its memory is free to the current stream's next tensor
    for out, mass in outs:
        tri.attn_decode(c.kv, 0, q, out, mass=mass, stream=side)
    torch.cuda.synchronize()
    for out, mass in outs:
        assert torch.equal(out, want) and torch.equal(mass, want_m)


@pytest.mark.parametrize("n_sink,window", [(0, 1), (0, 33), (4, 1), (4, 60), (70, 65), (1000, 3)])
@pytest.mark.parametrize("block", [0, 16, 64])
@pytest.mark.parametrize("d,dtype", [(64, torch.float32), (128, torch.float32), (64, torch.bfloat16)])
def test_prefill_and_mass_sinks_and_window(n_sink, window, block, d, dtype):
    check_prefill(Case([[200, 150], [70, 90]], d, dtype, L=1, block=block), 3, [66, 20], layer=0, n_sink=n_sink, window=window)


@pytest.mark.parametrize("block", [0, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_offsets_past_32_bits(block, dtype):
    """The last slices of a cache of more than 4 GB each of K and V give what a cache of those slices alone gives."""
    H, n, d, G = 2, 300, 128, 4
    c = Case([[n, n - 7]], d, dtype, L=1, block=block)
    per = c.n_cap
    elem = 2 if dtype == torch.bfloat16 else 4
    slices = (1 << 32) // (per * d * elem) + 50
    if block:
        nb, blocks = c.kv.k.shape[0], slices * per // (block * H)
        big = [torch.empty(blocks, 1, H, block, d, dtype=dtype, device="cuda") for _ in range(2)]
        for x, y in zip(big, (c.kv.k, c.kv.v)):
            x[blocks - nb:] = y
        kv = tri.PagedKVCache(*big, c.kv.block_table + (blocks - nb), c.kv.n_valid, c.kv.pos, c.kv.pos_out, c.status, post_rope=True)
        layer = 0
    else:
        L = slices // H
        big = [torch.empty(1, L, H, per, d, dtype=dtype, device="cuda") for _ in range(2)]
        for x, y in zip(big, (c.kv.k, c.kv.v)):
            x[:, L - 1:] = y
        nv = torch.zeros(L * H, dtype=torch.int32, device="cuda")
        nv[-H:] = c.kv.n_valid
        kv = tri.KVCache(*big, nv, None, None, c.status, post_rope=True)
        layer = L - 1
    assert big[0].numel() * elem > 1 << 32
    q = torch.randn(1, 70, H * G, d, generator=c.g, device="cuda").to(dtype)
    res = []
    for cache, lay in ((c.kv, 0), (kv, layer)):
        out, lse = torch.empty_like(q), torch.empty(1, 70, H * G, device="cuda")
        mass = torch.zeros(cache.n_slices, per, device="cuda")
        dec = torch.empty(1, H * G, d, dtype=dtype, device="cuda")
        tri.attn_prefill(cache, lay, q, out, lse=lse)
        tri.attn_mass(cache, lay, q, lse, mass)
        tri.attn_mass(cache, lay, q[:, -8:], lse[:, -8:], mass)
        tri.attn_decode(cache, lay, q[:, 69], dec, mass=mass)
        c.ok()
        res.append((out, lse, mass[-H:], dec))
    for x, y in zip(*res):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("what", ["nan", -1, 1 << 20])
def test_decode_blocks_out_of_sight(dtype, block, what):
    for lens, n_sink, window in (([[333, 700], [64, 200]], 4, 90), ([[9000]], 0, 33), ([[3000, 2900]], 130, 65)):
        c = Case(lens, 128, dtype, L=1, block=block)
        assert hide(c, [1] * c.B, n_sink, window, what) > 0
        check_decode(c, 4, layer=0, n_sink=n_sink, window=window, with_mass=True)
