"""Chunks over 4-bit caches in the launch shapes of long ones (tri_attn_prefill_q4: several query
tiles, a pair of them per CTA, rows shared by a cluster, more CTAs than SMs), and appending in the
shape of long prompts (several tokens per CTA, last tiles that are part empty), against the
definitions in 64 bits.

Tolerances as in test_gpu_q4.py (a chunk whose rows are written out) and test_gpu_append.py.
"""
import numpy as np
import pytest
import torch

import kv_cache_compression_tri_gb300 as tri
from q4_oracle import values
from test_gpu_append import Cache, check
from test_gpu_q4 import Case

pytestmark = pytest.mark.gpu
Q4 = torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tri.load_library()


def check_chunk(c, G, n_q, n_new=None, n_sink=0, window=0, seed=1):
    """check_prefill of test_gpu_q4.py for a chunk whose rows are written out, all queries of a slice at once."""
    B, H, d = c.B, c.H, c.d
    assert -(-n_q // (8 // G)) > 8  # passes of the decode kernel: too many
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(B, n_q, H * G, d, generator=g, device="cuda").bfloat16()
    out = torch.full((B, n_q, H * G, d), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, n_q, H * G), 9.0, device="cuda")
    nn = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device="cuda")
    need = tri.attn_prefill_workspace_bytes(c.kv)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    tri.attn_prefill(c.kv, 0, q, out, n_new=nn, n_sink=n_sink, window=window, lse=lse, workspace=ws[:need])
    c.ok()
    assert bool((ws[need:] == 0xFF).all())
    sc = d ** -0.5
    for b in range(B):
        new = n_q if n_new is None else n_new[b]
        assert bool((out[b, new:] == 9).all()) and bool((lse[b, new:] == 9).all())
        for h in range(H):
            n = int(c.lens[b, h])
            if new == 0:
                continue
            hs = slice(h * G, (h + 1) * G)
            got_o, got_l = out[b, :new, hs].double(), lse[b, :new, hs].double()
            row, col = (torch.arange(n - new, n, device="cuda")[:, None], torch.arange(n, device="cuda")[None])
            seen = col <= row
            if window:
                seen &= (col < n_sink) | (col > row - window)
            none = ~seen.any(1)
            assert bool((got_o[none] == 0).all()) and bool((got_l[none] == -np.inf).all())
            some = ~none
            if not bool(some.any()):
                continue
            k, v = (torch.from_numpy(values(x)).cuda() for x in c.slice_rows(b, 0, h))
            qd = q[b, :new, hs].double()[some]  # [queries, G, d]
            vis = seen[some][:, None]
            x = (sc * (qd @ k.T)).masked_fill(~vis, -np.inf)
            want_l = torch.logsumexp(x, -1)
            w = torch.exp(x - want_l[..., None])
            want_o = w @ v
            ex = ((d + 10) * 2.0 ** -23 + 2.0 ** -16) * sc * (qd.abs() @ k.abs().T).masked_fill(~vis, 0).amax(-1)
            ew = 2 * ex + 2.0 ** -20 + 2.0 ** -22 * x.masked_fill(~vis, 0).abs().amax(-1)
            most = (v.abs().amax(-1) * vis).amax(-1)
            tol = (w @ v.abs()) * (2 * ew + 2.0 ** -10 + n * 2.0 ** -24)[..., None] + (n * 2.0 ** -31 * most + 2.0 ** -25)[..., None] + 2.0 ** -8 * want_o.abs()
            off = (got_o[some] - want_o).abs() / tol
            assert bool((off <= 1).all()), (b, h, float(off.max()))
            off_l = (got_l[some] - want_l).abs() / (ex + ew + 2.0 ** -22 * want_l.abs().clamp(min=1))
            assert bool((off_l <= 1).all()), (b, h, float(off_l.max()))


# few CTAs: 1, 2, 4 and 8 of them share the rows of a pair of query tiles (d 128: 64 tokens at group 4)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q", [70, 131])
@pytest.mark.parametrize("rows", [[400, 131], [600, 577], [1100, 1029], [2200, 2113]])
def test_chunks_shared_by_a_cluster(d, n_q, rows):
    check_chunk(Case([rows], d, L=1), 4, n_q)


@pytest.mark.parametrize("d", [64, 128])
def test_chunks_with_a_window_shared_by_a_cluster(d):
    check_chunk(Case([[2200, 1500]], d, L=1, block=16), 4, 131, n_sink=5, window=1000)
    check_chunk(Case([[2200, 900], [300, 2113]], d, L=1, block=64), 4, 99, n_new=[65, 99], n_sink=130, window=64)


# more pairs of query tiles than half the SMs
@pytest.mark.parametrize("d,group,n_q", [(128, 4, 131), (64, 4, 131), (128, 1, 290), (64, 2, 301), (128, 7, 100)])
@pytest.mark.parametrize("n_sink,window,block", [(0, 0, 0), (5, 100, 16), (200, 77, 64)])
def test_chunks_of_many_tiles(d, group, n_q, n_sink, window, block):
    H = 8
    lens = np.random.default_rng(d + n_q).integers(n_q, 700, (4, H))
    lens[1, 0], lens[3, 2], lens[3, 3], lens[0, 1] = n_q, n_q - 30, 0, 512  # (tokens before the first row)
    check_chunk(Case(lens, d, L=1, block=block), group, n_q, n_new=[n_q, n_q // 2 + 3, 0, n_q - 1], n_sink=n_sink, window=window)


# more tokens than the SMs' first CTAs take: 4 of them per CTA at d 64, 2 at d 128
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, Q4])
@pytest.mark.parametrize("d,B,n_q,n_new", [(64, 3, 601, [601, 334, 599]), (128, 2, 401, [401, 200])])
def test_append_several_tokens_per_cta(dtype, d, B, n_q, n_new):
    c = Cache([[5, 0]] * (B - 1) + [[17, 30]], d, dtype, 640, L=1, block=16)
    check(c, n_q, 2, layer=0, n_new=n_new, half=d == 64, axes=[f % 2 for f in range(d // 2)])
    assert int(c.status) == 0


def test_append_several_tokens_and_head_tiles_per_cta():
    c = Cache([[3 * h for h in range(20)]], 64, Q4, 704, L=1)  # 16 heads, and 4
    check(c, 613, 1, layer=0, n_new=[611])
    assert int(c.status) == 0


@pytest.mark.parametrize("lens,d,group,n_q,n_sink,window", [([[700, 33]], 64, 4, 3, 0, 0), ([[20000]], 128, 2, 9, 0, 0), ([[9000, 8800]] * 8, 64, 1, 30, 0, 0),
                                                            ([[5000, 4990]], 128, 4, 16, 7, 3000), ([[200] * 6] * 9, 64, 8, 5, 0, 50)])
def test_scratch_of_few_tokens(lens, d, group, n_q, n_sink, window):
    c = Case(lens, d, L=1, block=64)
    q = torch.randn(c.B, n_q, c.H * group, d, device="cuda").bfloat16()
    need, full = tri.attn_prefill_workspace_bytes(c.kv, q, n_sink, window), tri.attn_prefill_workspace_bytes(c.kv)
    assert 16 <= need <= full
    outs = []
    for size in (need, full, None):
        out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:3], 9.0, device="cuda")
        ws = None if size is None else torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        tri.attn_prefill(c.kv, 0, q, out, n_sink=n_sink, window=window, lse=lse, workspace=None if size is None else ws[:size])
        c.ok()
        assert size is None or bool((ws[size:] == 0xA5).all())
        outs.append((out, lse))
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(outs[0], o))


def test_few_tokens_over_a_large_cache_need_little_memory():
    n_cap = 1 << 17  # 1.3 GB of rows, 6.4 GB if they were written out
    k = torch.zeros(8, 1, 8, n_cap, 80, dtype=torch.uint8, device="cuda")
    nv = torch.full((64,), 100, dtype=torch.int32, device="cuda")
    kv = tri.KVCache(k, k, nv, None, None, torch.zeros(1, dtype=torch.int32, device="cuda"), post_rope=True)
    q = torch.randn(8, 2, 32, 128, device="cuda").bfloat16()
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    tri.attn_prefill(kv, 0, q, out)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < 16 << 20
    assert not bool(out.any())
