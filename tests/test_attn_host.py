"""Host-side argument checks of the attention and mass-eviction calls (they
return before anything touches CUDA), the binding's own checks, and the 64-bit
definitions on cases worked by hand."""
import ctypes

import numpy as np
import pytest
import torch

from attn_oracle import attend, evict, visible
from test_abi_host import INVALID, PAGED, UNSUPPORTED, _kv, lib  # noqa: F401  (lib is a fixture)


def _q(**over):
    import kv_cache_compression_tri_gb300 as tri
    f = dict(q=0x10000, seq_stride=4 * 64, token_stride=4 * 64, n_new=None, n_q=1, group=2, layer=0, n_sink=0, window=0, scale=0.125)
    f.update(over)
    return tri._TriQueries(*f.values())


def _post(**over):
    return _kv(**{"key_layout": 1, **over})


BAD_Q = [
    (dict(q=None), INVALID),
    (dict(q=0x10008), INVALID),  # not 16-byte aligned
    (dict(n_q=0), INVALID),
    (dict(group=0), INVALID),
    (dict(group=9), INVALID),
    (dict(layer=-1), INVALID),
    (dict(layer=1), INVALID),  # the cache has one layer
    (dict(n_sink=-1), INVALID),
    (dict(window=-1), INVALID),
    (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(n_new=0x20002), INVALID),
    (dict(seq_stride=-8), INVALID),
    (dict(seq_stride=4), INVALID),  # rows not 16-byte aligned
    (dict(token_stride=4 * 64 + 4), INVALID),
]
BAD_KV = [
    (dict(key_layout=0), UNSUPPORTED),  # keys as cached: post-RoPE only
    (dict(head_dim=96), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED),
    (dict(v=None), INVALID),
    (dict(n_valid=None), INVALID),
    (dict(PAGED, block_size=24), INVALID),
]


def _calls(lib, kv, q, **o):  # noqa: F811
    kp, qp = ctypes.byref(kv), ctypes.byref(q)
    yield lib.tri_attn_decode(kp, qp, o.get("out", 0x30000), o.get("lse"), o.get("mass"), o.get("ws", 0x40000), o.get("ws_bytes", 1 << 40), None)
    yield lib.tri_attn_prefill(kp, qp, o.get("out", 0x30000), o.get("lse"), None)
    yield lib.tri_attn_mass(kp, qp, o.get("lse_in", 0x50000), 16, o.get("mass_in", 0x60000), None)


@pytest.mark.parametrize("over,code", BAD_Q)
def test_attention_rejects_bad_queries(lib, over, code):  # noqa: F811
    assert list(_calls(lib, _post(), _q(**over))) == [code] * 3


@pytest.mark.parametrize("over,code", BAD_KV)
def test_attention_rejects_bad_caches(lib, over, code):  # noqa: F811
    assert list(_calls(lib, _post(**over), _q())) == [code] * 3


def test_attention_rejects_bad_buffers(lib):  # noqa: F811
    kv, q = _post(), _q()
    for o in (dict(out=None), dict(out=0x30004), dict(lse=0x50002)):
        assert list(_calls(lib, kv, q, **o))[:2] == [INVALID] * 2
    dec = lambda **o: next(_calls(lib, kv, o.pop("q", q), **o))
    assert dec(mass=0x60002) == INVALID
    assert dec(ws=None) == INVALID
    assert dec(ws=0x40008) == INVALID
    need = lib.tri_attn_decode_workspace_bytes(ctypes.byref(kv), 2, 0)
    assert need > 0 and need % 16 == 0
    assert dec(ws_bytes=need - 1) == INVALID
    more = lib.tri_attn_decode_workspace_bytes(ctypes.byref(kv), 2, 1)
    assert more > need
    assert dec(mass=0x60000, ws_bytes=more - 1) == INVALID
    assert dec(q=_q(n_q=2)) == INVALID  # one token per sequence
    assert lib.tri_attn_decode_workspace_bytes(ctypes.byref(kv), 9, 0) == 0
    assert lib.tri_attn_decode_workspace_bytes(None, 2, 0) == 0
    mass = lambda **o: list(_calls(lib, kv, q, **o))[2]
    assert mass(lse_in=None) == INVALID
    assert mass(lse_in=0x50002) == INVALID
    assert mass(mass_in=None) == INVALID
    assert mass(mass_in=0x60002) == INVALID
    # a chunk's tokens may not overlap
    q2 = _q(n_q=2, token_stride=2 * 64)
    assert list(_calls(lib, kv, q2))[1:] == [INVALID] * 2
    assert lib.tri_attn_prefill(ctypes.byref(kv), None, 0x30000, None, None) == INVALID


def test_mass_evict_rejects_bad_args(lib):  # noqa: F811
    call = lambda **o: lib.tri_mass_evict(o.get("mass", 0x10000), o.get("mass_out", 0x20000), ctypes.byref(o.get("kv", _kv())), o.get("P", 0),
                                          o.get("W", 0), o.get("budget", 64), o.get("keep", 0x50000), None)
    assert call(mass=None) == INVALID
    assert call(mass=0x10002) == INVALID
    assert call(mass_out=None) == INVALID
    assert call(mass_out=0x20001) == INVALID
    assert call(keep=None) == INVALID
    assert call(P=40, W=40) == INVALID
    assert call(budget=0) == INVALID
    assert call(budget=129) == INVALID
    assert call(kv=_kv(pos_out=None)) == INVALID
    assert call(kv=_kv(v=None)) == INVALID
    assert call(kv=_kv(head_dim=96)) == UNSUPPORTED


def test_mass_evict_rejects_masses_that_overlap(lib):  # noqa: F811
    kv = _kv()
    nbytes = kv.n_seq * kv.n_layers * kv.n_kv_heads * kv.n_cap * 4
    call = lambda m0, m1: lib.tri_mass_evict(m0, m1, ctypes.byref(kv), 0, 0, 64, 0x50000, None)
    for off in (4, 4 * kv.n_cap, nbytes - 4):
        assert call(0x1000000, 0x1000000 + off) == INVALID
        assert call(0x1000000 + off, 0x1000000) == INVALID


def test_definitions_by_hand():
    # rows seen by row 9 with two sinks and a window of three
    assert visible(9, 12, 2, 3).nonzero()[0].tolist() == [0, 1, 7, 8, 9]
    assert visible(1, 12, 5, 3).nonzero()[0].tolist() == [0, 1]
    assert visible(-1, 12, 5, 3).sum() == 0
    # weights 1/3, 2/3 from logits log 1, log 2
    k, v = np.array([[0.0], [np.log(2.0)]]), np.array([[3.0], [6.0]])
    o, l, w = attend(np.array([1.0]), k, v, 1, 1.0)
    assert np.allclose(w, [1 / 3, 2 / 3]) and np.allclose(o, [5.0]) and np.isclose(l, np.log(3.0))
    o, l, w = attend(np.array([1.0]), k, v, -1, 1.0)
    assert o[0] == 0 and l == -np.inf and w.sum() == 0
    # masses 5 4 4 1 4 9: two protected ends, two kept of the rest, the lower of equal masses
    assert evict([5, 4, 4, 1, 4, 9], 6, 1, 1, 4).tolist() == [0, 1, 2, 5]
    assert evict([5, 4], 2, 1, 1, 4).tolist() == [0, 1]


def test_weights_are_derivatives_of_the_log_sum():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=8), rng.normal(size=(6, 8)), rng.normal(size=(6, 8))
    _, l, w = attend(q, k, v, 5, 0.5, 1, 3)
    for j in range(6):
        e = 1e-6
        k2 = k.copy()
        k2[j] += e * q / (0.5 * (q @ q))  # moves logit j by e
        assert np.isclose((attend(q, k2, v, 5, 0.5, 1, 3)[1] - l) / e, w[j], atol=1e-5)


def test_prompts_and_masses_refuse_more_rows_than_a_coordinate_numbers(lib):  # noqa: F811
    rows = dict(PAGED, num_blocks=1 << 27, block_stride=16 * 64, head_stride=(1 << 27) * 16 * 64, layer_stride=0)
    far = dict(slice_stride=((1 << 31) - 128) * 64)
    for over in (rows, far):
        kp, qp = ctypes.byref(_post(**over)), ctypes.byref(_q())
        assert lib.tri_attn_prefill(kp, qp, 0x30000, None, None) == UNSUPPORTED
        assert lib.tri_attn_mass(kp, qp, 0x50000, 16, 0x60000, None) == UNSUPPORTED
    # queries too, where no map of theirs fits their strides
    q = _q(n_q=3, token_stride=(1 << 36) + 8, seq_stride=0)
    assert lib.tri_attn_mass(ctypes.byref(_post()), ctypes.byref(q), 0x50000, 16, 0x60000, None) == UNSUPPORTED


def test_more_tokens_than_tiles_can_count(lib):  # noqa: F811
    for n_q in ((1 << 31) - 1, (1 << 31) - 256):  # (rounding up to tiles would leave the int range)
        assert list(_calls(lib, _post(), _q(n_q=n_q))) == [INVALID] * 3
