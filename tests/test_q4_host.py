"""Host-side argument checks of tri_append, tri_read_rows and the calls on 4-bit
caches (they return before anything touches CUDA), and the 64-bit definitions on
cases worked by hand."""
import ctypes

import numpy as np
import pytest

from q4_oracle import nibble, pack, quantise, rotate, values
from test_abi_host import INVALID, PAGED, UNSUPPORTED, _kv, lib  # noqa: F401  (lib is a fixture)
from test_attn_host import BAD_Q, _q

Q4 = dict(dtype=2, key_layout=1, slice_stride=128 * 48)  # two heads, d 64, 128 rows
Q4_PAGED = dict(PAGED, dtype=2, key_layout=1, block_stride=2 * 16 * 48, layer_stride=2 * 16 * 48, head_stride=16 * 48)
AXES = bytes([0, 1] * 16)


def _tok(**over):
    import kv_cache_compression_tri_gb300 as tri
    f = dict(k=0x100000, v=0x200000, k_seq_stride=3 * 128, k_token_stride=128, v_seq_stride=3 * 128, v_token_stride=128,
             q=0x300000, q_out=0x400000, q_seq_stride=3 * 256, q_token_stride=256, q_out_seq_stride=3 * 256, q_out_token_stride=256,
             positions=0x500000, band_axis=None, n_new=None, rope_theta=1e4, style=0, n_axes=1, n_q=3, group=2, layer=0)
    f.update(over)
    return tri._TriTokens(*f.values())


def _append(lib, kv, tok):  # noqa: F811
    return lib.tri_append(ctypes.byref(kv), ctypes.byref(tok), None)


@pytest.mark.parametrize("over,code", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=0x100008), INVALID), (dict(v=0x200008), INVALID),
    (dict(k_seq_stride=-128), INVALID), (dict(k_token_stride=120), INVALID),  # tokens overlap
    (dict(k_token_stride=132), INVALID),  # rows not 16-byte aligned
    (dict(v_token_stride=64), INVALID), (dict(v_seq_stride=4), INVALID),
    (dict(q=0x300008), INVALID), (dict(q_out=None), INVALID), (dict(q_out=0x400008), INVALID),
    (dict(q_token_stride=128), INVALID), (dict(q_out_token_stride=128), INVALID),
    (dict(group=0), INVALID), (dict(group=9), INVALID),
    (dict(q_out=0x300000, q_out_token_stride=512), INVALID),  # in place at other strides
    (dict(positions=None), INVALID), (dict(positions=0x500002), INVALID), (dict(n_new=0x600002), INVALID),
    (dict(n_axes=0), INVALID), (dict(n_axes=5), INVALID), (dict(n_axes=2), INVALID),  # bands without axes
    (dict(n_axes=1, band_axis=AXES), INVALID),  # an axis that is not there
    (dict(style=2), INVALID), (dict(rope_theta=1.0), INVALID), (dict(rope_theta=float("nan")), INVALID),
    (dict(rope_theta=float("inf")), INVALID), (dict(n_q=0), INVALID), (dict(n_q=(1 << 31) - 1), INVALID),
    (dict(layer=-1), INVALID), (dict(layer=1), INVALID),
])
def test_append_rejects_bad_tokens(lib, over, code):  # noqa: F811
    assert _append(lib, _kv(key_layout=1), _tok(**over)) == code


def test_append_rejects_results_that_overlap(lib):  # noqa: F811
    kv = _kv(key_layout=1, n_seq=2)
    for seq, token in ((0, 256), (256, 256), (2 * 256, 256), (2 * 256 + 8, 256)):
        assert _append(lib, kv, _tok(q_out_seq_stride=seq, q_out_token_stride=token)) == INVALID


@pytest.mark.parametrize("over,code", [
    (dict(head_dim=96), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(n_valid=None), INVALID), (dict(slice_stride=100), INVALID), (dict(PAGED, block_size=24), INVALID),
    (dict(Q4, key_layout=0), UNSUPPORTED),  # 4-bit rows of pre-RoPE keys
    (dict(Q4, slice_stride=128 * 48 - 16), INVALID), (dict(Q4, slice_stride=128 * 48 + 8), INVALID),
    (dict(Q4_PAGED, head_stride=15 * 48), INVALID), (dict(Q4_PAGED, block_stride=2 * 16 * 48 + 8), INVALID),
])
def test_append_rejects_bad_caches(lib, over, code):  # noqa: F811
    assert _append(lib, _kv(**over), _tok()) == code


def test_append_rejects_several_axes_before_the_rotation(lib):  # noqa: F811
    assert _append(lib, _kv(), _tok(n_axes=2, band_axis=AXES)) == UNSUPPORTED
    assert lib.tri_append(None, ctypes.byref(_tok()), None) == INVALID
    assert lib.tri_append(ctypes.byref(_kv()), None, None) == INVALID


@pytest.mark.parametrize("over", [Q4, Q4_PAGED])
def test_calls_that_4_bit_caches_do_not_have(lib, over):  # noqa: F811
    import kv_cache_compression_tri_gb300 as tri
    kv = _kv(**over)
    kp, qp = ctypes.byref(kv), ctypes.byref(_q())
    c = tri._TriCenters(0x10000, 0x20000, 0x30000)
    offs = ctypes.cast((ctypes.c_int32 * 1)(1), ctypes.c_void_p)
    assert lib.tri_score(kp, ctypes.byref(c), 1e4, 0, 0, offs, 1, 0x70000, 0, 0, 0x80000, None) == UNSUPPORTED
    assert lib.tri_score_heads(kp, ctypes.byref(c), 2, 1e4, 0, 0, offs, 1, 0x70000, 0x80000, 0x90000, 0xA0000, 1 << 40, None) == UNSUPPORTED
    assert lib.tri_compress(kp, ctypes.byref(c), 1e4, 0, 0, offs, 1, 0x70000, 0, 0, 64, 0x80000, 0x90000, 1 << 40, None) == UNSUPPORTED
    assert lib.tri_attn_prefill(kp, qp, 0x30000, None, None) == UNSUPPORTED
    assert lib.tri_attn_mass(kp, qp, 0x50000, 16, 0x60000, None) == UNSUPPORTED
    assert lib.tri_compress_workspace_bytes(kp) == 0
    assert lib.tri_score_heads_workspace_bytes(kp, 2) == 0


def _q4_calls(lib, kv, q, **o):  # noqa: F811
    kp, qp = ctypes.byref(kv), ctypes.byref(q)
    yield lib.tri_attn_decode(kp, qp, o.get("out", 0x30000), o.get("lse"), None, o.get("ws", 0x40000), o.get("ws_bytes", 1 << 40), None)
    yield lib.tri_attn_prefill_q4(kp, qp, o.get("out", 0x30000), o.get("lse"), o.get("ws", 0x40000), o.get("ws_bytes", 1 << 40), None)


@pytest.mark.parametrize("over,code", BAD_Q)
def test_attention_over_4_bits_rejects_bad_queries(lib, over, code):  # noqa: F811
    assert list(_q4_calls(lib, _kv(**Q4), _q(**over))) == [code] * 2


def test_attention_over_4_bits_rejects_bad_buffers(lib):  # noqa: F811
    kv = _kv(**Q4)
    for o in (dict(out=None), dict(out=0x30004), dict(lse=0x50002), dict(ws=None), dict(ws=0x40008), dict(ws_bytes=0)):
        assert list(_q4_calls(lib, kv, _q(), **o)) == [INVALID] * 2
    need = lib.tri_attn_prefill_q4_workspace_bytes(ctypes.byref(kv))
    assert need >= 3 * 2 * 128 * 64 * 2 and need % 16 == 0  # K twice and V of two heads, 16 bits
    assert list(_q4_calls(lib, kv, _q(), ws_bytes=need - 1))[1] == INVALID
    assert lib.tri_attn_prefill_q4_workspace_bytes(None) == 0
    for other in (_kv(key_layout=1), _kv(key_layout=1, dtype=0)):  # bf16 and fp32 caches have their own call
        assert lib.tri_attn_prefill_q4_workspace_bytes(ctypes.byref(other)) == 0
        assert lib.tri_attn_prefill_q4(ctypes.byref(other), ctypes.byref(_q()), 0x30000, None, 0x40000, 1 << 40, None) == UNSUPPORTED
    far = _kv(**dict(Q4_PAGED, n_cap=1 << 30, num_blocks=64))  # more rows than a chunk's copies number
    q = _q(n_q=100, token_stride=4 * 64)
    assert lib.tri_attn_prefill_q4(ctypes.byref(far), ctypes.byref(q), 0x30000, None, 0x40000, 1 << 60, None) == UNSUPPORTED


def test_read_rows_rejects_bad_args(lib):  # noqa: F811
    call = lambda layer=0, k=0x30000, v=0x40000, **kv: lib.tri_read_rows(ctypes.byref(_kv(**{**Q4, **kv})), layer, k, v, None)
    assert call(layer=-1) == INVALID
    assert call(layer=1) == INVALID
    assert call(k=None, v=None) == INVALID
    assert call(k=0x30008) == INVALID
    assert call(v=0x40008) == INVALID
    assert call(dtype=1, slice_stride=128 * 64) == UNSUPPORTED
    assert call(n_valid=None) == INVALID


def test_the_order_of_codes():
    for d in (64, 128):
        assert sorted(nibble(d, e) for e in range(d)) == list(range(d))
    # d 128: the first word holds elements 0 .. 7, the next the same of the second quarter
    assert [nibble(128, e) for e in (0, 7, 8, 32)] == [0, 7, 32, 8]
    # d 64: the first word: elements 0, 1 of quarters 0 and 1, then 2, 3
    assert [nibble(64, e) for e in (0, 1, 16, 17, 2, 3, 18, 19, 4, 32)] == [0, 1, 2, 3, 4, 5, 6, 7, 16, 8]


def test_quantisation_by_hand():
    x = np.zeros(64)
    x[:16] = np.arange(16) * 0.5 - 2  # scale 1/2, exactly
    x[16:32] = 7.0  # one value: scale 0
    x[32:48] = np.where(np.arange(16) % 2, 1e9, -1e9)  # saturates
    x[50] = np.nan
    codes, scale, low = quantise(x)
    assert scale[0] == 0.5 and low[0] == -2 and codes[:16].tolist() == list(range(16))
    assert scale[1] == 0 and low[1] == 7 and not codes[16:32].any()
    assert low[2] == -30656 and scale[2] == np.float16(2 * 30656 / 15) and set(codes[32:48]) == {0, 15}
    assert np.isnan(scale[3]) and np.isnan(low[3])
    v = values(pack(x))
    assert np.array_equal(v[:32], x[:32]) and np.isnan(v[48:]).all()
    # the error is at most half a step, and what the pair's rounding to fp16 moves (2^-11 of the minimum, 15 times that of the scale)
    y = np.random.default_rng(0).normal(size=128) * 3
    _, s, m = quantise(y)
    assert (np.abs(values(pack(y)) - y).reshape(4, 32) <= (s / 2 + np.abs(m) * 2.0 ** -11 + 15 * s * 2.0 ** -11)[:, None]).all()


def test_rotation_by_hand():
    x = np.array([1.0, 0.0, 0.0, 1.0])
    # d 4, theta 100: bands turn by p and p / 10
    r = rotate(x, [2], 100.0)
    assert np.allclose(r, [np.cos(2), np.sin(2), -np.sin(0.2), np.cos(0.2)])
    r = rotate(np.array([1.0, 0.0, 0.0, 1.0]), [2], 100.0, half=True)
    assert np.allclose(r, [np.cos(2), -np.sin(0.2), np.sin(2), np.cos(0.2)])
    r = rotate(x, [2, 5], 100.0, band_axis=[1, 0])
    assert np.allclose(r, [np.cos(5), np.sin(5), -np.sin(0.2), np.cos(0.2)])
    # the product of two rotated rows depends on their distance
    rng = np.random.default_rng(1)
    a, b = rng.normal(size=64), rng.normal(size=64)
    assert np.isclose(rotate(a, [1000], 1e4) @ rotate(b, [993], 1e4), rotate(a, [7], 1e4) @ b)


def test_more_than_a_launch_counts(lib):  # noqa: F811
    many = dict(key_layout=1, n_seq=1 << 24, n_kv_heads=64)
    tok = _tok(n_q=1 << 20, k_seq_stride=0, v_seq_stride=0, k_token_stride=64 * 64, v_token_stride=64 * 64, q=None)
    assert _append(lib, _kv(**many), tok) == UNSUPPORTED
    assert lib.tri_read_rows(ctypes.byref(_kv(**dict(Q4, n_seq=1 << 24, n_kv_heads=64, n_cap=1 << 20, slice_stride=48 << 20))), 0, 0x30000, None,
                             None) == UNSUPPORTED


def _few(lib, kv, q):  # noqa: F811
    return lib.tri_attn_prefill_q4_few_workspace_bytes(ctypes.byref(kv), ctypes.byref(q))


def _few_call(lib, kv, q, **o):  # noqa: F811
    return lib.tri_attn_prefill_q4_few(ctypes.byref(kv), ctypes.byref(q), o.get("out", 0x30000), o.get("lse"), o.get("ws", 0x40000),
                                       o.get("ws_bytes", 1 << 40), None)


def test_scratch_of_few_tokens_does_not_grow_with_the_cache(lib):  # noqa: F811
    q = lambda n, group=4: _q(n_q=n, group=group, seq_stride=n * 8 * group * 128, token_stride=8 * group * 128)
    sizes = []
    for n_cap in (4096, 32768, 1 << 20):
        kv = _kv(dtype=2, key_layout=1, head_dim=128, n_seq=16, n_kv_heads=8, n_cap=n_cap, slice_stride=n_cap * 80)
        few = [_few(lib, kv, q(n)) for n in (1, 2, 5, 16)]
        # sums and (m, l) of at most 16 runs of 8 columns for each of the passes
        assert all(0 < b <= 128 * passes * 16 * 8 * (128 * 4 + 8) for b, passes in zip(few, (1, 1, 3, 8))), few
        full = lib.tri_attn_prefill_q4_workspace_bytes(ctypes.byref(kv))
        assert full >= 6 * 128 * n_cap * 128 and max(few) <= full
        assert _few(lib, kv, q(17)) == 0  # nine passes: written out
        sizes.append(few[1])
    assert sizes[1] == sizes[2] and sizes[1] <= 8 << 20, sizes


@pytest.mark.parametrize("over,code", BAD_Q)
def test_few_tokens_reject_bad_queries(lib, over, code):  # noqa: F811
    kv, q = _kv(**Q4), _q(**over)
    assert _few_call(lib, kv, q) == code and _few(lib, kv, q) == 0


def test_few_tokens_reject_bad_buffers_and_other_calls(lib):  # noqa: F811
    kv, q = _kv(**Q4), _q()
    need = _few(lib, kv, q)
    assert 16 <= need <= lib.tri_attn_prefill_q4_workspace_bytes(ctypes.byref(kv)) and need % 16 == 0
    for o in (dict(out=None), dict(out=0x30004), dict(lse=0x50002), dict(ws=None), dict(ws=0x40008), dict(ws_bytes=need - 1)):
        assert _few_call(lib, kv, q, **o) == INVALID
    many = _q(n_q=100, token_stride=4 * 64)
    assert _few(lib, kv, many) == 0 and _few_call(lib, kv, many) == UNSUPPORTED
    for other in (_kv(key_layout=1), _kv(**dict(Q4, key_layout=0))):
        assert _few(lib, other, q) == 0 and _few_call(lib, other, q) == UNSUPPORTED
    assert lib.tri_attn_prefill_q4_few_workspace_bytes(None, None) == 0 and _few(lib, _kv(**dict(Q4, n_valid=None)), q) == 0


@pytest.mark.parametrize("d,n_seq,n_cap,passes", [(64, 4, 200, 8), (64, 64, 200, 2), (64, 16, 700, 4), (64, 64, 1400, 5), (64, 64, 2176, 7), (64, 32, 4096, 6), (64, 64, 8192, 8),
                                                  (128, 4, 200, 8), (128, 64, 200, 3), (128, 32, 700, 5), (128, 32, 1400, 6), (128, 16, 2176, 8)])
def test_passes_that_are_of_few_tokens(lib, d, n_seq, n_cap, passes):  # noqa: F811
    # 8 heads: slices and rows of which more passes were measured to take longer than rows written out
    kv = _kv(dtype=2, key_layout=1, head_dim=d, n_seq=n_seq, n_kv_heads=8, n_cap=n_cap, slice_stride=n_cap * (d // 2 + 16))
    for group, t in ((1, 8), (2, 4), (3, 2), (8, 1)):
        q = lambda n: _q(n_q=n, group=group, seq_stride=n * 8 * group * d, token_stride=8 * group * d)
        few = [n for n in range(1, 80) if _few(lib, kv, q(n)) > 0]
        assert few == list(range(1, passes * t + 1))


def test_attention_refuses_more_rows_than_it_counts(lib):  # noqa: F811
    from test_attn_host import _calls
    for n_cap in ((1 << 31) - 1, (1 << 31) - 64, (1 << 31) - 256):
        kv = _kv(**dict(Q4, n_cap=n_cap, slice_stride=n_cap * 48))
        assert list(_q4_calls(lib, kv, _q(), ws_bytes=1 << 62)) == [UNSUPPORTED] * 2 and _few(lib, kv, _q()) == 0
        assert list(_calls(lib, _kv(key_layout=1, n_cap=n_cap, slice_stride=n_cap * 64), _q())) == [UNSUPPORTED] * 3
