"""GB300 KV-cache compression: TriAttention scoring, budgeted selection,
in-place compaction, and Random Attention eviction.

This module is a thin ctypes binding over ``libtri.so`` (C ABI in
``include/tri.h``): it turns torch tensors into device pointers and the
current CUDA stream into a stream handle, and raises on a non-zero status.
Every step of the path runs in the library's CUDA kernels; there is no
fallback. If the library has not been built, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass

import torch

from ._build import LIB as _LIB_PATH

__all__ = [
    "TriError", "KVCache", "PagedKVCache", "select_compact", "rand_evict_compact", "paged_blocks_used", "Centers", "lib_path", "load_library", "calibrate_centers",
    "calibrate_workspace_bytes", "score", "select_topk", "compact_kv", "rand_evict",
    "compress", "compress_workspace_bytes", "score_heads", "score_heads_workspace_bytes",
    "select_topk_zmax", "select_union", "select_union_workspace_bytes", "rand_evict_scoped", "DRAW_PER_HEAD", "DRAW_PER_LAYER", "DRAW_PER_SEQUENCE",
    "launch_count", "ROPE_INTERLEAVED", "ROPE_HALF", "NORM_WEIGHTED", "NORM_UNWEIGHTED",
    "DEV_OK", "DEV_NVALID_OVER_CAP", "DEV_NAN_SCORE", "DEV_BAD_KEEP", "DEV_BAD_QUERY",
    "attn_decode", "attn_decode_workspace_bytes", "attn_prefill", "attn_mass", "mass_evict",
    "append", "read_rows", "attn_prefill_workspace_bytes", "q4_row_bytes",
]

ROPE_INTERLEAVED, ROPE_HALF = 0, 1
NORM_WEIGHTED, NORM_UNWEIGHTED = 0, 1
F32, BF16, Q4 = 0, 1, 2
(DEV_OK, DEV_NVALID_OVER_CAP, DEV_NAN_SCORE, DEV_BAD_KEEP, DEV_TIMEOUT, DEV_GROUP_NVALID, DEV_BAD_BLOCK,
 DEV_BAD_QUERY) = (0, 1, 2, 3, 4, 5, 6, 7)

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}
_KV_DTYPES = {**_DTYPES, torch.uint8: Q4}
_Q4_DIMS = {48: 64, 80: 128}  # head dimension of a 4-bit row of so many bytes


def q4_row_bytes(head_dim: int) -> int:
    """Bytes of a 4-bit row (TRI_Q4): codes, and scale and minimum of each quarter."""
    return head_dim // 2 + 16


class TriError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: status {status} ({msg})")
        self.status = status


class _TriKV(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pos", ctypes.c_void_p),
        ("pos_out", ctypes.c_void_p), ("n_valid", ctypes.c_void_p),
        ("slice_stride", ctypes.c_int64), ("n_seq", ctypes.c_int32),
        ("n_layers", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("n_cap", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int),
        ("dev_status", ctypes.c_void_p), ("key_layout", ctypes.c_int),
        ("block_table", ctypes.c_void_p), ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
        ("block_stride", ctypes.c_int64), ("layer_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
    ]


class _TriCenters(ctypes.Structure):
    _fields_ = [("center", ctypes.c_void_p), ("mean_norm", ctypes.c_void_p),
                ("mrl", ctypes.c_void_p)]


class _TriTokens(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_seq_stride", ctypes.c_int64), ("k_token_stride", ctypes.c_int64),
        ("v_seq_stride", ctypes.c_int64), ("v_token_stride", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
        ("q_seq_stride", ctypes.c_int64), ("q_token_stride", ctypes.c_int64),
        ("q_out_seq_stride", ctypes.c_int64), ("q_out_token_stride", ctypes.c_int64),
        ("positions", ctypes.c_void_p), ("band_axis", ctypes.c_char_p), ("n_new", ctypes.c_void_p),
        ("rope_theta", ctypes.c_double), ("style", ctypes.c_int), ("n_axes", ctypes.c_int32),
        ("n_q", ctypes.c_int32), ("group", ctypes.c_int32), ("layer", ctypes.c_int32),
    ]


class _TriQueries(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("seq_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
        ("n_new", ctypes.c_void_p), ("n_q", ctypes.c_int32), ("group", ctypes.c_int32),
        ("layer", ctypes.c_int32), ("n_sink", ctypes.c_int32), ("window", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


_lock = threading.Lock()
_lib = None


def lib_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libtri.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libtri.so is not built ({_LIB_PATH}); run __graft_entry__.build()")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i32, i64, u32, u64 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                  ctypes.c_uint32, ctypes.c_uint64)
        kvp = ctypes.POINTER(_TriKV)
        lib.tri_status_string.argtypes = [ctypes.c_int]
        lib.tri_status_string.restype = ctypes.c_char_p
        lib.tri_abi_version.restype = i32
        lib.tri_launch_count.restype = u64
        lib.tri_calibrate_workspace_bytes.argtypes = [i32, i32, i32, i32, i64]
        lib.tri_calibrate_workspace_bytes.restype = ctypes.c_size_t
        lib.tri_calibrate_centers.argtypes = [vp, ctypes.c_int, i32, i32, i32, i32, i64,
                                              ctypes.c_int, _TriCenters, vp, ctypes.c_size_t, vp]
        lib.tri_calibrate_centers.restype = ctypes.c_int
        lib.tri_score.argtypes = [kvp, ctypes.POINTER(_TriCenters), ctypes.c_double, ctypes.c_int,
                                  ctypes.c_int, vp, i32, vp, i32, i32, vp, vp]
        lib.tri_score.restype = ctypes.c_int
        lib.tri_select_topk.argtypes = [vp, kvp, i32, i32, i32, vp, vp]
        lib.tri_select_topk.restype = ctypes.c_int
        lib.tri_compact_kv.argtypes = [kvp, vp, i32, vp]
        lib.tri_compact_kv.restype = ctypes.c_int
        lib.rand_evict.argtypes = [kvp, u64, u32, i32, i32, i32, vp, vp]
        lib.rand_evict.restype = ctypes.c_int
        lib.rand_evict_scoped.argtypes = [kvp, u64, u32, ctypes.c_int, i32, i32, i32, vp, vp]
        lib.rand_evict_scoped.restype = ctypes.c_int
        lib.tri_compress_workspace_bytes.argtypes = [kvp]
        lib.tri_compress_workspace_bytes.restype = ctypes.c_size_t
        lib.tri_compress.argtypes = [kvp, ctypes.POINTER(_TriCenters), ctypes.c_double, ctypes.c_int,
                                     ctypes.c_int, vp, i32, vp, i32, i32, i32, vp, vp, ctypes.c_size_t, vp]
        lib.tri_compress.restype = ctypes.c_int
        lib.tri_score_heads_workspace_bytes.argtypes = [kvp, i32]
        lib.tri_score_heads_workspace_bytes.restype = ctypes.c_size_t
        lib.tri_score_heads.argtypes = [kvp, ctypes.POINTER(_TriCenters), i32, ctypes.c_double, ctypes.c_int,
                                        ctypes.c_int, vp, i32, vp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.tri_score_heads.restype = ctypes.c_int
        lib.tri_select_topk_zmax.argtypes = [vp, vp, i32, kvp, i32, i32, i32, vp, vp, vp]
        lib.tri_select_topk_zmax.restype = ctypes.c_int
        lib.tri_select_union_workspace_bytes.argtypes = [kvp, i32, i32, i32]
        lib.tri_select_union_workspace_bytes.restype = ctypes.c_size_t
        lib.tri_select_union.argtypes = [vp, kvp, i32, i32, i32, i32, vp, vp, vp, ctypes.c_size_t, vp]
        lib.tri_select_union.restype = ctypes.c_int
        lib.tri_select_compact.argtypes = [vp, kvp, i32, i32, i32, vp, vp]
        lib.tri_select_compact.restype = ctypes.c_int
        lib.rand_evict_compact.argtypes = [kvp, u64, u32, ctypes.c_int, i32, i32, i32, vp, vp]
        lib.rand_evict_compact.restype = ctypes.c_int
        qp = ctypes.POINTER(_TriQueries)
        lib.tri_attn_decode_workspace_bytes.argtypes = [kvp, i32, i32]
        lib.tri_attn_decode_workspace_bytes.restype = ctypes.c_size_t
        lib.tri_attn_decode.argtypes = [kvp, qp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.tri_attn_decode.restype = ctypes.c_int
        lib.tri_attn_prefill.argtypes = [kvp, qp, vp, vp, vp]
        lib.tri_attn_prefill.restype = ctypes.c_int
        lib.tri_attn_prefill_q4_workspace_bytes.argtypes = [kvp]
        lib.tri_attn_prefill_q4_workspace_bytes.restype = ctypes.c_size_t
        lib.tri_attn_prefill_q4.argtypes = [kvp, qp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.tri_attn_prefill_q4.restype = ctypes.c_int
        lib.tri_attn_prefill_q4_few_workspace_bytes.argtypes = [kvp, qp]
        lib.tri_attn_prefill_q4_few_workspace_bytes.restype = ctypes.c_size_t
        lib.tri_attn_prefill_q4_few.argtypes = [kvp, qp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.tri_attn_prefill_q4_few.restype = ctypes.c_int
        lib.tri_append.argtypes = [kvp, ctypes.POINTER(_TriTokens), vp]
        lib.tri_append.restype = ctypes.c_int
        lib.tri_read_rows.argtypes = [kvp, i32, vp, vp, vp]
        lib.tri_read_rows.restype = ctypes.c_int
        lib.tri_attn_mass.argtypes = [kvp, qp, vp, i64, vp, vp]
        lib.tri_attn_mass.restype = ctypes.c_int
        lib.tri_mass_evict.argtypes = [vp, vp, kvp, i32, i32, i32, vp, vp]
        lib.tri_mass_evict.restype = ctypes.c_int
        lib.tri_paged_blocks_used.argtypes = [kvp, vp, vp]
        lib.tri_paged_blocks_used.restype = ctypes.c_int
        lib.tri_selftest_wait_timeout.argtypes = [vp, u64, vp]
        lib.tri_selftest_wait_timeout.restype = ctypes.c_int
        _lib = lib
        return lib


def _check(fn: str, status: int):
    if status != 0:
        msg = load_library().tri_status_string(status).decode()
        raise TriError(fn, status, msg)


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    """Memory for a call on `stream` (None: the current one), from that stream's own: the current
    stream's may still be in use there, and be handed out there again before the call has run."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _scratch(nbytes: int, device, stream=None) -> torch.Tensor:
    return _empty(max(nbytes, 16), torch.uint8, device, stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def launch_count() -> int:
    """Kernels the library has launched in this process."""
    return int(load_library().tri_launch_count())


@dataclass
class Centers:
    """Per-(layer, KV head) query statistics (fp32, device): center
    [L*H][F][2], mean_norm [L*H][F], mrl [L*H][F]."""
    center: torch.Tensor
    mean_norm: torch.Tensor
    mrl: torch.Tensor

    def _abi(self) -> _TriCenters:
        for t in (self.center, self.mean_norm, self.mrl):
            assert t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()
        return _TriCenters(self.center.data_ptr(), self.mean_norm.data_ptr(), self.mrl.data_ptr())


@dataclass
class KVCache:
    """A batch of caches: k, v [n_seq, n_layers, n_kv_heads, n_cap, head_dim]
    (bf16 or fp32, device); n_valid [S] int32; pos / pos_out [S, n_cap] int32
    (pos may be None: position = slot index); dev_status [1] int32.
    post_rope: k holds RoPE-rotated keys (the score then ignores pos).
    4-bit rows (post_rope only): k, v uint8 with q4_row_bytes(head_dim) in place
    of head_dim."""
    k: torch.Tensor
    v: torch.Tensor
    n_valid: torch.Tensor
    pos: torch.Tensor | None
    pos_out: torch.Tensor | None
    dev_status: torch.Tensor | None = None
    post_rope: bool = False

    @property
    def shape(self):
        return tuple(self.k.shape)

    @property
    def n_slices(self) -> int:
        s = self.k.shape
        return s[0] * s[1] * s[2]

    @property
    def n_cap(self) -> int:
        return self.k.shape[3]

    @property
    def device(self):
        return self.k.device

    def _abi(self) -> _TriKV:
        k, v = self.k, self.v
        shape, strides, dtype = k.shape, k.stride(), k.dtype
        n_seq, L, H, n_cap, d = shape
        assert k.is_cuda and dtype in _KV_DTYPES
        assert dtype != torch.uint8 or d in _Q4_DIMS
        assert v.shape == shape and v.dtype == dtype
        # rows contiguous, slices evenly strided
        stride = strides[2]
        assert strides == (L * H * stride, H * stride, stride, d, 1)
        assert v.stride() == strides
        assert self.n_valid.dtype == torch.int32 and self.n_valid.numel() == n_seq * L * H
        for t in (self.pos, self.pos_out):
            if t is not None:
                assert t.dtype == torch.int32 and t.is_contiguous() and t.numel() == n_seq * L * H * n_cap
        return _TriKV(k.data_ptr(), v.data_ptr(), _ptr(self.pos), _ptr(self.pos_out),
                      self.n_valid.data_ptr(), stride, n_seq, L, H, n_cap, _Q4_DIMS[d] if dtype == torch.uint8 else d, _KV_DTYPES[dtype],
                      _ptr(self.dev_status), 1 if self.post_rope else 0, None, 0, 0, 0, 0, 0)


@dataclass
class PagedKVCache:
    """A paged batch of caches: k, v pools [num_blocks, n_layers, n_kv_heads,
    block_size, head_dim] (bf16 or fp32, device; any strides that keep each
    (block, layer, head) run of block_size rows contiguous); block_table
    [n_seq, blocks per sequence] int32 (physical block of each logical block,
    shared by the sequence's layers and heads); n_valid [S] int32; pos /
    pos_out [S, n_cap] int32 with n_cap = blocks per sequence * block_size.
    4-bit rows as in KVCache: uint8 pools, q4_row_bytes(head_dim) per row."""
    k: torch.Tensor
    v: torch.Tensor
    block_table: torch.Tensor
    n_valid: torch.Tensor
    pos: torch.Tensor | None
    pos_out: torch.Tensor | None
    dev_status: torch.Tensor | None = None
    post_rope: bool = False

    @property
    def n_seq(self) -> int:
        return self.block_table.shape[0]

    @property
    def n_slices(self) -> int:
        return self.n_seq * self.k.shape[1] * self.k.shape[2]

    @property
    def n_cap(self) -> int:
        return self.block_table.shape[1] * self.k.shape[3]

    @property
    def device(self):
        return self.k.device

    def _abi(self) -> _TriKV:
        k, v, table = self.k, self.v, self.block_table
        shape, strides, dtype = k.shape, k.stride(), k.dtype
        nb, L, H, bs, d = shape
        assert k.is_cuda and dtype in _KV_DTYPES
        assert dtype != torch.uint8 or d in _Q4_DIMS
        assert v.shape == shape and v.dtype == dtype
        assert v.stride() == strides
        assert strides[4] == 1 and strides[3] == d
        assert table.dtype == torch.int32 and table.is_contiguous()
        n_seq, blocks = table.shape
        S, n_cap = n_seq * L * H, blocks * bs
        assert self.n_valid.dtype == torch.int32 and self.n_valid.numel() == S
        for t in (self.pos, self.pos_out):
            if t is not None:
                assert t.dtype == torch.int32 and t.is_contiguous() and t.numel() == S * n_cap
        return _TriKV(k.data_ptr(), v.data_ptr(), _ptr(self.pos), _ptr(self.pos_out),
                      self.n_valid.data_ptr(), 0, n_seq, L, H, n_cap, _Q4_DIMS[d] if dtype == torch.uint8 else d, _KV_DTYPES[dtype],
                      _ptr(self.dev_status), 1 if self.post_rope else 0, table.data_ptr(), bs, nb,
                      strides[0], strides[1], strides[2])


def paged_blocks_used(kv: PagedKVCache, out: torch.Tensor, stream=None) -> torch.Tensor:
    """Blocks each sequence still uses after compaction (tri_paged_blocks_used);
    table entries from there on are free. out: [n_seq] int32."""
    lib = load_library()
    assert out.dtype == torch.int32 and out.is_contiguous() and out.numel() == kv.n_seq
    kvs = kv._abi()
    _check("tri_paged_blocks_used", lib.tri_paged_blocks_used(ctypes.byref(kvs), out.data_ptr(), _stream(stream)))
    return out


def selftest_wait_timeout(status: torch.Tensor, limit_ns: int, stream=None) -> torch.Tensor:
    """The kernels' failure path (tri_selftest_wait_timeout): a bounded wait
    on an mbarrier nothing arrives on runs out after limit_ns and sets
    status (device int32 [1]) to DEV_TIMEOUT."""
    lib = load_library()
    assert status.dtype == torch.int32 and status.is_cuda and status.numel() >= 1
    _check("tri_selftest_wait_timeout", lib.tri_selftest_wait_timeout(status.data_ptr(), int(limit_ns),
                                                                      _stream(stream)))
    return status


def calibrate_workspace_bytes(n_layers: int, n_q_heads: int, group: int, head_dim: int,
                              n_tok: int) -> int:
    return int(load_library().tri_calibrate_workspace_bytes(n_layers, n_q_heads, group, head_dim, n_tok))


def calibrate_centers(q: torch.Tensor, group: int, style: int = ROPE_INTERLEAVED,
                      out: Centers | None = None, workspace: torch.Tensor | None = None,
                      stream=None) -> Centers:
    """Per-KV-head query centre, mean norm and MRL from pre-RoPE queries q
    [L, Hq, n_tok, d] (tri_calibrate_centers)."""
    lib = load_library()
    L, Hq, n_tok, d = q.shape
    assert q.is_cuda and q.is_contiguous() and q.dtype in _DTYPES
    H, F = Hq // group, d // 2
    if out is None:
        out = Centers(*(_empty(shape, torch.float32, q.device, stream) for shape in ((L * H, F, 2), (L * H, F), (L * H, F))))
        if stream is not None:  # read on the current stream later on
            for t in (out.center, out.mean_norm, out.mrl):
                t.record_stream(torch.cuda.current_stream())
    ws_bytes = calibrate_workspace_bytes(L, Hq, group, d, n_tok)
    if workspace is None:
        workspace = _scratch(ws_bytes, q.device, stream)
    assert workspace.numel() >= ws_bytes
    _check("tri_calibrate_centers", lib.tri_calibrate_centers(
        q.data_ptr(), _DTYPES[q.dtype], L, Hq, group, d, n_tok, style, out._abi(),
        workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return out


def score(kv: KVCache, centers: Centers, rope_theta: float, offsets, p_cur: torch.Tensor,
          scores: torch.Tensor, n_prompt: int = 0, n_recent: int = 0,
          style: int = ROPE_INTERLEAVED, norm_mode: int = NORM_WEIGHTED, stream=None) -> torch.Tensor:
    """Offset-averaged TriAttention score of rows [n_prompt, n_valid - n_recent)
    of every slice into scores [S, n_cap] fp32 (tri_score)."""
    lib = load_library()
    offs = (ctypes.c_int32 * len(offsets))(*[int(o) for o in offsets])
    assert p_cur.dtype == torch.int64 and p_cur.is_cuda
    assert scores.dtype == torch.float32 and scores.is_contiguous()
    assert scores.numel() == kv.n_slices * kv.n_cap
    kvs, cs = kv._abi(), centers._abi()
    _check("tri_score", lib.tri_score(ctypes.byref(kvs), ctypes.byref(cs), float(rope_theta), style,
                                      norm_mode, ctypes.cast(offs, ctypes.c_void_p), len(offsets),
                                      p_cur.data_ptr(), n_prompt, n_recent, scores.data_ptr(),
                                      _stream(stream)))
    return scores


def select_topk(scores: torch.Tensor, kv: KVCache, n_prompt: int, n_recent: int, budget: int,
                keep: torch.Tensor, stream=None) -> torch.Tensor:
    """Protected top-budget keep lists [S, budget] int32, ascending (tri_select_topk)."""
    lib = load_library()
    assert keep.dtype == torch.int32 and keep.is_contiguous() and keep.numel() == kv.n_slices * budget
    kvs = kv._abi()
    _check("tri_select_topk", lib.tri_select_topk(scores.data_ptr(), ctypes.byref(kvs), n_prompt,
                                                  n_recent, budget, keep.data_ptr(), _stream(stream)))
    return keep


def rand_evict(kv: KVCache, seed: int, rnd: int, n_prompt: int, n_recent: int, budget: int,
               keep: torch.Tensor, stream=None) -> torch.Tensor:
    """Random Attention keep lists [S, budget] int32 (rand_evict)."""
    lib = load_library()
    assert keep.dtype == torch.int32 and keep.is_contiguous() and keep.numel() == kv.n_slices * budget
    kvs = kv._abi()
    _check("rand_evict", lib.rand_evict(ctypes.byref(kvs), seed, rnd, n_prompt, n_recent, budget,
                                        keep.data_ptr(), _stream(stream)))
    return keep


DRAW_PER_HEAD, DRAW_PER_LAYER, DRAW_PER_SEQUENCE = 0, 1, 2


def rand_evict_scoped(kv: KVCache, seed: int, rnd: int, scope: int, n_prompt: int, n_recent: int, budget: int,
                      keep: torch.Tensor, stream=None) -> torch.Tensor:
    """Random Attention keep lists with the draw shared by every KV head of a
    layer (DRAW_PER_LAYER) or of a sequence (DRAW_PER_SEQUENCE) (rand_evict_scoped)."""
    lib = load_library()
    assert keep.dtype == torch.int32 and keep.is_contiguous() and keep.numel() == kv.n_slices * budget
    kvs = kv._abi()
    _check("rand_evict_scoped", lib.rand_evict_scoped(ctypes.byref(kvs), seed, rnd, scope, n_prompt, n_recent,
                                                      budget, keep.data_ptr(), _stream(stream)))
    return keep


def compact_kv(kv: KVCache, keep: torch.Tensor, budget: int, stream=None) -> None:
    """In-place order-preserving compaction of K, V and positions (tri_compact_kv)."""
    lib = load_library()
    assert keep.dtype == torch.int32 and keep.is_contiguous() and keep.numel() == kv.n_slices * budget
    kvs = kv._abi()
    _check("tri_compact_kv", lib.tri_compact_kv(ctypes.byref(kvs), keep.data_ptr(), budget,
                                                _stream(stream)))


def select_compact(scores: torch.Tensor, kv, n_prompt: int, n_recent: int, budget: int, keep: torch.Tensor,
                   stream=None) -> torch.Tensor:
    """select_topk then compact_kv, one kernel (tri_select_compact)."""
    lib = load_library()
    assert keep.dtype == torch.int32 and keep.is_contiguous() and keep.numel() == kv.n_slices * budget
    kvs = kv._abi()
    _check("tri_select_compact", lib.tri_select_compact(scores.data_ptr(), ctypes.byref(kvs), n_prompt, n_recent,
                                                        budget, keep.data_ptr(), _stream(stream)))
    return keep


def rand_evict_compact(kv, seed: int, rnd: int, n_prompt: int, n_recent: int, budget: int, keep: torch.Tensor,
                       scope: int = 0, stream=None) -> torch.Tensor:
    """rand_evict_scoped then compact_kv, one kernel (rand_evict_compact)."""
    lib = load_library()
    assert keep.dtype == torch.int32 and keep.is_contiguous() and keep.numel() == kv.n_slices * budget
    kvs = kv._abi()
    _check("rand_evict_compact", lib.rand_evict_compact(ctypes.byref(kvs), seed, rnd, scope, n_prompt, n_recent,
                                                        budget, keep.data_ptr(), _stream(stream)))
    return keep


def compress_workspace_bytes(kv: KVCache) -> int:
    kvs = kv._abi()
    return int(load_library().tri_compress_workspace_bytes(ctypes.byref(kvs)))


def compress(kv: KVCache, centers: Centers, rope_theta: float, offsets, p_cur: torch.Tensor,
             n_prompt: int, n_recent: int, budget: int, keep: torch.Tensor,
             workspace: torch.Tensor | None = None, style: int = ROPE_INTERLEAVED,
             norm_mode: int = NORM_WEIGHTED, stream=None) -> torch.Tensor:
    """One compression event: score + select + compact (tri_compress)."""
    lib = load_library()
    offs = (ctypes.c_int32 * len(offsets))(*[int(o) for o in offsets])
    assert p_cur.dtype == torch.int64 and p_cur.is_cuda
    assert keep.dtype == torch.int32 and keep.is_contiguous() and keep.numel() == kv.n_slices * budget
    kvs, cs = kv._abi(), centers._abi()
    need = int(lib.tri_compress_workspace_bytes(ctypes.byref(kvs)))
    if workspace is None:
        workspace = _scratch(need, kv.device, stream)
    assert workspace.numel() >= need
    _check("tri_compress", lib.tri_compress(ctypes.byref(kvs), ctypes.byref(cs), float(rope_theta), style,
                                            norm_mode, ctypes.cast(offs, ctypes.c_void_p), len(offsets),
                                            p_cur.data_ptr(), n_prompt, n_recent, budget, keep.data_ptr(),
                                            workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return keep


def score_heads_workspace_bytes(kv: KVCache, group: int) -> int:
    kvs = kv._abi()
    return int(load_library().tri_score_heads_workspace_bytes(ctypes.byref(kvs), group))


def score_heads(kv: KVCache, centers: Centers, group: int, rope_theta: float, offsets, p_cur: torch.Tensor,
                scores_g: torch.Tensor, stats: torch.Tensor, workspace: torch.Tensor | None = None,
                style: int = ROPE_INTERLEAVED, norm_mode: int = NORM_WEIGHTED, stream=None):
    """Per-query-head scores [S, group, n_cap] of every valid row and their
    per-head (mean, std) [S, group, 2] (tri_score_heads). `centers` holds one
    row per query head (calibrate_centers with group=1)."""
    lib = load_library()
    offs = (ctypes.c_int32 * len(offsets))(*[int(o) for o in offsets])
    assert p_cur.dtype == torch.int64 and p_cur.is_cuda
    assert scores_g.dtype == torch.float32 and scores_g.is_contiguous()
    assert scores_g.numel() == kv.n_slices * group * kv.n_cap
    assert stats.dtype == torch.float32 and stats.is_contiguous() and stats.numel() == kv.n_slices * group * 2
    kvs, cs = kv._abi(), centers._abi()
    need = int(lib.tri_score_heads_workspace_bytes(ctypes.byref(kvs), group))
    if workspace is None:
        workspace = _scratch(need, kv.device, stream)
    assert workspace.numel() >= need
    _check("tri_score_heads", lib.tri_score_heads(
        ctypes.byref(kvs), ctypes.byref(cs), group, float(rope_theta), style, norm_mode,
        ctypes.cast(offs, ctypes.c_void_p), len(offsets), p_cur.data_ptr(), scores_g.data_ptr(),
        stats.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return scores_g, stats


def select_topk_zmax(scores_g: torch.Tensor, stats: torch.Tensor, group: int, kv: KVCache, n_prompt: int,
                     n_recent: int, budget: int, keep: torch.Tensor, final_scores: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Protected top-budget keep lists ranked by the GQA z-score maximum
    (tri_select_topk_zmax); optionally writes the final scores [S, n_cap]."""
    lib = load_library()
    assert keep.dtype == torch.int32 and keep.is_contiguous() and keep.numel() == kv.n_slices * budget
    if final_scores is not None:
        assert final_scores.dtype == torch.float32 and final_scores.is_contiguous()
        assert final_scores.numel() == kv.n_slices * kv.n_cap
    kvs = kv._abi()
    _check("tri_select_topk_zmax", lib.tri_select_topk_zmax(
        scores_g.data_ptr(), stats.data_ptr(), group, ctypes.byref(kvs), n_prompt, n_recent, budget,
        keep.data_ptr(), _ptr(final_scores), _stream(stream)))
    return keep


def select_union_workspace_bytes(kv: KVCache, n_prompt: int, n_recent: int, k_head: int) -> int:
    kvs = kv._abi()
    return int(load_library().tri_select_union_workspace_bytes(ctypes.byref(kvs), n_prompt, n_recent, k_head))


def select_union(scores: torch.Tensor, kv: KVCache, n_prompt: int, n_recent: int, budget: int, k_head: int,
                 keep: torch.Tensor, final_scores: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One keep list per (seq, layer) shared by its KV heads: union of every
    head's top k_head, ranked by the z-score maximum, topped up by it
    (tri_select_union). `scores` must cover every valid row."""
    lib = load_library()
    assert keep.dtype == torch.int32 and keep.is_contiguous() and keep.numel() == kv.n_slices * budget
    kvs = kv._abi()
    need = int(lib.tri_select_union_workspace_bytes(ctypes.byref(kvs), n_prompt, n_recent, k_head))
    if workspace is None:
        workspace = _scratch(need, kv.device, stream)
    assert workspace.numel() >= need
    if final_scores is not None:
        assert final_scores.dtype == torch.float32 and final_scores.is_contiguous()
    _check("tri_select_union", lib.tri_select_union(
        scores.data_ptr(), ctypes.byref(kvs), n_prompt, n_recent, budget, k_head, keep.data_ptr(),
        _ptr(final_scores), workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return keep


def _queries(kvs: _TriKV, kv, layer: int, q: torch.Tensor, shape, strides, n_new: torch.Tensor | None,
             scale: float | None, n_sink: int, window: int) -> _TriQueries:
    """Queries of shape [n_seq, n_q, Hq, d] (any sequence and token strides) of the cache's type (bf16 for one in 4
    bits) and device."""
    n_seq, n_q, Hq, d = shape
    dev = q.get_device()
    assert dev == kv.k.get_device() == torch.cuda.current_device(), "cache and queries on the current device"
    assert q.dtype == _token_dtype(kv) and d == kvs.head_dim and n_seq == kvs.n_seq and Hq % kvs.n_kv_heads == 0
    assert strides[3] == 1 and (strides[2] == d or Hq == 1)
    if n_new is not None:
        assert n_new.is_cuda and n_new.dtype == torch.int32 and n_new.is_contiguous() and n_new.numel() == n_seq
    # (the stride of a dimension of one may be anything)
    return _TriQueries(q.data_ptr(), strides[0] if n_seq > 1 else 0, strides[1] if n_q > 1 else Hq * d, _ptr(n_new), n_q,
                       Hq // kvs.n_kv_heads, layer, n_sink, window, d ** -0.5 if scale is None else scale)


def _token_dtype(kv) -> torch.dtype:
    """Type of queries, new rows and attention results: the cache's, bf16 for one in 4 bits."""
    return torch.bfloat16 if kv.k.dtype == torch.uint8 else kv.k.dtype


def _token_strides(t: torch.Tensor, shape, dtype: torch.dtype, device: int):
    """Sequence and token strides of rows [n_seq, n_q, heads, d] whose heads are contiguous."""
    a, b, c, e = t.stride()
    assert t.shape == shape and t.dtype == dtype and t.get_device() == device and e == 1 and (c == shape[3] or shape[2] == 1)
    # (the stride of a dimension of one may be anything)
    return a if shape[0] > 1 else 0, b if shape[1] > 1 else shape[2] * shape[3]


def append(kv, layer: int, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, rope_theta: float,
           q: torch.Tensor | None = None, q_out: torch.Tensor | None = None, n_new: torch.Tensor | None = None,
           band_axis=None, style: int = ROPE_INTERLEAVED, stream=None) -> torch.Tensor | None:
    """New tokens into one layer of the cache (tri_append): k, v [n_seq, n_q, H, d]
    (any sequence and token strides: views of a fused projection's output) go
    behind the rows of the layer's slices, k rotated at the tokens' positions
    [n_seq, n_q] or [n_seq, n_q, axes] int32 if the cache is post-RoPE; n_valid
    grows by n_new [n_seq] int32 (None: n_q each), kv.pos gets the first axis. q
    [n_seq, n_q, Hq, d] is rotated into q_out (q itself, or apart from it; None: a
    new tensor), which is returned. band_axis: the axis of each of the d / 2 bands.
    A 4-bit cache takes bf16 tokens."""
    lib = load_library()
    kvs = kv._abi()
    dev, dtype, d, H, n_seq = kv.k.get_device(), _token_dtype(kv), kvs.head_dim, kvs.n_kv_heads, kvs.n_seq
    assert dev == torch.cuda.current_device(), "cache and tokens on the current device"
    n_q = k.shape[1]
    shape = (n_seq, n_q, H, d)
    ks, vs = _token_strides(k, shape, dtype, dev), _token_strides(v, shape, dtype, dev)
    at = positions.shape
    n_axes = at[2] if len(at) == 3 else 1
    assert at[0] == n_seq and at[1] == n_q and len(at) <= 3
    assert positions.get_device() == dev and positions.dtype == torch.int32 and positions.is_contiguous()
    if n_new is not None:
        assert n_new.get_device() == dev and n_new.dtype == torch.int32 and n_new.is_contiguous() and n_new.numel() == n_seq
    axes = None
    if band_axis is not None:
        axes = bytes(band_axis)
        assert len(axes) == d // 2
    qs, qos, group = (0, 0), (0, 0), 0
    if q is not None:
        Hq = q.shape[2]
        assert Hq % H == 0
        group, shape = Hq // H, (n_seq, n_q, Hq, d)
        qs = _token_strides(q, shape, dtype, dev)
        if q_out is None:
            q_out = _empty(shape, dtype, q.device, stream)
            if stream is not None:  # read on the current stream later on
                q_out.record_stream(torch.cuda.current_stream())
        qos = qs if q_out is q else _token_strides(q_out, shape, dtype, dev)
    else:
        assert q_out is None
    tok = _TriTokens(k.data_ptr(), v.data_ptr(), *ks, *vs, _ptr(q), _ptr(q_out), *qs, *qos, positions.data_ptr(), axes,
                     _ptr(n_new), rope_theta, style, n_axes, n_q, group, layer)
    _check("tri_append", lib.tri_append(ctypes.byref(kvs), ctypes.byref(tok),
                                        stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)))
    return q_out


def read_rows(kv, layer: int, k_out: torch.Tensor | None, v_out: torch.Tensor | None, stream=None) -> None:
    """The values that one layer's rows of a 4-bit cache stand for (tri_read_rows):
    k_out, v_out [n_seq, H, n_cap, d] bf16 (either may be None); rows from n_valid
    on are left as they were."""
    lib = load_library()
    kvs = kv._abi()
    assert kv.k.get_device() == torch.cuda.current_device()
    for t in (k_out, v_out):
        if t is not None:
            assert t.get_device() == kv.k.get_device() and t.dtype == torch.bfloat16 and t.is_contiguous()
            assert t.shape == (kvs.n_seq, kvs.n_kv_heads, kvs.n_cap, kvs.head_dim)
    _check("tri_read_rows", lib.tri_read_rows(ctypes.byref(kvs), layer, _ptr(k_out), _ptr(v_out), _stream(stream)))


def _check_mass(kvs: _TriKV, mass: torch.Tensor):
    assert mass.is_cuda and mass.dtype == torch.float32 and mass.is_contiguous()
    assert mass.numel() == kvs.n_seq * kvs.n_layers * kvs.n_kv_heads * kvs.n_cap


def attn_decode_workspace_bytes(kv, group: int, with_mass: bool = False) -> int:
    kvs = kv._abi()
    return int(load_library().tri_attn_decode_workspace_bytes(ctypes.byref(kvs), group, int(with_mass)))


def attn_decode(kv, layer: int, q: torch.Tensor, out: torch.Tensor, n_new: torch.Tensor | None = None,
                scale: float | None = None, n_sink: int = 0, window: int = 0, lse: torch.Tensor | None = None,
                mass: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of one new token per sequence, q [n_seq, Hq, d], over one layer
    of a post-RoPE cache that already holds the token's row (tri_attn_decode):
    out [n_seq, Hq, d]; lse [n_seq, Hq] fp32; mass [S, n_cap] fp32 gets every
    row's weight added. window > 0: the first n_sink and newest `window` rows
    only. n_new [n_seq] int32: 0 leaves a sequence out. scale: d ** -0.5."""
    lib = load_library()
    kvs = kv._abi()
    shape, strides = q.shape, q.stride()
    n_seq, Hq, d = shape
    qs = _queries(kvs, kv, layer, q, (n_seq, 1, Hq, d), (strides[0], strides[0], strides[1], strides[2]), n_new, scale,
                  n_sink, window)
    assert out.is_cuda and out.is_contiguous() and out.shape == shape and out.dtype == q.dtype
    if lse is not None:
        assert lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous() and lse.numel() == n_seq * Hq
    if mass is not None:
        _check_mass(kvs, mass)
    if workspace is None:
        need = int(lib.tri_attn_decode_workspace_bytes(ctypes.byref(kvs), qs.group, int(mass is not None)))
        workspace = _scratch(need, kv.device, stream)
    assert workspace.is_cuda and workspace.is_contiguous()
    _check("tri_attn_decode", lib.tri_attn_decode(ctypes.byref(kvs), ctypes.byref(qs), out.data_ptr(), _ptr(lse),
                                                  _ptr(mass), workspace.data_ptr(), workspace.nbytes, _stream(stream)))
    return out


def attn_prefill_workspace_bytes(kv, q: torch.Tensor | None = None, n_sink: int = 0, window: int = 0) -> int:
    """Scratch of attn_prefill: one layer's rows written out for a 4-bit cache, none otherwise. q (with the call's n_sink
    and window): what a call with these queries needs, much less where they are few tokens."""
    lib, kvs = load_library(), kv._abi()
    if q is not None and kvs.dtype == Q4:
        few = lib.tri_attn_prefill_q4_few_workspace_bytes(
            ctypes.byref(kvs), ctypes.byref(_queries(kvs, kv, 0, q, q.shape, q.stride(), None, None, n_sink, window)))
        if few:
            return int(few)
    return int(lib.tri_attn_prefill_q4_workspace_bytes(ctypes.byref(kvs)))


def attn_prefill(kv, layer: int, q: torch.Tensor, out: torch.Tensor, n_new: torch.Tensor | None = None,
                 scale: float | None = None, n_sink: int = 0, window: int = 0, lse: torch.Tensor | None = None,
                 stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention of a chunk of new tokens, q [n_seq, n_q, Hq, d] (any
    sequence and token strides), over one layer of a post-RoPE cache whose
    newest rows they are (tri_attn_prefill): out [n_seq, n_q, Hq, d]; lse
    [n_seq, n_q, Hq] fp32. n_new [n_seq] int32: tokens of each sequence (rows of
    out past them stay as they were). A 4-bit cache (tri_attn_prefill_q4) needs
    attn_prefill_workspace_bytes(kv, q, n_sink, window) of workspace."""
    lib = load_library()
    kvs = kv._abi()
    shape = q.shape
    qs = _queries(kvs, kv, layer, q, shape, q.stride(), n_new, scale, n_sink, window)
    assert out.is_cuda and out.is_contiguous() and out.shape == shape and out.dtype == q.dtype
    if lse is not None:
        assert lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous() and lse.shape == shape[:3]
    if kvs.dtype == Q4:
        few = lib.tri_attn_prefill_q4_few_workspace_bytes(ctypes.byref(kvs), ctypes.byref(qs))
        if workspace is None:
            workspace = _scratch(int(few or lib.tri_attn_prefill_q4_workspace_bytes(ctypes.byref(kvs))), kv.device, stream)
        assert workspace.is_cuda and workspace.is_contiguous()
        call = lib.tri_attn_prefill_q4_few if few else lib.tri_attn_prefill_q4
        _check("tri_attn_prefill_q4", call(ctypes.byref(kvs), ctypes.byref(qs), out.data_ptr(), _ptr(lse), workspace.data_ptr(),
                                           workspace.nbytes, _stream(stream)))
        return out
    _check("tri_attn_prefill", lib.tri_attn_prefill(ctypes.byref(kvs), ctypes.byref(qs), out.data_ptr(), _ptr(lse),
                                                    _stream(stream)))
    return out


def attn_mass(kv, layer: int, q: torch.Tensor, lse: torch.Tensor, mass: torch.Tensor,
              n_new: torch.Tensor | None = None, scale: float | None = None, n_sink: int = 0, window: int = 0,
              stream=None) -> torch.Tensor:
    """Add to mass [S, n_cap] the weight every cached row of one layer gets from
    a chunk of queries, q [n_seq, n_q, Hq, d] with their lse [n_seq, n_q, Hq] from
    attn_prefill (tri_attn_mass). Both may be the last n_q tokens of a longer
    chunk (q[:, -n:], lse[:, -n:]): an observation window."""
    lib = load_library()
    kvs = kv._abi()
    shape, ls = q.shape, lse.stride()
    qs = _queries(kvs, kv, layer, q, shape, q.stride(), n_new, scale, n_sink, window)
    assert lse.is_cuda and lse.dtype == torch.float32 and lse.shape == shape[:3]
    assert ls[2] == 1 and (ls[1] == shape[2] or shape[1] == 1)
    _check_mass(kvs, mass)
    _check("tri_attn_mass", lib.tri_attn_mass(ctypes.byref(kvs), ctypes.byref(qs), lse.data_ptr(), ls[0],
                                              mass.data_ptr(), _stream(stream)))
    return mass


def mass_evict(kv, mass: torch.Tensor, mass_out: torch.Tensor, n_prompt: int, n_recent: int, budget: int,
               keep: torch.Tensor, stream=None) -> torch.Tensor:
    """Eviction by accumulated attention weight (tri_mass_evict): select_compact
    with mass [S, n_cap] as the scores, the masses moved with their rows into
    mass_out (mass itself or apart from it), the freed rows' masses set to 0."""
    lib = load_library()
    kvs = kv._abi()
    assert kv.k.get_device() == mass.get_device() == mass_out.get_device() == torch.cuda.current_device()
    assert keep.dtype == torch.int32 and keep.is_contiguous() and keep.numel() == kv.n_slices * budget
    _check_mass(kvs, mass)
    _check_mass(kvs, mass_out)
    _check("tri_mass_evict", lib.tri_mass_evict(mass.data_ptr(), mass_out.data_ptr(), ctypes.byref(kvs), n_prompt,
                                                n_recent, budget, keep.data_ptr(), _stream(stream)))
    return keep
