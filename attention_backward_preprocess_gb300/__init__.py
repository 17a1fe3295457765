"""GB300 (sm_103a) fused exact-softmax attention backward.

Thin ctypes binding of the C ABI in ``include/fa.h`` (``libfa_gb300.so``,
built in-tree by ``attention_backward_preprocess_gb300.build``).  This module
only marshals arguments: every step of the computation runs in the library's
CUDA kernels.  PyTorch supplies device memory and streams.  There is no CPU
fallback: when the library is missing or cannot load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa_gb300.so")
SHORT_PATH = os.path.join(_PKG, "_fa_torch.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
FA_ERR_SCRATCH_LIMIT = 5
FA_BF16, FA_FP16 = 0, 1

# entry points declared in include/fa.h and include/fa_selftest.h
EXPORTED = [
    "fa_bwd", "fa_bwd_workspace_bytes", "fa_bwd_with_workspace", "fa_bwd_preprocess",
    "fa_bwd_main", "fa_bwd_postprocess", "fa_bwd_workspace_layout", "fa_fwd",
    "fa_device_status", "fa_set_wait_timeout_ns", "fa_status_string",
    "fa_selftest_umma", "fa_selftest_semaphore", "fa_selftest_tmem_layout", "fa_bwd_noalloc",
    "fa_bwd_noalloc_scratch_bytes", "fa_fwd_ext", "fa_bwd_ext", "fa_bwd_stages_ext", "fa_bwd_workspace_sync_layout",
    "fa_bwd_noalloc_status", "fa_mask_ranges", "fa_mask_ranges_bytes", "fa_ext_bytes",
    "fa_kvcache_append", "fa_fwd_kvcache", "fa_fwd_kvcache_workspace_bytes",
    "fa_kvcache4_append", "fa_kvcache4_read", "fa_fwd_kvcache4", "fa_fwd_kvcache4_workspace_bytes",
    "fa_rope", "fa_rope_frequencies", "fa_rope_steps",
]


class FaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (what, status_string(status), status))


_lib = None
_lock = threading.Lock()

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_SHAPE = [_i] * 6   # B, Sq, Sk, Hq, Hkv, D


class FaExt(ctypes.Structure):
    """fa_ext of include/fa.h: local window, ALiBi slopes, used lengths."""
    _fields_ = [("window_left", ctypes.c_int), ("window_right", ctypes.c_int),
                ("alibi_slopes", ctypes.c_void_p), ("alibi_batch_stride", ctypes.c_int),
                ("seqused_q", ctypes.c_void_p), ("seqused_k", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("bias_batch_stride", ctypes.c_longlong),
                ("bias_head_stride", ctypes.c_longlong), ("bias_row_stride", ctypes.c_longlong),
                ("dbias", ctypes.c_void_p), ("dropout_p", ctypes.c_float),
                ("dropout_seed", ctypes.c_ulonglong), ("dropout_offset", ctypes.c_uint),
                ("dropout_mask", ctypes.c_void_p), ("total_q", ctypes.c_longlong),
                ("total_k", ctypes.c_longlong), ("head_dim_v", ctypes.c_int),
                ("softcap", ctypes.c_float), ("mask_ranges", ctypes.c_void_p),
                ("mask_ranges_bytes", ctypes.c_size_t)] + [
                    (n + "_stride", ctypes.c_longlong * 3) for n in ("q", "k", "v", "o", "dout")]


def dropout_mask_shape(q, k, cu_seqlens_q=None, max_seqlen_k=None):
    """Shape of the int32 keep-flag buffer fa_fwd / fa_bwd take with dropout:
    [B, Hq, Sq, W] (dense) or [Hq, total_q, W] (varlen), W = ceil(Sk / 32)
    words of 32 keys per query row, Sk the key length (max_seqlen_k)."""
    if cu_seqlens_q is not None:
        Sk = int(max_seqlen_k)
        return (q.shape[1], q.shape[0], (Sk + 31) // 32)
    return (q.shape[0], q.shape[2], q.shape[1], (k.shape[1] + 31) // 32)


def _ext(Hq, window=None, alibi_slopes=None, seqused_q=None, seqused_k=None, bias=None,
         dbias=None, dropout=None, totals=None, head_dim_v=0, softcap=0.0, mask_ranges=None,
         sizes=None, strides=None, rows=0, dtype=None):
    """A pointer to an FaExt, or None when no extension is asked for.

    ``bias``: [B or 1, Hq or 1, Sq, >= Sk] in the input dtype, last axis
    contiguous (a size-1 batch / head axis broadcasts).  ``dbias``: a
    contiguous [B, Hq, Sq, Sk] output of the input dtype (backward only).
    ``dropout``: (p, seed, offset), or (p, seed, offset, mask) with ``mask`` an
    int32 tensor of ``dropout_mask_shape(...)`` that fa_fwd fills with the keep
    flags and fa_bwd reads back; see fa_ext in include/fa.h.  ``totals``:
    (total_q, total_k), the packed row counts of a varlen call (cu_seqlens[B]),
    so that the library need not read them back (no stream synchronisation).
    ``head_dim_v``: the value head dim when it differs from q's (else 0).
    ``softcap``: scores become softcap * tanh(score / softcap) (0: none).
    ``mask_ranges``: a MaskRanges of the call's ``sizes`` (B, Sq, Sk, GPU); ``rows``
    query rows of type ``dtype`` in all.
    ``strides``: what ``_inputs`` said of inputs that are not contiguous."""
    if (window is None and alibi_slopes is None and seqused_q is None and seqused_k is None
            and bias is None and dbias is None and dropout is None and totals is None
            and not head_dim_v and softcap == 0.0 and mask_ranges is None and not strides):
        return None
    e = FaExt(-1, -1)   # the rest 0
    B, Sq, Sk, at = sizes

    def reaches(name, t, n, dtype=None):
        """``t`` is on the call's GPU and holds the n elements the kernels may read or write."""
        if t.get_device() != at or t.numel() < n or (dtype is not None and t.dtype != dtype):
            raise ValueError("%s: at least %d elements%s on q's GPU" % (name, n, "" if dtype is None else " of %s" % dtype))
    if strides:
        for name, s in strides.items():
            setattr(e, name + "_stride", s)
    e.softcap = float(softcap)
    if mask_ranges is not None:
        m = mask_ranges
        if not isinstance(m, MaskRanges) or sizes != (m.B, m.S, m.S, m.buffer.get_device()):
            raise ValueError("mask_ranges: what mask_ranges(B, S, ...) returned, for this call's B, S = Sq = Sk and GPU")
        e.mask_ranges, e.mask_ranges_bytes = mask_ranges.buffer.data_ptr(), mask_ranges.buffer.numel()
    e.head_dim_v = int(head_dim_v)
    if totals is not None:
        e.total_q, e.total_k = int(totals[0]), int(totals[1])
    if dropout is not None:
        e.dropout_p, e.dropout_seed, e.dropout_offset = (float(dropout[0]), int(dropout[1]),
                                                         int(dropout[2]))
        if len(dropout) > 3 and dropout[3] is not None:
            m = dropout[3]
            if m.dtype != torch.int32 or not m.is_contiguous():
                raise ValueError("dropout mask: a contiguous int32 tensor of dropout_mask_shape(...)")
            reaches("dropout mask", m, rows * Hq * ((Sk + 31) // 32))
            e.dropout_mask = m.data_ptr()
    if window is not None:
        e.window_left, e.window_right = int(window[0]), int(window[1])
    if alibi_slopes is not None:
        if alibi_slopes.dtype != torch.float32 or not alibi_slopes.is_contiguous():
            raise ValueError("alibi_slopes: contiguous fp32 [Hq] or [B, Hq]")
        reaches("alibi_slopes", alibi_slopes, Hq * (B if alibi_slopes.dim() == 2 else 1))
        e.alibi_slopes = alibi_slopes.data_ptr()
        e.alibi_batch_stride = Hq if alibi_slopes.dim() == 2 else 0
    for name, t in (("seqused_q", seqused_q), ("seqused_k", seqused_k)):
        if t is not None:
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError(name + ": contiguous int32 [B]")
            reaches(name, t, B)
            setattr(e, name, t.data_ptr())
    if bias is not None:
        if bias.dim() != 4 or bias.stride(3) != 1:
            raise ValueError("bias: [B or 1, Hq or 1, Sq, Sk] with a contiguous last axis")
        reaches("bias", bias, 0, dtype)
        if any(n != 1 and n < m for n, m in zip(bias.shape[:2], (B, Hq))) or bias.shape[2] < Sq or bias.shape[3] < Sk:
            raise ValueError("bias: [B or 1, Hq or 1, Sq, Sk], got %r" % (tuple(bias.shape),))
        e.bias = bias.data_ptr()
        e.bias_batch_stride = 0 if bias.shape[0] == 1 else bias.stride(0)
        e.bias_head_stride = 0 if bias.shape[1] == 1 else bias.stride(1)
        e.bias_row_stride = bias.stride(2)
    if dbias is not None:
        if not dbias.is_contiguous():
            raise ValueError("dbias: a contiguous [B, Hq, Sq, Sk] tensor")
        reaches("dbias", dbias, B * Hq * Sq * Sk, dtype)
        e.dbias = dbias.data_ptr()
    return ctypes.pointer(e)


class _KvCacheStruct(ctypes.Structure):
    """fa_kv_cache of include/fa.h, and fa_kv_cache4, whose fields are the same."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("D", ctypes.c_int)]


class _PagedCache:
    """What the two kinds of cache share: the tensors, held, and their struct."""
    # read only: the library holds the addresses of these very tensors
    k, v, k_scale, v_scale, block_table = (property(lambda self, i=i: self._tensors[i]) for i in range(5))

    def _hold(self, k, v, k_scale, v_scale, block_table, P, ps, H, D):
        self._tensors = k, v, k_scale, v_scale, block_table
        self._c = _KvCacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                 block_table.data_ptr(), P, ps, block_table.shape[1], H, D)
        self._at = ctypes.addressof(self._c)

    def _check(self, name, t, dtype, shape):
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != self.device \
                or self.device < 0:
            raise ValueError("%s: contiguous %s %r on the cache's GPU" % (name, dtype, tuple(shape)))


def _kind(cache, cls):
    """The library reads a cache of another kind, or none, past its end.  (What stands in for a
    KvCache with its fields, a wrapper say, is one.)"""
    if not isinstance(cache, cls) and not (
            cls is KvCache and getattr(getattr(cache, "k", None), "dtype", None) == torch.float8_e4m3fn):
        raise ValueError("cache: a %s" % cls.__name__)


class KvCache(_PagedCache):
    """An 8-bit paged key / value cache over the caller's tensors: ``k``
    float8_e4m3fn [pages, Hkv, page, D], ``v`` float8_e4m3fn [pages, Hkv, D,
    page], ``k_scale`` / ``v_scale`` float32 [pages, Hkv], ``block_table``
    int32 [B, max_pages]; see fa_kv_cache in include/fa.h.  Keeps the tensors,
    copies nothing.  Their contents may change; other tensors (a wider block
    table) make another KvCache."""

    def __init__(self, k, v, k_scale, v_scale, block_table):
        if k.dim() != 4 or block_table.dim() != 2:
            raise ValueError("k: [pages, Hkv, page, D], block_table: [B, max_pages]")
        P, H, ps, D = k.shape
        self.B = block_table.shape[0]
        self.device = k.get_device()   # index, -1: not on a GPU
        if self.device < 0 or not _binding().cache(k, v, k_scale, v_scale, block_table):
            for name, t, dt, shape in (("k", k, torch.float8_e4m3fn, (P, H, ps, D)),
                                       ("v", v, torch.float8_e4m3fn, (P, H, D, ps)),
                                       ("k_scale", k_scale, torch.float32, (P, H)),
                                       ("v_scale", v_scale, torch.float32, (P, H)),
                                       ("block_table", block_table, torch.int32, block_table.shape)):
                self._check(name, t, dt, shape)
        self._hold(k, v, k_scale, v_scale, block_table, P, ps, H, D)


def kvcache_append(cache, cache_len, k_new, v_new, cu_new=None, max_new=None, stream=None):
    """Quantises new keys and values into ``cache`` (a KvCache) behind the
    ``cache_len`` (int32 [B]) tokens each sequence holds: fa_kvcache_append.

    ``k_new`` / ``v_new``: [B, T, Hkv, D], or [total, Hkv, D] with ``cu_new``
    (int32 [B + 1] prefix sums) and ``max_new``, the most tokens of one
    sequence.  The cache's tensors are updated in place."""
    _kind(cache, KvCache)
    if stream is None:
        r = _binding().append(cache._at, cache.B, cache.device, cache_len, k_new, v_new, cu_new, max_new)
        if r is not None:
            _done(r, "fa_kvcache_append")
            return
    _append("fa_kvcache_append", cache, cache_len, k_new, v_new, cu_new, max_new, stream)


def _append(what, cache, cache_len, k_new, v_new, cu_new, max_new, stream):
    """An append through ctypes, to either kind of cache."""
    B, c = cache.B, cache._c
    cache._check("cache_len", cache_len, torch.int32, (B,))
    if cu_new is None:
        if k_new.dim() != 4:
            raise ValueError("k_new: [B, T, Hkv, D]")
        max_new = k_new.shape[1]
        shape = (B, max_new, c.Hkv, c.D)
    else:
        cache._check("cu_new", cu_new, torch.int32, (B + 1,))
        if max_new is None:
            raise ValueError("max_new: the most new tokens of one sequence")
        shape = (k_new.shape[0], c.Hkv, c.D)
    code = _dtype_code(k_new)
    if not (k_new.is_contiguous() and v_new.is_contiguous()):
        k_new, v_new = _dense(stream, k_new=k_new, v_new=v_new)
    cache._check("k_new", k_new, k_new.dtype, shape)
    cache._check("v_new", v_new, k_new.dtype, shape)
    with _on(cache.device):
        _check(getattr(lib(), what)(ctypes.byref(c), cache_len.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
                                    _ptr(cu_new), k_new.numel() // (c.Hkv * c.D), B, int(max_new), code,
                                    _stream(stream)), what)


def fa_fwd_kvcache(q, cache, cache_len, softmax_scale=None, softcap=0.0, window_left=-1, workspace=None,
                   out=None, stream=None):
    """Attention of each sequence's last tokens over an 8-bit paged cache:
    returns (o, lse).  ``q``: [B, Sq, Hq, D], the last Sq tokens of each
    sequence, whose own keys and values are in the cache already; ``cache_len``
    (int32 [B]) counts them.  ``workspace``: a uint8 CUDA tensor of
    ``fa_fwd_kvcache_workspace_bytes(D)`` (allocated when not given); ``out``:
    (o, lse) to write into.  See fa_fwd_kvcache in include/fa.h."""
    _kind(cache, KvCache)
    if stream is None and out is None and workspace is None:
        r = _binding().attend(cache._at, cache.B, cache.device, q, cache_len, softmax_scale, softcap, window_left)
        if r is not None:
            return _done(r, "fa_fwd_kvcache")
    return _attend("fa_fwd_kvcache", q, cache, cache_len, softmax_scale, softcap, window_left, workspace, out, stream)


def _attend(what, q, cache, cache_len, softmax_scale, softcap, window_left, workspace, out, stream):
    """An attention over either kind of cache through ctypes."""
    c = cache._c
    if q.dim() != 4:
        raise ValueError("q: [B, Sq, Hq, D]")
    B, Sq, Hq, D = q.shape
    if not q.is_contiguous():
        (q,) = _dense(stream, q=q)
    code = _dtype_code(q)
    cache._check("q", q, q.dtype, (cache.B, Sq, Hq, c.D))
    cache._check("cache_len", cache_len, torch.int32, (B,))
    scale = default_scale(D) if softmax_scale is None else float(softmax_scale)
    with _on(cache.device):
        with _memory(stream):
            if out is None:
                out = torch.empty_like(q), q.new_empty((B, Hq, Sq), dtype=torch.float32)
            else:
                cache._check("out[0]", out[0], q.dtype, q.shape)
                cache._check("out[1]", out[1], torch.float32, (B, Hq, Sq))
            if workspace is None:
                workspace = q.new_empty(getattr(lib(), what + "_workspace_bytes")(int(D)), dtype=torch.uint8)
            else:
                _scratch(workspace, cache.device)
        _check(getattr(lib(), what)(q.data_ptr(), ctypes.byref(c), cache_len.data_ptr(), out[0].data_ptr(),
                                    out[1].data_ptr(), B, Sq, Hq, scale, softcap, window_left, code,
                                    workspace.data_ptr(), workspace.numel(), _stream(stream)), what)
    return out


def fa_fwd_kvcache_workspace_bytes(D) -> int:
    """Bytes of workspace fa_fwd_kvcache needs (0: a head dim it does not take)."""
    return int(lib().fa_fwd_kvcache_workspace_bytes(int(D)))


class KvCache4(_PagedCache):
    """A 4-bit paged key / value cache over the caller's tensors: ``k`` and
    ``v`` uint8 [pages, Hkv, page, D / 2], ``k_scale`` and ``v_scale`` bfloat16
    [pages, Hkv, page, D / 64, 2] (scale, middle), ``block_table`` int32 [B,
    max_pages]; see fa_kv_cache4 in include/fa.h.  Otherwise as KvCache."""

    def __init__(self, k, v, k_scale, v_scale, block_table):
        if k.dim() != 4 or block_table.dim() != 2:
            raise ValueError("k: [pages, Hkv, page, D / 2], block_table: [B, max_pages]")
        self.B = block_table.shape[0]
        self.device = k.get_device()   # index, -1: not on a GPU
        raw = _binding().cache4(k, v, k_scale, v_scale, block_table) if self.device >= 0 else None
        if raw is not None:
            self._tensors = k, v, k_scale, v_scale, block_table
            self._c = _KvCacheStruct.from_buffer_copy(raw)
            self._at = ctypes.addressof(self._c)
            return
        P, H, ps, D = k.shape
        D *= 2
        for name, t, dt, shape in (("k", k, torch.uint8, (P, H, ps, D // 2)),
                                   ("v", v, torch.uint8, (P, H, ps, D // 2)),
                                   ("k_scale", k_scale, torch.bfloat16, (P, H, ps, D // 64, 2)),
                                   ("v_scale", v_scale, torch.bfloat16, (P, H, ps, D // 64, 2)),
                                   ("block_table", block_table, torch.int32, block_table.shape)):
            self._check(name, t, dt, shape)
        self._hold(k, v, k_scale, v_scale, block_table, P, ps, H, D)


def kvcache4_append(cache, cache_len, k_new, v_new, cu_new=None, max_new=None, stream=None):
    """Quantises new keys and values into ``cache`` (a KvCache4) behind the
    ``cache_len`` tokens each sequence holds: fa_kvcache4_append.  Arguments as
    for kvcache_append."""
    _kind(cache, KvCache4)
    if stream is None:
        r = _binding().append4(cache._at, cache.B, cache.device, cache_len, k_new, v_new, cu_new, max_new)
        if r is not None:
            _done(r, "fa_kvcache4_append")
            return
    _append("fa_kvcache4_append", cache, cache_len, k_new, v_new, cu_new, max_new, stream)


def fa_fwd_kvcache4(q, cache, cache_len, softmax_scale=None, softcap=0.0, window_left=-1, workspace=None,
                    out=None, stream=None):
    """Attention of each sequence's last tokens over a 4-bit paged cache (a
    KvCache4): returns (o, lse).  Arguments as for fa_fwd_kvcache, ``workspace``
    of ``fa_fwd_kvcache4_workspace_bytes(D)``."""
    _kind(cache, KvCache4)
    if stream is None and out is None and workspace is None:
        r = _binding().attend4(cache._at, cache.B, cache.device, q, cache_len, softmax_scale, softcap, window_left)
        if r is not None:
            return _done(r, "fa_fwd_kvcache4")
    return _attend("fa_fwd_kvcache4", q, cache, cache_len, softmax_scale, softcap, window_left, workspace, out, stream)


def fa_fwd_kvcache4_workspace_bytes(D) -> int:
    """Bytes of workspace fa_fwd_kvcache4 needs (0: a head dim it does not take)."""
    return int(lib().fa_fwd_kvcache4_workspace_bytes(int(D)))


def kvcache4_read(cache, cache_len, cu_rows, rows, dtype=torch.bfloat16, first=None, out=None, stream=None):
    """Tokens of a 4-bit cache (a KvCache4) as 16-bit tensors (k, v), each [rows,
    Hkv, D]: rows ``cu_rows[b] .. cu_rows[b + 1]`` (int32 [B + 1] prefix sums, in
    all ``rows``) are sequence b's tokens from ``first[b]`` (int32 [B]; None: 0)
    on, of the ``cache_len[b]`` held.  They are what fa_fwd takes with
    ``cu_seqlens_k``.  ``out``: (k, v) to write into; rows behind the last
    sequence's are left as they are.  See fa_kvcache4_read in include/fa.h."""
    _kind(cache, KvCache4)
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("dtype: bf16 or fp16, got %s" % dtype)
    if stream is None and out is None:
        r = _binding().read4(cache._at, cache.B, cache.device, cache_len, cu_rows, rows, dtype == torch.bfloat16, first)
        if r is not None:
            return _done(r, "fa_kvcache4_read")
    c, B, rows = cache._c, cache.B, int(rows)
    cache._check("cache_len", cache_len, torch.int32, (B,))
    cache._check("cu_rows", cu_rows, torch.int32, (B + 1,))
    if first is not None:
        cache._check("first", first, torch.int32, (B,))
    if rows <= 0:
        raise ValueError("rows: the rows of k and v, at least one")
    with _on(cache.device):
        with _memory(stream):
            if out is None:
                out = tuple(torch.empty((rows, c.Hkv, c.D), dtype=dtype, device=cache.k.device) for _ in range(2))
            else:
                for i in range(2):
                    cache._check("out[%d]" % i, out[i], dtype, (rows, c.Hkv, c.D))
        _check(lib().fa_kvcache4_read(ctypes.byref(c), cache_len.data_ptr(), _ptr(first), cu_rows.data_ptr(), rows, B,
                                      out[0].data_ptr(), out[1].data_ptr(), FA_BF16 if dtype == torch.bfloat16 else FA_FP16,
                                      _stream(stream)), "fa_kvcache4_read")
    return out


# ------------------------------------------------------------ rotary positions
class _RopeTensor(ctypes.Structure):
    """fa_rope_tensor of include/fa.h."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("in_stride", ctypes.c_longlong * 3), ("out_stride", ctypes.c_longlong * 3)]


class RopeTable:
    """What turns a head's pairs of dims: ``steps``, int64 CUDA tensor
    [rotary_dim / 2], the part of a turn that pair i makes per position in
    2^-64ths (as unsigned numbers), and the ``factor`` that the turned dims are
    multiplied by.  Made by rope_table or RopeTable.of; see fa_rope in
    include/fa.h."""

    def __init__(self, steps, factor=1.0):
        self.steps, self.factor = steps, float(factor)

    @property
    def rotary_dim(self):
        return 2 * self.steps.numel()

    @staticmethod
    def of(frequencies, factor=1.0, device="cuda"):
        """From radians per position (numbers or a tensor, one per pair)."""
        w = torch.as_tensor(frequencies, dtype=torch.float64).cpu().contiguous()
        if w.dim() != 1 or w.numel() == 0:
            raise ValueError("frequencies: one per pair of dims")
        steps = torch.empty(w.numel(), dtype=torch.int64)
        _check(lib().fa_rope_steps(w.data_ptr(), w.numel(), steps.data_ptr()), "fa_rope_steps")
        return RopeTable(steps.to(device), factor)


_SCALINGS = {"linear": 1, "ntk": 2, "yarn": 3}


def rope_frequencies(rotary_dim, base=10000.0, scaling=None):
    """(radians per position of every pair, a float64 CPU tensor; factor).
    ``scaling``: None, ("linear", scale), ("ntk", scale) or ("yarn", scale,
    trained_len[, beta_fast, beta_slow]); see fa_rope_frequencies in include/fa.h.
    YaRN's ramp is its paper's, linear in a pair's turns over ``trained_len``.  For
    a model that was stretched with another one (linear between two pairs' numbers,
    as some are), make the frequencies that way and hand them to RopeTable.of."""
    kind, args = 0, ()
    if scaling is not None:
        if scaling[0] not in _SCALINGS:
            raise ValueError("scaling: one of %s, got %r" % (", ".join(sorted(_SCALINGS)), scaling[0]))
        kind, args = _SCALINGS[scaling[0]], tuple(float(x) for x in scaling[1:])
        if len(args) not in ((2, 4) if kind == 3 else (1,)):
            raise ValueError("scaling: (kind, scale), for yarn (kind, scale, trained_len[, beta_fast, beta_slow])")
    args += (1.0, 1.0, 32.0, 1.0)[len(args):]
    w, factor = torch.empty(max(int(rotary_dim) // 2, 0), dtype=torch.float64), ctypes.c_double()
    _check(lib().fa_rope_frequencies(int(rotary_dim), float(base), kind, *args, w.data_ptr(), ctypes.byref(factor)),
           "fa_rope_frequencies")
    return w, factor.value


def rope_table(rotary_dim, base=10000.0, scaling=None, device="cuda"):
    """The RopeTable of rope_frequencies(rotary_dim, base, scaling)."""
    return RopeTable.of(*rope_frequencies(rotary_dim, base, scaling), device=device)


def rope(q, k, table, positions=None, offsets=None, interleaved=False, out=None, stream=None):
    """q and k (or None) turned by their rows' positions: (q, k), new tensors or
    ``out``, which may be the inputs themselves (in place).

    ``q`` / ``k``: [B, S, heads, D] or packed [total, heads, D]; slices of a
    joint projection are read (and with ``out`` written) where they lie.  The
    first ``table.rotary_dim`` dims of a head are turned, as pairs of its halves
    or ``interleaved``; the rest is copied.  A row's position is
    ``positions[b, s]`` (int32 [B, S]; packed: [total]), or ``offsets[b] + s``
    (int32 [B]), or s.  See fa_rope in include/fa.h."""
    return _rope(q, k, table, positions, offsets, interleaved, False, out, stream)


def rope_bwd(dq, dk, table, positions=None, offsets=None, interleaved=False, out=None, stream=None):
    """The gradients of rope's inputs from those of its results: (dq, dk).
    Arguments as for rope, of which it is the transpose."""
    return _rope(dq, dk, table, positions, offsets, interleaved, True, out, stream)


def _rope(q, k, table, positions, offsets, interleaved, inverse, out, stream):
    if out is None and stream is None:
        r = _binding().rope(q, k, table.steps, table.factor, positions, offsets, interleaved, inverse)
        if r is not None:
            return _done(r, "fa_rope")
    at = q.get_device()
    if at < 0:
        raise ValueError("q: not on a GPU")
    if q.dim() not in (3, 4):
        raise ValueError("q: [B, S, heads, D] or [total, heads, D]")
    code, D = _dtype_code(q), q.shape[-1]
    rows = tuple(q.shape[:-2])
    B, S = rows if len(rows) == 2 else (1, rows[0])
    if out is not None and (len(out) != 2 or (out[1] is None) != (k is None)):
        raise ValueError("out: (q, k) as the inputs are")
    given = [("q", q), ("k", k)] + ([] if out is None else [("out[0]", out[0]), ("out[1]", out[1])])
    for i, (name, t) in enumerate(given):
        if t is not None and (t.dim() != q.dim() or t.shape[:-2] != rows or t.shape[-1] != D or t.dtype != q.dtype
                              or t.get_device() != at or (i > 1 and t.shape != given[i - 2][1].shape)):
            raise ValueError("%s: %r of q's type on q's GPU" % (name, rows + ("heads", D)))
    for name, t, shape in (("positions", positions, rows), ("offsets", offsets, (B,))):
        if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous() or t.get_device() != at):
            raise ValueError("%s: contiguous int32 %r on q's GPU" % (name, shape))
    steps = table.steps
    if steps.dtype != torch.int64 or steps.dim() != 1 or not steps.is_contiguous() or steps.get_device() != at:
        raise ValueError("table: its steps, contiguous int64, on q's GPU")
    heads = [t.shape[-2] for t in (q, k) if t is not None]
    if B * S == 0 or 0 in heads:
        raise ValueError("q: empty")

    def lies(name, t, must):
        """(batch, row, head) strides as the library takes them; None where it cannot."""
        st = ((t.shape[0] * t.stride(0),) if t.dim() == 3 else ()) + t.stride()
        use = [8 if n == 1 else x for n, x in zip(((1,) if t.dim() == 3 else ()) + tuple(t.shape[:-1]), st[:3])]
        if st[3] == 1 and t.data_ptr() % 16 == 0 and all(0 < x < 1 << 39 and x % 8 == 0 for x in use):
            return use
        if must:
            raise ValueError(name + ": D contiguous, other strides multiples of 8, 16-byte aligned")
        return None
    with _on(at), _memory(stream):
        made, args = [], []
        for i, (name, t) in enumerate((("q", q), ("k", k))):
            if t is None:
                made.append(None)
                args.append(None)
                continue
            into = _like(t) if out is None else out[i]
            st = lies(name, t, False)
            if st is None:
                if out is not None and into.data_ptr() == t.data_ptr():
                    raise ValueError(name + ": cannot be turned in place as it lies")
                (t,) = _dense(stream, **{name: t})
                st = lies(name, t, True)
            r = _RopeTensor(t.data_ptr(), into.data_ptr(), t.shape[-2])
            r.in_stride[:], r.out_stride[:] = st, lies("out", into, True)
            made.append((into, t))   # (a copy lives until the call is made)
            args.append(ctypes.pointer(r))
        _check(lib().fa_rope(args[0], args[1], B, S, D, table.rotary_dim, steps.data_ptr(), table.factor,
                             int(bool(interleaved)), int(bool(inverse)), _ptr(positions), _ptr(offsets), code,
                             _stream(stream)), "fa_rope")
    return tuple(None if m is None else m[0] for m in made)


class _Here:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on(index):
    """A context in which GPU ``index`` (None: the current one) is current."""
    return _HERE if index is None or index == torch._C._cuda_getDevice() else torch.cuda.device(index)


def _gpu(t):
    """The index of the GPU a tensor lies on (None: on none)."""
    return t.get_device() if t.is_cuda else None


def _memory(stream):
    """A context in which memory is allocated for work on ``stream``: a block
    of the current stream's may still be in use there, and given back it would
    be used there again, both without regard to the other stream."""
    if stream is None:
        return _HERE
    if not isinstance(stream, torch.cuda.Stream):
        at = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(at) if at else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


class MaskRanges:
    """Visible-key intervals of a batch (``mask_ranges``): ``buffer``, a uint8
    CUDA tensor, for ``B`` sequences of ``S`` tokens."""

    def __init__(self, buffer, B, S):
        self.buffer, self.B, self.S = buffer, B, S


def _ranges(r):
    """A MaskRanges' buffer, B and S (None, 0, 0 without one)."""
    return (r.buffer, r.B, r.S) if isinstance(r, MaskRanges) else (r, 0, 0)


def mask_ranges(B, S, doc_ids=None, prefix_len=None, causal=True, window=None, device=None, out=None,
                stream=None):
    """Visible keys of every query row of a dense self-attention batch, for the
    ``mask_ranges`` keyword of fa_fwd and fa_bwd (see fa_mask_ranges in
    include/fa.h); built once per batch, read by every layer.

    ``doc_ids``: int32 [B, S], documents are runs of equal ids, a negative id
    is padding.  ``prefix_len``: int32 [B] (one prefix length for every
    document of a sequence) or [B, S] (read at a document's first token): the
    leading tokens every row of the document sees; with ``causal`` and without
    a window only.  ``window=(left, right)``, -1 = unbounded.  ``out``: a
    MaskRanges of the same B and S to fill again (a captured graph's)."""
    if window is None and device is None and out is None and stream is None:
        r = _binding().mask_ranges(B, S, doc_ids, prefix_len, causal)
        if r is not None:
            return MaskRanges(_done(r, "fa_mask_ranges"), int(B), int(S))
    at = None if device is None else torch.device(device).index   # None: the current GPU
    if out is not None:
        if not isinstance(out, MaskRanges) or (out.B, out.S) != (B, S):
            raise ValueError("out: a MaskRanges of the same B and S")
        at = _ranges_device(at, "out", out.buffer)
    if doc_ids is not None:
        at = _ranges_device(at, "doc_ids", doc_ids)
        if doc_ids.dtype != torch.int32 or doc_ids.shape != (B, S):
            raise ValueError("doc_ids: int32 [B, S]")
    if prefix_len is not None:
        at = _ranges_device(at, "prefix_len", prefix_len)
        if prefix_len.dtype != torch.int32 or (prefix_len.shape != (B, S) and prefix_len.shape != (B,)):
            raise ValueError("prefix_len: int32 [B] or [B, S]")
    wl, wr = (-1, -1) if window is None else (int(window[0]), int(window[1]))
    L = lib()
    need = L.fa_mask_ranges_bytes(B, S)
    if need == 0:
        raise FaError(FA_ERR_INVALID_ARG, "fa_mask_ranges")
    with _on(at):
        if out is None:
            with _memory(stream):
                out = MaskRanges(torch.empty(need, dtype=torch.uint8, device="cuda"), B, S)
        per_token = 1 if prefix_len is not None and prefix_len.dim() == 2 else 0
        _check(L.fa_mask_ranges(_ptr(doc_ids), _ptr(prefix_len), per_token, B, S, 1 if causal else 0, wl, wr,
                                out.buffer.data_ptr(), out.buffer.numel(), _stream(stream)), "fa_mask_ranges")
    return out


def _ranges_device(at, name, t):
    """The GPU of one of mask_ranges' tensors, which is ``at`` when that is known."""
    d = t.get_device()
    if d < 0 or not t.is_contiguous() or (at is not None and at != d):
        raise ValueError(name + ": a contiguous CUDA tensor, all on one GPU")
    return d


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libfa_gb300.so is not built (run attention_backward_preprocess_gb300.build."
                "build()); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        # (a library built before its header changed would read another struct)
        size = getattr(L, "fa_ext_bytes", None)
        if size is not None:
            size.restype = _sz
        if size is None or size() != ctypes.sizeof(FaExt):
            raise RuntimeError("libfa_gb300.so was built from another include/fa.h (run "
                               "attention_backward_preprocess_gb300.build.build()); there is no fallback path")
        L.fa_bwd.argtypes = [_vp] * 9 + _SHAPE + [_f, _i, _vp, _vp, _i, _i, _vp]
        L.fa_bwd_workspace_bytes.argtypes = _SHAPE + [_i, _i]
        L.fa_bwd_workspace_bytes.restype = _sz
        L.fa_bwd_with_workspace.argtypes = ([_vp] * 9 + _SHAPE + [_f, _i, _vp, _vp, _i, _i, _vp,
                                                                  _sz, _vp])
        L.fa_bwd_preprocess.argtypes = [_vp] * 3 + _SHAPE + [_vp, _vp, _i, _i, _vp, _sz, _vp]
        L.fa_bwd_main.argtypes = [_vp] * 6 + _SHAPE + [_f, _i, _vp, _vp, _i, _i, _vp, _sz, _vp]
        L.fa_bwd_postprocess.argtypes = [_vp] + _SHAPE + [_f, _vp, _vp, _i, _i, _vp, _sz, _vp]
        L.fa_bwd_workspace_layout.argtypes = _SHAPE + [_i, _i] + [ctypes.POINTER(_sz)] * 4
        L.fa_fwd.argtypes = [_vp] * 5 + _SHAPE + [_f, _i, _vp, _vp, _i, _vp]
        _ep = ctypes.POINTER(FaExt)
        L.fa_fwd_ext.argtypes = [_vp] * 5 + _SHAPE + [_f, _i, _vp, _vp, _ep, _i, _vp]
        L.fa_bwd_ext.argtypes = ([_vp] * 9 + _SHAPE + [_f, _i, _vp, _vp, _ep, _i, _i, _vp, _sz,
                                                       _vp])
        L.fa_bwd_stages_ext.argtypes = ([_i] + [_vp] * 9 + _SHAPE +
                                        [_f, _i, _vp, _vp, _ep, _i, _i, _vp, _sz, _vp])
        L.fa_device_status.argtypes = [_vp, _vp]
        L.fa_set_wait_timeout_ns.argtypes = [ctypes.c_longlong]
        L.fa_set_wait_timeout_ns.restype = ctypes.c_longlong
        L.fa_status_string.argtypes = [_i]
        L.fa_status_string.restype = ctypes.c_char_p
        L.fa_bwd_noalloc.argtypes = [_vp] * 9 + _SHAPE + [_f, _i, _vp, _vp, _i, _i, _vp]
        L.fa_bwd_noalloc.restype = _i
        L.fa_bwd_noalloc_scratch_bytes.argtypes = []
        L.fa_bwd_noalloc_scratch_bytes.restype = _sz
        L.fa_bwd_noalloc_status.argtypes = [_vp]
        L.fa_bwd_noalloc_status.restype = _i
        L.fa_bwd_workspace_sync_layout.argtypes = _SHAPE + [_i, _i] + [ctypes.POINTER(_sz)] * 3
        L.fa_bwd_workspace_sync_layout.restype = _i
        _kp = ctypes.POINTER(_KvCacheStruct)
        L.fa_kvcache_append.argtypes = [_kp] + [_vp] * 4 + [_i] * 4 + [_vp]
        L.fa_fwd_kvcache_workspace_bytes.argtypes = [_i]
        L.fa_fwd_kvcache_workspace_bytes.restype = _sz
        L.fa_fwd_kvcache.argtypes = [_vp, _kp, _vp, _vp, _vp] + [_i] * 3 + [_f, _f, _i, _i, _vp, _sz, _vp]
        L.fa_kvcache4_append.argtypes = L.fa_kvcache_append.argtypes
        L.fa_kvcache4_read.argtypes = [_kp] + [_vp] * 3 + [_i] * 2 + [_vp, _vp, _i, _vp]
        L.fa_fwd_kvcache4_workspace_bytes.argtypes = [_i]
        L.fa_fwd_kvcache4_workspace_bytes.restype = _sz
        L.fa_fwd_kvcache4.argtypes = L.fa_fwd_kvcache.argtypes
        _d, _rp = ctypes.c_double, ctypes.POINTER(_RopeTensor)
        L.fa_rope_frequencies.argtypes = [_i, _d, _i] + [_d] * 4 + [_vp, _vp]
        L.fa_rope_steps.argtypes = [_vp, _i, _vp]
        L.fa_rope.argtypes = [_rp, _rp] + [_i] * 4 + [_vp, _f, _i, _i, _vp, _vp, _i, _vp]
        L.fa_mask_ranges_bytes.argtypes = [_i, _i]
        L.fa_mask_ranges_bytes.restype = _sz
        L.fa_mask_ranges.argtypes = [_vp, _vp] + [_i] * 6 + [_vp, _sz, _vp]
        L.fa_selftest_umma.argtypes = [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]
        L.fa_selftest_semaphore.argtypes = [_vp, _i, ctypes.c_longlong, _vp, _vp]
        L.fa_selftest_tmem_layout.argtypes = [_i, _vp, _vp]
        for name in ("fa_bwd", "fa_bwd_with_workspace", "fa_bwd_preprocess", "fa_bwd_main",
                     "fa_bwd_postprocess", "fa_bwd_workspace_layout", "fa_fwd", "fa_fwd_ext",
                     "fa_bwd_ext", "fa_mask_ranges", "fa_kvcache_append", "fa_fwd_kvcache",
                     "fa_kvcache4_append", "fa_kvcache4_read", "fa_fwd_kvcache4", "fa_rope",
                     "fa_rope_frequencies", "fa_rope_steps",
                     "fa_device_status", "fa_selftest_umma", "fa_selftest_semaphore",
                     "fa_selftest_tmem_layout"):
            getattr(L, name).restype = _i
        _lib = L
        return _lib


_short = None


class _NoShortWay:
    """Stands in for the compiled short way in: every call goes on the Python way."""

    def __getattr__(self, name):
        return lambda *a: None


def _binding():
    """The compiled short way in (fa_torch.cpp): less host time for the ordinary
    call, the same library behind it.  Where it is not built, or does not load (built
    against another torch), the calls go through ctypes, after a warning."""
    global _short
    if _short is None:
        lib()
        import importlib.machinery
        import importlib.util
        loader = importlib.machinery.ExtensionFileLoader("_fa_torch", SHORT_PATH)
        try:
            mod = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_fa_torch", SHORT_PATH,
                                                                                         loader=loader))
            loader.exec_module(mod)
        except (ImportError, OSError) as e:
            import warnings
            warnings.warn("%s: %s; calls take 10 to 30 us more on the host (run "
                          "attention_backward_preprocess_gb300.build.build())" % (SHORT_PATH, e), RuntimeWarning)
            mod = _NoShortWay()
        _short = mod
    return _short


def _done(r, what):
    """A short call's result: None for the Python path to take over, else the
    result; a status raises."""
    if type(r) is int:
        _check(r, what)
    return r


def status_string(status: int) -> str:
    return lib().fa_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != FA_OK:
        raise FaError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        # the current stream's handle itself: building torch's stream object
        # took 2.8 of a decoding step's 27 us on the host
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float16:
        return FA_FP16
    raise ValueError("q/k/v/o/dout must be bf16 or fp16, got %s" % t.dtype)


def _shape(q, k, cu_q, max_seqlen_q, max_seqlen_k):
    """(B, Sq, Sk, Hq, Hkv, D) from dense [B,S,H,D] or packed [total,H,D] tensors."""
    if cu_q is None:
        if q.dim() != 4 or k.dim() != 4:
            raise ValueError("dense q/k are [B, S, H, D]")
        B, Sq, Hq, D = q.shape
        return B, Sq, k.shape[1], Hq, k.shape[2], D
    if q.dim() != 3 or k.dim() != 3 or max_seqlen_q is None or max_seqlen_k is None:
        raise ValueError("varlen q/k are [total, H, D] with max_seqlen_q / max_seqlen_k")
    return cu_q.numel() - 1, int(max_seqlen_q), int(max_seqlen_k), q.shape[1], k.shape[1], q.shape[2]


def _agree(q, k, v, cu_q=None, cu_k=None, o=None, dout=None, lse=None, dq=None, dk=None, dv=None, Dv=None):
    """The tensors of a call have the shapes, types and GPU that q and k say: the
    kernels take sizes from those two and read and write as far as they go."""
    if (Dv is None or v.shape[-1] == Dv) and _binding().agree(q, k, v, o, dout, dq, dk, dv, lse, cu_q, cu_k):
        return
    at = q.get_device()   # below: the same, with its messages
    rows, kv = q.shape[:-1], k.shape[:-1]
    ok_k = k.dim() == q.dim() and k.shape[-1] == q.shape[-1] and (q.dim() == 3 or k.shape[0] == q.shape[0])
    out = rows + v.shape[-1:]
    if Dv is not None and v.shape[-1] != Dv:
        raise ValueError("v: this call takes no head dim of its own for the values")
    for name, t, shape in (("k", k, k.shape if ok_k else None), ("v", v, kv + v.shape[-1:]), ("o", o, out),
                           ("dout", dout, out), ("dq", dq, q.shape), ("dk", dk, k.shape), ("dv", dv, v.shape)):
        if t is not None and (t.shape != shape or t.dtype != q.dtype or t.get_device() != at):
            raise ValueError("%s: %s of q's type on q's GPU, got %r" % (
                name, "q's batch and head dim" if shape is None else list(shape), tuple(t.shape)))
    if lse is not None:
        # (varlen: its rows are cu_seqlens_q[B], which only the device knows)
        n, most = lse.numel(), rows.numel()
        if (n != most and (q.dim() == 4 or n > most or n % rows[1])) or lse.dtype != torch.float32 \
                or lse.get_device() != at:
            raise ValueError("lse: fp32 [B, Hq, Sq] or [Hq, total_q] on q's GPU")
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_seqlens_q and cu_seqlens_k: both or neither")
    for name, t in (("cu_seqlens_q", cu_q), ("cu_seqlens_k", cu_k)):
        if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or t.shape != cu_q.shape or not t.is_contiguous()
                              or t.get_device() != at):
            raise ValueError(name + ": contiguous int32 [B + 1] on q's GPU")
    if at < 0:
        raise ValueError("q: not on a GPU")


def _value_dim(D, v) -> int:
    """head_dim_v of fa_ext: v's last axis when it differs from the query /
    key head dim, else 0."""
    return 0 if v.shape[-1] == D else int(v.shape[-1])


def _inputs(stream, **tensors):
    """The named inputs as the library can read them, and {name: (batch, row,
    head) element strides} of those that are not contiguous.  The tensor loads
    take any strides that are multiples of 16 bytes; a tensor that lies
    otherwise is copied on the current stream -- with another ``stream`` the
    copy and the call would not be in order, so that is refused."""
    out, strides = [], {}
    for name, t in tensors.items():
        if not t.is_contiguous():
            st = t.stride()
            st = ((0,) if t.dim() == 3 else ()) + st
            # an axis of one entry may carry any stride: a step of 8 serves
            size = ((1,) if t.dim() == 3 else ()) + tuple(t.shape)
            use = [8 if n == 1 else x for n, x in zip(size[:3], st[:3])]
            if t.dim() in (3, 4) and st[3] == 1 and all(0 < x < 1 << 39 and x % 8 == 0 for x in use) \
                    and t.data_ptr() % 16 == 0:
                strides[name] = tuple(use)
            else:
                t = _dense(stream, **{name: t})[0]
        out.append(t)
    return out, strides


def _dense(stream, **tensors):
    """The named tensors, each contiguous: copied on the current stream where
    they are not, refused where the call goes to another ``stream``."""
    out = []
    for name, t in tensors.items():
        if not t.is_contiguous():
            if stream is not None:
                raise ValueError(name + ": must be contiguous when a stream is given")
            t = t.contiguous()
        out.append(t)
    return out


def _like(t):
    """A new contiguous tensor of t's shape, dtype and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _scratch(workspace, at):
    """A caller's workspace lies on the call's GPU (its size is the library's to check)."""
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()
                                  or workspace.get_device() != at):
        raise ValueError("workspace: a contiguous uint8 tensor on q's GPU")


def _outputs(**tensors):
    for name, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError(name + ": must be contiguous")


def default_scale(D: int) -> float:
    return 1.0 / (D ** 0.5)


def fa_fwd(q, k, v, causal=False, softmax_scale=None, cu_seqlens_q=None, cu_seqlens_k=None,
           max_seqlen_q=None, max_seqlen_k=None, stream=None, window=None, alibi_slopes=None,
           seqused_q=None, seqused_k=None, bias=None, dropout=None, totals=None, softcap=0.0,
           mask_ranges=None):
    """Forward pass: returns (o, lse); lse fp32 [B,Hq,Sq] or [Hq,total_q].

    ``window=(left, right)`` (-1 = unbounded side), ``alibi_slopes`` (fp32
    [Hq] or [B, Hq]), ``seqused_q`` / ``seqused_k`` (int32 [B]) and ``bias``
    (see ``_ext``) and ``dropout=(p, seed, offset)`` select fa_fwd_ext; rows
    past the used lengths are left as allocated.  ``totals=(total_q, total_k)``
    (varlen: cu_seqlens_q[B], cu_seqlens_k[B]) spares the read-back of the
    packed totals, so the call does not synchronise the stream.  ``softcap``
    caps the scores, softcap * tanh(score / softcap); ``mask_ranges`` (from the
    function of that name) takes the place of ``causal`` and ``window``, which
    must be off with it.
    """
    if cu_seqlens_q is None and stream is None and window is None and alibi_slopes is None and seqused_q is None \
            and seqused_k is None and bias is None and dropout is None and totals is None:
        r = _binding().fwd(q, k, v, softmax_scale, causal, softcap, *_ranges(mask_ranges))
        if r is not None:
            return _done(r, "fa_fwd_ext")
    B, Sq, Sk, Hq, Hkv, D = _shape(q, k, cu_seqlens_q, max_seqlen_q, max_seqlen_k)
    _agree(q, k, v, cu_seqlens_q, cu_seqlens_k)
    (q, k, v), strides = _inputs(stream, q=q, k=k, v=v)
    scale = default_scale(D) if softmax_scale is None else float(softmax_scale)
    with _on(_gpu(q)), _memory(stream):
        o = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
        if cu_seqlens_q is None:
            lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
        else:
            lse = torch.empty((Hq, q.shape[0]), dtype=torch.float32, device=q.device)
        ext = _ext(Hq, window, alibi_slopes, seqused_q, seqused_k, bias, dropout=dropout,
                   totals=totals, head_dim_v=_value_dim(D, v), softcap=softcap, mask_ranges=mask_ranges,
                   sizes=(B, Sq, Sk, q.get_device()), strides=strides, rows=q.shape[:-2].numel(), dtype=q.dtype)
        args = [_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Sq, Sk, Hq, Hkv, D, scale,
                int(bool(causal)), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k)]
        if ext is None:
            _check(lib().fa_fwd(*args, _dtype_code(q), _stream(stream)), "fa_fwd")
        else:
            _check(lib().fa_fwd_ext(*args, ext, _dtype_code(q), _stream(stream)), "fa_fwd_ext")
    return o, lse


def fa_bwd(q, k, v, o, dout, lse, causal=False, softmax_scale=None, cu_seqlens_q=None,
           cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None, deterministic=False,
           dq=None, dk=None, dv=None, workspace=None, stream=None, window=None,
           alibi_slopes=None, seqused_q=None, seqused_k=None, bias=None, dbias=None,
           dropout=None, totals=None, softcap=0.0, mask_ranges=None):
    """Backward pass through the C ABI; returns (dq, dk, dv).

    Outputs are allocated when not given.  ``workspace`` (a uint8 CUDA tensor
    of at least ``workspace_bytes(...)``) selects fa_bwd_with_workspace,
    otherwise the call takes its scratch from the library's memory pool, so
    that calls may overlap on different streams.  The extension keywords
    (as for fa_fwd, plus ``dbias``, an output tensor filled with dBias = dS)
    select fa_bwd_ext, and so does ``totals=(total_q, total_k)`` (varlen: the
    packed row counts, which spare the stream synchronisation of reading them
    back).  ``softcap`` and ``mask_ranges`` as the forward had them.
    """
    if cu_seqlens_q is None and stream is None and window is None and alibi_slopes is None and seqused_q is None \
            and seqused_k is None and bias is None and dropout is None and totals is None and not deterministic \
            and dq is None and dk is None and dv is None and workspace is None and dbias is None:
        r = _binding().bwd(q, k, v, softmax_scale, causal, softcap, *_ranges(mask_ranges), o, dout, lse)
        if r is not None:
            return _done(r, "fa_bwd_ext")
    B, Sq, Sk, Hq, Hkv, D = _shape(q, k, cu_seqlens_q, max_seqlen_q, max_seqlen_k)
    _agree(q, k, v, cu_seqlens_q, cu_seqlens_k, o, dout, lse, dq, dk, dv)
    (q, k, v, o, dout), strides = _inputs(stream, q=q, k=k, v=v, o=o, dout=dout)
    (lse,) = _dense(stream, lse=lse)
    _outputs(dq=dq, dk=dk, dv=dv)
    _scratch(workspace, q.get_device())
    scale = default_scale(D) if softmax_scale is None else float(softmax_scale)
    with _on(_gpu(q)), _memory(stream):
        dq, dk, dv = (_like(t) if g is None else g for t, g in ((q, dq), (k, dk), (v, dv)))
        args = [_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                _ptr(dv), B, Sq, Sk, Hq, Hkv, D, scale, int(bool(causal)), _ptr(cu_seqlens_q),
                _ptr(cu_seqlens_k), int(bool(deterministic)), _dtype_code(q)]
        ext = _ext(Hq, window, alibi_slopes, seqused_q, seqused_k, bias, dbias, dropout, totals,
                   _value_dim(D, v), softcap, mask_ranges, (B, Sq, Sk, q.get_device()), strides,
                   q.shape[:-2].numel(), q.dtype)
        if ext is not None:
            st = lib().fa_bwd_ext(*args[:19], ext, *args[19:], _ptr(workspace),
                                  0 if workspace is None else workspace.numel(), _stream(stream))
            _check(st, "fa_bwd_ext")
        elif workspace is None:
            st = lib().fa_bwd(*args, _stream(stream))
            _check(st, "fa_bwd")
        else:
            st = lib().fa_bwd_with_workspace(*args, _ptr(workspace), workspace.numel(),
                                              _stream(stream))
            _check(st, "fa_bwd_with_workspace")
    return dq, dk, dv


def noalloc_scratch_bytes() -> int:
    """Size of the fixed scratch array fa_bwd_noalloc works in."""
    return int(lib().fa_bwd_noalloc_scratch_bytes())


def fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, causal=False, softmax_scale=None,
                   cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None,
                   deterministic=False, stream=None) -> int:
    """fa_bwd without any device allocation, for callers that cannot allocate
    device memory at call time (its scratch is a fixed array inside the
    library; see include/fa.h).  The outputs must be given.  Returns the
    status (FA_OK, or FA_ERR_SCRATCH_LIMIT for a problem too large)."""
    B, Sq, Sk, Hq, Hkv, D = _shape(q, k, cu_seqlens_q, max_seqlen_q, max_seqlen_k)
    _agree(q, k, v, cu_seqlens_q, cu_seqlens_k, o, dout, lse, dq, dk, dv, D)
    _outputs(q=q, k=k, v=v, o=o, dout=dout, lse=lse, dq=dq, dk=dk, dv=dv)
    scale = default_scale(D) if softmax_scale is None else float(softmax_scale)
    return int(lib().fa_bwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
        B, Sq, Sk, Hq, Hkv, D, scale, int(bool(causal)), _ptr(cu_seqlens_q),
        _ptr(cu_seqlens_k), int(bool(deterministic)), _dtype_code(q), _stream(stream)))


def noalloc_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the error status of
    the fixed scratch array fa_bwd_noalloc works in."""
    return int(lib().fa_bwd_noalloc_status(_stream(stream)))


def workspace_sync_layout(B, Sq, Sk, Hq, Hkv, D, varlen=False, deterministic=False) -> dict:
    """Byte offsets of the error word and of the deterministic-order
    semaphores inside a workspace, and the number of semaphores."""
    vals = [_sz() for _ in range(3)]
    st = lib().fa_bwd_workspace_sync_layout(B, Sq, Sk, Hq, Hkv, D, int(bool(varlen)),
                                            int(bool(deterministic)),
                                            *[ctypes.byref(x) for x in vals])
    _check(st, "fa_bwd_workspace_sync_layout")
    return dict(err=vals[0].value, sem=vals[1].value, n_sem=vals[2].value)


def workspace_bytes(B, Sq, Sk, Hq, Hkv, D, varlen=False, deterministic=False) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, Sq, Sk, Hq, Hkv, D, int(bool(varlen)),
                                            int(bool(deterministic))))


def workspace_layout(B, Sq, Sk, Hq, Hkv, D, varlen=False, deterministic=False) -> dict:
    """fp32-element offsets of Dv, LSE2 and the dQ accumulator inside a workspace."""
    vals = [_sz() for _ in range(4)]
    st = lib().fa_bwd_workspace_layout(B, Sq, Sk, Hq, Hkv, D, int(bool(varlen)),
                                       int(bool(deterministic)), *[ctypes.byref(x) for x in vals])
    _check(st, "fa_bwd_workspace_layout")
    return dict(dvec=vals[0].value, lse2=vals[1].value, dqacc=vals[2].value, rows=vals[3].value)


def fa_bwd_stages(q, k, v, o, dout, lse, workspace, causal=False, softmax_scale=None,
                  cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None,
                  deterministic=False, dq=None, dk=None, dv=None, stages=("pre", "main", "post"),
                  stream=None, totals=None, window=None, softcap=0.0, mask_ranges=None):
    """Runs the chosen stages (preprocess / main / postprocess) on ``workspace``.

    ``totals=(total_q, total_k)`` (varlen) goes through fa_bwd_stages_ext with
    the packed row counts, so that no stage synchronises the stream; so do
    ``window``, ``softcap`` and ``mask_ranges`` (as for fa_bwd).  Stages in
    separate calls share no copies, so every tensor must be contiguous."""
    B, Sq, Sk, Hq, Hkv, D = _shape(q, k, cu_seqlens_q, max_seqlen_q, max_seqlen_k)
    _agree(q, k, v, cu_seqlens_q, cu_seqlens_k, o, dout, lse, dq, dk, dv, D)
    _outputs(q=q, k=k, v=v, o=o, dout=dout, lse=lse, dq=dq, dk=dk, dv=dv)
    _scratch(workspace, q.get_device())
    scale = default_scale(D) if softmax_scale is None else float(softmax_scale)
    dq, dk, dv = (_like(t) if g is None else g for t, g in ((q, dq), (k, dk), (v, dv)))
    shape = [B, Sq, Sk, Hq, Hkv, D]
    ext = _ext(Hq, window, totals=totals, softcap=softcap, mask_ranges=mask_ranges, sizes=(B, Sq, Sk, q.get_device()))
    if ext is not None:
        mask = ((1 if "pre" in stages else 0) | (2 if "main" in stages else 0) |
                (4 if "post" in stages else 0))
        _check(lib().fa_bwd_stages_ext(mask, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout),
                                       _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), *shape, scale,
                                       int(bool(causal)), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                       ext, int(bool(deterministic)), _dtype_code(q),
                                       _ptr(workspace), workspace.numel(), _stream(stream)),
               "fa_bwd_stages_ext")
        return dq, dk, dv
    cu = [_ptr(cu_seqlens_q), _ptr(cu_seqlens_k)]
    det, dt = int(bool(deterministic)), _dtype_code(q)
    ws = [_ptr(workspace), workspace.numel(), _stream(stream)]
    L = lib()
    if "pre" in stages:
        _check(L.fa_bwd_preprocess(_ptr(o), _ptr(dout), _ptr(lse), *shape, *cu, det, dt, *ws),
               "fa_bwd_preprocess")
    if "main" in stages:
        _check(L.fa_bwd_main(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dk), _ptr(dv), *shape,
                             scale,
                             int(bool(causal)), *cu, det, dt, *ws), "fa_bwd_main")
    if "post" in stages:
        _check(L.fa_bwd_postprocess(_ptr(dq), *shape, scale, *cu, det, dt, *ws),
               "fa_bwd_postprocess")
    return dq, dk, dv


def device_status(workspace=None, stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error status."""
    return int(lib().fa_device_status(_ptr(workspace), _stream(stream)))


def set_wait_timeout_ns(ns: int) -> int:
    return int(lib().fa_set_wait_timeout_ns(int(ns)))


def selftest_umma(mode: int, A: torch.Tensor, B: torch.Tensor, N: int, K: int, stream=None):
    """One-CTA tcgen05 GEMM in one of the kernel's operand forms (see fa_selftest.h)."""
    C = torch.empty((128, N), dtype=torch.float32, device=A.device)
    err = torch.zeros(1, dtype=torch.int32, device=A.device)
    st = lib().fa_selftest_umma(mode, N, K, int(A.dtype == torch.bfloat16), _ptr(A), _ptr(B),
                                _ptr(C), _ptr(err), _stream(stream))
    if st != 0:
        raise RuntimeError("fa_selftest_umma returned %d" % st)
    return C, err


def selftest_tmem_layout(which: int, device="cuda", stream=None):
    """The 16-lane tensor-memory access shapes' layout probe (see fa_selftest.h);
    returns the [128, 32] uint32 result as int64."""
    out = torch.zeros((128, 32), dtype=torch.int32, device=device)
    st = lib().fa_selftest_tmem_layout(int(which), _ptr(out), _stream(stream))
    if st != 0:
        raise RuntimeError("fa_selftest_tmem_layout returned %d" % st)
    return out.cpu().to(torch.int64) & 0xFFFFFFFF


def selftest_semaphore(sem: torch.Tensor, target: int, budget_ns: int, stream=None):
    err = torch.zeros(1, dtype=torch.int32, device=sem.device)
    st = lib().fa_selftest_semaphore(_ptr(sem), int(target), int(budget_ns), _ptr(err),
                                     _stream(stream))
    if st != 0:
        raise RuntimeError("fa_selftest_semaphore returned %d" % st)
    return err
