"""Python binding of the operators around the 4-bit paged KV cache.

``qk_norm_rope`` makes the Q and K that the scorer takes; ``cache_reserve``
and ``cache_release`` keep block tables and slot maps on the device;
``q4_append``, ``q4_read`` and ``q4_compact`` move rows between bf16 and the
4-bit pages; ``q4_decode_attention`` is one decode step over them.
:class:`Q4Cache` owns the tensors of one such cache.  Contracts:
``include/waits.h``.  Like :mod:`.api` this module only checks tensors,
allocates outputs and passes pointers and the current stream.
"""

from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import _lib


_BF16, _I32, _U8 = torch.bfloat16, torch.int32, torch.uint8
_CONTIGUOUS = torch.contiguous_format


def _device(name, t):
    """Index of the CUDA device that ``t`` is on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _dense(name, t, dtype, device, shape=None):
    """``t``: a contiguous ``dtype`` tensor on CUDA device ``device``.  The
    first test is the whole cost of a good argument: these checks run at
    every step of a decode loop."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device \
            and t.is_contiguous() and (shape is None or t.shape == shape):
        return
    if _device(name, t) != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _rows(name, t, device, shape=None):
    """Token stride of a bf16 ``[tokens, heads, head_dim]`` tensor whose heads
    are dense."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        _device(name, t)
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have shape {shape or '[tokens, heads, head_dim]'}, "
                         f"got {tuple(t.shape)}")
    T, H, d = t.shape
    st, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and H > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return st if T > 1 else H * d


def _table(block_table, device, nseq):
    _dense("block_table", block_table, _I32, device)
    if block_table.dim() != 2 or block_table.shape[0] != nseq:
        raise ValueError(f"block_table must be [{nseq}, max_blocks]")
    return block_table.shape[1]


_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _call(name, device, *args):
    """Run a C entry on CUDA device ``device``'s current stream."""
    fn = getattr(_lib.load(), name)
    if device == _current_device():
        st = fn(*args, _current_stream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _current_stream(device))
    if st:
        _lib.check(name, st)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _status(t, device):
    if t is None:
        return None
    _dense("status", t, _I32, device)
    if t.numel() != 1:
        raise ValueError("status must hold one int32")
    return t.data_ptr()


def rotary_inv_freq(rotary_dim: int, theta: float) -> torch.Tensor:
    """``theta ** (-2 i / rotary_dim)``, the CPU float64 tensor that
    :func:`qk_norm_rope` takes (scaled or interpolated ones are made from it)."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    return float(theta) ** (-2.0 * i / rotary_dim)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor,
                 inv_freq: torch.Tensor, *, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False,
                 out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """Head norms and rotary positions in one pass (``waits_qk_norm_rope``).

    ``q`` bf16 ``[T, Hq, d]``, ``k`` bf16 ``[T, Hkv, d]`` (views of a fused
    projection fit), ``positions`` int32 ``[T]``, ``inv_freq`` CPU float64
    ``[rotary_dim / 2]``; ``q_weight``, ``k_weight`` bf16 ``[d]`` or both
    None (rotation only).  Returns ``(q_out, k_out)``: new contiguous
    tensors, or ``out``, which may be ``(q, k)`` themselves.
    """
    dev = _device("q", q)
    q_stride = _rows("q", q, dev)
    k_stride = _rows("k", k, dev)
    T, Hq, d = q.shape
    Tk, Hkv, dk = k.shape
    if Tk != T or dk != d:
        raise ValueError("k must be [T, Hkv, d] like q's [T, Hq, d]")
    _dense("positions", positions, _I32, dev, (T,))
    if inv_freq.dtype is not torch.float64 or inv_freq.is_cuda or inv_freq.dim() != 1 \
            or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous 1-D float64 CPU tensor")
    qw = kw = None
    if q_weight is not None or k_weight is not None:
        if q_weight is None or k_weight is None:
            raise ValueError("q_weight and k_weight come together")
        _dense("q_weight", q_weight, _BF16, dev, (d,))
        _dense("k_weight", k_weight, _BF16, dev, (d,))
        qw, kw = q_weight.data_ptr(), k_weight.data_ptr()
    if out is None:
        q_out = torch.empty_like(q, memory_format=_CONTIGUOUS)
        k_out = torch.empty_like(k, memory_format=_CONTIGUOUS)
        qo_stride, ko_stride = Hq * d, Hkv * d
    else:
        q_out, k_out = out
        qo_stride = _rows("out[0]", q_out, dev, (T, Hq, d))
        ko_stride = _rows("out[1]", k_out, dev, (T, Hkv, d))
    _call("waits_qk_norm_rope", dev, T, Hq, Hkv, d, 2 * inv_freq.numel(), interleaved,
          q.data_ptr(), q_stride, k.data_ptr(), k_stride, positions.data_ptr(),
          inv_freq.data_ptr(), qw, kw, eps, q_out.data_ptr(), qo_stride, k_out.data_ptr(),
          ko_stride)
    return q_out, k_out


def cache_reserve(new_len: torch.Tensor, cache_len: torch.Tensor, block_table: torch.Tensor,
                  free_list: torch.Tensor, free_count: torch.Tensor, *, block_size: int,
                  max_new: int, in_place: bool = True,
                  status: Optional[torch.Tensor] = None):
    """Blocks and slots for ``new_len`` more tokens of every sequence
    (``waits_cache_reserve``), all int32 on the device.

    Returns ``(slot_map [max_new], cu_new [nseq + 1], cache_len,
    free_count)``; ``block_table`` gets its new entries in place, the lengths
    and the count too unless ``in_place`` is False, which returns new tensors
    for them.  A refused sequence keeps its length and gets -1 slots.
    """
    dev = _device("cache_len", cache_len)
    nseq = cache_len.numel()
    _dense("cache_len", cache_len, _I32, dev, (nseq,))
    _dense("new_len", new_len, _I32, dev, (nseq,))
    width = _table(block_table, dev, nseq)
    _dense("free_list", free_list, _I32, dev)
    _dense("free_count", free_count, _I32, dev)
    if free_count.numel() != 1:
        raise ValueError("free_count must hold one int32")
    slots = torch.empty(max_new, dtype=_I32, device=dev)
    cu = torch.empty(nseq + 1, dtype=_I32, device=dev)
    len_out = cache_len if in_place else torch.empty_like(cache_len)
    count_out = free_count if in_place else torch.empty_like(free_count)
    _call("waits_cache_reserve", dev, nseq, block_size, width, free_list.numel(), max_new,
          new_len.data_ptr(), cache_len.data_ptr(), block_table.data_ptr(), free_list.data_ptr(),
          free_count.data_ptr(), len_out.data_ptr(), count_out.data_ptr(),
          slots.data_ptr() or None, cu.data_ptr(), _status(status, dev))
    return slots, cu, len_out, count_out


def cache_release(ended: torch.Tensor, cache_len: torch.Tensor, block_table: torch.Tensor,
                  free_list: torch.Tensor, free_count: torch.Tensor, *, block_size: int,
                  status: Optional[torch.Tensor] = None) -> None:
    """Give the blocks of the sequences with ``ended != 0`` (int32 ``[nseq]``)
    back to the free list (``waits_cache_release``), in place."""
    dev = _device("cache_len", cache_len)
    nseq = cache_len.numel()
    _dense("cache_len", cache_len, _I32, dev, (nseq,))
    _dense("ended", ended, _I32, dev, (nseq,))
    width = _table(block_table, dev, nseq)
    _dense("free_list", free_list, _I32, dev)
    _dense("free_count", free_count, _I32, dev)
    if free_count.numel() != 1:
        raise ValueError("free_count must hold one int32")
    _call("waits_cache_release", dev, nseq, block_size, width, free_list.numel(),
          ended.data_ptr(), cache_len.data_ptr(), block_table.data_ptr(), free_list.data_ptr(),
          free_count.data_ptr(), _status(status, dev))


def q4_page_bytes(block_size: int, head_dim: int) -> int:
    """Bytes of one KV head's page of ``block_size`` tokens."""
    return block_size * head_dim * 9 // 8


def _cache(pool: torch.Tensor, device: int, head_dim: int):
    _dense("pool", pool, _U8, device)
    if pool.dim() != 3:
        raise ValueError("pool must be uint8 [num_blocks, Hkv, page_bytes]")
    num_blocks, heads, page = pool.shape
    bs = page * 8 // (9 * head_dim) if head_dim > 0 else 0
    if bs * head_dim * 9 != page * 8:
        raise ValueError(f"a page of {page} bytes is no whole number of tokens of "
                         f"head_dim {head_dim}")
    return ctypes.byref(_lib.Q4Cache(num_blocks, bs, heads, head_dim, pool.data_ptr()))


def q4_append(K: torch.Tensor, V: torch.Tensor, slot_map: torch.Tensor, pool: torch.Tensor, *,
              status: Optional[torch.Tensor] = None) -> None:
    """Quantise the rows of ``K``, ``V`` (bf16 ``[n, Hkv, d]``, views with
    dense heads fit) into the slots ``slot_map`` (int32 ``[n]``, negative:
    skipped) of ``pool`` (``waits_q4_append``)."""
    dev = _device("K", K)
    ks = _rows("K", K, dev)
    vs = _rows("V", V, dev, K.shape)
    n, Hkv, d = K.shape
    c = _cache(pool, dev, d)
    if pool.shape[1] != Hkv:
        raise ValueError("pool must have K's heads")
    _dense("slot_map", slot_map, _I32, dev, (n,))
    _call("waits_q4_append", dev, c, n, K.data_ptr(), ks, V.data_ptr(), vs, slot_map.data_ptr(),
          _status(status, dev))


def q4_read(pool: torch.Tensor, slot_map: torch.Tensor, head_dim: int, *,
            status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``(K, V)`` bf16 ``[n, Hkv, d]`` of the slots (``waits_q4_read``);
    zero rows for negative slots."""
    dev = _device("pool", pool)
    c = _cache(pool, dev, head_dim)
    n = slot_map.numel()
    _dense("slot_map", slot_map, _I32, dev, (n,))
    K = torch.empty(n, pool.shape[1], head_dim, dtype=_BF16, device=dev)
    V = torch.empty_like(K)
    _call("waits_q4_read", dev, c, n, slot_map.data_ptr(), K.data_ptr(), V.data_ptr(),
          _status(status, dev))
    return K, V


def q4_compact(K: torch.Tensor, V: torch.Tensor, cu_seqlens: torch.Tensor, idx: torch.Tensor,
               kept_len: torch.Tensor, block_table: torch.Tensor, pool: torch.Tensor, *,
               status: Optional[torch.Tensor] = None) -> None:
    """The rows ``idx`` keeps (``select``'s ``[nseq, Hkv, B]``), quantised
    into the first ``kept_len`` slots of every sequence's table row
    (``waits_q4_compact``)."""
    dev = _device("K", K)
    _dense("K", K, _BF16, dev)
    if K.dim() != 3:
        raise ValueError("K must be [T, Hkv, d]")
    T, Hkv, d = K.shape
    _dense("V", V, _BF16, dev, K.shape)
    _dense("idx", idx, _I32, dev)
    if idx.dim() != 3 or idx.shape[1] != Hkv:
        raise ValueError("idx must be [nseq, Hkv, B]")
    nseq, _, B = idx.shape
    _dense("cu_seqlens", cu_seqlens, _I32, dev, (nseq + 1,))
    _dense("kept_len", kept_len, _I32, dev, (nseq,))
    width = _table(block_table, dev, nseq)
    c = _cache(pool, dev, d)
    shape = _lib.Shape(nseq, T, T, Hkv, Hkv, d, cu_seqlens.data_ptr())
    _call("waits_q4_compact", dev, ctypes.byref(shape), K.data_ptr(), V.data_ptr(),
          idx.data_ptr(), kept_len.data_ptr(), B, c, block_table.data_ptr(), width,
          _status(status, dev))


@functools.lru_cache(maxsize=256)
def _decode_workspace(num_blocks, block_size, heads, head_dim, nseq, num_q_heads):
    c = _lib.Q4Cache(num_blocks, block_size, heads, head_dim, None)
    n = ctypes.c_size_t(0)
    _lib.check("waits_q4_decode_workspace_size", _lib.load().waits_q4_decode_workspace_size(
        ctypes.byref(c), nseq, num_q_heads, ctypes.byref(n)))
    return int(n.value)


def q4_decode_workspace_bytes(pool: torch.Tensor, nseq: int, num_q_heads: int,
                              head_dim: int) -> int:
    """Bytes of :func:`q4_decode_attention`'s workspace."""
    num_blocks, heads, page = pool.shape
    return _decode_workspace(num_blocks, page * 8 // (9 * head_dim), heads, head_dim, nseq,
                             num_q_heads)


def q4_decode_attention(q: torch.Tensor, pool: torch.Tensor, block_table: torch.Tensor,
                        cache_len: torch.Tensor, with_lse: bool = False, *,
                        workspace: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None):
    """One decode step over the 4-bit paged cache
    (``waits_q4_decode_attention``): ``q`` bf16 ``[nseq, Hq, d]``,
    ``block_table`` int32 ``[nseq, max_blocks]``, ``cache_len`` int32
    ``[nseq]``.  Returns bf16 ``[nseq, Hq, d]`` (and the fp32 ``[nseq, Hq]``
    row LSE).  ``workspace``: a uint8 tensor of
    :func:`q4_decode_workspace_bytes` to reuse; made here otherwise."""
    dev = _device("q", q)
    _dense("q", q, _BF16, dev)
    if q.dim() != 3:
        raise ValueError("q must be [nseq, Hq, d]")
    nseq, Hq, d = q.shape
    c = _cache(pool, dev, d)
    width = _table(block_table, dev, nseq)
    _dense("cache_len", cache_len, _I32, dev, (nseq,))
    if workspace is None:
        workspace = torch.empty(q4_decode_workspace_bytes(pool, nseq, Hq, d), dtype=_U8,
                                device=dev)
    else:
        _dense("workspace", workspace, _U8, dev)
    out = torch.empty_like(q)
    lse = torch.empty(nseq, Hq, dtype=torch.float32, device=dev) if with_lse else None
    _call("waits_q4_decode_attention", dev, c, nseq, Hq, width, q.data_ptr(),
          block_table.data_ptr(), cache_len.data_ptr(), out.data_ptr(), _ptr(lse),
          workspace.data_ptr(), workspace.numel(), _status(status, dev))
    return (out, lse) if with_lse else out


class Q4Cache:
    """The tensors of one layer's 4-bit paged cache for ``nseq`` sequences.

    ``num_blocks`` blocks of ``block_size`` tokens, shared by the sequences;
    at most ``max_blocks`` each.  All state (pool, block table, lengths, free
    stack, status) stays on the device and keeps its addresses, so calls may
    be captured in a CUDA graph and replayed; calls on one cache share its
    state and its workspace and must not overlap on the GPU.
    """

    def __init__(self, nseq: int, num_q_heads: int, num_kv_heads: int, head_dim: int, *,
                 num_blocks: int, max_blocks: int, block_size: int = 64, device="cuda"):
        dev = torch.empty(0, device=device).device
        i32 = dict(dtype=torch.int32, device=dev)
        self.block_size, self.head_dim, self.num_q_heads = block_size, head_dim, num_q_heads
        self.pool = torch.zeros((num_blocks, num_kv_heads, q4_page_bytes(block_size, head_dim)),
                                dtype=torch.uint8, device=dev)
        self.block_table = torch.full((nseq, max_blocks), -1, **i32)
        self.cache_len = torch.zeros((nseq,), **i32)
        self.free_list = torch.arange(num_blocks - 1, -1, -1, **i32)
        self.free_count = torch.full((1,), num_blocks, **i32)
        self.status = torch.zeros((1,), **i32)
        self.workspace = torch.empty(
            (q4_decode_workspace_bytes(self.pool, nseq, num_q_heads, head_dim),),
            dtype=torch.uint8, device=dev)

    def reserve(self, new_len: torch.Tensor, max_new: int):
        """``(slot_map, cu_new)`` for ``new_len`` more tokens a sequence."""
        slots, cu, _, _ = cache_reserve(
            new_len, self.cache_len, self.block_table, self.free_list, self.free_count,
            block_size=self.block_size, max_new=max_new, status=self.status)
        return slots, cu

    def release(self, ended: torch.Tensor) -> None:
        """Frees the blocks of sequences with ``ended != 0``."""
        cache_release(ended, self.cache_len, self.block_table, self.free_list, self.free_count,
                      block_size=self.block_size, status=self.status)

    def append(self, K: torch.Tensor, V: torch.Tensor, slot_map: torch.Tensor) -> None:
        q4_append(K, V, slot_map, self.pool, status=self.status)

    def compact(self, K: torch.Tensor, V: torch.Tensor, cu_seqlens: torch.Tensor,
                idx: torch.Tensor, kept_len: torch.Tensor) -> None:
        """Reserves ``kept_len`` slots of every empty sequence and writes the
        rows that ``idx`` keeps into them: ``select``'s output, e.g.
        ``compress``'s, becomes the cache.  A sequence that holds tokens
        already stays as it is, and one that is refused (see ``status``)
        stays empty."""
        nseq, _, B = idx.shape
        fresh = self.cache_len == 0
        self.reserve(torch.where(fresh, kept_len, 0), nseq * B)
        q4_compact(K, V, cu_seqlens, idx, torch.where(fresh, self.cache_len, 0),
                   self.block_table, self.pool, status=self.status)

    def attend(self, q: torch.Tensor, with_lse: bool = False):
        return q4_decode_attention(q, self.pool, self.block_table, self.cache_len, with_lse,
                                   workspace=self.workspace, status=self.status)

    def read(self, slot_map: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        return q4_read(self.pool, slot_map, self.head_dim, status=self.status)

    def device_status(self) -> int:
        """The ``WAITS_DEV_*`` bits seen so far (synchronises); clears them."""
        v = int(self.status.item())
        self.status.zero_()
        return v
