"""Python binding of the attention half of include/fd.h: rotary positions, the append to a paged
key/value cache and the attention over it. Argument marshalling only, like kernels.py."""

from __future__ import annotations

import math
import struct

import torch

from . import _lib
from .kernels import _check_tensor, _device_of, _on_device, _ptr, _stream_handle

# fd_heads, fd_paged_cache and fd_paged_batch of include/fd.h, packed as the C compiler lays them out
_HEADS = struct.Struct("=Qqqi4x")
_CACHE = struct.Struct("=QQqqqqqqiiii")
_BATCH = struct.Struct("=QQQiiiii4x")


def _heads(name: str, t: torch.Tensor, tokens: int | None = None, heads: int | None = None,
           head_dim: int | None = None) -> bytes:
    """The fd_heads of a bf16 [tokens, heads, head_dim] tensor (any token and head strides)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the fd kernels have no CPU path)")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    n, h, d = t.shape
    if (tokens is not None and n != tokens) or (heads is not None and h != heads) or \
            (head_dim is not None and d != head_dim):
        raise ValueError(f"{name} must have shape {(tokens or n, heads or h, head_dim or d)}, got {(n, h, d)}")
    ts, hs, ds = t.stride()
    if ds != 1 and d > 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    return _HEADS.pack(t.data_ptr(), ts if n > 1 else 0, hs if h > 1 else 0, h)


def _cache(k: torch.Tensor, v: torch.Tensor) -> tuple[bytes, int, int, int]:
    """(fd_paged_cache, kv_heads, head_dim, page_size) of bf16 [num_pages, page_size, kv_heads, head_dim] tensors."""
    for name, t in (("k_cache", k), ("v_cache", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the fd kernels have no CPU path)")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [num_pages, page_size, kv_heads, head_dim], got {tuple(t.shape)}")
        if t.stride(3) != 1:
            raise ValueError(f"{name} must have unit stride along head_dim")
    if k.shape != v.shape:
        raise ValueError(f"k_cache and v_cache differ in shape: {tuple(k.shape)}, {tuple(v.shape)}")
    pages, page, heads, d = k.shape
    a, b = k.stride(), v.stride()
    return (_CACHE.pack(k.data_ptr(), v.data_ptr(), a[0], a[1], a[2], b[0], b[1], b[2], pages, page, heads, d),
            heads, d, page)


def _batch(q_start, kv_len, block_table, total_q: int, max_q: int) -> bytes:
    if not isinstance(kv_len, torch.Tensor) or kv_len.dim() != 1:
        raise ValueError("kv_len must be an int32 [batch] tensor")
    batch = kv_len.shape[0]
    _check_tensor("q_start", q_start, torch.int32, (batch + 1,))
    _check_tensor("kv_len", kv_len, torch.int32)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError("block_table must be an int32 [batch, max_pages] tensor")
    if not block_table.is_cuda:
        raise ValueError("block_table must be a CUDA tensor (the fd kernels have no CPU path)")
    if block_table.dtype != torch.int32:
        raise TypeError(f"block_table must be torch.int32, got {block_table.dtype}")
    pages = block_table.shape[1]
    row, col = block_table.stride()
    if pages > 1 and col != 1:
        raise ValueError("block_table must have unit stride along a sequence's pages")
    return _BATCH.pack(q_start.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(),
                       row if batch > 1 else pages, batch, total_q, max_q, pages)


def _inv_freq(inv_freq: torch.Tensor, head_dim: int) -> int:
    _check_tensor("inv_freq", inv_freq, torch.float64)
    if inv_freq.dim() != 1 or not 1 <= inv_freq.shape[0] <= head_dim // 2:
        raise ValueError(f"inv_freq must be [rot_dim / 2] with 2 <= rot_dim <= head_dim={head_dim}")
    return 2 * inv_freq.shape[0]


def rope(
    q: torch.Tensor,
    k: torch.Tensor | None,
    positions: torch.Tensor,
    inv_freq: torch.Tensor,
    interleaved: bool = False,
    scale: float = 1.0,
    q_out: torch.Tensor | None = None,
    k_out: torch.Tensor | None = None,
    stream: torch.cuda.Stream | None = None,
) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(q_out, k_out): rotary positions on q and k (fd_rope in include/fd.h).

    q, k: bf16 [tokens, heads, head_dim], views of a wider row allowed (unit stride along
    head_dim); k may be None. positions: int32 [tokens]. inv_freq: float64 [rot_dim / 2] and
    scale, from ``rope_inv_freq``; the first rot_dim elements of a head are rotated, in pairs
    (2i, 2i + 1) if interleaved, else (i, i + rot_dim / 2). q_out, k_out: allocated if None; q
    and k themselves for a rotation in place.
    """
    qb = _heads("q", q)
    n, h, d = q.shape
    _check_tensor("positions", positions, torch.int32, (n,))
    rot = _inv_freq(inv_freq, d)
    if q_out is None:
        q_out = torch.empty((n, h, d), dtype=torch.bfloat16, device=q.device)
    qo = _heads("q_out", q_out, n, h, d)
    kb = ko = None
    if k is not None:
        kb = _heads("k", k, n, None, d)
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=k.device)
        ko = _heads("k_out", k_out, n, k.shape[1], d)
        dev = _device_of(q, k, q_out, k_out, positions, inv_freq)
    elif k_out is not None:
        raise ValueError("k_out without k")
    else:
        dev = _device_of(q, q_out, positions, inv_freq)
    lib = _lib.load()
    with _on_device(dev):
        st = lib.fd_rope(qb, kb, qo, ko, _ptr(positions), _ptr(inv_freq), n, d, rot,
                         int(bool(interleaved)), scale, _stream_handle(stream, dev))
    _lib.check(st)
    return q_out, k_out


def rope_append(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    k_cache: torch.Tensor,
    v_cache: torch.Tensor,
    q_start: torch.Tensor,
    kv_len: torch.Tensor,
    block_table: torch.Tensor,
    inv_freq: torch.Tensor,
    positions: torch.Tensor | None = None,
    interleaved: bool = False,
    scale: float = 1.0,
    q_out: torch.Tensor | None = None,
    stream: torch.cuda.Stream | None = None,
) -> torch.Tensor:
    """q_out, the rotated queries; the rotated keys and the values go to their places in the
    cache (fd_rope_append in include/fd.h).

    q: bf16 [total_q, q_heads, head_dim]; k, v: [total_q, kv_heads, head_dim]; k_cache, v_cache:
    bf16 [num_pages, page_size, kv_heads, head_dim], written in place (any strides: a
    [num_pages, kv_heads, page_size, head_dim] cache is passed transposed). q_start int32
    [batch + 1], kv_len int32 [batch] (the new tokens included) and block_table int32 [batch,
    max_pages] say where each token goes; positions int32 [total_q] (default: the token's number
    in its cache). q_out: allocated if None; may be q (in place). Rows past q_start[batch] are not
    written.
    """
    cache, hk, d, _ = _cache(k_cache, v_cache)
    qb = _heads("q", q, None, None, d)
    n, h, _ = q.shape
    kb = _heads("k", k, n, hk, d)
    vb = _heads("v", v, n, hk, d)
    rot = _inv_freq(inv_freq, d)
    batch = _batch(q_start, kv_len, block_table, n, n)
    if positions is not None:
        _check_tensor("positions", positions, torch.int32, (n,))
    if q_out is None:
        q_out = torch.empty((n, h, d), dtype=torch.bfloat16, device=q.device)
    qo = _heads("q_out", q_out, n, h, d)
    dev = _device_of(q, k, v, k_cache, v_cache, q_start, kv_len, block_table, inv_freq, q_out,
                     *(() if positions is None else (positions,)))
    lib = _lib.load()
    with _on_device(dev):
        st = lib.fd_rope_append(qb, kb, vb, qo, cache, batch,
                                None if positions is None else _ptr(positions), _ptr(inv_freq), rot,
                                int(bool(interleaved)), scale, _stream_handle(stream, dev))
    _lib.check(st)
    return q_out


def paged_attention_scratch(batch: int, total_q: int, q_heads: int, kv_heads: int, head_dim: int,
                            max_q: int, device=None) -> torch.Tensor:
    """A zeroed scratch buffer for ``paged_attention`` calls of at most these sizes; every
    completed call leaves it ready for the next. One per stream (and per graph that may run at
    the same time as another)."""
    n = _lib.load().fd_paged_attention_scratch_bytes(batch, total_q, q_heads, kv_heads, head_dim, max_q)
    if n == 0:
        raise ValueError("paged_attention does not take these sizes (see fd_paged_attention in include/fd.h)")
    return torch.zeros(n, dtype=torch.uint8, device=device if device is not None else "cuda")


def paged_attention(
    q: torch.Tensor,
    k_cache: torch.Tensor,
    v_cache: torch.Tensor,
    q_start: torch.Tensor,
    kv_len: torch.Tensor,
    block_table: torch.Tensor,
    max_q: int,
    scratch: torch.Tensor,
    scale: float | None = None,
    causal: bool = True,
    window: int = 0,
    softcap: float = 0.0,
    out: torch.Tensor | None = None,
    lse: torch.Tensor | None = None,
    stream: torch.cuda.Stream | None = None,
) -> torch.Tensor:
    """out: attention of each sequence's new tokens over its pages (fd_paged_attention in
    include/fd.h).

    q: bf16 [total_q, q_heads, head_dim]; the cache and the batch's index tensors as in
    ``rope_append``; max_q: no sequence has more new tokens (1 when decoding). scratch:
    ``paged_attention_scratch``. scale: of the scores (default head_dim^-0.5). causal: a token
    sees itself and what is before it; window > 0: only the last ``window`` of those; softcap >
    0: scores s become softcap * tanh(s / softcap). out: allocated if None (rows past
    q_start[batch] are then undefined, they are not written); lse: optional float32 [total_q,
    q_heads] output, the log of each row's sum of exponentials. A row that sees no key gives zeros
    and -inf.
    """
    cache, hk, d, _ = _cache(k_cache, v_cache)
    qb = _heads("q", q, None, None, d)
    n, h, _ = q.shape
    if h % hk:
        raise ValueError(f"q has {h} heads: not a multiple of the cache's {hk}")
    if max_q < 0 or window < 0:
        raise ValueError("max_q and window must not be negative")
    batch = _batch(q_start, kv_len, block_table, n, min(max_q, n))
    _check_tensor("scratch", scratch, torch.uint8)
    if out is None:
        out = torch.empty((n, h, d), dtype=torch.bfloat16, device=q.device)
    ob = _heads("out", out, n, h, d)
    more = ()
    if lse is not None:
        _check_tensor("lse", lse, torch.float32, (n, h))
        more = (lse,)
    dev = _device_of(q, k_cache, v_cache, q_start, kv_len, block_table, scratch, out, *more)
    lib = _lib.load()
    with _on_device(dev):
        st = lib.fd_paged_attention(qb, cache, batch, ob, None if lse is None else _ptr(lse),
                                    1.0 / math.sqrt(d) if scale is None else scale, int(bool(causal)),
                                    min(int(window), 2**31 - 1), softcap, _ptr(scratch), scratch.numel(),
                                    _stream_handle(stream, dev))
    _lib.check(st)
    return out
