"""Python binding of the attention half of include/fd.h: rotary positions, the append to a paged
key/value cache and the attention over it. Argument marshalling only, like kernels.py."""

from __future__ import annotations

import ctypes
import struct
import sys

import torch

from . import _lib
from .kernels import _on_device, _stream_handle

# These calls are a few microseconds on the GPU when decoding, so what the host does for them
# counts. Calls whose arguments are plainly in order are made by csrc/fd_torch.cpp (_fast); the
# others, and all where it has not been built, here: checks read each attribute once, structures
# are packed without ctypes objects, and what exactly is wrong with an argument is looked into only
# when something is.

_Tensor, _BF16, _I32 = torch.Tensor, torch.bfloat16, torch.int32

# fd_heads, fd_paged_cache and fd_paged_batch of include/fd.h, packed as the C compiler lays them out
_HEADS = struct.Struct("=Qqqi4x")
_CACHE = struct.Struct("=QQqqqqqqiiii")
_BATCH = struct.Struct("=QQQiiiii4x")

_fast = None  # csrc/fd_torch.cpp, from the first call on (False: not built, or for another torch or Python)


def _load():
    """The library; its first call also loads the C++ form of the calls below."""
    global _fast
    lib = _lib.load()
    if _fast is None:
        try:
            from . import _fd_torch
        except ImportError:
            _fast = False
        else:
            python = getattr(_fd_torch, "python_version", None)
            if _fd_torch.torch_version == torch.__version__ and python == "%d.%d" % sys.version_info[:2]:
                _fd_torch.init(*(ctypes.cast(f, ctypes.c_void_p).value
                                 for f in (lib.fd_rope, lib.fd_rope_append, lib.fd_paged_attention)))
                _fast = _fd_torch
            else:
                _fast = False
    return lib


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _refuse(name: str, t, dtype: torch.dtype, shape, dims: str) -> Exception:
    """What is wrong with tensor argument `name` (`shape`: its sizes, None where any will do)."""
    if not isinstance(t, _Tensor):
        return TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        return ValueError(f"{name} must be a CUDA tensor (the fd kernels have no CPU path)")
    if t.dtype != dtype:
        return TypeError(f"{name} must be {dtype}, got {t.dtype}")
    got = tuple(t.shape)
    if len(got) != len(shape) or any(w is not None and w != g for w, g in zip(shape, got)):
        want = ", ".join("*" if w is None else str(w) for w in shape)
        return ValueError(f"{name} must be {dims} of shape [{want}], got {got}")
    return ValueError(f"{name} must have unit stride along its last dimension and be on the device of the "
                      f"call's other tensors, got strides {t.stride()} on {t.device}")


def _device(t) -> int:
    """The device index of a call's first tensor (-1: not a CUDA tensor, which its own check refuses)."""
    return t.get_device() if isinstance(t, _Tensor) else -1


def _heads(name: str, t: _Tensor, dev: int, n=None, h=None, d=None) -> bytes:
    """The fd_heads of a bf16 [tokens, heads, head_dim] tensor (any token and head strides)."""
    if isinstance(t, _Tensor) and t.dtype is _BF16 and t.get_device() == dev >= 0:
        shape, stride = t.shape, t.stride()
        if len(shape) == 3 and stride[2] == 1 and (n is None or shape[0] == n) and (h is None or shape[1] == h) \
                and (d is None or shape[2] == d):
            return _HEADS.pack(t.data_ptr(), stride[0] if shape[0] > 1 else 0,
                               stride[1] if shape[1] > 1 else 0, shape[1])
    raise _refuse(name, t, _BF16, (n, h, d), "[tokens, heads, head_dim]")


def _new(like: _Tensor, shape: torch.Size, stream) -> tuple[_Tensor, bytes]:
    """A new contiguous bf16 [tokens, heads, head_dim] tensor beside `like`, of the stream that the call
    is made on, and its fd_heads."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _new(like, shape, None)
    # (the likeness of a dense tensor is the cheaper call)
    t = torch.empty_like(like) if like.is_contiguous() else torch.empty(shape, dtype=_BF16, device=like.device)
    n, h, d = shape
    return t, _HEADS.pack(t.data_ptr(), h * d, d, h)


def _flat(name: str, t: _Tensor, dev: int, dtype: torch.dtype, n=None) -> int:
    """The address of a contiguous one-dimensional tensor."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev >= 0:
        shape = t.shape
        if len(shape) == 1 and (n is None or shape[0] == n) and t.is_contiguous():
            return t.data_ptr()
    raise _refuse(name, t, dtype, (n,), "a contiguous vector")


def _cache(k: _Tensor, v: _Tensor, dev: int) -> tuple[bytes, int, int]:
    """(fd_paged_cache, kv_heads, head_dim) of bf16 [num_pages, page_size, kv_heads, head_dim] tensors."""
    if isinstance(k, _Tensor) and isinstance(v, _Tensor) and k.dtype is _BF16 and v.dtype is _BF16 \
            and k.get_device() == dev >= 0 and v.get_device() == dev:
        shape = k.shape
        if len(shape) == 4 and v.shape == shape:
            pages, page, heads, d = shape
            a0, a1, a2, a3 = k.stride()
            b0, b1, b2, b3 = v.stride()
            if a3 == 1 and b3 == 1:
                return (_CACHE.pack(k.data_ptr(), v.data_ptr(), a0, a1, a2, b0, b1, b2, pages, page, heads, d),
                        heads, d)
    for name, t in (("k_cache", k), ("v_cache", v)):
        if not (isinstance(t, _Tensor) and t.dtype is _BF16 and t.get_device() == dev >= 0 and t.dim() == 4
                and t.stride(3) == 1):
            raise _refuse(name, t, _BF16, (None,) * 4, "[num_pages, page_size, kv_heads, head_dim]")
    raise ValueError(f"k_cache and v_cache differ in shape: {tuple(k.shape)}, {tuple(v.shape)}")


def _batch(q_start, kv_len, block_table, dev: int, total_q: int, max_q: int) -> bytes:
    kv = _flat("kv_len", kv_len, dev, _I32)
    batch = kv_len.shape[0]
    start = _flat("q_start", q_start, dev, _I32, batch + 1)
    if isinstance(block_table, _Tensor) and block_table.dtype is _I32 and block_table.get_device() == dev:
        shape, stride = block_table.shape, block_table.stride()
        if len(shape) == 2 and shape[0] == batch and (stride[1] == 1 or shape[1] <= 1):
            return _BATCH.pack(start, kv, block_table.data_ptr(), stride[0] if batch > 1 else shape[1], batch,
                               total_q, max_q, shape[1])
    raise _refuse("block_table", block_table, _I32, (batch, None), "[batch, max_pages]")


def _inv_freq(inv_freq: _Tensor, dev: int, head_dim: int) -> tuple[int, int]:
    ptr = _flat("inv_freq", inv_freq, dev, torch.float64)
    pairs = inv_freq.shape[0]
    if not 1 <= pairs <= head_dim // 2:
        raise ValueError(f"inv_freq must be [rot_dim / 2] with 2 <= rot_dim <= head_dim={head_dim}, got [{pairs}]")
    return ptr, 2 * pairs


def _stream(stream, dev: int) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream_handle(stream, torch.device("cuda", dev)).value


def _call(dev: int, fn, *args):
    """fn(*args) with `dev` as the current device."""
    if dev == torch.cuda.current_device():
        st = fn(*args)
    else:
        with _on_device(torch.device("cuda", dev)):
            st = fn(*args)
    if st:
        _lib.check(st)


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
    if _fast and stream is None:
        r = _fast.rope(q, k, positions, inv_freq, interleaved, scale, q_out, k_out)
        if r is not None:
            return r if r.__class__ is tuple else _lib.check(r)
    lib = _load()
    dev = _device(q)
    qb = _heads("q", q, dev)
    shape = n, _, d = q.shape
    pos = _flat("positions", positions, dev, _I32, n)
    freq, rot = _inv_freq(inv_freq, dev, d)
    kb = ko = None
    if k is not None:
        kb = _heads("k", k, dev, n, None, d)
        if k_out is None:
            k_out, ko = _new(k, k.shape, stream)
        else:
            ko = _heads("k_out", k_out, dev, *k.shape)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if q_out is None:
        q_out, qo = _new(q, shape, stream)
    else:
        qo = _heads("q_out", q_out, dev, *shape)
    _call(dev, lib.fd_rope, qb, kb, qo, ko, pos, freq, n, d, rot, 1 if interleaved else 0, scale,
          _stream(stream, dev))
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
    if _fast and stream is None:
        r = _fast.rope_append(q, k, v, k_cache, v_cache, q_start, kv_len, block_table, inv_freq, positions,
                              interleaved, scale, q_out)
        if r is not None:
            return r if r.__class__ is _Tensor else _lib.check(r)
    lib = _load()
    dev = _device(q)
    cache, hk, d = _cache(k_cache, v_cache, dev)
    qb = _heads("q", q, dev, None, None, d)
    shape = n, _, _ = q.shape
    kb = _heads("k", k, dev, n, hk, d)
    vb = _heads("v", v, dev, n, hk, d)
    freq, rot = _inv_freq(inv_freq, dev, d)
    batch = _batch(q_start, kv_len, block_table, dev, n, n)
    pos = None if positions is None else _flat("positions", positions, dev, _I32, n)
    if q_out is None:
        q_out, qo = _new(q, shape, stream)
    else:
        qo = _heads("q_out", q_out, dev, *shape)
    _call(dev, lib.fd_rope_append, qb, kb, vb, qo, cache, batch, pos, freq, rot,
          1 if interleaved else 0, scale, _stream(stream, dev))
    return q_out


def paged_attention_scratch(batch: int, total_q: int, q_heads: int, kv_heads: int, head_dim: int,
                            max_q: int, device=None) -> torch.Tensor:
    """A zeroed scratch buffer for ``paged_attention`` calls with these heads and head_dim and at
    most these batch, total_q and max_q; every completed call leaves it ready for the next. One per
    stream (and per graph that may run at the same time as another)."""
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
    if _fast and stream is None:
        r = _fast.paged_attention(q, k_cache, v_cache, q_start, kv_len, block_table, max_q, scratch, scale, causal,
                                  window, softcap, out, lse)
        if r is not None:
            return r if r.__class__ is _Tensor else _lib.check(r)
    lib = _load()
    dev = _device(q)
    cache, hk, d = _cache(k_cache, v_cache, dev)
    qb = _heads("q", q, dev, None, None, d)
    shape = n, h, _ = q.shape
    if hk == 0 or h % hk:
        raise ValueError(f"q has {h} heads: not a multiple of the cache's {hk}")
    if max_q < 0 or window < 0:
        raise ValueError("max_q and window must not be negative")
    if softcap and not ctypes.c_float(softcap).value:
        raise ValueError(f"softcap {softcap} is 0, which means none, in 32 bits")
    batch = _batch(q_start, kv_len, block_table, dev, n, min(max_q, n))
    work = _flat("scratch", scratch, dev, torch.uint8)
    if out is None:
        out, ob = _new(q, shape, stream)
    else:
        ob = _heads("out", out, dev, *shape)
    lse_ptr = None
    if lse is not None:
        if not isinstance(lse, _Tensor) or lse.dtype != torch.float32 or lse.get_device() != dev \
                or lse.shape != shape[:2] or not lse.is_contiguous():
            raise _refuse("lse", lse, torch.float32, (n, h), "contiguous [total_q, q_heads]")
        lse_ptr = lse.data_ptr()
    _call(dev, lib.fd_paged_attention, qb, cache, batch, ob, lse_ptr,
          d**-0.5 if scale is None else scale, 1 if causal else 0, min(window, 2**31 - 1), softcap, work,
          scratch.shape[0], _stream(stream, dev))
    return out
