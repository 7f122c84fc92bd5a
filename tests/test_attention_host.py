"""Host-side tests (no GPU) of rotary positions, the cache append and paged attention: every
refusal comes before any CUDA call, frequencies follow their formulas, the references the GPU
tests compare with agree with a second way of computing them."""

import ctypes
import math
import re
from pathlib import Path

import pytest
import torch

import memory_bound_decode_fd_gb300 as fd
from attn_check import Batch, check_attention, check_rope
from memory_bound_decode_fd_gb300 import _lib, attention

HEADER = Path(__file__).resolve().parent.parent / "include" / "fd.h"

# Fake device addresses, far apart; nothing is dereferenced.
Q, K, V, O, P, F, KC, VC, QS, KL, BT, L, S = (0x100000000000 + i * 0x1000000000 for i in range(13))
NULL, SHAPE, ALIGN, UNSUP, OVER, OK = (_lib.FD_ERR_NULL, _lib.FD_ERR_SHAPE, _lib.FD_ERR_ALIGN,
                                       _lib.FD_ERR_UNSUPPORTED, _lib.FD_ERR_OVERLAP, _lib.FD_OK)
BIG = 1 << 40


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ts", ctypes.c_longlong), ("hs", ctypes.c_longlong),
                ("heads", ctypes.c_int)]


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (n, ctypes.c_longlong) for n in ("kp", "kt", "kh", "vp", "vt", "vh")] + [
        (n, ctypes.c_int) for n in ("pages", "page", "heads", "d")]


class PagedBatch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q_start", "kv_len", "table")] + [
        (n, ctypes.c_int) for n in ("stride", "batch", "total_q", "max_q", "max_pages")]


def heads(data, ts=4096, hs=128, n=32):
    return Heads(data, ts, hs, n)


def cache(**kw):
    c = dict(k=KC, v=VC, kp=16 * 1024, kt=1024, kh=128, vp=16 * 1024, vt=1024, vh=128, pages=100, page=16,
             heads=8, d=128)
    c.update(kw)
    return Cache(*[c[n] for n, _ in Cache._fields_])


def batch(**kw):
    c = dict(q_start=QS, kv_len=KL, table=BT, stride=10, batch=4, total_q=8, max_q=4, max_pages=10)
    c.update(kw)
    return PagedBatch(*[c[n] for n, _ in PagedBatch._fields_])


@pytest.fixture
def no_launch(fdlib):
    """Calls that pass every check end as a failed launch, without calling CUDA."""
    prev = fdlib.fd_get_launch_flags()
    fdlib.fd_set_launch_flags(prev | _lib.FD_LAUNCH_TEST_FAIL)
    yield fdlib
    fdlib.fd_set_launch_flags(prev)


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_structures_match_the_packed_ones():
    assert ctypes.sizeof(Heads) == attention._HEADS.size == 32
    assert ctypes.sizeof(Cache) == attention._CACHE.size == 80
    assert ctypes.sizeof(PagedBatch) == attention._BATCH.size == 48
    assert bytes(heads(Q, 8, 16, 3))[:28] == attention._HEADS.pack(Q, 8, 16, 3)[:28]
    assert bytes(cache()) == attention._CACHE.pack(*[getattr(cache(), n) for n, _ in Cache._fields_])
    assert bytes(batch())[:44] == attention._BATCH.pack(*[getattr(batch(), n) for n, _ in PagedBatch._fields_])[:44]


def test_header_constants_match_binding():
    text = HEADER.read_text()
    for name in ("FD_MAX_PAGE_SIZE", "FD_MAX_BATCH", "FD_MAX_HEADS", "FD_MAX_ROPE_DIM", "FD_MAX_SEQ",
                 "FD_DEVICE_STATUS_BAD_PAGE"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(_lib, name)


def rope(lib, q=heads(Q), k=heads(K, 1024, 128, 8), qo=heads(O), ko=heads(V, 1024, 128, 8), pos=P, f=F,
         tokens=4, d=128, rot=128, scale=1.0):
    return lib.fd_rope(ref(q), ref(k), ref(qo), ref(ko), pos, f, tokens, d, rot, 0, scale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(), _lib.FD_ERR_CUDA),
    (dict(k=None, ko=None), _lib.FD_ERR_CUDA),
    (dict(qo=heads(Q), ko=heads(K, 1024, 128, 8)), _lib.FD_ERR_CUDA),            # in place
    (dict(q=heads(Q, 6144), k=heads(Q + 8192, 6144, 128, 8), qo=heads(Q, 6144),
          ko=heads(Q + 8192, 6144, 128, 8)), _lib.FD_ERR_CUDA),                   # in place, parts of one row
    (dict(q=heads(Q, 0)), _lib.FD_ERR_CUDA),                                      # an input may repeat
    (dict(tokens=0, q=None, qo=None), OK),
    (dict(tokens=-1), SHAPE), (dict(d=100, rot=64), SHAPE), (dict(rot=3), SHAPE), (dict(rot=0), SHAPE),
    (dict(rot=130), SHAPE), (dict(scale=math.inf), SHAPE), (dict(scale=math.nan), SHAPE),
    (dict(q=None), NULL), (dict(ko=None), NULL), (dict(k=None), NULL), (dict(pos=None), NULL), (dict(f=None), NULL),
    (dict(q=heads(None)), NULL),
    (dict(d=264, rot=64), UNSUP), (dict(tokens=1 << 29), UNSUP), (dict(q=heads(Q, 4096, 128, 1025)), UNSUP),
    (dict(q=heads(Q, BIG)), UNSUP),
    (dict(q=heads(Q, 4100)), SHAPE), (dict(q=heads(Q, -4096)), SHAPE), (dict(q=heads(Q, n=0)), SHAPE),
    (dict(qo=heads(O, n=16)), SHAPE),
    (dict(q=heads(Q + 8)), ALIGN), (dict(ko=heads(V + 2, 1024, 128, 8)), ALIGN), (dict(pos=P + 2), ALIGN),
    (dict(f=F + 4), ALIGN),
    (dict(qo=heads(O, 0)), OVER), (dict(qo=heads(O, 4096, 64)), OVER), (dict(qo=heads(O, 2048)), OVER),
    (dict(qo=heads(Q + 16)), OVER), (dict(qo=heads(Q, 8192)), OVER), (dict(ko=heads(O, 1024, 128, 8)), OVER),
    (dict(ko=heads(Q, 1024, 128, 8)), OVER), (dict(qo=heads(K)), OVER), (dict(pos=O + 64), OVER), (dict(f=O + 64), OVER),
    # parts of one row that overlap by a head
    (dict(q=heads(Q, 6144), qo=heads(Q, 6144), k=heads(Q + 8192 - 256, 6144, 128, 8),
          ko=heads(Q + 8192 - 256, 6144, 128, 8)), OVER),
])
def test_rope_refusals(no_launch, kw, status):
    assert rope(no_launch, **kw) == status


def append(lib, q=heads(Q), k=heads(K, 1024, 128, 8), v=heads(V, 1024, 128, 8), qo=heads(O), c=cache(),
           b=batch(), pos=None, f=F, rot=128, scale=1.0):
    return lib.fd_rope_append(ref(q), ref(k), ref(v), ref(qo), ref(c), ref(b), pos, f, rot, 0, scale, None)


FUSED = 2 * 16 * 1024  # keys and values of a page side by side


@pytest.mark.parametrize("kw,status", [
    (dict(), _lib.FD_ERR_CUDA), (dict(qo=heads(Q)), _lib.FD_ERR_CUDA), (dict(pos=P), _lib.FD_ERR_CUDA),
    (dict(c=cache(kh=16 * 128, kt=128, vh=16 * 128, vt=128)), _lib.FD_ERR_CUDA),          # heads before tokens
    (dict(c=cache(v=KC + FUSED, kp=FUSED, vp=FUSED)), _lib.FD_ERR_CUDA),
    (dict(c=cache(v=KC + 2048, kt=2048, vt=2048, kp=FUSED, vp=FUSED)), _lib.FD_ERR_CUDA),  # K and V of a token
    (dict(b=batch(total_q=0), q=None), OK), (dict(b=batch(batch=0), q=None), OK),
    (dict(c=None), NULL), (dict(b=None), NULL), (dict(q=None), NULL), (dict(v=None), NULL), (dict(f=None), NULL),
    (dict(c=cache(k=None)), NULL), (dict(b=batch(q_start=None)), NULL), (dict(b=batch(table=None)), NULL),
    (dict(rot=130), SHAPE), (dict(rot=7), SHAPE), (dict(scale=math.nan), SHAPE),
    (dict(c=cache(page=24)), SHAPE), (dict(c=cache(page=8)), SHAPE), (dict(c=cache(pages=0)), SHAPE),
    (dict(c=cache(page=2048)), UNSUP), (dict(c=cache(d=96), rot=64), UNSUP),
    (dict(c=cache(kt=1020)), SHAPE), (dict(c=cache(kt=0)), SHAPE), (dict(c=cache(kp=16 * 1024 + 8)), SHAPE),
    (dict(c=cache(vp=BIG)), UNSUP),
    (dict(c=cache(k=KC + 8)), ALIGN), (dict(c=cache(heads=4)), SHAPE), (dict(k=heads(K, 1024, 128, 4)), SHAPE),
    (dict(b=batch(batch=-1)), SHAPE), (dict(b=batch(stride=9)), SHAPE), (dict(b=batch(batch=4097)), UNSUP),
    (dict(b=batch(max_pages=1 << 21, stride=1 << 21)), UNSUP), (dict(b=batch(kv_len=KL + 2)), ALIGN),
    (dict(c=cache(kp=8 * 1024)), OVER),                      # pages over one another
    (dict(c=cache(v=KC)), OVER), (dict(c=cache(v=KC + 1024)), OVER),
    (dict(c=cache(v=KC + FUSED - 2048, kp=FUSED, vp=FUSED)), OVER),
    (dict(c=cache(k=Q)), OVER), (dict(c=cache(v=O + 64)), OVER), (dict(qo=heads(V)), OVER),
    (dict(qo=heads(Q + 256)), OVER),
])
def test_append_refusals(no_launch, kw, status):
    assert append(no_launch, **kw) == status


def attend(lib, q=heads(Q), c=cache(), b=batch(), o=heads(O), lse=L, scale=0.1, window=0, cap=0.0, s=S, n=None):
    need = lib.fd_paged_attention_scratch_bytes(4, 8, 32, 8, 128, 4)
    return lib.fd_paged_attention(ref(q), ref(c), ref(b), ref(o), lse, scale, 1, window, cap, s,
                                  need if n is None else n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(), _lib.FD_ERR_CUDA), (dict(lse=None), _lib.FD_ERR_CUDA), (dict(window=5, cap=30.0), _lib.FD_ERR_CUDA),
    (dict(c=cache(v=KC)), _lib.FD_ERR_CUDA),                # one tensor as both is fine to read
    (dict(b=batch(total_q=0), q=None, s=None), OK), (dict(b=batch(batch=0), o=None), OK),
    (dict(q=None), NULL), (dict(o=None), NULL), (dict(s=None), NULL), (dict(c=None), NULL), (dict(b=None), NULL),
    (dict(scale=math.inf), SHAPE), (dict(window=-1), SHAPE), (dict(cap=-1.0), SHAPE), (dict(cap=math.nan), SHAPE),
    (dict(scale=2e30), UNSUP), (dict(scale=-2e30), UNSUP), (dict(cap=2e30), UNSUP), (dict(cap=1e-32), UNSUP),
    (dict(b=batch(max_q=0), q=None, o=None), OK),
    (dict(cap=math.inf), SHAPE), (dict(n=1000), SHAPE), (dict(q=heads(Q, 4096, 128, 20), o=heads(O, 4096, 128, 20)), SHAPE),
    (dict(o=heads(O, n=16)), SHAPE), (dict(c=cache(page=48)), SHAPE), (dict(b=batch(max_q=-1)), SHAPE),
    (dict(c=cache(d=256)), UNSUP), (dict(s=S + 8), ALIGN), (dict(lse=L + 2), ALIGN), (dict(q=heads(Q + 4)), ALIGN),
    (dict(o=heads(Q)), OVER), (dict(o=heads(O, 0)), OVER), (dict(o=heads(KC)), OVER), (dict(o=heads(VC + 256)), OVER),
    (dict(lse=O + 64), OVER), (dict(lse=Q), OVER), (dict(lse=KC), OVER), (dict(s=Q), OVER), (dict(s=O), OVER),
    (dict(s=KC), OVER), (dict(lse=S + 16), OVER),
])
def test_attention_refusals(no_launch, kw, status):
    assert attend(no_launch, **kw) == status


def test_scratch_sizes(fdlib):
    f = fdlib.fd_paged_attention_scratch_bytes
    assert f(1, 1, 32, 8, 128, 1) > 0 and f(0, 0, 8, 8, 64, 0) > 0
    for bad in ((-1, 1, 8, 8, 64, 1), (4097, 1, 8, 8, 64, 1), (1, 1, 9, 8, 64, 1), (1, 1, 8, 8, 96, 1),
                (1, 1, 0, 8, 64, 1), (1, 1, 8, 0, 64, 1), (1, -1, 8, 8, 64, 1), (1, 1, 2048, 8, 64, 1)):
        assert f(*bad) == 0
    with pytest.raises(ValueError):
        fd.paged_attention_scratch(1, 1, 8, 8, 96, 1)
    # room for the smaller call in the larger one's scratch
    assert f(4, 8, 32, 8, 128, 4) >= f(3, 5, 16, 4, 128, 2)


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pos, f = torch.zeros(2, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    c = torch.zeros(3, 16, 4, 64, dtype=torch.bfloat16)
    ix = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fd.rope(q, q, pos, f)
    with pytest.raises(ValueError, match="CUDA"):
        fd.rope_append(q, q, q, c, c, ix, ix[:1], ix[None], f)
    with pytest.raises(ValueError, match="CUDA"):
        fd.paged_attention(q, c, c, ix, ix[:1], ix[None], 1, torch.zeros(8, dtype=torch.uint8))


# ------------------------------------------------------------------------------ frequencies


def test_inv_freq_plain_and_linear():
    f, m = fd.rope_inv_freq(8, 10000.0)
    assert m == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14, atol=0)
    g, m = fd.rope_inv_freq(8, 10000.0, "linear", 4.0)
    assert m == 1.0 and torch.equal(g * 4, f)


def test_inv_freq_banded():
    f, _ = fd.rope_inv_freq(128, 500000.0)
    g, m = fd.rope_inv_freq(128, 500000.0, "banded", 8.0, 8192)
    turns = 8192 * f / (2 * math.pi)
    assert m == 1.0
    assert torch.equal(g[turns > 4], f[turns > 4]) and torch.equal(g[turns < 1], f[turns < 1] / 8)
    mid = (turns >= 1) & (turns <= 4)
    assert mid.any() and bool((g[mid] <= f[mid]).all()) and bool((g[mid] >= f[mid] / 8).all())
    s = (turns[mid] - 1) / 3
    assert torch.allclose(g[mid], (1 - s) * f[mid] / 8 + s * f[mid], rtol=1e-14, atol=0)


def test_inv_freq_ramp():
    f, _ = fd.rope_inv_freq(64, 10000.0)
    g, m = fd.rope_inv_freq(64, 10000.0, "ramp", 16.0, 4096)
    assert m == pytest.approx(0.1 * math.log(16) + 1)
    pair = lambda n: 64 * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(10000))  # noqa: E731
    lo, hi = math.floor(pair(32)), math.ceil(pair(1))
    i = torch.arange(32)
    assert torch.equal(g[i <= lo], f[i <= lo])
    assert torch.allclose(g[i >= hi], f[i >= hi] / 16, rtol=1e-14, atol=0)
    assert bool((g.diff() < 0).all())


@pytest.mark.parametrize("kw", [dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, base=1.0),
                                dict(rot_dim=8, scaling="other"), dict(rot_dim=8, scaling="linear", factor=0.5),
                                dict(rot_dim=8, scaling="banded", factor=2.0, low=4.0, high=1.0),
                                dict(rot_dim=8, scaling="ramp", factor=math.inf)])
def test_inv_freq_refusals(kw):
    with pytest.raises(ValueError):
        fd.rope_inv_freq(**kw)


# --------------------------------------------------------- the references of the GPU tests


def test_rope_reference_keeps_lengths_and_angles():
    x = torch.randn(5, 2, 16, dtype=torch.float64).to(torch.bfloat16)
    pos = torch.tensor([0, 1, 7, 100000, -4])
    f, _ = fd.rope_inv_freq(16)
    z = torch.complex(x.double()[..., :8], x.double()[..., 8:])
    z = z * torch.exp(1j * pos.double()[:, None, None] * f)
    check_rope(torch.cat((z.real, z.imag), -1).to(torch.bfloat16), x, pos, f, 16, False, 1.0)
    with pytest.raises(AssertionError):  # one position off
        check_rope(torch.cat((z.real, z.imag), -1).to(torch.bfloat16), x, pos + 1, f, 16, False, 1.0)


@pytest.mark.parametrize("kw", [dict(), dict(window=5), dict(cap=3.0), dict(causal=False)])
def test_attention_reference_against_loops(kw):
    b = Batch(4, 2, 64, [3, 1, 4], [20, 1, 2], device="cpu", fused_kv=True)
    out, lse = torch.zeros_like(b.q), torch.zeros(8, 4)
    row = 0
    for s, (n, t) in enumerate(zip(b.q_lens, b.kv_lens)):
        for i in range(n):
            p = t - n + i
            for h in range(4):
                keys = [j for j in range(t) if (kw.get("causal", True) is False or j <= p) and
                        (not kw.get("window") or j > p - kw["window"])]
                sc = [float(b.q[row, h].double() @ b.keys[s][j, h // 2].double()) / 8 for j in keys]
                if kw.get("cap"):
                    sc = [kw["cap"] * math.tanh(x / kw["cap"]) for x in sc]
                e = [math.exp(x) for x in sc]
                lse[row, h] = math.log(sum(e)) if e else -math.inf
                if e:
                    out[row, h] = sum(x * b.values[s][j, h // 2].double() for x, j in zip(e, keys)) / sum(e)
            row += 1
    check_attention(b, out, lse, **kw)
    wrong = out.clone()
    wrong[0, 1] += 0.1
    with pytest.raises(AssertionError):
        check_attention(b, wrong, lse, **kw)
