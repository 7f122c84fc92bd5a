"""Capped scores against 64 bits, with bounds that follow the scores, whatever the cap.

The bounds of attn_check.py, but for the cap's own error: cap and tanh take a score to within
16 u32 of its size (u32 = 2^-24; below the cap: the factors' roundings and a polynomial, 8 u32 at most;
above it: of tanh >= 0.76 the argument's rounding 1.3 u32, ex2.approx 0.9, the quotient's two units 4
and the sums 3, less than 13 u32 in all). So
dp = ds + 17 u32 max|s| + 2^-21 + n 2^-26, where attn_check.py has 8 u32 c + u32 max|s|."""

import math

import pytest
import torch

import memory_bound_decode_fd_gb300 as fd
from attn_check import U16, U32, Batch
from memory_bound_decode_fd_gb300 import attention

pytestmark = pytest.mark.gpu


def check(b, cap, scale=None, window=0):
    scale = 1.0 / math.sqrt(b.d) if scale is None else scale
    n, h, d = b.q.shape
    scratch = fd.paged_attention_scratch(len(b.q_lens), n, b.hq, b.hk, b.d, b.max_q)
    lse = torch.full((n, h), 5.0, device="cuda")
    fd.device_status()
    out = fd.paged_attention(b.q, *b.args(), b.max_q, scratch, scale=scale, softcap=cap, window=window, lse=lse)
    assert fd.device_status() == 0
    g = b.hq // b.hk
    row = 0
    for nq, t, k, v in zip(b.q_lens, b.kv_lens, b.keys, b.values):
        q = b.q[row:row + nq].double().view(nq, b.hk, g, d)
        k, v = k.double(), v.double()
        i = torch.arange(t - nq, t, device="cuda")[:, None]
        j = torch.arange(t, device="cuda")[None, :]
        seen = (j <= i) & (j > i - (window or 1 << 30))
        s = torch.einsum("nhgd,thd->nhgt", q, k) * scale
        mag = torch.einsum("nhgd,thd->nhgt", q.abs(), k.abs()) * abs(scale)
        s = cap * torch.tanh(s / cap)
        hidden = ~seen[:, None, None, :]
        big = s.masked_fill(hidden, 0.0).abs().amax(-1)
        ds = mag.masked_fill(hidden, 0.0).amax(-1) * (d / 16 + 8) * 2.0**-22
        dp = ds + 17 * U32 * big + 2.0**-21 + t * 2.0**-26
        s = s.masked_fill(hidden, -math.inf)
        l = torch.logsumexp(s, -1)
        p = torch.exp(s - l[..., None])
        ref, room = torch.einsum("nhgt,thd->nhgd", p, v), torch.einsum("nhgt,thd->nhgd", p, v.abs())
        bound = U16 * ref.abs() + ((U16 + 2 * dp) * (1 + 2.0**-6))[..., None] * room
        err = (out[row:row + nq].double().view(nq, b.hk, g, d) - ref).abs()
        e = (lse[row:row + nq].double().view(nq, b.hk, g) - l).abs()
        row += nq
        assert bool((e <= dp + 4 * U32 * l.abs()).all()), ("lse", nq, t, float((e / dp).max()))
        assert bool((err <= bound).all()), ("out", nq, t, float((err - bound).max()))


# rows of one pass of the decoding kernel (with a negative scale several), and chunks
SHAPES = [([1, 1, 1], [1, 5, 400], 0.3), ([1, 1], [4097, 130], None), ([9], [40], -0.2)]
CHUNKS = [([40, 1], [40, 300], 0.3), ([90, 300], [400, 300], None)]


@pytest.mark.parametrize("cap", [1e4, 1e5, 1e7, 1e10, 1e30])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens,scale", SHAPES)
def test_caps_far_above_the_scores_of_tokens(cuda_device, q_lens, kv_lens, scale, d, cap):
    check(Batch(8, 2, d, q_lens, kv_lens, 16, seed=41, q_std=2.0), cap, scale)
    check(Batch(8, 2, d, q_lens, kv_lens, 16, seed=42, q_std=2.0), cap, scale, window=1)


@pytest.mark.parametrize("cap", [5.0, 1e4, 1e7, 1e10, 1e30])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens,scale", CHUNKS)
def test_caps_far_above_the_scores_of_chunks(cuda_device, q_lens, kv_lens, scale, d, cap):
    # ordinary scores, and ones of about 100 (of which 2^s does not fit 32 bits)
    for std in (2.0, 40.0):
        check(Batch(8, 2, d, q_lens, kv_lens, 16, seed=43, q_std=std), cap, scale)


@pytest.mark.parametrize("q_lens,kv_lens", [([4], [60]), ([40], [90])])
@pytest.mark.parametrize("d", [64, 128])
def test_small_scores_beside_ones_past_the_cap(cuda_device, q_lens, kv_lens, d):
    # one token's scores pass the cap, the other rows' are ordinary: these lose nothing by it
    b = Batch(4, 1, d, q_lens, kv_lens, 16, seed=44)
    b.q[1] *= 65536.0
    check(b, 1e4)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [3, 300]), ([40], [90])])
@pytest.mark.parametrize("d", [64, 128])
def test_scale_far_below_the_cap(cuda_device, q_lens, kv_lens, d):
    # scale / cap is no 32-bit number, the scores are ordinary
    check(Batch(8, 2, d, q_lens, kv_lens, 16, seed=45, q_std=2.0**60), 1e30, 2.0**-60 / math.sqrt(d))


@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("cap", [1e-46, -1e-46, 5e-324])
def test_a_cap_that_32_bits_take_for_none_is_refused(cuda_device, monkeypatch, cap, fast):
    attention._load()
    if not fast:
        monkeypatch.setattr(attention, "_fast", False)
    b = Batch(4, 2, 64, [1, 1], [20, 30])
    scratch = fd.paged_attention_scratch(2, 2, 4, 2, 64, 1)
    with pytest.raises(ValueError, match="softcap"):
        fd.paged_attention(b.q, *b.args(), 1, scratch, softcap=cap)
