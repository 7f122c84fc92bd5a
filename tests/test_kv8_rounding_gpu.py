"""What the first kernel over a cache in 8 bits rounds: queries to fp16, each row scaled to its largest
element, and probabilities to fp16 with the scales of their values; against 64 bits, and against the
kernel over a bf16 cache of the same values."""

import math

import pytest
import torch

import memory_bound_decode_fd_gb300 as fd
from attn_check import U16, U32
from kv8_batch import E4M3, INT8, Kv8Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [1, 16, 32])
@pytest.mark.parametrize("largest,small", [(1.0, 2.0**-38), (1.0, -(2.0**-38)), (1.0, 1.5 * 2.0**-38), (1.0, 2.0**-39),
                                           (1.9921875, 1.25 * 2.0**-37), (2.0**20, 2.0**-18), (2.0**-60, 2.0**-98),
                                           (2.0**-110, 2.0**-133)])
def test_small_elements_of_queries(cuda_device, dtype, d, hq, largest, small):
    # A row's largest element meets zeros in the keys, the others are 2^-37 to 2^-39 of it (or the smallest that
    # bf16 has) and the keys so large that they decide the score: lse is the score of the one key that there is.
    # An element is off by 2^-39 of the row's largest at most, the sum in 32 bits by d / 16 + 8 steps of 2^-22.
    up = min(-math.frexp(small)[1], 100)  # keys of 2^up: their scale byte stays in range
    scale = 2.0 ** (-math.frexp(small)[1] - up) * 8 / d
    q = torch.full((1, hq, d), small, dtype=torch.float64, device="cuda")
    q[..., 0] = largest
    assert torch.equal(q, q.to(torch.bfloat16).double())
    codes = torch.ones(1, 16, 1, d, device="cuda")
    codes[..., 0] = 0
    codes = codes.to(dtype)
    scales = torch.full((1, 1, 1), 127 + up, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    scratch = fd.paged_attention_scratch(1, 1, hq, 1, d, 1)
    lse = torch.empty(1, hq, device="cuda")
    fd.paged_attention_kv8(q.to(torch.bfloat16), codes, codes, scales, scales, torch.tensor([0, 1], **i32),
                           torch.tensor([1], **i32), torch.zeros(1, 1, **i32), 1, scratch, scale=scale, lse=lse)
    k = codes[0, 0, 0].double() * 2.0**up
    want = scale * (q[0] @ k)
    mag = float(scale * (q[0].abs() @ k.abs()).max())
    bound = scale * largest * 2.0**-39 * float(k.sum()) + mag * ((d / 16 + 8) * 2.0**-22 + 4 * U32)
    assert float((lse[0].double() - want).abs().max()) <= bound


def parts(b, softmax_scale):
    """Per sequence and key head: reference, sum of p |v|, and what of a probability is off beside its rounding."""
    row = 0
    for t, keys, values in zip(b.kv_lens, b.keys, b.values):
        q = b.q[row].double().view(b.hk, b.hq // b.hk, b.d)
        for h in range(b.hk):
            k, v = keys[:, h].double(), values[:, h].double()
            s = q[h] @ k.T * softmax_scale
            mag = (q[h].abs() @ k.abs().T).amax(-1) * softmax_scale
            flat = q[h].abs().amax(-1) * k.abs().sum(-1).amax() * softmax_scale * 2.0**-39
            # scores; the exponents' rounding, of the sum's and of the values' own maximum; a factor each time that
            # a maximum grows, at most once a tile, and when the warps meet; sums of t terms
            dp = mag * (b.d / 16 + 8) * 2.0**-22 + flat + (4 * s.abs().amax(-1) + 512) * U32 + (t / 256 + 8) * 2.0**-20 + t * 2.0**-26
            p = torch.softmax(s, -1)
            floor = 2.0**-40 * t * (p * v.abs().amax(-1)).amax(-1)
            yield (row, h), p @ v, p @ v.abs(), dp, floor
        row += 1


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (16, 1, 64), (32, 1, 128)])
@pytest.mark.parametrize("gains", [0.0, 1.0])
def test_results_of_single_tokens(cuda_device, dtype, hq, hk, d, gains):
    # to 64 bits, and to the kernel over a bf16 cache that holds the same values (which are exact in bf16)
    b = Kv8Batch(hq, hk, d, [1] * 5, [700, 90, 1, 17, 3000], dtype=dtype, seed=10, gains=gains)
    scratch = fd.paged_attention_scratch(5, 5, hq, hk, d, 1)
    k, v = (torch.zeros(c.shape, dtype=torch.bfloat16, device="cuda") for c in (b.k_cache, b.v_cache))
    for s, (pg, off) in enumerate(b.slots):
        k[pg, off], v[pg, off] = b.keys[s].to(torch.bfloat16), b.values[s].to(torch.bfloat16)
        assert torch.equal(k[pg, off].double(), b.keys[s]) and torch.equal(v[pg, off].double(), b.values[s])
    got = fd.paged_attention_kv8(b.q, *b.args(), 1, scratch).double().view(5, hk, hq // hk, d)
    over_bf16 = fd.paged_attention(b.q, k, v, b.q_start, b.kv_len, b.block_table, 1, scratch).double().view(5, hk, hq // hk, d)
    for at, ref, room, dp, floor in parts(b, 1 / math.sqrt(d)):
        # one rounding of the result (2^-8), probabilities in fp16 (2^-11, the smallest step apart), the sum's error
        own = U16 * ref.abs() + ((2.0**-11 + 2 * dp) * (1 + 2.0**-6))[:, None] * room + floor[:, None]
        assert bool(((got[at] - ref).abs() <= own).all()), at
        other = U16 * ref.abs() + ((U16 + 2 * dp) * (1 + 2.0**-6))[:, None] * room
        assert bool(((got[at] - over_bf16[at]).abs() <= own + other).all()), at
