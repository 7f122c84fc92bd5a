"""What the first kernel over a cache in 8 bits rounds: queries to fp16, each row scaled to its largest
element."""

import math

import pytest
import torch

import memory_bound_decode_fd_gb300 as fd
from attn_check import U32
from kv8_batch import E4M3, INT8

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
