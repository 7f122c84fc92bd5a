"""Angles of rotary positions at both ends of the positions and at frequencies of many turns, against
exact ones: products and remainders in fractions, pi to 60 digits.

The positions are those, of many, whose cosine is nearest to 0, where a bf16 result has digits to
show an angle's error by; the bound is the rounding of the result and the 1e-6 radians that the angle may
be off by."""

import math
import random
from fractions import Fraction

import pytest
import torch

import memory_bound_decode_fd_gb300 as fd
from attn_check import U16

pytestmark = pytest.mark.gpu

TURNS_OF_RADIAN = 1 / (2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459"))
FREQS = [1.0, 2.9, 7.5, -31.7, 1000.0, 123456.789, 1e9, -1e15]


def angle(position, freq):
    """position * freq radians, less whole turns."""
    t = position * Fraction(freq) * TURNS_OF_RADIAN
    return float(t - round(t)) * 2 * math.pi


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("append", [False, True])
def test_angles_near_their_cosines_zeros(cuda_device, interleaved, append):
    rng = random.Random(7)
    positions = []
    for f in FREQS:
        some = [rng.choice((1, -1)) * rng.randrange(2**31 - 2**24, 2**31) for _ in range(3000)]
        some.sort(key=lambda p: abs(math.cos(angle(p, f))))
        positions += some[:8]
    n, half, d = len(positions), len(FREQS), 64
    ref = torch.tensor([[[math.cos(angle(p, f)) for f in FREQS], [math.sin(angle(p, f)) for f in FREQS]]
                        for p in positions], dtype=torch.float64)
    p0 = torch.arange(half) * 2 if interleaved else torch.arange(half)
    p1 = p0 + 1 if interleaved else p0 + half
    x = torch.zeros(n, 1, d, dtype=torch.bfloat16)
    x[..., p0] = 1.0
    x = x.cuda()
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    freq = torch.tensor(FREQS, dtype=torch.float64, device="cuda")
    if append:
        cache = [torch.zeros(1, 64, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
        start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        out = fd.rope_append(x, x, x, *cache, start, start[1:], table, freq, positions=pos, interleaved=interleaved)
        assert torch.equal(cache[0][0, :n], out)
    else:
        out = fd.rope(x, None, pos, freq, interleaved=interleaved)[0]
    out = out.double().cpu()[:, 0]
    for got, want in ((out[:, p0], ref[:, 0]), (out[:, p1], ref[:, 1])):
        err = (got - want).abs() - U16 * want.abs()
        assert bool((err <= 1e-6).all()), [float(e) for e in err.amax(0)]
