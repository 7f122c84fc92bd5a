"""Plain 64-bit references of rotary positions and paged attention, and the bounds that the
kernels' arithmetic gives.

Bounds, per element (u16 = 2^-8, half a bf16 step relative to the value; u32 = 2^-24):
  * rope: the angle is off by less than 1e-6 (2^-24 of a half turn, pi 2^-24 < 2e-7 radians, and
    sincospif's few u32), two products and a sum in 32 bits, one rounding:
    |y - ref| <= u16 |ref| + 2e-6 scale (|x0| + |x1|).
  * attention: a score is a sum of d products in 32 bits, in steps of 16 that may truncate (2^-22
    of the running magnitude each, as for the library's other tensor-core sums):
    ds = |scale| max_j sum_d |q_d k_jd| (d / 16 + 8) 2^-22. With a cap c the score passes through
    c (1 - 2 / (e^2y + 1)), whose error is below 8 u32 c. Probabilities, relative: the exponent's
    error, ex2.approx (2^-22) and the exponent's own rounding (|s| u32, times ln 2 <= 1), on
    top of that u16 for the rounding to bf16 that only the numerator has; the denominator again
    without it; the sums of n terms in 32 bits, in steps of 16 in order, n / 16 2^-22:
    |o - ref| <= u16 |ref| + (u16 + 2 dp) (1 + 2^-6) sum_j p_j |v_j|,
    dp = ds + 8 u32 c + max|s| u32 + 2^-21 + n 2^-26.
    lse: |l - ref| <= dp + 4 u32 |ref|.
"""

from __future__ import annotations

import math

import torch

U16, U32 = 2.0**-8, 2.0**-24


def rope_ref(x, positions, inv_freq, rot, interleaved, scale):
    """(ref, |x0| + |x1| per element) in float64 of x [tokens, heads, d]."""
    x = x.double()
    a = positions.double()[:, None, None] * inv_freq.double()[None, None, :]
    c, s = torch.cos(a) * scale, torch.sin(a) * scale
    i = torch.arange(rot // 2, device=x.device)
    p0, p1 = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., p0] = x[..., p0] * c - x[..., p1] * s
    y[..., p1] = x[..., p0] * s + x[..., p1] * c
    mag[..., p0] = mag[..., p1] = x[..., p0].abs() + x[..., p1].abs()
    return y, mag


def check_rope(got, x, positions, inv_freq, rot, interleaved, scale):
    ref, mag = rope_ref(x, positions, inv_freq, rot, interleaved, scale)
    bound = U16 * ref.abs() + 2e-6 * abs(scale) * mag
    bound[..., rot:] = 0.0  # copied
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


class Batch:
    """A cache of `pages` pages and a batch over it; every place that no sequence has a token
    in holds NaN, and unneeded entries of the table lie far outside the cache."""

    def __init__(self, hq, hk, d, q_lens, kv_lens, page=16, head_major=False, seed=0, device="cuda",
                 spare_rows=0, q_std=1.0, fused_kv=False, max_pages=None):
        g = torch.Generator(device=device).manual_seed(seed)
        self.hq, self.hk, self.d, self.page, self.device = hq, hk, d, page, device
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        counts = [(t + page - 1) // page for t in kv_lens]
        n_pages = max(1, sum(counts)) + 2
        order = torch.randperm(n_pages, generator=g, device=device).tolist()
        width = max(max(counts), 1) if max_pages is None else max_pages
        table = torch.full((len(q_lens), width), 1 << 30, dtype=torch.int32)
        at = 0
        self.slots = []  # per sequence: (pages, places) of its tokens
        for b, (t, c) in enumerate(zip(kv_lens, counts)):
            mine = order[at:at + c]
            at += c
            table[b, :c] = torch.tensor(mine, dtype=torch.int32)
            pos = torch.arange(t, device=device)
            self.slots.append((torch.tensor(mine + [0], device=device)[pos // page], pos % page))
        self.block_table = table.to(device)
        self.q_start = torch.tensor([sum(q_lens[:i]) for i in range(len(q_lens) + 1)], dtype=torch.int32,
                                    device=device)
        self.kv_len = torch.tensor(kv_lens, dtype=torch.int32, device=device)
        self.max_q = max(max(q_lens), 1)

        def normal(*shape, std=1.0):
            return torch.empty(shape, dtype=torch.bfloat16, device=device).normal_(0, std, generator=g)

        shape = (n_pages, hk, page, d) if head_major else (n_pages, page, hk, d)
        if fused_kv:
            buf = torch.full((n_pages, 2) + shape[1:], float("nan"), dtype=torch.bfloat16, device=device)
            caches = [buf[:, 0], buf[:, 1]]
        else:
            caches = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device=device) for _ in range(2)]
        self.k_cache, self.v_cache = (c.transpose(1, 2) if head_major else c for c in caches)
        self.keys, self.values = [], []
        for t, (pg, off) in zip(kv_lens, self.slots):
            k, v = normal(t, hk, d), normal(t, hk, d)
            self.k_cache[pg, off], self.v_cache[pg, off] = k, v
            self.keys.append(k)
            self.values.append(v)
        self.q = normal(sum(q_lens) + spare_rows, hq, d, std=q_std)

    def args(self):
        return self.k_cache, self.v_cache, self.q_start, self.kv_len, self.block_table


def check_attention(b: Batch, out, lse=None, scale=None, causal=True, window=0, cap=0.0):
    """Every row of `out` (and `lse`) against the 64-bit definition."""
    scale = 1.0 / math.sqrt(b.d) if scale is None else scale
    g = b.hq // b.hk
    row = 0
    for n, t, k, v in zip(b.q_lens, b.kv_lens, b.keys, b.values):
        q = b.q[row:row + n].double().view(n, b.hk, g, b.d)
        got = out[row:row + n].double().view(n, b.hk, g, b.d)
        got_l = None if lse is None else lse[row:row + n].double().view(n, b.hk, g)
        row += n
        if n == 0:
            continue
        i = torch.arange(t - n, t, device=b.device)[:, None]
        j = torch.arange(t, device=b.device)[None, :]
        seen = torch.ones((n, t), dtype=torch.bool, device=b.device)
        if causal:
            seen &= j <= i
        if window:
            seen &= j > i - window
        some = seen.any(-1)
        for h in range(b.hk):
            kd, vd = k[:, h].double(), v[:, h].double()
            s = torch.einsum("ngd,td->ngt", q[:, h], kd) * scale
            mag = torch.einsum("ngd,td->ngt", q[:, h].abs(), kd.abs()) * abs(scale)
            ds = (mag.amax(-1) if t else mag.new_zeros(n, g)) * (b.d / 16 + 8) * 2.0**-22
            if cap:
                s = cap * torch.tanh(s / cap)
            s = s.masked_fill(~seen[:, None, :], -math.inf)
            big = s.masked_fill(~seen[:, None, :], 0.0).abs().amax(-1) if t else mag.new_zeros(n, g)
            dp = ds + 8 * U32 * cap + big * U32 + 2.0**-21 + t * 2.0**-26
            l = torch.logsumexp(s, -1) if t else mag.new_full((n, g), -math.inf)
            p = torch.exp(s - torch.where(some[:, None], l, torch.zeros_like(l))[..., None])
            ref = torch.einsum("ngt,td->ngd", p, vd)
            room = torch.einsum("ngt,td->ngd", p, vd.abs())
            bound = U16 * ref.abs() + ((U16 + 2 * dp) * (1 + 2.0**-6))[..., None] * room
            err = (got[:, h] - ref).abs()
            assert bool((err <= bound).all()), ("out", n, t, h, float((err - bound).max()))
            assert bool((got[:, h][~some] == 0).all())
            if got_l is not None:
                assert bool((got_l[:, h][~some] == -math.inf).all())
                e = (got_l[:, h][some] - l[some]).abs()
                assert bool((e <= dp[some] + 4 * U32 * l[some].abs()).all()), ("lse", n, t, h, float(e.max()))
