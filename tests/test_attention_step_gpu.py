"""The attention half of a layer as it is used: add-RMSNorm beside the QKV product, rotary positions
and the append in place on its rows, attention over the pages; prompts of two sequences first, then
tokens one by one, replayed as one captured graph with new lengths. Every part is checked: the cache
against a 64-bit rotation of the rows that went in, the attention against a 64-bit one over what the
cache holds."""

import numpy as np
import pytest
import torch

import memory_bound_decode_fd_gb300 as fd
from attn_check import Batch, check_attention, check_rope
from memory_bound_decode_fd_gb300 import inputs

pytestmark = pytest.mark.gpu

HQ, HK, D, HIDDEN, PAGE = 8, 2, 128, 1024, 16
N = (HQ + 2 * HK) * D


def u8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    """Buffers of one layer for up to `rows` tokens, and its calls."""

    def __init__(self, rows, batch, max_pages, k_cache, v_cache, inv_freq, scale):
        e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.x, self.res, self.normed, self.qkv = e(rows, HIDDEN), e(rows, HIDDEN), e(rows, HIDDEN), e(rows, N)
        self.out = e(rows, HQ, D)
        self.weight = torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")
        i = inputs.nvfp4_inputs(rows, HIDDEN, N, seed=rows)
        self.fp4 = [u8(i[n]) for n in ("x", "x_sf", "w", "w_sf")]
        self.alpha = torch.ones(1, device="cuda")
        self.q = self.qkv[:, :HQ * D].view(rows, HQ, D)
        self.k = self.qkv[:, HQ * D:(HQ + HK) * D].view(rows, HK, D)
        self.v = self.qkv[:, (HQ + HK) * D:].view(rows, HK, D)
        self.before = e(rows, N)
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.q_start, self.kv_len = i32(batch + 1), i32(batch)
        self.block_table = torch.full((batch, max_pages), -1, dtype=torch.int32, device="cuda")
        self.cache = k_cache, v_cache
        self.inv_freq, self.scale = inv_freq, scale
        self.max_q = rows
        self.scratch = fd.paged_attention_scratch(batch, rows, HQ, HK, D, rows)

    def run(self):
        fd.add_rmsnorm(self.x, self.res, self.weight, 1e-5, out=self.normed, residual_out=self.res)
        fd.nvfp4_scaled_mm(*self.fp4, self.alpha, out=self.qkv)
        fd.copy(self.before, self.qkv)
        fd.rope_append(self.q, self.k, self.v, *self.cache, self.q_start, self.kv_len, self.block_table,
                       self.inv_freq, scale=self.scale, q_out=self.q)
        fd.paged_attention(self.q, *self.cache, self.q_start, self.kv_len, self.block_table, self.max_q,
                           self.scratch, out=self.out)

    def check(self, new, lengths):
        """After a run: new tokens and lengths of the sequences."""
        view = lambda t, a, b: t[:, a * D:b * D].view(-1, b - a, D)  # noqa: E731
        pos = torch.cat([torch.arange(t - n, t, device="cuda") for n, t in zip(new, lengths)])
        n = sum(new)
        check_rope(self.q[:n], view(self.before, 0, HQ)[:n], pos, self.inv_freq, D, False, self.scale)
        b = Batch.__new__(Batch)
        b.hq, b.hk, b.d, b.device, b.q = HQ, HK, D, "cuda", self.q
        b.q_lens, b.kv_lens, b.keys, b.values = new, lengths, [], []
        row = 0
        for s, (m, t) in enumerate(zip(new, lengths)):
            p = torch.arange(t, device="cuda")
            page = self.block_table[s].long()[p // PAGE]
            b.keys.append(self.cache[0][page, p % PAGE])
            b.values.append(self.cache[1][page, p % PAGE])
            check_rope(b.keys[-1][t - m:], view(self.before, HQ, HQ + HK)[row:row + m], p[t - m:], self.inv_freq, D,
                       False, self.scale)
            assert torch.equal(b.values[-1][t - m:], view(self.before, HQ + HK, HQ + 2 * HK)[row:row + m])
            row += m
        check_attention(b, self.out)


@pytest.mark.parametrize("pdl", [False, True])
def test_prompts_then_tokens(cuda_device, pdl):
    pages = 12
    caches = [torch.full((pages, PAGE, HK, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[:10].view(2, 5).int()
    inv_freq, scale = fd.rope_inv_freq(D, 500000.0, "banded", 8.0, device="cuda")
    prompts = [37, 5]
    fd.device_status()
    prev = fd.set_pdl(pdl)
    try:
        first = Layer(sum(prompts), 2, 5, *caches, inv_freq, scale)
        first.block_table.copy_(table)
        first.q_start.copy_(torch.tensor([0, 37, 42], dtype=torch.int32))
        first.kv_len.copy_(torch.tensor(prompts, dtype=torch.int32))
        # scores of ordinary size whatever the product's
        first.run()
        torch.cuda.synchronize()
        first.alpha /= first.before.float().std()
        first.run()
        torch.cuda.synchronize()
        first.check(prompts, prompts)

        step = Layer(2, 2, 5, *caches, inv_freq, scale)
        step.alpha.copy_(first.alpha)
        step.block_table.copy_(table)
        step.q_start.copy_(torch.tensor([0, 1, 2], dtype=torch.int32))
        lengths = list(prompts)
        # captured with lengths of zero, as a padded batch: nothing is written to the cache
        graph = torch.cuda.CUDAGraph()
        step.run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            step.run()
        for n in range(20):
            lengths = [t + 1 for t in lengths]
            step.kv_len.copy_(torch.tensor(lengths, dtype=torch.int32))
            step.fp4[0].copy_(step.fp4[0].roll(n + 1, 1))  # another token
            graph.replay()
            torch.cuda.synchronize()
            step.check([1, 1], lengths)
    finally:
        fd.set_pdl(prev)
    assert fd.device_status() == 0


def test_calls_from_python_and_from_cpp_agree(cuda_device, monkeypatch):
    # attention.py hands a call whose arguments are in order to its C++ form, and makes it itself where
    # that has not been built: the same results, new outputs and given ones, and the same refusals
    from memory_bound_decode_fd_gb300 import attention

    attention._load()
    assert attention._fast, "csrc/fd_torch.cpp is not built"
    b = Batch(4, 2, 64, [1, 5, 0], [40, 33, 0], 16, seed=3, spare_rows=1)
    n = b.q.shape[0]
    gen = torch.Generator(device="cuda").manual_seed(5)
    row = torch.randn(n, 8, 64, device="cuda", generator=gen).to(torch.bfloat16)
    k, v = row[:, 4:6], row[:, 6:]
    inv_freq, _ = fd.rope_inv_freq(32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    scratch = fd.paged_attention_scratch(3, n, 4, 2, 64, b.max_q)
    caches = b.k_cache.clone(), b.v_cache.clone()
    index = b.q_start, b.kv_len, b.block_table

    def results():
        kc, vc = caches[0].clone(), caches[1].clone()
        new = torch.zeros(n, 4, 64, dtype=torch.bfloat16, device="cuda")
        lse, out = torch.zeros(n, 4, device="cuda"), new.clone()
        r = [*fd.rope(row[:, :4], k, pos, inv_freq, True, 1.5)]
        r += [fd.rope(row[:, :4], None, pos, inv_freq)[0], *fd.rope(row[:, :4], k, pos, inv_freq, q_out=new)]
        assert r[-2] is new
        r += [fd.rope_append(row[:, :4], k, v, kc, vc, *index, inv_freq)[:6], kc, vc]
        r += [fd.rope_append(row[:, :4], k, v, kc, vc, *index, inv_freq, pos, True, 2.0)[:6], kc, vc]
        r += [fd.paged_attention(b.q, *caches, *index, b.max_q, scratch)[:6]]
        assert fd.paged_attention(b.q, *caches, *index, b.max_q, scratch, 0.3, False, 9, 5.0, out, lse) is out
        r += [out, lse]
        stream = torch.cuda.current_stream()
        r += [fd.paged_attention(b.q, *caches, *index, b.max_q, scratch, stream=stream)[:6]]
        return [t.clone() for t in r]

    def refusals():
        got = []
        for call in (lambda: fd.rope(row, k, pos[1:], inv_freq), lambda: fd.rope(row[..., :63], None, pos, inv_freq),
                     lambda: fd.rope(row.float(), None, pos, inv_freq), lambda: fd.rope(row, None, pos.cpu(), inv_freq),
                     lambda: fd.rope(row, None, pos, inv_freq, scale=float("inf")), lambda: fd.rope(3, None, pos, inv_freq),
                     lambda: fd.rope(row[:, :4], row[:, 3:5], pos, inv_freq, q_out=row[:, :4], k_out=row[:, 3:5]),
                     lambda: fd.rope_append(row[:, :4], k, v, caches[0], caches[0], *index, inv_freq),
                     lambda: fd.rope_append(row[:, :4], k, v, *caches, *index, inv_freq.repeat(3)),
                     lambda: fd.paged_attention(b.q, *caches, *index, -1, scratch),
                     lambda: fd.paged_attention(b.q[:, :3], *caches, *index, 5, scratch),
                     lambda: fd.paged_attention(b.q, *caches, *index, 5, scratch[:64]),
                     lambda: fd.paged_attention(b.q, *caches, *index, 5, scratch, out=b.q),
                     lambda: fd.paged_attention(b.q, *caches, *index, 5, scratch, lse=torch.zeros(4, n, device="cuda"))):
            with pytest.raises((TypeError, ValueError, fd.FdError)) as e:
                call()
            got.append((type(e.value), str(e.value)))
        return got

    cpp, cpp_refusals = results(), refusals()
    monkeypatch.setattr(attention, "_fast", False)
    for x, y in zip(cpp, results()):
        assert x.shape == y.shape and x.stride() == y.stride()
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert refusals() == cpp_refusals
