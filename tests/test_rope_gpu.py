"""Rotary positions and the append to a paged cache against a plain 64-bit computation."""

import math

import pytest
import torch

import memory_bound_decode_fd_gb300 as fd
from attn_check import Batch, check_rope

pytestmark = pytest.mark.gpu


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)


# d and rot that take 16-element units, and ones that do not (pairs one by one)
@pytest.mark.parametrize("tokens", [1, 3, 700])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 16), (256, 256), (80, 32), (96, 24),
                                   (72, 72), (64, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(cuda_device, tokens, d, rot, interleaved):
    hq, hk = 5, 2
    q, k = normal((tokens, hq, d), tokens), normal((tokens, hk, d), tokens + 1)
    pos = torch.randint(-5000, 200000, (tokens,), dtype=torch.int32, device="cuda")
    f, _ = fd.rope_inv_freq(rot, device="cuda")
    qo, ko = fd.rope(q, k, pos, f, interleaved=interleaved, scale=1.25)
    check_rope(qo, q, pos, f, rot, interleaved, 1.25)
    check_rope(ko, k, pos, f, rot, interleaved, 1.25)


@pytest.mark.parametrize("tokens", [1, 37, 2500])
def test_rope_in_place_on_views_of_one_row(cuda_device, tokens):
    hq, hk, d = 8, 2, 128
    qkv = normal((tokens, (hq + 2 * hk) * d), 3)
    before = qkv.clone()
    view = lambda t: (t[:, :hq * d].view(tokens, hq, d), t[:, hq * d:(hq + hk) * d].view(tokens, hk, d))  # noqa: E731
    q, k = view(qkv)
    pos = torch.arange(100, 100 + tokens, dtype=torch.int32, device="cuda")
    f, _ = fd.rope_inv_freq(d, 500000.0, device="cuda")
    qo, ko = fd.rope(q, k, pos, f, q_out=q, k_out=k)
    assert qo is q and ko is k
    q0, k0 = view(before)
    check_rope(q, q0, pos, f, d, False, 1.0)
    check_rope(k, k0, pos, f, d, False, 1.0)
    assert torch.equal(qkv[:, (hq + hk) * d:].view(torch.int16), before[:, (hq + hk) * d:].view(torch.int16))


def test_rope_queries_alone_and_strides(cuda_device):
    # heads outermost, and every token the same row (stride 0)
    q = normal((3, 9, 64), 5).transpose(0, 1)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    f, _ = fd.rope_inv_freq(64, device="cuda")
    out, none = fd.rope(q, None, pos, f)
    assert none is None
    check_rope(out, q, pos, f, 64, False, 1.0)
    one = normal((1, 3, 64), 6).expand(9, 3, 64)
    out, _ = fd.rope(one, None, pos, f, interleaved=True)
    check_rope(out, one, pos, f, 64, True, 1.0)
    dst = torch.zeros(3, 9, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    fd.rope(q, None, pos, f, q_out=dst)
    check_rope(dst, q, pos, f, 64, False, 1.0)


def test_rope_far_positions(cuda_device):
    # the largest and smallest int32, and a frequency of exactly one: the angle itself
    pos = torch.tensor([2**31 - 1, -2**31, 2**30 + 1, 16777217, 0, -1], dtype=torch.int32, device="cuda")
    q = normal((6, 2, 64), 7)
    f, _ = fd.rope_inv_freq(64, device="cuda")
    f = f.clone()
    f[1] = 0.0
    f[2] = 7.5  # more than one turn a position
    out, _ = fd.rope(q, None, pos, f)
    check_rope(out, q, pos, f, 64, False, 1.0)
    # position 0 and a zero frequency rotate nothing
    assert torch.equal(out[4], q[4]) and torch.equal(out[:, :, [1, 33]], q[:, :, [1, 33]])


def test_rope_empty(cuda_device):
    f, _ = fd.rope_inv_freq(64, device="cuda")
    q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, k = fd.rope(q, q, torch.empty(0, dtype=torch.int32, device="cuda"), f)
    assert out.shape == (0, 2, 64) and k.shape == (0, 2, 64)


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("banded", 8.0), ("ramp", 16.0)])
def test_rope_scalings(cuda_device, scaling, factor):
    f, m = fd.rope_inv_freq(128, 10000.0, scaling, factor, 4096, device="cuda")
    q = normal((50, 4, 128), 8)
    pos = torch.arange(60000, 60050, dtype=torch.int32, device="cuda")
    out, _ = fd.rope(q, None, pos, f, scale=m)
    check_rope(out, q, pos, f, 128, False, m)


APPENDS = [
    # hq, hk, d, rot, page, head_major, fused, q_lens, kv_lens
    (4, 2, 128, 128, 16, False, False, [1], [1]),
    (32, 8, 128, 128, 16, False, False, [1, 1, 1], [17, 16, 100]),
    (7, 1, 64, 32, 32, True, False, [5, 0, 40, 1], [5, 3, 90, 33]),
    (4, 4, 64, 48, 64, False, True, [700, 1, 3], [700, 5, 3]),
    (4, 2, 128, 90, 128, True, True, [3, 129], [200, 129]),   # rot not a multiple of 16
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hk,d,rot,page,head_major,fused,q_lens,kv_lens", APPENDS)
def test_append(cuda_device, hq, hk, d, rot, page, head_major, fused, q_lens, kv_lens, interleaved):
    b = Batch(hq, hk, d, q_lens, kv_lens, page, head_major, seed=sum(kv_lens), fused_kv=fused, spare_rows=2)
    n = sum(q_lens)
    qkv = normal((n + 2, (hq + 2 * hk) * d), 11)
    q = qkv[:, :hq * d].view(n + 2, hq, d)
    k = qkv[:, hq * d:(hq + hk) * d].view(n + 2, hk, d)
    v = qkv[:, (hq + hk) * d:].view(n + 2, hk, d)
    f, m = fd.rope_inv_freq(rot, 500000.0, "ramp", 8.0, device="cuda")
    kc, vc = b.k_cache.clone(), b.v_cache.clone()
    q_out = torch.full((n + 2, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    fd.device_status()
    fd.rope_append(q, k, v, *b.args(), f, interleaved=interleaved, scale=m, q_out=q_out)
    assert fd.device_status() == 0
    row = 0
    for nq, t, (pg, off) in zip(q_lens, kv_lens, b.slots):
        pos = torch.arange(t - nq, t, device="cuda")
        s = slice(row, row + nq)
        row += nq
        check_rope(q_out[s], q[s], pos, f, rot, interleaved, m)
        check_rope(b.k_cache[pg[t - nq:], off[t - nq:]], k[s], pos, f, rot, interleaved, m)
        assert torch.equal(b.v_cache[pg[t - nq:], off[t - nq:]], v[s])
        kc[pg[t - nq:], off[t - nq:]] = b.k_cache[pg[t - nq:], off[t - nq:]]
        vc[pg[t - nq:], off[t - nq:]] = v[s]
    # nothing else was written: the rest of the cache, and the rows behind the last sequence
    assert torch.equal(b.k_cache.contiguous().view(torch.int16), kc.contiguous().view(torch.int16))
    assert torch.equal(b.v_cache.contiguous().view(torch.int16), vc.contiguous().view(torch.int16))
    assert bool((q_out[n:] == 3.0).all())


def test_append_given_positions_and_in_place(cuda_device):
    b = Batch(4, 2, 128, [3, 2], [20, 40])
    q, k, v = normal((5, 4, 128), 1), normal((5, 2, 128), 2), normal((5, 2, 128), 3)
    q0 = q.clone()
    pos = torch.tensor([5, 5, 1000000, -3, 0], dtype=torch.int32, device="cuda")
    f, _ = fd.rope_inv_freq(128, device="cuda")
    assert fd.rope_append(q, k, v, *b.args(), f, positions=pos, q_out=q) is q
    check_rope(q, q0, pos, f, 128, False, 1.0)
    pg, off = b.slots[0]
    check_rope(b.k_cache[pg[17:], off[17:]], k[:3], pos[:3], f, 128, False, 1.0)


def test_append_without_a_place(cuda_device):
    # a padded sequence (kv_len 0), a bad page, and a length above the table's pages
    b = Batch(2, 1, 64, [1, 1, 1], [1, 17, 16], page=16)
    b.kv_len = torch.tensor([0, 17, 33], dtype=torch.int32, device="cuda")
    b.block_table[1, 1] = -1
    kc, vc = b.k_cache.clone(), b.v_cache.clone()
    q, k, v = normal((3, 2, 64), 1), normal((3, 1, 64), 2), normal((3, 1, 64), 3)
    f, _ = fd.rope_inv_freq(64, device="cuda")
    fd.device_status()
    q_out = fd.rope_append(q, k, v, *b.args(), f)
    assert fd.device_status() == fd.FD_DEVICE_STATUS_BAD_PAGE
    assert fd.device_status() == 0
    # sequence 2's length counts as 32 (two pages): its last place lies in a page the table does
    # not have, nothing of it is written either
    assert torch.equal(b.k_cache.view(torch.int16), kc.view(torch.int16))
    assert torch.equal(b.v_cache.view(torch.int16), vc.view(torch.int16))
    check_rope(q_out, q, torch.tensor([-1, 16, 31], device="cuda"), f, 64, False, 1.0)


def test_append_past_the_table_writes_nothing(cuda_device):
    # all pages there, one token more than they hold: no place, and no other's place either
    b = Batch(2, 1, 64, [2, 1], [32, 20], page=16)
    b.kv_len = torch.tensor([33, 20], dtype=torch.int32, device="cuda")
    kc = b.k_cache.clone()
    q, k, v = normal((3, 2, 64), 1), normal((3, 1, 64), 2), normal((3, 1, 64), 3)
    f, _ = fd.rope_inv_freq(64, device="cuda")
    fd.device_status()
    fd.rope_append(q, k, v, *b.args(), f)
    assert fd.device_status() == fd.FD_DEVICE_STATUS_BAD_PAGE
    changed = (b.k_cache.view(torch.int16) != kc.view(torch.int16)).any(-1).flatten().nonzero().tolist()
    assert changed == [[int(b.block_table[1, 1]) * 16 + 3]]


def test_append_offsets_past_32_bits(cuda_device):
    # a cache of more than 2^31 elements, its last pages used
    hk, d, page = 8, 128, 64
    pages = 2**31 // (hk * d * page) + 5
    kc = torch.empty((pages, page, hk, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    kv_len = torch.tensor([page * 2 + 3], dtype=torch.int32, device="cuda")
    q_start = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    q, k, v = normal((5, 8, d), 1), normal((5, hk, d), 2), normal((5, hk, d), 3)
    f, _ = fd.rope_inv_freq(d, device="cuda")
    fd.rope_append(q, k, v, kc, vc, q_start, kv_len, table, f)
    pos = torch.arange(page * 2 - 2, page * 2 + 3, device="cuda")
    got = torch.cat((kc[0, -2:], kc[pages - 2, :3]))
    check_rope(got, k, pos, f, d, False, 1.0)
    assert torch.equal(torch.cat((vc[0, -2:], vc[pages - 2, :3])), v)


def test_rope_on_another_stream_and_in_a_graph(cuda_device):
    q, k = normal((40, 4, 128), 1), normal((40, 2, 128), 2)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    f, _ = fd.rope_inv_freq(128, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qo, ko = fd.rope(q, k, pos, f, stream=side)
    side.synchronize()
    check_rope(qo, q, pos, f, 128, False, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.rope(q, k, pos, f, q_out=qo, k_out=ko)
    pos += 77777
    q.normal_()
    graph.replay()
    torch.cuda.synchronize()
    check_rope(qo, q, pos, f, 128, False, 1.0)
    check_rope(ko, k, pos, f, 128, False, 1.0)
    assert math.isfinite(float(qo.float().sum()))
