"""Attention over a paged cache against a plain 64-bit computation: decoding, chunks, masks that
leave rows empty, group sizes, layouts, NaN behind the last token, bad pages, graphs and streams."""

import pytest
import torch

import memory_bound_decode_fd_gb300 as fd
from attn_check import Batch, check_attention
from memory_bound_decode_fd_gb300 import _lib

pytestmark = pytest.mark.gpu


def run(b, scratch=None, out=None, with_lse=True, **kw):
    n, h, d = b.q.shape
    if scratch is None:
        scratch = fd.paged_attention_scratch(len(b.q_lens), n, b.hq, b.hk, b.d, b.max_q)
    if out is None:
        out = torch.full((n, h, d), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, h), 5.0, device="cuda") if with_lse else None
    fd.paged_attention(b.q, *b.args(), b.max_q, scratch, out=out, lse=lse, **kw)
    return out, lse


def checked(b, **kw):
    fd.device_status()
    scratch = fd.paged_attention_scratch(len(b.q_lens), b.q.shape[0], b.hq, b.hk, b.d, b.max_q)
    out, lse = run(b, scratch, **kw)
    assert fd.device_status() == 0
    args = {"cap" if k == "softcap" else k: v for k, v in kw.items()}
    check_attention(b, out, lse, **args)
    n = sum(b.q_lens)  # rows behind the last sequence stay as they were
    assert bool((out[n:] == 5.0).all()) and bool((lse[n:] == 5.0).all())
    assert not scratch[:16384].any()  # counters are zero again
    again, lse2 = run(b, scratch, **kw)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


DECODE = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(8, 2), (1, 1), (7, 1), (6, 2), (16, 1), (32, 1), (40, 2)])
def test_decode_lengths(cuda_device, d, hq, hk):
    checked(Batch(hq, hk, d, [1] * len(DECODE), DECODE, seed=hq, spare_rows=1))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
@pytest.mark.parametrize("head_major,fused", [(False, False), (True, False), (False, True), (True, True)])
def test_page_sizes_and_layouts(cuda_device, page, head_major, fused):
    checked(Batch(4, 2, 128, [1, 3, 70], [1030, 200, 1025], page, head_major, seed=page, fused_kv=fused))


@pytest.mark.parametrize("kv", [4097, 30000])
def test_decode_long(cuda_device, kv):
    # every SM works on the same sequence: the joining of partial results
    checked(Batch(32, 8, 128, [1], [kv], seed=kv, q_std=2.0))


def test_decode_ragged_batch(cuda_device):
    lens = [1 + (37 * i * i) % 3001 for i in range(70)]
    checked(Batch(8, 2, 64, [1] * 70, lens, 32, True, seed=1))


def test_empty_rows_and_sequences(cuda_device):
    # no keys at all; no new tokens; fewer keys than new tokens (the first rows see nothing)
    checked(Batch(4, 2, 128, [1, 0, 3, 1, 40, 0], [0, 5, 2, 70, 17, 0], spare_rows=3))
    checked(Batch(4, 2, 128, [200, 1], [100, 0]))


CHUNKS = [
    ([2], [2]), ([4], [1000]), ([5, 1, 16, 3], [5, 300, 129, 64]), ([64], [64]), ([33, 130, 1], [64, 300, 17]),
    ([257], [1000]), ([300, 129, 128], [300, 640, 128]), ([1000, 1, 7], [1000, 513, 2000]),
]


@pytest.mark.parametrize("q_lens,kv_lens", CHUNKS)
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (2, 2, 64), (7, 1, 128), (20, 4, 64), (32, 1, 64)])
def test_chunks(cuda_device, q_lens, kv_lens, hq, hk, d):
    checked(Batch(hq, hk, d, q_lens, kv_lens, seed=len(q_lens), spare_rows=2))


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [1, 100, 777]), ([9, 300], [400, 700]), ([1000], [1000])])
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=16), dict(window=200), dict(softcap=5.0),
                                dict(window=100, softcap=30.0), dict(causal=False),
                                dict(causal=False, window=50), dict(scale=0.5), dict(scale=-0.1),
                                dict(scale=0.0), dict(softcap=0.5, scale=1.0)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (7, 1, 64)])
def test_options(cuda_device, q_lens, kv_lens, kw, hq, hk, d):
    checked(Batch(hq, hk, d, q_lens, kv_lens, 16, seed=3, q_std=2.0), **kw)


def test_large_scores(cuda_device):
    # probabilities of nearly one key each, and maxima that keep rising along the keys
    b = Batch(8, 2, 128, [1, 60], [900, 900], seed=4, q_std=8.0)
    ramp = torch.linspace(0, 4, 900, device="cuda")[:, None, None].to(torch.bfloat16)
    for k, (pg, off) in zip(b.keys, b.slots):
        k.mul_(ramp)
        b.k_cache[pg, off] = k
    checked(b)


def test_pages_shared_by_sequences(cuda_device):
    # a common prefix: the second sequence's first pages are the first one's
    b = Batch(4, 2, 128, [1, 20], [100, 120], 16, seed=5)
    b.block_table[1, :5] = b.block_table[0, :5]
    pg, off = b.slots[1]
    pg[:80], b.keys[1][:80], b.values[1][:80] = b.slots[0][0][:80], b.keys[0][:80], b.values[0][:80]
    checked(b)


def test_nothing_past_the_window_is_needed(cuda_device):
    # pages before the window are gone from the table
    b = Batch(4, 2, 128, [1, 30], [600, 500], 16, seed=6)
    b.block_table[0, :(600 - 64) // 16] = -1
    b.block_table[1, :(500 - 30 + 1 - 64) // 16] = 1 << 29
    checked(b, window=64)


@pytest.mark.parametrize("q_len", [1, 100])
def test_bad_page_reads_zeros_and_is_reported(cuda_device, q_len):
    b = Batch(4, 2, 64, [q_len], [300], 32, seed=7)
    b.block_table[0, 3] = b.k_cache.shape[0]
    fd.device_status()
    out, lse = run(b)
    assert fd.device_status() == fd.FD_DEVICE_STATUS_BAD_PAGE
    b.keys[0][96:128] = 0
    b.values[0][96:128] = 0
    check_attention(b, out, lse)


def test_length_above_the_table_counts_as_its_end(cuda_device):
    b = Batch(4, 2, 64, [1], [64], 16, seed=8)
    b.kv_len += 1000
    out, lse = run(b)
    check_attention(b, out, lse)


def test_strided_views(cuda_device):
    b = Batch(4, 2, 128, [1, 40], [77, 90], 16, seed=9)
    n = b.q.shape[0]
    row = torch.zeros((n, 4 * 128 + 256), dtype=torch.bfloat16, device="cuda")
    row[:, :512] = b.q.view(n, 512)
    q = row[:, :512].view(n, 4, 128)
    out = torch.zeros((4, n, 128), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    scratch = fd.paged_attention_scratch(2, n, 4, 2, 128, 40)
    table = torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
    table[:, :b.block_table.shape[1]] = b.block_table
    fd.paged_attention(q, b.k_cache, b.v_cache, b.q_start, b.kv_len, table[:, :b.block_table.shape[1]], 40,
                       scratch, out=out)
    check_attention(b, out)


def test_offsets_past_32_bits(cuda_device):
    # the last pages of a cache of more than 2^31 elements
    hk, d, page = 8, 128, 64
    pages = 2**31 // (hk * d * page) + 5
    small = Batch(8, hk, d, [1, 30], [150, 100], page, seed=10)
    kc = torch.empty((pages, page, hk, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    n = small.k_cache.shape[0]
    kc[-n:], vc[-n:] = small.k_cache, small.v_cache
    used = small.block_table < n
    small.block_table[used] += pages - n
    small.k_cache, small.v_cache = kc, vc
    out, lse = run(small)
    check_attention(small, out, lse)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [700, 90]), ([200, 3], [700, 90])])
def test_graph_replayed_with_new_lengths(cuda_device, q_lens, kv_lens):
    b = Batch(8, 2, 128, q_lens, kv_lens, 16, seed=11)
    scratch = fd.paged_attention_scratch(2, b.q.shape[0], 8, 2, 128, b.max_q)
    out, lse = run(b, scratch)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.paged_attention(b.q, *b.args(), b.max_q, scratch, out=out, lse=lse)
    for cut in (0, 5, 80):
        b.kv_len.copy_(torch.tensor([t - cut for t in kv_lens], dtype=torch.int32))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        c = Batch.__new__(Batch)
        c.__dict__ = dict(b.__dict__, kv_lens=[t - cut for t in kv_lens],
                          keys=[k[:t - cut] for k, t in zip(b.keys, kv_lens)],
                          values=[v[:t - cut] for v, t in zip(b.values, kv_lens)])
        check_attention(c, out, lse)


def test_two_streams_with_a_scratch_each(cuda_device):
    b = Batch(32, 8, 128, [1], [3000], seed=12)
    streams = [torch.cuda.Stream() for _ in range(2)]
    scratch = [fd.paged_attention_scratch(1, 1, 32, 8, 128, 1) for _ in range(2)]
    outs = [torch.zeros_like(b.q) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, sc, o in zip(streams, scratch, outs):
            fd.paged_attention(b.q, *b.args(), 1, sc, out=o, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        check_attention(b, o)


def test_back_to_back_with_programmatic_launch(cuda_device):
    # calls that share a scratch, each started before the last has ended
    b = Batch(32, 8, 128, [1, 1], [3000, 40], seed=13)
    scratch = fd.paged_attention_scratch(2, 2, 32, 8, 128, 1)
    prev = fd.set_pdl(True)
    try:
        outs = [run(b, scratch)[0] for _ in range(10)]
    finally:
        fd.set_pdl(prev)
    check_attention(b, outs[0])
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


# ---------------------------------------------------------------- how the work is dealt out


def test_many_sequences_of_chunks(cuda_device):
    # more sequences than a CTA lists: an item a CTA, some of them empty
    q_lens = [(7 * i) % 10 for i in range(200)]
    kv_lens = [n + (i * i) % 150 for i, n in enumerate(q_lens)]
    checked(Batch(8, 2, 128, q_lens, kv_lens, 16, seed=20, spare_rows=2))


def test_many_decoded_sequences(cuda_device):
    # several sequences for each thread of the list, some empty
    lens = [0 if i % 7 == 3 else 1 + (i * 37) % 90 for i in range(1500)]
    checked(Batch(4, 1, 64, [1 if t else 0 for t in lens], lens, 16, seed=21))


def test_more_pairs_than_a_list(cuda_device):
    # 32 heads a key head: four tokens a half
    checked(Batch(32, 1, 64, [700, 650, 1, 0, 33], [700, 900, 50, 3, 33], 32, seed=22))


@pytest.mark.parametrize("q_len,kv", [(20, 20000), (130, 9001), (40, 3000)])
@pytest.mark.parametrize("hq,hk,d", [(4, 1, 128), (8, 2, 64)])
def test_one_chunk_over_many_ctas(cuda_device, q_len, kv, hq, hk, d):
    # the joining of many parts of few items
    checked(Batch(hq, hk, d, [q_len], [kv], 64, seed=kv, q_std=2.0))


def test_parts_without_keys(cuda_device):
    # long caches of which a window leaves little, and rows that see nothing among rows that do
    checked(Batch(4, 1, 128, [200, 60], [5000, 40], 64, seed=23), window=100)


@pytest.mark.parametrize("q_lens,kv_lens", [([5, 1, 2], [300, 20, 2]), ([1, 1], [4000, 17])])
def test_more_query_heads_than_a_tile(cuda_device, q_lens, kv_lens):
    checked(Batch(130, 1, 64, q_lens, kv_lens, 16, seed=24, spare_rows=1))


@pytest.mark.parametrize("q_len", [1, 90])
@pytest.mark.parametrize("cap", [1.0, 8.0, 200.0])
@pytest.mark.parametrize("d", [64, 128])
def test_caps_inside_and_beyond_the_scores(cuda_device, q_len, cap, d):
    # every score far below the cap, every one far above it, and both in one tile
    for std in (0.2, 6.0):
        b = Batch(8, 2, d, [q_len, q_len], [400, 150], 16, seed=25, q_std=std)
        checked(b, softcap=cap)


def test_heads_and_pages_of_one(cuda_device):
    # dimensions of one entry, whatever their strides say
    b = Batch(3, 1, 128, [1, 17], [15, 16], 16, seed=26)
    b.k_cache = b.k_cache.as_strided(b.k_cache.shape, (b.k_cache.stride(0), b.k_cache.stride(1), 999, 1))
    checked(b)
    one = Batch(4, 2, 64, [5], [16], 16, seed=27, max_pages=1)
    page = one.slots[0][0][:1]
    one.k_cache, one.v_cache = one.k_cache[page].contiguous(), one.v_cache[page].contiguous()
    one.block_table.fill_(0)
    checked(one)


def test_refusals_of_the_binding(cuda_device):
    b = Batch(4, 2, 128, [1, 1], [20, 30])
    scratch = fd.paged_attention_scratch(2, 2, 4, 2, 128, 1)
    ok = dict(q=b.q, k_cache=b.k_cache, v_cache=b.v_cache, q_start=b.q_start, kv_len=b.kv_len,
              block_table=b.block_table, max_q=1, scratch=scratch)
    fd.paged_attention(**ok)
    for change, error in ((dict(q=b.q.float()), TypeError), (dict(q=b.q[0]), ValueError), (dict(q=b.q[:, :3]), ValueError),
                          (dict(kv_len=b.kv_len.long()), TypeError), (dict(q_start=b.q_start[:2]), ValueError),
                          (dict(block_table=b.block_table.cpu()), ValueError), (dict(max_q=-1), ValueError),
                          (dict(k_cache=b.k_cache[..., :64]), ValueError), (dict(scratch=scratch[:100]), fd.FdError),
                          (dict(out=b.q[:1]), ValueError), (dict(lse=torch.zeros(2, 3, device="cuda")), ValueError),
                          (dict(k_cache=b.k_cache.transpose(2, 3)), ValueError), (dict(window=-2), ValueError),
                          (dict(out=b.q), fd.FdError), (dict(scale=float("nan")), fd.FdError)):
        with pytest.raises(error):
            fd.paged_attention(**{**ok, **change})


def test_no_new_tokens_at_all(cuda_device):
    b = Batch(4, 2, 64, [1, 2], [30, 40])
    out = torch.full_like(b.q, 5.0)
    scratch = fd.paged_attention_scratch(2, 3, 4, 2, 64, 0)
    fd.paged_attention(b.q, *b.args(), 0, scratch, out=out)
    torch.cuda.synchronize()
    assert bool((out == 5.0).all())


@pytest.mark.parametrize("q_len", [1, 40])
def test_a_cap_far_below_all_scores(cuda_device, q_len):
    b = Batch(4, 1, 64, [q_len], [70], seed=31)
    v = b.values[0].double()[:, 0]
    i = torch.arange(70 - q_len, 70, device="cuda")
    # a cap so small that all visible keys count the same
    out, lse = run(b, scale=1.0, softcap=1e-30)
    n = (i + 1).double()
    mean = v.cumsum(0)[i] / n[:, None]
    room = v.abs().cumsum(0)[i] / n[:, None]
    # each probability and the result rounded to bf16 once, sums of 70 in fp32
    assert bool(((out[:q_len].double() - mean[:, None]).abs() <= (2.0**-8 * room + 2.0**-8 * mean.abs() + 1e-5)[:, None]).all())
    assert torch.allclose(lse[:q_len].double(), n.log()[:, None].expand(-1, 4), atol=1e-5)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [5000, 3, 700]), ([300, 2], [4000, 90]), ([40] * 200, [50] * 200)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_that_runs_out_is_reported(cuda_device, q_lens, kv_lens, d):
    # a copy that is never made (the launch flag for it): no fault, no hang, and the scratch as good
    # as before
    lib = fd.load_library()
    b = Batch(8, 2, d, q_lens, kv_lens, 16, seed=33)
    scratch = fd.paged_attention_scratch(len(q_lens), b.q.shape[0], 8, 2, d, b.max_q)
    run(b, scratch)
    assert fd.device_status() == 0
    flags = lib.fd_get_launch_flags()
    assert lib.fd_set_launch_flags(flags | _lib.FD_LAUNCH_TEST_WAIT_TIMEOUT) == _lib.FD_OK
    try:
        out, lse = run(b, scratch)
        torch.cuda.synchronize()
    finally:
        lib.fd_set_launch_flags(flags)
    assert bool(out.isnan().all()) and bool(lse.isnan().all())
    assert fd.device_status() == _lib.FD_DEVICE_STATUS_WAIT_TIMEOUT
    assert fd.device_status() == 0
    out, lse = run(b, scratch)
    check_attention(b, out, lse)
    assert fd.device_status() == 0
