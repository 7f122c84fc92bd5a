"""Outputs of calls on a given stream: their memory is that stream's, so that what is freed while the
call is still to run is not given to work on another stream."""

import pytest
import torch

import memory_bound_decode_fd_gb300 as fd
from attn_check import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("op", ["rope", "rope_append", "paged_attention"])
def test_outputs_belong_to_the_stream_of_the_call(cuda_device, op, strided):
    b = Batch(4, 2, 64, [1, 5], [30, 40], 16, seed=1)
    n = b.q.shape[0]
    row = torch.zeros(n, 8, 64, dtype=torch.bfloat16, device="cuda")
    q = row[:, :4] if strided else b.q
    k, v = row[:, 4:6].clone(), row[:, 6:].clone()
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    freq, _ = fd.rope_inv_freq(64, device="cuda")
    scratch = fd.paged_attention_scratch(2, n, 4, 2, 64, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    if op == "rope":
        outs = fd.rope(q, k, pos, freq, stream=side)
    elif op == "rope_append":
        outs = (fd.rope_append(q, k, v, *b.args(), freq, stream=side),)
    else:
        outs = (fd.paged_attention(q, *b.args(), b.max_q, scratch, stream=side),)
    sizes = [(t.shape, t.data_ptr()) for t in outs]
    del outs  # the call may still be running
    for shape, at in sizes:
        here = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        assert here.data_ptr() != at
    with torch.cuda.stream(side):
        again = {torch.empty(shape, dtype=torch.bfloat16, device="cuda").data_ptr() for shape, _ in sizes}
    assert again & {at for _, at in sizes}
    torch.cuda.synchronize()
