"""Outputs over the arrays that say where things go: refused before any CUDA call, to the last byte."""

import pytest

from memory_bound_decode_fd_gb300 import _lib
from test_attention_host import (BT, F, KC, KL, O, OVER, P, QS, S, VC, append, attend, batch, cache, heads,  # noqa: F401
                                 no_launch)

RUNS = _lib.FD_ERR_CUDA  # past every check, a failed launch
OUT = 7 * 4096 * 2 + 32 * 128 * 2                    # bytes of q_out, heads(O): 8 tokens
KEYS = (99 * 16 * 1024 + 15 * 1024 + 7 * 128 + 128) * 2  # of the keys, cache()
TABLE = (3 * 10 + 10) * 4                            # of the block table, batch()


@pytest.mark.parametrize("kw,status", [
    (dict(b=batch(q_start=O + 64)), OVER), (dict(b=batch(kv_len=O + 64)), OVER), (dict(b=batch(table=O + 64)), OVER),
    (dict(f=O + 64), OVER), (dict(pos=O + 64), OVER),
    (dict(b=batch(q_start=KC + 64)), OVER), (dict(b=batch(kv_len=VC + 64)), OVER), (dict(b=batch(table=KC + 64)), OVER),
    (dict(f=VC + 64), OVER), (dict(pos=KC + 64), OVER),
    # the last bytes, and the first behind and before
    (dict(b=batch(q_start=O + OUT - 4)), OVER), (dict(b=batch(q_start=O + OUT)), RUNS),
    (dict(b=batch(q_start=O - 20)), RUNS), (dict(b=batch(q_start=O - 16)), OVER),
    (dict(b=batch(kv_len=O - 16)), RUNS), (dict(b=batch(kv_len=O - 12)), OVER),
    (dict(b=batch(table=O - TABLE)), RUNS), (dict(b=batch(table=O - TABLE + 4)), OVER),
    (dict(b=batch(table=O, max_pages=0)), RUNS),     # no entry of it is read
    (dict(pos=O - 32), RUNS), (dict(pos=O - 28), OVER), (dict(f=O - 512), RUNS), (dict(f=O - 504), OVER),
    (dict(pos=KC + KEYS - 4), OVER), (dict(pos=KC + KEYS), RUNS),
])
def test_append_over_its_index(no_launch, kw, status):  # noqa: F811
    assert append(no_launch, **kw) == status


LSE = 8 * 32 * 4


@pytest.mark.parametrize("kw,status", [
    (dict(b=batch(q_start=O + 64)), OVER), (dict(b=batch(kv_len=O + 64)), OVER), (dict(b=batch(table=O + 64)), OVER),
    (dict(b=batch(q_start=S + 64)), OVER), (dict(b=batch(kv_len=S + 64)), OVER), (dict(b=batch(table=S + 64)), OVER),
    (dict(lse=QS), OVER), (dict(lse=KL), OVER), (dict(lse=BT), OVER),
    (dict(lse=QS - LSE), RUNS), (dict(lse=QS - LSE + 4), OVER), (dict(lse=QS + 20), RUNS), (dict(lse=QS + 16), OVER),
    (dict(lse=KL + 16), RUNS), (dict(lse=KL + 12), OVER), (dict(lse=BT + TABLE), RUNS), (dict(lse=BT + TABLE - 4), OVER),
    (dict(b=batch(table=O, max_pages=0)), RUNS),
    (dict(b=batch(q_start=KC), c=cache()), RUNS),    # what is only read may be anywhere
])
def test_attention_over_its_index(no_launch, kw, status):  # noqa: F811
    assert attend(no_launch, **kw) == status
