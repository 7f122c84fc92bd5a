"""Chunks over a cache in 8 bits of which many rows see no key: items without a tile, several one after the
other in a CTA, between items with tiles (padded sequences, more new tokens than the cache has, parts of the
list that are an item's beginning alone)."""

import pytest

from kv8_batch import E4M3, INT8, Kv8Batch
from test_kv8_attention_gpu import checked

pytestmark = pytest.mark.gpu


# the list's items key head by key head, pair of halves by pair: some sequences without keys, or with few
@pytest.mark.parametrize("hq,hk,d,q_lens,kv_lens,dtype", [
    (16, 8, 64, [282, 300, 176, 300, 300], [4262, 3229, 2431, 0, 2099], INT8),
    (48, 8, 128, [213, 300, 300, 300, 300], [3501, 1393, 4637, 4748, 0], E4M3),
    (64, 4, 64, [130, 93, 0, 130, 130, 1, 130, 0, 130], [1128, 1, 0, 4458, 1634, 4892, 2091, 799, 4839], E4M3),
    (136, 8, 64, [16, 16, 1, 16, 16, 16, 1, 16], [733, 0, 722, 1050, 3, 1135, 746, 188], INT8),
    (8, 2, 128, [200, 900, 70, 900], [1000, 5, 600, 0], E4M3),
    (32, 1, 128, [40, 400, 40, 400], [900, 0, 30, 17], INT8),
])
@pytest.mark.parametrize("kw", [dict(), dict(window=100, sinks=20), dict(causal=False, softcap=30.0, window=500)])
def test_sequences_without_keys(cuda_device, hq, hk, d, q_lens, kv_lens, dtype, kw):
    checked(Kv8Batch(hq, hk, d, q_lens, kv_lens, 64, dtype=dtype, seed=len(q_lens), spare_rows=2), **kw)


# more pairs than a list has: whole items, those with keys first in every CTA
@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_more_new_tokens_than_keys(cuda_device, dtype, d):
    checked(Kv8Batch(64, 4, d, [2600], [300], dtype=dtype, seed=1, spare_rows=1))
    checked(Kv8Batch(64, 4, d, [1300, 1300], [40, 200], 32, dtype=dtype, seed=2), window=20, sinks=3)
