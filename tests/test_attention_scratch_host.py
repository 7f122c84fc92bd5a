"""The bytes of scratch that the header states are enough for every size, and not far above them."""

import re

import pytest

from test_attention_host import HEADER


@pytest.fixture(scope="module")
def stated():
    text = re.search(r"/\* Bytes of scratch that suffice.*?\*/", HEADER.read_text(), re.S).group(0)
    few, many = (float(x) * 1e6 for x in re.findall(r"([\d.]+) MB", text))
    return few, many


HEADS = [(1, 1), (8, 8), (32, 8), (16, 1), (17, 1), (32, 1), (128, 1), (129, 1), (256, 2), (1024, 8), (1024, 1)]


@pytest.mark.parametrize("max_q", [0, 1, 2, 4, 5, 16, 17, 4096, 1 << 28])
def test_stated_sizes_are_enough(fdlib, stated, max_q):
    for hq, hk in HEADS:
        few = max_q * (hq // hk) <= 16 or hq // hk > 128
        for d in (64, 128):
            for batch in (0, 1, 4096):
                n = fdlib.fd_paged_attention_scratch_bytes(batch, batch * max_q if max_q < 1 << 16 else max_q, hq, hk, d, max_q)
                assert 0 < n <= stated[0 if few else 1], (hq, hk, d, batch)


def test_stated_sizes_are_the_largest(fdlib, stated):
    f = fdlib.fd_paged_attention_scratch_bytes
    assert f(1, 1, 32, 8, 128, 1) > stated[0] - 0.1e6
    assert f(1, 1, 32, 1, 128, 1) > stated[1] - 0.1e6   # a single token of 32 heads on one
