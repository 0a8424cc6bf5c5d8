"""Scratch sizes of the cache operators, without a GPU."""

import pytest

from full_attention_decode_gb300 import binding as B
from full_attention_decode_gb300 import synth


@pytest.mark.parametrize("capacity,block,rows", [(0, 16, 4), ((1 << 31) + 16, 16, 4), ((1 << 32) - 16, 0, 1), (256, 24, 4),
                                                 (256, 8, 4), (256, 2048, 4), (256, 16, 0), (256, 16, (1 << 20) + 1)])
def test_sizes_that_the_calls_reject_have_no_scratch(capacity, block, rows):
    assert B.qwen35_cache_scratch_bytes(B.make_config(synth.config("4b")), capacity, block, rows) == 0


def test_scratch_grows_with_the_selection_only():
    c = B.make_config(synth.config("4b"))
    small = B.qwen35_cache_scratch_bytes(c, 1 << 31, 0, 1 << 20)
    assert 0 < small < 4 << 20
    assert small == B.qwen35_cache_scratch_bytes(c, 256, 0, 1)
    assert B.qwen35_cache_scratch_bytes(c, 1 << 31, 1024, 1) > small
    assert B.qwen35_cache_scratch_bytes(c, 1 << 17, 16, 2048) == B.qwen35_cache_scratch_bytes(c, 1 << 17, 16, 1 << 20)
