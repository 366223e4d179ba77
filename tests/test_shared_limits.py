"""CPU checks of pa_shared_prefix_groups at its limits: thresholds up to the largest int."""
import numpy as np
import pytest

from paged_kv_cache_25_gb300 import binding as pa
from paged_kv_cache_25_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    return pa.lib()


def pairs(blocks, own=1):
    """tables and lengths of two sequences for each entry: that many common blocks, then their own"""
    width = max(blocks) + own
    tables = np.full((2 * len(blocks), width), -1, np.int32)
    at = 0
    for i, n in enumerate(blocks):
        tables[2 * i:2 * i + 2, :n] = np.arange(at, at + n)
        at += n
        for s in (2 * i, 2 * i + 1):
            tables[s, n:n + own] = np.arange(at, at + own)
            at += own
    return tables, (np.repeat(blocks, 2) + own).astype(np.int32) * 16


@pytest.mark.parametrize("least", [2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 17])
def test_a_threshold_near_the_largest_int_leaves_no_group(least):
    tables, lens = pairs([2, 5])
    group, prefix = pa.pa_shared_prefix_groups(tables, lens, 16, least)
    assert len(prefix) == 0 and (group == -1).all()
