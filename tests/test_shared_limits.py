"""CPU checks of pa_shared_prefix_groups at its limits: thresholds up to the
largest int, more pairs than a call has groups."""
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


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2048])
def test_as_many_groups_as_a_call_takes(n):
    blocks = 1 + np.random.default_rng(n).permutation(n) % 7
    tables, lens = pairs(blocks)
    group, prefix = pa.pa_shared_prefix_groups(tables, lens, 16)
    kept = min(n, 1024)
    assert len(prefix) == kept
    assert pa.pa_decode_shared_workspace_size(len(lens), 8, 2, 64, 16, 1 << 14, len(prefix)) > 0
    # the groups that save the most, numbered without gaps, and each member's prefix its own
    assert sorted(prefix // 16) == sorted(blocks)[n - kept:]
    assert np.array_equal(np.unique(group[group >= 0]), np.arange(kept))
    for s, g in enumerate(group):
        assert g == group[s ^ 1]
        assert g < 0 or prefix[g] == 16 * blocks[s // 2]


def test_what_a_dropped_pair_saves_is_the_least():
    """A group of many members on one block outweighs a pair on several."""
    tables, lens = pairs([3] * 1024)
    more = np.full((9, tables.shape[1]), -1, np.int32)
    more[:, 0] = tables.max() + 1
    more[:, 1] = tables.max() + 2 + np.arange(9)
    group, prefix = pa.pa_shared_prefix_groups(np.concatenate([tables, more]),
                                               np.concatenate([lens, np.full(9, 32, np.int32)]), 16)
    assert len(prefix) == 1024 and (group < 0).sum() == 2
    assert len(set(group[-9:])) == 1 and prefix[group[-1]] == 16


@pytest.mark.parametrize("least", [2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 17])
def test_a_threshold_near_the_largest_int_leaves_no_group(least):
    tables, lens = pairs([2, 5])
    group, prefix = pa.pa_shared_prefix_groups(tables, lens, 16, least)
    assert len(prefix) == 0 and (group == -1).all()
