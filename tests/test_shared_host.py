"""CPU checks of the shared-prefix decode: the grouping of a batch's tables against
brute force, workspace rules and refusals before any launch."""
import ctypes as C
import functools

import numpy as np
import pytest

from paged_kv_cache_25_gb300 import binding as pa
from paged_kv_cache_25_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    return pa.lib()


def _full(tables, lens, bs):
    out = []
    for row, n in zip(tables, lens):
        r = []
        for b in row[:min(max(n, 0) // bs, len(row))]:
            if b < 0:
                break
            r.append(int(b))
        out.append(tuple(r))
    return out


def _best_saving(rows, need):
    """most block reads that nested choices of groups save"""
    @functools.lru_cache(None)
    def best(members, depth):
        if len(members) < 2:
            return 0
        run = depth
        while all(len(rows[m]) > run for m in members) and len({rows[m][run] for m in members}) == 1:
            run += 1
        own = (len(members) - 1) * run if run >= need else 0
        by = {}
        for m in members:
            if len(rows[m]) > run:
                by.setdefault(rows[m][run], []).append(m)
        return max(own, sum(best(tuple(v), run) for v in by.values()))
    return best(tuple(range(len(rows))), 0)


@pytest.mark.parametrize("seed", range(40))
def test_groups_save_the_most(seed):
    rng = np.random.default_rng(seed)
    bs = int(rng.choice([16, 32]))
    B, mb = int(rng.integers(1, 30)), int(rng.integers(1, 12))
    # tables of a random tree: a sequence copies a random earlier one's leading blocks
    tables = rng.permutation(B * mb).reshape(B, mb).astype(np.int32)
    for s in range(1, B):
        n = int(rng.integers(0, mb + 1))
        tables[s, :n] = tables[rng.integers(0, s), :n]
    lens = rng.integers(0, mb * bs + 1, B).astype(np.int32)
    for s in range(B):
        tables[s, -(-int(lens[s]) // bs):] = -1
    need = int(rng.choice([0, 0, 2 * bs - 1]))
    group, prefix = pa.pa_shared_prefix_groups(tables, lens, bs, need)
    rows = _full(tables, lens, bs)
    saved = 0
    for g in range(len(prefix)):
        who = np.flatnonzero(group == g)
        n = int(prefix[g]) // bs
        assert len(who) >= 2 and prefix[g] % bs == 0 and prefix[g] >= max(need, 1)
        assert len({rows[s][:n] for s in who}) == 1 and all(len(rows[s]) >= n for s in who)
        saved += (len(who) - 1) * n
    assert group.min() >= -1 and group.max() < len(prefix)
    assert saved == _best_saving(rows, max(1, -(-need // bs)))


def test_groups_of_a_deep_chain_and_of_nothing():
    n = 3000                     # every sequence one block deeper than the one before
    tables = np.tile(np.arange(n, dtype=np.int32), (n, 1))
    lens = (np.arange(n, dtype=np.int32) + 1) * 16
    group, prefix = pa.pa_shared_prefix_groups(tables, lens, 16)
    rows = _full(tables, lens, 16)
    for g in range(len(prefix)):
        who = np.flatnonzero(group == g)
        assert len(who) >= 2 and all(len(rows[s]) * 16 >= prefix[g] for s in who)
    assert len(prefix) >= 1
    assert len(pa.pa_shared_prefix_groups(np.zeros((0, 4), np.int32), [], 16)[1]) == 0
    group, prefix = pa.pa_shared_prefix_groups([[0, 1], [2, 3], [-1, -1]], [32, 32, 0], 16)
    assert len(prefix) == 0 and (group == -1).all()


def test_grouping_refusals():
    f = pa.lib().pa_shared_prefix_groups
    assert f(None, 4, None, 2, 16, 0, None, None) == -1
    assert f(None, 0, None, 2, 16, 0, None, None) == -1
    assert f(None, 4, None, -1, 16, 0, None, None) == -1
    assert f(None, 4, None, 0, 16, 0, None, None) == 0


def _call(dt=2, d=128, B=4, groups=2, gos=0x7000, pl=0x8000, ws=0x10000, ws_bytes=1 << 26, **kw):
    desc = pa._Desc(64, 16, 8, d, dt, 1.0, 1.0, 2)
    a = dict(out=0x1000, q=0x2000, kc=0x3000, vc=0x4000, bt=0x5000, cl=0x6000, n_q=32, scale=0.1,
             bs=16, mb=16)
    a.update(kw)
    return pa.lib().pa_decode_shared(a["out"], 0, a["q"], a["kc"], a["vc"], C.byref(desc), a["bt"],
                                     a["mb"], a["cl"], B, a["n_q"], a["scale"], a["bs"], gos, pl,
                                     groups, ws, ws_bytes, None)


def test_refusals_before_any_launch():
    assert _call(gos=None) == pa.PA_ERR_INVALID_ARG
    assert _call(pl=None) == pa.PA_ERR_INVALID_ARG
    assert _call(gos=0x7002) == pa.PA_ERR_INVALID_ARG
    assert _call(groups=-1) == pa.PA_ERR_INVALID_ARG
    assert _call(groups=1025) == pa.PA_ERR_UNSUPPORTED
    assert _call(dt=0) == pa.PA_ERR_UNSUPPORTED
    assert _call(d=96) == pa.PA_ERR_UNSUPPORTED
    assert _call(q=0x2004) == pa.PA_ERR_INVALID_ARG
    assert _call(n_q=30) == pa.PA_ERR_INVALID_ARG
    assert _call(scale=float("inf")) == pa.PA_ERR_INVALID_ARG
    need = pa.pa_decode_shared_workspace_size(4, 32, 8, 128, 16, 256, 2)
    assert _call(ws_bytes=need - 1) == pa.PA_ERR_WORKSPACE
    assert _call(ws=0x10010) == pa.PA_ERR_INVALID_ARG
    assert _call(B=0) == pa.PA_OK


def test_workspace_rules():
    size = pa.pa_decode_shared_workspace_size
    assert size(256, 32, 8, 128, 16, 4096, 0) == pa.pa_decode_workspace_size(256, 32, 8, 128, 16, 4096)
    # a partial of every row for each range of the prefix (at most 152 / 8 = 19 of them here)
    assert size(256, 32, 8, 128, 16, 4096, 1) >= 256 * 32 * (19 + 4) * 130 * 4
    assert size(256, 32, 8, 128, 16, 4096, 1025) == 0
    assert size(256, 32, 8, 128, 16, 4096, -1) == 0
    assert size(256, 30, 8, 128, 16, 4096, 1) == 0
