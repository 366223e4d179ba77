"""CPU check of pa_decode_scored's workspace: one sized without a window serves every window."""
import random

import pytest

from paged_kv_cache_25_gb300 import binding as pa
from paged_kv_cache_25_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    return pa.lib()


SHAPES = [(32, 2, 1, 1, 32, 8192, 2259), (4, 1, 8, 1, 16, 32768, 18759), (1, 4, 8, 4, 16, 32768, 18903)]


@pytest.mark.parametrize("seed", range(8))
def test_a_workspace_without_a_window_is_enough_for_any(seed):
    rng = random.Random(seed)
    shapes = list(SHAPES)
    for _ in range(4000):
        n_kv, bs = rng.choice([1, 2, 4, 8]), rng.choice([16, 32])
        shapes.append((rng.choice([1, 2, 4, 8, 16, 32, 64, 100, 256, 1000]), rng.choice([1, 1, 2, 4, 16]),
                       n_kv * rng.choice([1, 2, 4, 8]), n_kv, bs,
                       rng.choice([512, 1000, 2048, 4096, 10000, 32768, 10 ** 6]) // bs * bs, rng.randint(1, 40000)))
    for B, nq, n_q, n_kv, bs, ctx, window in shapes:
        size = lambda w: pa.pa_decode_scored_workspace_size(B, nq, n_q, n_kv, 128, bs, ctx, w)  # noqa: E731
        assert 256 <= size(window) <= size(0), (B, nq, n_q, n_kv, bs, ctx, window)
