"""NaN in chunked prefills, whose key tiles are split over a cluster or not: the rows that see one are NaN, the others are not."""
import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests import fp4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("scored", [False, True], ids=["fp4", "scored"])
@pytest.mark.parametrize("chunk,ctx", [(70, 5000), (300, 300)], ids=["split", "whole"])
def test_a_nan_query_row_gives_a_nan_row(chunk, ctx, scored):
    p = ref.Pools(3, [ctx + chunk], 2, 128, 16)
    start = torch.tensor([0, chunk], dtype=torch.int32, device="cuda")
    q = ref.draw_q(4, (chunk, 8, 128), torch.bfloat16)
    out = torch.zeros(q.shape, device="cuda")
    bad = torch.zeros(chunk, 8, dtype=torch.bool, device="cuda")
    bad[3, 5] = bad[chunk - 1, 0] = True
    q[3, 5, 17] = q[chunk - 1, 0, 100] = float("nan")
    if scored:
        kc, vc = (torch.randn(*p.kc.shape[:3], 128, device="cuda").bfloat16() for _ in range(2))
        pa.pa_prefill_scored(out, q, kc, vc, p.tables, start, p.context, chunk, pa.ScoreMod(window=100000), 0.09, 16)
    else:
        pa.pa_prefill_chunk(out, q, p.kc, p.vc, p.tables, start, p.context, chunk, 0.09, 16, **p.scales)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad)


@pytest.mark.parametrize("token", [0, 3000, 5069])
@pytest.mark.parametrize("of", ["k", "v"])
def test_a_nan_key_reaches_the_rows_that_see_it(token, of):
    """one range of a call that is split over clusters"""
    p = ref.Pools(3, [5070], 2, 128, 16)
    pool = p.kc if of == "k" else p.vc
    pool[int(p.host_tables[0, token // 16]), 1, token % 16, 64 + 7] = 0x7F        # KV head 1, elements 112 - 127
    q = ref.draw_q(4, (70, 8, 128), torch.bfloat16)
    if token == 0 and of == "v":     # beside a key so far above it that its range weighs nothing
        q[:, 4:] = 0
        q[:, 4:, :16] = 64
        b = int(p.host_tables[0, 4000 // 16])
        p.kc[b, 1, 4000 % 16, :8], p.kc[b, 1, 4000 % 16, 64] = 0x77, 0x7E
    start = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    out = torch.zeros(q.shape, device="cuda")
    pa.pa_prefill_chunk(out, q, p.kc, p.vc, p.tables, start, p.context, 70, 0.09, 16, **p.scales)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    nan = out.isnan().cpu().numpy()
    sees = np.arange(5000, 5070) >= token
    assert not nan[:, :4].any()
    if of == "k":
        assert (nan[:, 4:] == sees[:, None, None]).all()
    else:          # (a V row that holds NaN in the rows' last key tile may reach rows before it: its probability is 0)
        assert nan[sees][:, 4:, 112:].all() and not nan[:, 4:, :112].any()
