"""Shared decode of a batch with more pairs than a call has groups, grouped from its tables,
against fp64 attention.  Tolerances: see scored_ref."""
import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests import test_gpu_shared as shared
from tests.scored_ref import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("form", ["fp16-g2-d64", "fp8-g8-d64"])
def test_more_pairs_than_groups(form):
    n_q, n_kv, d, bs, dtype, fp8 = shared.FORMS[form]
    c = shared.Case(800, [(16 * (1 + i % 5), [1 + i % 30, 3]) for i in range(1100)], [50], n_q, n_kv, d, bs, dtype,
                    fp8=fp8)
    group, prefix = pa.pa_shared_prefix_groups(c.p.tables, c.p.lens, bs)
    assert len(prefix) == 1024 and (group < 0).sum() == 2201 - 2048
    c.gd, c.pd = torch.from_numpy(group).cuda(), torch.from_numpy(prefix).cuda()
    size = pa.pa_decode_shared_workspace_size(len(group), n_q, n_kv, d, bs, c.p.max_ctx, len(prefix))
    c.ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    out = c.run()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    check(out, c.ref(), 2e-3)
