"""4-bit pools: lengths past the block table, on both sides of the number of rows that the decode kernel takes."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests import fp4_ref as ref

pytestmark = pytest.mark.gpu
ACT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("width,bs", [(12, 16), (9, 32), (41, 16)])
@pytest.mark.parametrize("rows,n_q,n_kv,d,act,seqs", [
    (1, 8, 2, 128, "bf16", 3), (16, 1, 1, 64, "fp16", 3), (1, 40, 1, 128, "bf16", 3), (16, 6, 2, 64, "bf16", 3), (5, 8, 1, 128, "fp16", 90)])
def test_rows_past_the_table_are_clamped_away(rows, n_q, n_kv, d, act, seqs, width, bs):
    """a query row sees the table's keys up to its own position, whatever the number of rows a KV head"""
    full = width * bs
    p = ref.Pools(rows + d, [full] * seqs, n_kv, d, bs)
    lens = [full + x for x in ((5, 0, 300) * seqs)[:seqs]]
    p.context.copy_(torch.tensor(lens, dtype=torch.int32))
    scale = 1 / math.sqrt(d)
    q = ref.draw_q(2, (seqs, rows, n_q, d), ACT[act])
    out = torch.full(q.shape, float("nan"), device="cuda")
    ws = torch.empty(pa.pa_decode_verify_workspace_size(seqs, rows, n_q, n_kv, d, bs, full), dtype=torch.uint8, device="cuda")
    pa.pa_decode_verify(out, q, p.kc, p.vc, p.tables, p.context, scale, bs, ws, **p.scales)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    q64 = q.double().cpu().numpy()
    want = np.stack([ref.attend(q64[s], p.k[s], p.v[s], n - rows + np.arange(rows), scale) for s, n in enumerate(lens)])
    # (as fp4_ref derives it, with 2^-11 for half a step of an fp16 part, and 2^-32 a key)
    ref.check(out, want, p.vmax * (2 * 5e-5 + 2.0 ** -20 + 2.0 ** -11 + full * 2.0 ** -32), torch.float32)
