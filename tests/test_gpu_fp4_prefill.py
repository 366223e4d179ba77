"""Chunked prefill over 4-bit pools, against softmax attention in fp64 (fp4_ref.py derives the tolerance)."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests import fp4_ref as ref

pytestmark = pytest.mark.gpu
ACT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


def run(p, chunks, n_q, act, out, max_q=None, seed=3):
    start = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    scale = 1 / math.sqrt(p.d)
    q = ref.draw_q(seed, (int(start[-1]), n_q, p.d), ACT[act])
    o = torch.full((len(q) + 3, n_q, p.d), 9.0, dtype=ACT[out], device="cuda")
    pa.pa_prefill_chunk(o[:len(q)], q, p.kc, p.vc, p.tables, torch.from_numpy(start).cuda(), p.context,
                        max(chunks) if max_q is None else max_q, scale, p.bs, **p.scales)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    assert (o[len(q):] == 9).all()                           # rows behind the last request
    q64 = q.double().cpu().numpy()
    want = [ref.attend(q64[start[r]:start[r + 1]], p.k[r], p.v[r], n - chunks[r] + np.arange(chunks[r]), scale)
            for r, n in enumerate(p.lens) if chunks[r]]
    ref.check(o[:len(q)], np.concatenate(want), ref.tolerance(p.vmax), ACT[out])


@pytest.mark.parametrize("chunks,ctx", [([1], [0]), ([1], [500]), ([16, 1, 33], [0, 130, 15]), ([129], [127]),
                                        ([300, 0, 7], [100, 64, 900]), ([257, 64], [1500, 1]), ([5] * 70, [3] * 70)],
                         ids=lambda x: str(x[:3]))
@pytest.mark.parametrize("n_q,n_kv,d,bs,act", [(8, 2, 128, 16, "bf16"), (8, 2, 128, 32, "fp16"), (16, 4, 64, 16, "fp16"),
                                               (3, 1, 64, 32, "bf16")])
def test_prefill(chunks, ctx, n_q, n_kv, d, bs, act):
    p = ref.Pools(sum(chunks) + d, [a + b for a, b in zip(chunks, ctx)], n_kv, d, bs)
    run(p, chunks, n_q, act, "fp32")


@pytest.mark.parametrize("chunks,ctx", [([70], [5000]), ([5, 70], [0, 4500]), ([300], [2100]), ([1, 1, 1], [2047, 2048, 3])],
                         ids=str)
@pytest.mark.parametrize("n_q,n_kv,d,bs,act,out", [(8, 2, 128, 16, "bf16", "fp32"), (4, 1, 64, 32, "fp16", "fp16"),
                                                   (5, 1, 128, 32, "fp16", "fp32"), (8, 2, 64, 16, "bf16", "bf16")])
def test_few_rows_over_long_contexts(chunks, ctx, n_q, n_kv, d, bs, act, out):
    """calls whose key tiles are split over clusters of up to 8 blocks, some of whose ranges are empty"""
    run(ref.Pools(sum(ctx) + d, [a + b for a, b in zip(chunks, ctx)], n_kv, d, bs), chunks, n_q, act, out)


@pytest.mark.parametrize("act,out", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp16"), ("fp16", "bf16")])
def test_outputs_in_16_bits(act, out):
    run(ref.Pools(4, [200, 333], 2, 128, 16), [150, 40], 8, act, out)


def test_full_multi_head_and_a_loose_bound():
    run(ref.Pools(6, [400, 77], 6, 64, 16), [90, 77], 6, "bf16", "fp32", max_q=513)


def test_chunk_longer_than_its_bound_is_flagged():
    p = ref.Pools(8, [100], 1, 64, 16)
    q = ref.draw_q(1, (100, 4, 64), torch.bfloat16)
    o = torch.zeros(100, 4, 64, device="cuda")
    pa.pa_prefill_chunk(o, q, p.kc, p.vc, p.tables, torch.tensor([0, 100], dtype=torch.int32, device="cuda"), p.context,
                        64, 0.125, 16, **p.scales)
    assert pa.pa_get_device_error() == pa.PA_ERR_OUT_OF_RANGE


def test_block_ids_outside_the_pool_are_flagged():
    p = ref.Pools(10, [100, 60], 1, 64, 16)
    p.tables[0, 1] = -3
    q = ref.draw_q(1, (30, 4, 64), torch.bfloat16)
    o = torch.zeros(30, 4, 64, device="cuda")
    start = torch.tensor([0, 20, 30], dtype=torch.int32, device="cuda")
    pa.pa_prefill_chunk(o, q, p.kc, p.vc, p.tables, start, p.context, 20, 0.125, 16, **p.scales)
    assert pa.pa_get_device_error() == pa.PA_ERR_OUT_OF_RANGE
    want = ref.attend(q[20:].double().cpu().numpy(), p.k[1], p.v[1], 50 + np.arange(10), 0.125)
    ref.check(o[20:], want, ref.tolerance(p.vmax), torch.float32)
