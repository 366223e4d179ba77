"""Attention over 4-bit pools whose scores are far apart: keys that move a row's reference again and again, and pieces of a
row with very different maxima.

Tolerances (fp32 outputs, |v| <= vmax): a probability enters P V as one fp16 part, off by at most half a step, 2^-11
of itself, or, below the smallest normal number, by 2^-25 under a reference that lies 7 powers of two below the row's
largest score: 2^-32.  So an output moves by at most (2^-11 + keys 2^-32) vmax.  A score is a sum of exact products
whose magnitudes add up to A (in nats); each of at most 136 additions rounds or cuts off 2^-23 A at most, and an
output moves by at most twice the error of the scores, times vmax."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests import fp4_ref as ref

pytestmark = pytest.mark.gpu
ACT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LOG2E = 1 / math.log(2)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


FACTORS = np.array([1, 0.5, -1, 0.25])      # of the heads: how strongly a query sees the planted keys

# the planted keys' heights above the rest (powers of two of their weights), in the order of their places, of the sequences
# in turn: one late key, rising, falling, mixed ones
HEIGHTS = [9.5], [12, 30, 60, 95, 150], [150, 95, 60, 30, 12], [20, 140, 9, 60, 141, 30]


def plant(p, seed):
    """K rows of every sequence: small ones, and one per height at places of its own (in order), whose first 16 elements
    make the height for a query of ones"""
    rng = np.random.default_rng(seed)
    scale, ks = 1 / math.sqrt(p.d), p.scales["k_scale"]
    for s, n in enumerate(p.lens):
        heights = HEIGHTS[s % len(HEIGHTS)]
        rows = 0.25 * rng.standard_normal((n, p.n_kv, p.d)).astype(np.float32)
        rows[..., :16] = 0
        at = np.sort(rng.choice(n, min(n, len(heights)), replace=False))
        if len(heights) == 1:
            at[:] = n - 1 - n // 50
        for t, h in zip(at, heights):
            rows[t, :, :16] = h / (16 * scale * LOG2E)
        data, t = ref.quantise(rows, ks), np.arange(n)
        p.host_pools[0][p.host_tables[s, t // p.bs], :, t % p.bs] = data
        p.k[s] = ref.values(data, ks)
    p.kc.copy_(torch.from_numpy(p.host_pools[0]))


def queries(seed, shape, act):
    """N(0, 1) but for the first 16 elements: one of FACTORS by the head"""
    q = ref.draw_q(seed, shape, torch.float32)
    q[..., :16] = torch.from_numpy(FACTORS[np.arange(shape[-2]) % 4]).float().cuda()[:, None]
    return q.to(ACT[act])


def tolerance(p, scale, q):
    # A: the planted part (a group's scale is off by 1/16 at most), and of the others no more than |q| |k|
    a = max(map(max, HEIGHTS)) / LOG2E * 1.1
    a += scale * q.float()[..., 16:].norm(dim=-1).max().item() * max(np.linalg.norm(k[..., 16:], axis=-1).max() for k in p.k)
    return p.vmax * (2 * 136 * 2.0 ** -23 * a + 2.0 ** -20 + 2.0 ** -11 + max(p.lens) * 2.0 ** -32)


def attend(q, k, v, pos, scale):
    """as fp4_ref.attend, by matrix products"""
    rows, n_q, d = q.shape
    n_kv, g = k.shape[1], n_q // k.shape[1]
    z = q.reshape(rows, n_kv, g, d).transpose(1, 0, 2, 3).reshape(n_kv, rows * g, d) @ k.transpose(1, 2, 0) * scale
    z = np.where(np.arange(len(k)) <= np.repeat(pos, g)[:, None], z, -np.inf)
    p = np.exp(z - z.max(-1, keepdims=True))
    o = p @ v.transpose(1, 0, 2) / p.sum(-1, keepdims=True)
    return o.reshape(n_kv, rows, g, d).transpose(1, 0, 2, 3).reshape(q.shape)


def workspace(p, rows, n_q):
    n = pa.pa_decode_verify_workspace_size(len(p.lens), rows, n_q, p.n_kv, p.d, p.bs, p.max_ctx)
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def run_decode(p, rows, n_q, act):
    scale = 1 / math.sqrt(p.d)
    plant(p, rows + n_q)
    q = queries(rows, (len(p.lens), rows, n_q, p.d), act)
    out = torch.full(q.shape, float("nan"), device="cuda")
    if rows == 1:
        pa.pa_decode(out[:, 0], q[:, 0], p.kc, p.vc, p.tables, p.context, scale, p.bs, workspace(p, 1, n_q), **p.scales)
    else:
        pa.pa_decode_verify(out, q, p.kc, p.vc, p.tables, p.context, scale, p.bs, workspace(p, rows, n_q), **p.scales)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    q64 = q.double().cpu().numpy()
    want = np.stack([attend(q64[s], p.k[s], p.v[s], n - rows + np.arange(rows), scale) for s, n in enumerate(p.lens)])
    ref.check(out, want, tolerance(p, scale, q), torch.float32)


# rows of a KV head: 4, 8 and 16 a unit of work, and more than the decode kernel takes
@pytest.mark.parametrize("rows,n_q,n_kv,d,bs,act", [(1, 8, 2, 128, 16, "bf16"), (1, 16, 2, 64, 32, "fp16"), (1, 16, 1, 128, 32, "bf16"),
                                                    (3, 4, 4, 64, 16, "bf16"), (4, 4, 2, 128, 16, "fp16"), (5, 6, 2, 64, 16, "bf16"),
                                                    (8, 12, 2, 128, 16, "bf16")])
def test_rows_split_over_blocks(rows, n_q, n_kv, d, bs, act):
    """few rows: a piece is one stage, and the merge sees the maxima"""
    run_decode(ref.Pools(rows + d, [700, 3000, 2500, 1700, 150 + rows, 160, 900, 2100], n_kv, d, bs), rows, n_q, act)


@pytest.mark.parametrize("rows,n_q,n_kv,d,bs,act", [(1, 32, 8, 128, 16, "bf16"), (1, 64, 8, 64, 16, "fp16"), (2, 16, 8, 64, 32, "bf16"),
                                                    (4, 32, 8, 128, 32, "bf16"), (3, 10, 10, 128, 16, "fp16")])
def test_runs_of_several_stages(rows, n_q, n_kv, d, bs, act):
    """more work than thread blocks: a block's reference moves within its runs"""
    run_decode(ref.Pools(rows + d, [40 + (i * 613) % 2900 for i in range(40)], n_kv, d, bs), rows, n_q, act)


@pytest.mark.parametrize("chunks,ctx,n_q,n_kv,d,bs,act", [
    ([9, 70, 1], [100, 5000, 4000], 8, 2, 128, 16, "bf16"), ([5, 40, 7, 3], [100, 4500, 900, 2000], 4, 1, 64, 32, "fp16"),   # split over clusters
    ([300, 257, 30, 70], [1000, 64, 3000, 500], 32, 8, 128, 16, "bf16"), ([290, 90] * 3, [700, 1500] * 3, 16, 8, 64, 16, "fp16")])
def test_prefill(chunks, ctx, n_q, n_kv, d, bs, act):
    p = ref.Pools(sum(chunks), [a + b for a, b in zip(chunks, ctx)], n_kv, d, bs)
    scale = 1 / math.sqrt(d)
    plant(p, d)
    start = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    q = queries(3, (int(start[-1]), n_q, d), act)
    out = torch.full(q.shape, float("nan"), device="cuda")
    pa.pa_prefill_chunk(out, q, p.kc, p.vc, p.tables, torch.from_numpy(start).cuda(), p.context, max(chunks), scale, bs, **p.scales)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    q64 = q.double().cpu().numpy()
    want = [attend(q64[start[r]:start[r + 1]], p.k[r], p.v[r], n - chunks[r] + np.arange(chunks[r]), scale)
            for r, n in enumerate(p.lens)]
    ref.check(out, np.concatenate(want), tolerance(p, scale, q), torch.float32)
