"""Decode and multi-row decode over 4-bit pools, against softmax attention in fp64 (fp4_ref.py derives the
tolerance)."""
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


def workspace(p, rows, n_q):
    n = pa.pa_decode_verify_workspace_size(len(p.lens), rows, n_q, p.n_kv, p.d, p.bs, p.max_ctx)
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def call(p, q, out, ws, scale, **kw):
    f = pa.pa_decode if q.dim() == 3 else pa.pa_decode_verify
    f(out, q, p.kc, p.vc, p.tables, p.context, scale, p.bs, ws, **p.scales, **kw)


def want(p, q, scale):
    q = q.double().cpu().numpy()
    q = q[:, None] if q.ndim == 3 else q
    nq = q.shape[1]
    return np.stack([ref.attend(q[s], p.k[s], p.v[s], n - nq + np.arange(nq), scale)
                     for s, n in enumerate(p.lens)])


def run(p, rows, n_q, act, out, scale=None, seed=3):
    scale = 1 / math.sqrt(p.d) if scale is None else scale
    shape = (len(p.lens), n_q, p.d) if rows == 1 else (len(p.lens), rows, n_q, p.d)
    q = ref.draw_q(seed, shape, ACT[act])
    o = torch.full(shape, float("nan"), dtype=ACT[out], device="cuda")
    call(p, q, o, workspace(p, rows, n_q), scale)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    ref.check(o, want(p, q, scale).reshape(shape), ref.tolerance(p.vmax), ACT[out])


@pytest.mark.parametrize("lens", [[1], [2, 15, 16, 17], [31, 32, 33, 1, 64], [127, 128, 129], [1023, 1024, 1025],
                                  [3000, 1, 700, 16], [5000]], ids=str)
@pytest.mark.parametrize("n_q,n_kv,d,bs,act", [(8, 2, 128, 16, "bf16"), (32, 4, 64, 16, "bf16"),
                                               (3, 3, 64, 32, "fp16"), (10, 2, 128, 32, "fp16"),
                                               (16, 1, 128, 16, "bf16"), (24, 2, 64, 16, "fp16")])
def test_decode(lens, n_q, n_kv, d, bs, act):
    run(ref.Pools(sum(lens) + d, lens, n_kv, d, bs), 1, n_q, act, "fp32")


@pytest.mark.parametrize("out", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["bf16", "fp16"])
def test_outputs_in_16_bits(act, out):
    run(ref.Pools(5, [300, 17, 2050], 2, 128, 16), 1, 8, act, out)


@pytest.mark.parametrize("rows", [2, 3, 4, 5, 8, 13, 16])
@pytest.mark.parametrize("n_q,n_kv,d,bs,act", [(4, 4, 128, 16, "fp16"), (8, 2, 64, 16, "bf16"),
                                               (5, 1, 128, 32, "bf16"), (16, 2, 64, 32, "fp16")])
def test_several_rows(rows, n_q, n_kv, d, bs, act):
    lens = [rows, rows + 1, 16 + rows, 130, 1029, 2500]
    run(ref.Pools(rows + d, lens, n_kv, d, bs), rows, n_q, act, "fp32")


@pytest.mark.parametrize("rows,n_q,n_kv,d,bs,act", [(1, 32, 8, 128, 16, "bf16"), (1, 8, 8, 128, 32, "fp16"),
                                                    (3, 16, 8, 128, 16, "fp16"), (1, 32, 8, 64, 32, "bf16"),
                                                    (7, 10, 10, 64, 16, "bf16"), (5, 24, 6, 128, 32, "bf16")])
def test_batches_with_long_runs_of_whole_and_split_rows(rows, n_q, n_kv, d, bs, act):
    """more work than thread blocks: runs of several rows, begun and ended inside rows, with ragged ends"""
    run(ref.Pools(rows + d, [20 + (i * 613) % 2900 for i in range(48)], n_kv, d, bs), rows, n_q, act, "fp32")


def test_many_sequences_of_all_lengths():
    lens = [1 + (i * 7919) % 260 for i in range(1100)]      # more than the kernel keeps prefix sums for
    run(ref.Pools(9, lens, 1, 64, 16), 1, 4, "bf16", "fp32")


def test_wide_table_and_long_context():
    p = ref.Pools(11, [40000, 33], 1, 64, 16, max_blocks=4000)
    run(p, 1, 2, "bf16", "fp32")


@pytest.mark.parametrize("k_scale,v_scale,scale", [(3.0, 1.0 / 512, 0.02), (2.0 ** -12, 7.5, 40.0), (1 / 16, 1 / 32, 0.0),
                                                   (1 / 16, 1 / 32, -0.1)])
def test_scales(k_scale, v_scale, scale):
    # (the rows are N(0, 1) whatever the pool's scales: these move the groups' scales)
    run(ref.Pools(21, [200, 1029], 2, 128, 16, k_scale, v_scale), 1, 8, "bf16", "fp32",
        scale=scale if abs(scale) < 1 else 0.09)


def test_large_and_tiny_queries():
    """bf16 queries far outside fp16's range (scores near zero or one-hot)"""
    p = ref.Pools(31, [65], 1, 128, 16)
    for factor, scale in ((2.0 ** 100, 2.0 ** -103), (2.0 ** -90, 2.0 ** 87)):
        q = (ref.draw_q(5, (1, 4, 128), torch.float32) * factor).to(torch.bfloat16)
        o = torch.empty(1, 4, 128, device="cuda")
        call(p, q, o, workspace(p, 1, 4), scale)
        assert pa.pa_get_device_error() == 0
        ref.check(o, want(p, q, scale)[:, 0], ref.tolerance(p.vmax), torch.float32)


def test_a_nan_row_reaches_the_sequences_that_see_it():
    p = ref.Pools(41, [50, 50], 1, 64, 16)
    b, o = p.host_tables[0, 1], 3
    p.vc[b, 0, o, 32] = 0x7F                 # token 19, elements 0 - 15 of V
    q = ref.draw_q(6, (2, 4, 64), torch.bfloat16)
    out = torch.empty(2, 4, 64, device="cuda")
    call(p, q, out, workspace(p, 1, 4), 0.125)
    got = out.cpu().numpy()
    assert np.isnan(got[0, :, :16]).all() and np.isfinite(got[0, :, 16:]).all() and np.isfinite(got[1]).all()


def test_block_ids_outside_the_pool_are_flagged():
    p = ref.Pools(51, [100, 40], 2, 128, 16)
    p.tables[0, 2] = p.kc.shape[0]
    q = ref.draw_q(7, (2, 8, 128), torch.bfloat16)
    out = torch.zeros(2, 8, 128, device="cuda")
    call(p, q, out, workspace(p, 1, 8), 0.1)
    assert pa.pa_get_device_error() == pa.PA_ERR_OUT_OF_RANGE
    ref.check(out[1], want(p, q, 0.1)[1, 0], ref.tolerance(p.vmax), torch.float32)


def test_fewer_keys_than_rows_is_flagged():
    p = ref.Pools(61, [3, 40], 2, 128, 16)
    q = ref.draw_q(8, (2, 4, 8, 128), torch.bfloat16)
    out = torch.full((2, 4, 8, 128), 5.0, device="cuda")
    call(p, q, out, workspace(p, 4, 8), 0.1)
    assert pa.pa_get_device_error() == pa.PA_ERR_OUT_OF_RANGE
    assert (out[0] == 5).all()
    ref.check(out[1], ref.attend(q[1].double().cpu().numpy(), p.k[1], p.v[1], 36 + np.arange(4), 0.1),
              ref.tolerance(p.vmax), torch.float32)


def test_results_do_not_change_from_call_to_call():
    p = ref.Pools(71, [2000, 5, 900, 4100], 4, 128, 16)
    q = ref.draw_q(9, (4, 16, 128), torch.bfloat16)
    ws = workspace(p, 1, 16)
    outs = []
    for _ in range(3):
        o = torch.empty(4, 16, 128, device="cuda")
        call(p, q, o, ws, 0.09)
        outs.append(o)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("rows,n_q,n_kv,d,bs,act,out,seqs", [
    (1, 40, 1, 128, 16, "bf16", "bf16", 5), (1, 48, 1, 64, 32, "fp16", "fp32", 3), (16, 8, 2, 128, 16, "bf16", "fp32", 5),
    (16, 32, 1, 64, 16, "fp16", "fp16", 4), (9, 8, 2, 128, 32, "fp16", "fp32", 70), (11, 3, 1, 64, 16, "bf16", "fp32", 1),
    (16, 64, 4, 128, 16, "bf16", "bf16", 2), (16, 17, 1, 128, 16, "bf16", "fp32", 3)])
def test_more_rows_than_the_decode_kernel_takes(rows, n_q, n_kv, d, bs, act, out, seqs):
    lens = [rows + (i * 811) % 2600 for i in range(seqs)]
    run(ref.Pools(rows + n_q, lens, n_kv, d, bs), rows, n_q, act, out)


@pytest.mark.parametrize("rows,n_q", [(4, 8), (16, 8)])
def test_padded_batches(rows, n_q):
    """sequences of length 0 (padding) are no error, and the others are what they are without them; too short
    ones are flagged and left alone"""
    p = ref.Pools(81, [700, 40, 40, 40, 95], 2, 128, 16)
    p.context[2:4] = 0
    q = ref.draw_q(8, (5, rows, n_q, 128), torch.bfloat16)
    out = torch.full(q.shape, 5.0, device="cuda")
    call(p, q, out, workspace(p, rows, n_q), 0.1)
    assert pa.pa_get_device_error() == 0
    for s in (0, 1, 4):
        w = ref.attend(q[s].double().cpu().numpy(), p.k[s], p.v[s], p.lens[s] - rows + np.arange(rows), 0.1)
        ref.check(out[s], w, ref.tolerance(p.vmax), torch.float32)
    p.context[2] = rows - 1
    out.fill_(5.0)
    call(p, q, out, workspace(p, rows, n_q), 0.1)
    assert pa.pa_get_device_error() == pa.PA_ERR_OUT_OF_RANGE
    assert (out[2] == 5).all()
    ref.check(out[4], w, ref.tolerance(p.vmax), torch.float32)


def test_lengths_of_a_captured_call_of_many_rows():
    p = ref.Pools(83, [1500, 300], 1, 64, 16)
    q = ref.draw_q(9, (2, 16, 4, 64), torch.bfloat16)
    out, ws = torch.zeros(q.shape, device="cuda"), workspace(p, 16, 4)
    call(p, q, out, ws, 0.125)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(p, q, out, ws, 0.125)
    for lens in ([1500, 300], [16, 299], [1000, 17]):
        p.context.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        for s, n in enumerate(lens):
            w = ref.attend(q[s].double().cpu().numpy(), p.k[s][:n], p.v[s][:n], n - 16 + np.arange(16), 0.125)
            ref.check(out[s], w, ref.tolerance(p.vmax), torch.float32)
    assert pa.pa_get_device_error() == 0
