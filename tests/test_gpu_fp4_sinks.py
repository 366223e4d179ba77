"""Attention over 4-bit pools of one key far above a long flat rest, whose probabilities are each next to nothing and together
are not.

One key lies 17.4 nats above all others: e^-17.4 = 2^-25.1 is nothing in fp16.  Queries are ones; the key's row starts with 16
elements of 6 and its v is 0, the others' K is 0 and their v is 1.  All scores are exact.

Tolerance: a probability enters P V as one fp16 part, off by half a step, 2^-11 of itself, or, below the smallest normal
number, by 2^-25 under a reference that lies 7 powers of two below the row's largest score: 2^-32.  A row's rest weighs
w = (keys - 1) e^-17.4, and its output is w / (1 + w): it moves by 2^-11 of itself, by 2^-32 a key, and by the sums' roundings
(2^-23 of the output a key at worst)."""
import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa

pytestmark = pytest.mark.gpu
NATS = 17.4


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


def sink_pool(blocks, n_kv, d, bs, token):
    """one sequence's K and V in blocks 0 .. blocks - 1 (scales 1.0: 0x38)"""
    kc, vc = (torch.zeros(blocks, n_kv, bs, 9 * d // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    kc[..., d // 2:] = vc[..., d // 2:] = 0x38
    vc[..., :d // 2] = 0x22
    kc[token // bs, :, token % bs, :8] = 0x77
    vc[token // bs, :, token % bs, :d // 2] = 0
    return kc, vc


def check_sink(out, keys, scale):
    """keys: of each row (broadcast over the heads)"""
    keys = np.asarray(keys, np.float64)
    w = (keys - 1) * np.exp(-96 * np.float64(np.float32(scale)))
    want = w / (1 + w)
    tol = want * (2.0 ** -11 + keys * 2.0 ** -23) + keys * 2.0 ** -32
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - want.reshape(want.shape + (1,) * (out.dim() - want.ndim)))
    worst = err.reshape(*want.shape, -1).max(-1)
    assert np.isfinite(worst).all() and (worst <= tol).all(), (worst.max(), (worst / tol).max())


@pytest.mark.parametrize("rows,n_q,n_kv,d,seqs,blocks", [(1, 8, 8, 64, 64, 32768), (2, 16, 4, 128, 64, 16384), (1, 32, 2, 64, 128, 32768),
                                                         (5, 8, 1, 64, 160, 8192)])
def test_a_long_flat_rest_below_one_key(rows, n_q, n_kv, d, seqs, blocks):
    """long runs of a block (the last: through the prefill's kernel)"""
    bs = 16
    n, scale = blocks * bs - 3, NATS / 96
    kc, vc = sink_pool(blocks, n_kv, d, bs, 5)
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    lens = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    q = torch.ones(seqs, rows, n_q, d, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(q.shape, device="cuda")
    ws = torch.empty(pa.pa_decode_verify_workspace_size(seqs, rows, n_q, n_kv, d, bs, blocks * bs), dtype=torch.uint8, device="cuda")
    pa.pa_decode_verify(out, q, kc, vc, tables, lens, scale, bs, ws, k_scale=1.0, v_scale=1.0)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    check_sink(out, np.broadcast_to(n - rows + 1 + np.arange(rows), (seqs, rows)), scale)


def far_pool(seqs, bs, d=64):
    """two keys a sequence, 128 tokens apart, whose raw scores are 16 * 64 * 2688 and half more (the others 0); all v are 1.
    scale: the scores are then 2^25 powers of two, where a product's rounding is worth 2, and the keys lie 6 apart"""
    blocks = 256 // bs
    kc, vc = (torch.zeros(seqs * blocks, 1, bs, 9 * d // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    kc[..., d // 2:], vc[..., d // 2:], vc[..., :d // 2] = 0x38, 0x38, 0x22
    for token in (3, 131):
        b = torch.arange(seqs, device="cuda") * blocks + token // bs
        kc[b, 0, token % bs, :8], kc[b, 0, token % bs, d // 2] = 0x77, 0x7E           # 16 elements of 6 * 448
    kc[b, 0, token % bs, 8] = 0x01                                                     # one of 0.5
    q = torch.ones(seqs, 4, d, dtype=torch.bfloat16, device="cuda")
    q[..., :16] = 64
    tables = torch.arange(seqs * blocks, dtype=torch.int32, device="cuda").view(seqs, blocks)
    return kc, vc, q, tables, 2.0 ** 25 / (16 * 64 * 2688) * np.log(2)


@pytest.mark.parametrize("seqs", [3, 700])
def test_scores_far_from_zero(seqs):
    """weights stay finite where the reference's own rounding is worth several powers of two"""
    kc, vc, q, tables, scale = far_pool(seqs, 16)
    lens = torch.full((seqs,), 256, dtype=torch.int32, device="cuda")
    out = torch.empty(q.shape, device="cuda")
    ws = torch.empty(pa.pa_decode_workspace_size(seqs, 4, 1, 64, 16, 256), dtype=torch.uint8, device="cuda")
    pa.pa_decode(out, q, kc, vc, tables, lens, scale, 16, ws, k_scale=1.0, v_scale=1.0)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    assert ((out - 1).abs() <= 2.0 ** -11 + 256 * 2.0 ** -23).all()


@pytest.mark.parametrize("reqs,n_kv,d,act", [(20, 8, 128, "bfloat16"), (20, 8, 64, "float16"), (2, 1, 64, "bfloat16")])
def test_prefill_of_a_long_flat_rest_below_one_key(reqs, n_kv, d, act):
    """(the last: key tiles split over clusters)"""
    bs, blocks, chunk = 32, 4096, 3
    n, scale = blocks * bs, NATS / 96
    kc, vc = sink_pool(blocks, n_kv, d, bs, 700)
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda").repeat(reqs, 1)
    lens = torch.full((reqs,), n, dtype=torch.int32, device="cuda")
    start = torch.arange(reqs + 1, dtype=torch.int32, device="cuda") * chunk
    q = torch.ones(reqs * chunk, 2 * n_kv, d, dtype=getattr(torch, act), device="cuda")
    out = torch.empty(q.shape, device="cuda")
    pa.pa_prefill_chunk(out, q, kc, vc, tables, start, lens, chunk, scale, bs, k_scale=1.0, v_scale=1.0)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    check_sink(out, np.tile(n - chunk + 1 + np.arange(chunk), reqs), scale)


def test_prefill_of_scores_far_from_zero():
    kc, vc, q, tables, scale = far_pool(160, 32)
    lens = torch.full((160,), 256, dtype=torch.int32, device="cuda")
    start = torch.arange(161, dtype=torch.int32, device="cuda")
    out = torch.empty(q.shape, device="cuda")
    pa.pa_prefill_chunk(out, q, kc, vc, tables, start, lens, 1, scale, 32, k_scale=1.0, v_scale=1.0)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    assert ((out - 1).abs() <= 2.0 ** -11 + 256 * 2.0 ** -23).all()
