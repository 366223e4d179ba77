"""Serving calls launched one behind the other see what the calls before them wrote: steps of
new rows, lengths, groups and queries, enqueued without a wait in between, give bit for bit what
the same steps give with a synchronisation after every launch."""
import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests import test_gpu_shared as shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


STEPS = 40


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("form", ["bf16-g4", "fp8-g4", "fp16-g2-d64"])
def test_steps_without_a_wait_in_between(form, graph):
    n_q, n_kv, d, bs, dtype, fp8 = shared.FORMS[form]
    c = shared.Case(700, [(256, [60, 300, 45]), (1024, [50, 900, 41, 40, 77])], [500, 90, 1300], n_q, n_kv, d, bs,
                    dtype, fp8=fp8)
    rng = np.random.default_rng(5)
    g = torch.Generator(device="cuda").manual_seed(6)
    B, long = len(c.p.lens), c.p.lens.astype(np.int64)
    lens, slots, groups = [], [], []
    for _ in range(STEPS):
        n = long - rng.integers(0, 40, B)                 # (the newest row is never the prefix's)
        at = n - 1
        lens.append(torch.from_numpy(n.astype(np.int32)).cuda())
        slots.append(torch.from_numpy(c.p.tables[np.arange(B), at // bs].astype(np.int64) * bs + at % bs).cuda())
        groups.append(torch.where(torch.from_numpy(rng.random(B) < 0.2).cuda(), -1, c.gd))
    qkv = torch.randn(STEPS, B, (n_q + 2 * n_kv) * d, device="cuda", generator=g).to(dtype)
    table = pa.pa_rope_table(2000, d).cuda()
    now = qkv[0].clone()
    q, k, v = (t.unflatten(1, (-1, d)) for t in now.split([n_q * d, n_kv * d, n_kv * d], 1))
    cl, slot, gd = lens[0].clone(), slots[0].clone(), groups[0].clone()
    q_out = torch.empty(B, n_q, d, dtype=dtype, device="cuda")
    mod = pa.ScoreMod(softcap=30.0, window=400)
    ws = torch.empty(pa.pa_decode_scored_workspace_size(B, 1, n_q, n_kv, d, bs, c.p.max_ctx, 400),
                     dtype=torch.uint8, device="cuda")
    out, scored = (torch.empty(B, n_q, d, device="cuda") for _ in range(2))

    def calls():
        pa.pa_rope_and_cache(q_out, q, k, v, cl, table, c.p.kc, c.p.vc, slot, **c.p.scales)
        yield
        pa.pa_decode_shared(out, q_out, c.p.kc, c.p.vc, c.tables, cl, gd, c.pd, c.p.scale, bs, c.ws, **c.p.scales)
        yield
        pa.pa_decode_scored(scored, q_out, c.p.kc, c.p.vc, c.tables, cl, mod, c.p.scale, bs, ws, **c.p.scales)
        yield

    def inputs(i):
        now.copy_(qkv[i])
        cl.copy_(lens[i])
        slot.copy_(slots[i])
        gd.copy_(groups[i])

    kc, vc = c.p.kc.clone(), c.p.vc.clone()
    ref = []
    for i in range(STEPS):
        inputs(i)
        for _ in calls():
            torch.cuda.synchronize()
        ref.append((out.clone(), scored.clone()))
    assert pa.pa_get_device_error() == 0
    assert any(not torch.equal(ref[0][0], a) for a, _ in ref)
    c.p.kc.copy_(kc)
    c.p.vc.copy_(vc)
    replay = None
    if graph:
        replay = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(replay):
            list(calls())
    torch.cuda.synchronize()
    got = []
    for i in range(STEPS):
        inputs(i)
        if graph:
            replay.replay()
        else:
            list(calls())
        got.append((out.clone(), scored.clone()))
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for a, b in zip(ref, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
