"""The serving operators in one run, as a model's layers use them: rotary embedding
with the append, scored chunked prefill, prefix groups of the prefix cache's tables,
shared-prefix and scored decode; and a step of the mixed workload that shares its
prefix.  Tolerances: see scored_ref; rotations are made exact (below), so stored rows
are those of the reference bit for bit."""
import dataclasses

import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from paged_kv_cache_25_gb300 import inputs
from tests.helpers import max_err, oracle_decode, oracle_prefill_all
from tests.scored_ref import attend64, check, slopes_of

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


N_Q, N_KV, D, BS, ROT, NB = 8, 2, 64, 16, 32, 200
SCALE = float(np.float32(D ** -0.5))


class Model:
    """One layer's pool, rotation table and rows.  q, k are multiples of 2^-6 up to 4 and the
    table's values multiples of 2^-7, so x cos - y sin is exact in fp32 (17 bits) and its
    rounding to bf16 the same everywhere."""

    def __init__(self, seed):
        self.rng = np.random.default_rng(seed)
        self.table = torch.round(pa.pa_rope_table(1000, ROT) * 128) / 128
        self.kc = torch.full((NB, N_KV, BS, D), float("nan"), dtype=BF, device="cuda")
        self.vc = torch.full_like(self.kc, float("nan"))
        self.keys, self.values = {}, {}        # sequence -> stored rows, fp64

    def rows(self, n):
        x = np.clip(np.round(self.rng.standard_normal((n, (N_Q + 2 * N_KV) * D)) * 64) / 64, -4, 4)
        return torch.from_numpy(x).to(BF)

    def stored(self, qkv, pos):
        """(rotated q, rotated k, v) of the rows as bf16 keeps them, in fp64"""
        x = qkv.double().numpy().reshape(len(qkv), -1, D)
        cs = self.table.double().numpy()[pos][:, None]
        y = x[:, :N_Q + N_KV].copy()
        a, b, c, s = y[..., :ROT // 2].copy(), y[..., ROT // 2:ROT].copy(), cs[..., :ROT // 2], cs[..., ROT // 2:]
        y[..., :ROT // 2], y[..., ROT // 2:ROT] = a * c - b * s, b * c + a * s
        y = torch.from_numpy(y).to(BF).double().numpy()
        return y[:, :N_Q], y[:, N_Q:], x[:, N_Q + N_KV:]

    def append(self, qkv, pos, slots):
        d = qkv.cuda()
        q, k, v = (t.unflatten(1, (-1, D)) for t in d.split([N_Q * D, N_KV * D, N_KV * D], 1))
        q_out = torch.empty(len(qkv), N_Q, D, dtype=BF, device="cuda")
        pa.pa_rope_and_cache(q_out, q, k, v, torch.from_numpy(pos.astype(np.int32)).cuda(),
                             self.table.cuda(), self.kc, self.vc, torch.from_numpy(slots).cuda())
        return q_out

    def remember(self, s, k, v):
        self.keys[s] = np.concatenate([self.keys.get(s, k[:0]), k])
        self.values[s] = np.concatenate([self.values.get(s, v[:0]), v])


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def test_prompt_cache_prefill_and_decode_steps():
    m = Model(5)
    cache = pa.PrefixCache(NB, BS, m.rng.permutation(NB).astype(np.int32))
    system = m.rng.integers(0, 1000, 70).astype(np.int32)          # 4 full blocks and a rest
    prompts = [np.concatenate([system, m.rng.integers(0, 1000, n).astype(np.int32)]) for n in (5, 40, 90, 1)]
    prompts += [m.rng.integers(0, 1000, 33).astype(np.int32)]     # one that shares nothing
    B, max_blocks, steps = len(prompts), 16, 6
    tables = np.full((B, max_blocks), -1, np.int32)
    cached = []
    slopes = slopes_of(N_Q)
    mod = dict(softcap=15.0, alibi_slopes=torch.from_numpy(slopes).cuda(), window=60)
    # prompts, one after the other: hit blocks are not computed again
    for s, p in enumerate(prompts):
        hit, tables[s] = cache.acquire(p, max_blocks)
        n0 = hit * BS
        cached.append(n0)
        if n0:
            m.remember(s, m.keys[0][:n0], m.values[0][:n0])
        pos = np.arange(n0, len(p))
        qkv = m.rows(len(pos))
        q64, k64, v64 = m.stored(qkv, pos)
        m.remember(s, k64, v64)
        slots = tables[s, pos // BS].astype(np.int64) * BS + pos % BS
        q = m.append(qkv, pos, slots)
        out = torch.full(q.shape, float("nan"), device="cuda")
        pa.pa_prefill_scored(out, q, m.kc, m.vc, dev(tables[s:s + 1]), dev([0, len(pos)]), dev([len(p)]),
                             len(pos), pa.ScoreMod(**mod), SCALE, BS)
        check(out, attend64(q64, m.keys[s], m.values[s], pos, np.maximum(pos - 59, 0), pos, SCALE, 15.0,
                            slopes), 2e-3)
        cache.commit(p, tables[s])
    assert cached == [0, 64, 64, 64, 0]
    # room for the tokens to come
    lens = np.array([len(p) for p in prompts], np.int32)
    for s in range(B):
        have = -(-int(lens[s]) // BS)
        want = -(-int(lens[s] + steps) // BS)
        tables[s, have:want] = cache.alloc(want - have) if want > have else []
    group, prefix = pa.pa_shared_prefix_groups(tables, lens, BS)
    assert list(prefix) == [64] and list(group) == [0, 0, 0, 0, -1]
    # decode steps: one captured graph, replayed over the step's tensors
    # (tables as wide as the longest sequence that the server takes)
    wide = 2048
    bt, gd, pd = dev(np.pad(tables, ((0, 0), (0, wide - max_blocks)), constant_values=-1)), dev(group), dev(prefix)
    cl, posd = dev(lens), dev(lens)
    slot = torch.zeros(B, dtype=torch.int64, device="cuda")
    qkv_d = torch.zeros(B, (N_Q + 2 * N_KV) * D, dtype=BF, device="cuda")
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv_d.split([N_Q * D, N_KV * D, N_KV * D], 1))
    q_out = torch.empty(B, N_Q, D, dtype=BF, device="cuda")
    table_d = m.table.cuda()
    shared, scored = (torch.empty(B, N_Q, D, device="cuda") for _ in range(2))
    ws = torch.empty(pa.pa_decode_shared_workspace_size(B, N_Q, N_KV, D, BS, wide * BS, 1),
                     dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(pa.pa_decode_scored_workspace_size(B, 1, N_Q, N_KV, D, BS, wide * BS, 60),
                      dtype=torch.uint8, device="cuda")

    def step():
        pa.pa_rope_and_cache(q_out, q, k, v, posd, table_d, m.kc, m.vc, slot)
        pa.pa_decode_shared(shared, q_out, m.kc, m.vc, bt, cl, gd, pd, SCALE, BS, ws)
        pa.pa_decode_scored(scored, q_out, m.kc, m.vc, bt, cl, pa.ScoreMod(**mod), SCALE, BS, ws2)

    graph = None
    for i in range(steps):
        pos = lens + i
        qkv = m.rows(B)
        q64, k64, v64 = m.stored(qkv, pos)
        for s in range(B):
            m.remember(s, k64[s:s + 1], v64[s:s + 1])
        qkv_d.copy_(qkv)
        posd.copy_(dev(pos))
        cl.copy_(dev(pos + 1))
        slot.copy_(torch.from_numpy(pa.pa_slot_mapping(tables, BS, np.arange(B), pos)))
        if i == 0:
            step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            shared.fill_(float("nan"))
            scored.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        for s in range(B):
            p = np.array([pos[s]])
            check(shared[s:s + 1], attend64(q64[s:s + 1], m.keys[s], m.values[s], p, [0], p, SCALE), 2e-3)
            check(scored[s:s + 1], attend64(q64[s:s + 1], m.keys[s], m.values[s], p,
                                            np.maximum(p - 59, 0), p, SCALE, 15.0, slopes), 2e-3)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("name", ["mixed-llama3-8b-bf16", "mixed-llama3-8b-fp8"])
def test_a_step_of_the_mixed_workload_shares_its_prefix(name):
    from paged_kv_cache_25_gb300.step import PagedStep
    wl = dataclasses.replace(inputs.get(name), name="mixed-small", batch=24, lens_args=(5.0, 1.0, 16, 900),
                             pool="scale", pool_arg=1.5, shared_prefix_tokens=256, shared_fraction=0.5,
                             prefill_requests=2, prefill_chunk=40, prefill_ctx_range=(10, 90))
    st = PagedStep(wl, out_dtype=torch.float32, prefill_out_dtype=torch.float32, share_prefix=True)
    assert st.prefix_lens.tolist() == [256]
    assert np.array_equal(st.group_of_seq.cpu().numpy() >= 0, st.sharers)
    st.step()
    st.step()                                     # the workspace is used again
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    assert max_err(st.out, oracle_decode(st)) <= 2e-3
    assert max_err(st.p_out, oracle_prefill_all(st)) <= 2e-3
