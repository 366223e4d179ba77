"""Scored decode (soft cap, distance bias, window, document mask; one or several
query rows) against fp64 attention over the drawn rows.  Tolerances: see scored_ref."""
import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests.scored_ref import Pools, attend64, check, slopes_of, tolerance

pytestmark = pytest.mark.gpu
BF, FH, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


class Case:
    def __init__(self, seed, lens, n_q, n_kv, d, bs, dtype, nq=1, softcap=0.0, alibi=False,
                 window=0, doc=0, fp8=False, first=None, spoil=True, max_blocks=None):
        self.p = p = Pools(seed, lens, n_kv, d, bs, dtype, fp8, max_blocks=max_blocks)
        B = len(p.lens)
        g = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn(B, nq, n_q, d, generator=g).to(dtype)
        self.dtype, self.nq, self.n_q, self.softcap, self.window = dtype, nq, n_q, softcap, window
        self.alibi = alibi
        self.slopes = slopes_of(n_q) if alibi else None
        pos = p.lens[:, None].astype(np.int64) - nq + np.arange(nq)
        self.first = first if first is not None else (pos // doc * doc if doc else None)
        self.lo = np.zeros_like(pos) if not window else np.maximum(pos - window + 1, 0)
        if self.first is not None:
            self.lo = np.maximum(self.lo, self.first)
        self.pos = pos
        if spoil:
            for s in range(B):
                p.spoil(s, min(self.lo[s].min(), p.lens[s] - 1))
        self.tables, self.lens = p.dev()
        self.mod = pa.ScoreMod(
            softcap=softcap, window=window,
            alibi_slopes=torch.from_numpy(self.slopes).cuda() if alibi else None,
            first_key=torch.from_numpy(self.first.astype(np.int32)).cuda()
            if self.first is not None else None)
        size = pa.pa_decode_scored_workspace_size(B, nq, n_q, n_kv, d, bs, p.max_ctx, window)
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.qd = self.q.cuda()

    def run(self, out_dtype=FF, out=None):
        out = torch.full(self.q.shape, float("nan"), dtype=out_dtype, device="cuda") if out is None else out
        pa.pa_decode_scored(out, self.qd, self.p.kc, self.p.vc, self.tables, self.lens, self.mod,
                            self.p.scale, self.p.bs, self.ws, **self.p.scales)
        return out

    def ref(self):
        q = self.qd.double().cpu().numpy()
        return np.stack([attend64(q[s], self.p.k64[s], self.p.v64[s], self.pos[s], self.lo[s],
                                  self.pos[s], self.p.scale, self.softcap, self.slopes)
                         for s in range(len(self.p.lens))])

    def test(self):
        out = self.run()
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == 0
        check(out, self.ref(), tolerance(self.dtype, self.softcap, self.alibi))


# heads and pools of each kernel form: (n_q, n_kv, d, bs, dtype, nq, fp8)
FORMS = {
    "bf16-g4": (8, 2, 128, 16, BF, 1, False),
    "fp16-mha-d64-bs32": (3, 3, 64, 32, FH, 1, False),
    "bf16-g12": (12, 1, 128, 32, BF, 1, False),          # two sub-groups of rows
    "bf16-q4": (8, 2, 128, 16, BF, 4, False),            # 16-row units
    "fp16-q2-d64": (6, 2, 64, 32, FH, 2, False),         # 8-row units
    "fp8-g4": (8, 2, 128, 16, BF, 1, True),              # transposed
    "fp8-g2-d64-bs32": (4, 2, 64, 32, FH, 1, True),      # transposed
    "fp8-g8": (16, 2, 128, 32, BF, 1, True),
    "fp8-q3": (8, 2, 64, 16, BF, 3, True),
    "fp32-d64": (4, 2, 64, 16, FF, 1, False),            # CUDA-core path
    "fp32-d96": (3, 1, 96, 32, FF, 1, False),
    "bf16-d256": (4, 2, 256, 16, BF, 1, False),
}
MODS = {
    "none": {},
    "cap": dict(softcap=20.0),
    "bias": dict(alibi=True),
    "cap-bias": dict(softcap=5.0, alibi=True),
    "window1": dict(window=1),
    "window16": dict(window=16),
    "window37-cap": dict(window=37, softcap=50.0),
    "window700-bias": dict(window=700, alibi=True),
    "doc": dict(doc=45),
    "doc-window-cap-bias": dict(doc=130, window=100, softcap=30.0, alibi=True),
    "window-huge": dict(window=2 ** 31 - 1),
}
LENS = [17, 1, 16, 33, 64, 129, 300, 1000, 1501]


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("form", FORMS)
def test_scored_decode(form, mod):
    n_q, n_kv, d, bs, dtype, nq, fp8 = FORMS[form]
    lens = [max(L, nq) for L in LENS]
    Case(sorted(FORMS).index(form) * 100 + sorted(MODS).index(mod), lens, n_q, n_kv, d, bs, dtype,
         nq, fp8=fp8, **MODS[mod]).test()


@pytest.mark.parametrize("form", ["bf16-g4", "bf16-q4", "fp8-g4", "fp8-g8", "fp32-d64", "fp16-q2-d64"])
def test_a_row_that_sees_no_key_is_zero(form):
    n_q, n_kv, d, bs, dtype, nq, fp8 = FORMS[form]
    lens = [max(L, nq) for L in LENS]
    pos = np.array(lens)[:, None] - nq + np.arange(nq)
    first = np.maximum(pos - 20, 0)
    first[2] = pos[2] + 1            # every row of sequence 2
    first[7, 0] = lens[7] + 5        # the first row of sequence 7
    first[8] = 2 ** 30
    first[1] = -3                    # before the sequence: its first key
    c = Case(7, lens, n_q, n_kv, d, bs, dtype, nq, fp8=fp8, first=first, spoil=False)
    c.test()
    out = c.run()
    assert not out[2].any() and not out[7, 0].any() and not out[8].any()


@pytest.mark.parametrize("out_dtype", [BF, FH])
def test_low_precision_output(out_dtype):
    c = Case(8, [40, 700, 1300], 8, 2, 128, 16, BF, softcap=30.0, window=500)
    check(c.run(out_dtype), c.ref(), tolerance(BF), out_dtype)


def test_without_a_modification_it_is_decode():
    c = Case(9, [40, 700, 1300, 5], 8, 2, 128, 16, BF)
    out, plain = c.run(), torch.empty(4, 8, 128, device="cuda")
    ws = torch.empty(pa.pa_decode_workspace_size(4, 8, 2, 128, 16, c.p.max_ctx), dtype=torch.uint8,
                     device="cuda")
    pa.pa_decode(plain, c.qd[:, 0].contiguous(), c.p.kc, c.p.vc, c.tables, c.lens, c.p.scale, 16, ws)
    assert torch.equal(out[:, 0], plain)


def test_large_scores_saturate_at_the_cap():
    """q of 2^12: the tanh saturates on both sides (an uncapped softmax would be one-hot)."""
    c = Case(10, [50, 900], 8, 2, 64, 16, BF, softcap=2.0)
    c.qd = (c.q.float() * 4096).to(BF).cuda()
    c.test()


def test_many_sequences():
    """More sequences than the partition prefix table holds, several partitions each."""
    rng = np.random.default_rng(5)
    lens = rng.integers(1, 300, 1100)
    lens[::50] = 1300
    Case(11, lens, 2, 1, 64, 16, BF, window=200, softcap=20.0).test()


def test_empty_batch_and_refusals():
    c = Case(12, [40, 100], 8, 2, 64, 16, BF, nq=2, window=30)
    call = lambda **kw: pa.pa_decode_scored(**{**dict(  # noqa: E731
        out=torch.empty(2, 2, 8, 64, device="cuda"), q=c.qd, k_cache=c.p.kc, v_cache=c.p.vc,
        block_tables=c.tables, context_lens=c.lens, mod=c.mod, scale=0.1, block_size=16,
        workspace=c.ws), **kw})
    call(q=c.qd[:0], out=torch.empty(0, 2, 8, 64, device="cuda"))
    with pytest.raises(pa.PAError) as e:
        call(workspace=c.ws[:128])
    assert e.value.status == pa.PA_ERR_WORKSPACE
    with pytest.raises(pa.PAError):
        call(mod=pa.ScoreMod(prefix_lens=torch.ones(2, dtype=torch.int32, device="cuda")))
    with pytest.raises(ValueError):
        call(mod=pa.ScoreMod(first_key=torch.ones(3, dtype=torch.int32, device="cuda")))
    with pytest.raises(ValueError):
        call(mod=pa.ScoreMod(alibi_slopes=torch.ones(2, device="cuda")))
    with pytest.raises(TypeError):
        call(mod=pa.ScoreMod(alibi_slopes=torch.ones(8, device="cuda", dtype=torch.float64)))
    assert pa.pa_get_device_error() == 0


def test_a_table_entry_in_sight_is_checked():
    c = Case(13, [200, 100], 8, 2, 64, 16, BF, window=60)
    c.tables[0, 10] = -1                               # inside the window: flagged
    c.run()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == pa.PA_ERR_OUT_OF_RANGE


def test_two_streams_with_workspaces_of_their_own_and_a_replayed_graph():
    a = Case(14, [900, 1500, 3], 8, 2, 128, 16, BF, softcap=20.0)
    b = Case(15, [100, 2000], 16, 2, 128, 32, BF, window=1000, fp8=True)
    ra, rb = a.ref(), b.ref()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            oa = a.run()
        with torch.cuda.stream(s2):
            ob = b.run()
        outs.append((oa, ob))
    torch.cuda.synchronize()
    for oa, ob in outs:
        check(oa, ra, 2e-3)
        check(ob, rb, 2e-3)
    out = torch.zeros(a.q.shape, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(out=out)
    a.qd.copy_(a.qd.flip(0))
    a.lens.copy_(torch.tensor([700, 20, 2], dtype=torch.int32))    # new lengths under the same tables
    graph.replay()
    torch.cuda.synchronize()
    a.p.lens = np.array([700, 20, 2], np.int32)
    a.p.k64 = [k[:n] for k, n in zip(a.p.k64, a.p.lens)]
    a.p.v64 = [v[:n] for v, n in zip(a.p.v64, a.p.lens)]
    a.pos = a.p.lens[:, None].astype(np.int64) - 1
    check(out, a.ref(), 2e-3)
    assert pa.pa_get_device_error() == 0


CUDA_CORE = {   # (n_q, n_kv, d, bs, dtype): one, two and four heads a block, chunks with spare heads
    "fp32-d128-g4": (8, 2, 128, 16, FF),
    "fp32-d128-g2": (4, 2, 128, 32, FF),
    "fp32-d128-mha": (3, 3, 128, 16, FF),
    "fp32-d32-g5": (10, 2, 32, 16, FF),
    "fp32-d64-g7": (7, 1, 64, 32, FF),
    "fp32-d256-g3": (6, 2, 256, 16, FF),
    "fp16-d32-g3": (6, 2, 32, 32, FH),
    "bf16-d96-mha": (3, 3, 96, 16, BF),
    "fp16-d96-g6": (6, 1, 96, 16, FH),
    "fp16-d256-mha": (2, 2, 256, 32, FH),
}


@pytest.mark.parametrize("mod", ["none", "cap-bias", "window1", "window37-cap", "window700-bias"])
@pytest.mark.parametrize("form", CUDA_CORE)
def test_cuda_core_decode(form, mod):
    n_q, n_kv, d, bs, dtype = CUDA_CORE[form]
    Case(2000 + 10 * sorted(CUDA_CORE).index(form) + sorted(MODS).index(mod), LENS, n_q, n_kv, d, bs,
         dtype, **MODS[mod]).test()


@pytest.mark.parametrize("form", ["fp32-d128-g4", "bf16-d96-mha"])
def test_cuda_core_rows_without_a_key_and_bad_blocks(form):
    n_q, n_kv, d, bs, dtype = CUDA_CORE[form]
    first = np.zeros((3, 1), np.int64)
    first[1] = 2 ** 30                              # sees nothing
    c = Case(2200, [300, 40, 77], n_q, n_kv, d, bs, dtype, first=first, spoil=False)
    c.test()
    assert not c.run()[1].any()
    c.tables[2, 1] = c.p.nb                         # the other sequences are not touched by it
    out = c.run()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == pa.PA_ERR_OUT_OF_RANGE
    check(out[:2], c.ref()[:2], tolerance(dtype))


@pytest.mark.parametrize("mod", ["none", "cap-bias", "window1", "window37-cap", "window700-bias"])
@pytest.mark.parametrize("form", [(8, 2, 128, 16, BF, 4), (8, 2, 128, 32, FH, 4), (16, 1, 128, 16, BF, 2),
                                  (10, 2, 64, 16, BF, 2), (6, 2, 64, 32, FH, 7)],
                         ids=lambda f: "-".join(map(str, f)))
def test_sixteen_rows_over_an_fp8_pool(form, mod):
    n_q, n_kv, d, bs, dtype, nq = form
    c = Case(2300 + sorted(MODS).index(mod), [max(L, nq) for L in LENS], n_q, n_kv, d, bs, dtype, nq,
             fp8=True, max_blocks=2 ** 15 // bs, **MODS[mod])     # (a table that wide counts as much work)
    if mod == "none" and dtype == BF:      # rows of very different size: each has its own scale
        grow = 2.0 ** torch.arange(-12, 12, 24 / (nq * n_q)).view(1, nq, n_q, 1)[:, :nq]
        small = c.q.float() * grow.clamp(max=1.0)
        c.q = small.to(BF)
        c.qd = c.q.cuda()
    c.test()
