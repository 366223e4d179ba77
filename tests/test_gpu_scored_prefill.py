"""Scored chunked prefill (soft cap, distance bias, window, document and prefix
masks) against fp64 attention over the drawn rows.  Tolerances: see scored_ref."""
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
    def __init__(self, seed, reqs, n_q, n_kv, d, bs, dtype, softcap=0.0, alibi=False, window=0,
                 doc=0, prefix=0, fp8=False, first=None, spoil=True, kscale=1.0):
        """reqs: (chunk, context length with the chunk) of each request"""
        lens = [L for _, L in reqs]
        self.p = p = Pools(seed, lens, n_kv, d, bs, dtype, fp8)
        self.rows = rows = np.array([c for c, _ in reqs])
        g = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn(int(rows.sum()), n_q, d, generator=g).to(dtype)
        self.dtype, self.softcap, self.alibi = dtype, softcap, alibi
        self.slopes = slopes_of(n_q) if alibi else None
        self.start = np.concatenate([[0], np.cumsum(rows)])
        self.pos = np.concatenate([np.arange(L - c, L) for c, L in reqs]).astype(np.int64)
        req = np.repeat(np.arange(len(reqs)), rows)
        self.first = first if first is not None else (self.pos // doc * doc if doc else None)
        self.lo = np.maximum(self.pos - window + 1, 0) if window else np.zeros_like(self.pos)
        if self.first is not None:
            self.lo = np.maximum(self.lo, self.first)
        self.hi = np.maximum(self.pos, np.minimum(prefix, np.array(lens)[req]) - 1) if prefix else self.pos
        for r in range(len(reqs)):
            mine = req == r
            if spoil and mine.any():
                p.spoil(r, min(self.lo[mine].min(), lens[r] - 1))
        self.tables, self.lens = p.dev()
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731
        self.q_start = dev(self.start)
        self.mod = pa.ScoreMod(softcap=softcap, window=window,
                               alibi_slopes=torch.from_numpy(self.slopes).cuda() if alibi else None,
                               first_key=dev(self.first) if self.first is not None else None,
                               prefix_lens=dev(np.full(len(reqs), prefix)) if prefix else None)
        self.qd = self.q.cuda()

    def run(self, out_dtype=FF, out=None, max_q=None):
        out = torch.full(self.q.shape, float("nan"), dtype=out_dtype, device="cuda") if out is None else out
        pa.pa_prefill_scored(out, self.qd, self.p.kc, self.p.vc, self.tables, self.q_start, self.lens,
                             int(self.rows.max()) if max_q is None else max_q, self.mod, self.p.scale,
                             self.p.bs, **self.p.scales)
        return out

    def ref(self):
        q = self.qd.double().cpu().numpy()
        out = []
        for r in range(len(self.rows)):
            a, b = self.start[r], self.start[r + 1]
            out.append(attend64(q[a:b], self.p.k64[r], self.p.v64[r], self.pos[a:b], self.lo[a:b],
                                self.hi[a:b], self.p.scale, self.softcap, self.slopes))
        return np.concatenate(out)

    def test(self):
        out = self.run()
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == 0
        check(out, self.ref(), tolerance(self.dtype, self.softcap, self.alibi))


# (n_q, n_kv, d, bs, dtype, fp8)
FORMS = {
    "bf16-g4": (8, 2, 128, 16, BF, False),
    "bf16-mha-d64-bs32": (3, 3, 64, 32, BF, False),
    "fp16-g3": (6, 2, 128, 32, FH, False),               # a group that 256 is no multiple of
    "fp16-g2-d64": (4, 2, 64, 16, FH, False),
    "fp8-g4": (8, 2, 128, 16, BF, True),                 # score products on the codes themselves
    "fp8-fp16-g2": (4, 2, 128, 32, FH, True),            # converters for K and V
    "fp8-g8-d64": (8, 1, 64, 16, BF, True),
}
MODS = {
    "none": {},
    "cap": dict(softcap=20.0),
    "bias": dict(alibi=True),
    "cap-bias": dict(softcap=5.0, alibi=True),
    "window1": dict(window=1),
    "window100-cap": dict(window=100, softcap=50.0),
    "window300-bias": dict(window=300, alibi=True),
    "doc": dict(doc=45),
    "prefix": dict(prefix=150),
    "prefix-past-the-end-bias": dict(prefix=5000, alibi=True),
    "prefix-window-doc-cap": dict(prefix=200, window=170, doc=260, softcap=30.0),
    "window-huge": dict(window=2 ** 31 - 1),
}
REQS = [(1, 1), (5, 5), (1, 400), (130, 130), (77, 500), (200, 333)]


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("form", FORMS)
def test_scored_prefill(form, mod):
    n_q, n_kv, d, bs, dtype, fp8 = FORMS[form]
    Case(sorted(FORMS).index(form) * 100 + sorted(MODS).index(mod), REQS, n_q, n_kv, d, bs, dtype,
         fp8=fp8, **MODS[mod]).test()


@pytest.mark.parametrize("mod", ["cap", "window100-cap", "cap-bias", "prefix"])
@pytest.mark.parametrize("form", ["bf16-g4", "fp8-g4"])
def test_long_context(form, mod):
    n_q, n_kv, d, bs, dtype, fp8 = FORMS[form]
    Case(31, [(140, 3000), (70, 2049)], n_q, n_kv, d, bs, dtype, fp8=fp8, **MODS[mod]).test()


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("form", FORMS)
def test_a_row_that_sees_no_key_is_zero(form, alibi):
    n_q, n_kv, d, bs, dtype, fp8 = FORMS[form]
    pos = np.concatenate([np.arange(L - c, L) for c, L in REQS])
    first = np.maximum(pos - 50, -9)
    none = np.zeros(len(pos), bool)
    none[[1, 9, 300]] = True
    none[7:137] = True               # all of request 3
    none[-60:] = True                # the last rows of request 5
    first[none] = pos[none] + np.arange(none.sum()) + 1
    c = Case(32, REQS, n_q, n_kv, d, bs, dtype, fp8=fp8, first=first, spoil=False, alibi=alibi)
    c.test()
    out = c.run()
    assert not out[torch.from_numpy(none).cuda()].any()


@pytest.mark.parametrize("out_dtype", [BF, FH])
def test_low_precision_output(out_dtype):
    c = Case(33, REQS, 8, 2, 128, 16, BF, softcap=30.0, window=150)
    check(c.run(out_dtype), c.ref(), tolerance(BF), out_dtype)


@pytest.mark.parametrize("fp8", [False, True])
def test_without_a_modification_it_is_the_plain_prefill(fp8):
    c = Case(34, REQS, 8, 2, 128, 16, BF, fp8=fp8)
    out, plain = c.run(), torch.empty(c.q.shape, device="cuda")
    pa.pa_prefill_chunk(plain, c.qd, c.p.kc, c.p.vc, c.tables, c.q_start, c.lens, 200, c.p.scale, 16,
                        **c.p.scales)
    assert torch.equal(out, plain)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_other_scales(scale):
    c = Case(35, REQS, 8, 2, 64, 16, BF, softcap=2.0, alibi=True, window=90)
    type(c.p).scale, keep = scale, type(c.p).scale
    try:
        c.test()
    finally:
        type(c.p).scale = keep


def test_more_requests_than_are_ranked_and_a_chunk_beyond_the_grid():
    reqs = [(1 + i % 7, 10 + 5 * i) for i in range(70)]
    c = Case(36, reqs, 4, 2, 64, 16, BF, window=33, softcap=20.0)
    c.test()
    c.run(max_q=6)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == pa.PA_ERR_OUT_OF_RANGE
    assert pa.pa_get_device_error() == 0


def test_rows_behind_the_last_request_are_left_alone():
    c = Case(38, REQS, 8, 2, 64, 16, BF, window=50)
    n = c.q.shape[0]
    c.qd = torch.cat([c.qd, torch.full((9, 8, 64), float("nan"), dtype=BF, device="cuda")])
    out = torch.full(c.qd.shape, 7.0, device="cuda")
    c.run(out=out)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    c.qd = c.qd[:n]
    check(out[:n], c.ref(), 2e-3)
    assert (out[n:] == 7).all()


def test_replayed_graph():
    c = Case(37, REQS, 8, 2, 128, 16, BF, softcap=20.0, doc=100)
    out = torch.zeros(c.q.shape, device="cuda")
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out)
    c.qd.copy_(c.qd.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    check(out, c.ref(), 2e-3)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("mod", ["none", "cap-bias", "window300-bias", "doc", "prefix-window-doc-cap"])
@pytest.mark.parametrize("form", FORMS)
def test_few_rows_over_long_contexts(form, mod):
    """Key tiles split over a cluster of eight blocks, with requests too short for all of them."""
    n_q, n_kv, d, bs, dtype, fp8 = FORMS[form]
    Case(41, [(40, 4200), (3, 90), (1, 1)], n_q, n_kv, d, bs, dtype, fp8=fp8, **MODS[mod]).test()


@pytest.mark.parametrize("out_dtype", [BF, FH])
@pytest.mark.parametrize("form", ["bf16-g4", "fp16-g2-d64", "fp8-g4"])
def test_split_prefill_output_types_and_replay(form, out_dtype):
    n_q, n_kv, d, bs, dtype, fp8 = FORMS[form]
    c = Case(42, [(140, 3000), (9, 700)], n_q, n_kv, d, bs, dtype, fp8=fp8, softcap=20.0)
    check(c.run(out_dtype), c.ref(), tolerance(dtype, 20.0), out_dtype)
    out = torch.zeros(c.q.shape, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out)
        c.run(out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, c.run())
    assert pa.pa_get_device_error() == 0
