"""Decode of batches whose sequences share prefixes, against fp64 attention over the
drawn rows.  Tolerances: see scored_ref."""
import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests.scored_ref import Pools, attend64, check

pytestmark = pytest.mark.gpu
BF, FH, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


WORTH = 64 << 20      # bytes of the tables' blocks above which prefixes are read apart


class Case:
    """groups: list of (prefix tokens, [own tokens of each member]); loners: lengths."""

    def __init__(self, seed, groups, loners, n_q, n_kv, d, bs, dtype, fp8=False, shuffle=True):
        lens, of, pre, gid = [], [], [], []
        for g, (p, own) in enumerate(groups):
            lead = len(lens)
            for i, n in enumerate(own):
                lens.append(p + n); of.append(lead if i else -1); pre.append(p); gid.append(g)
        for n in loners:
            lens.append(n); of.append(-1); pre.append(0); gid.append(-1)
        # the longest member first, so that the others can copy their whole part
        self.p = p = Pools(seed, lens, n_kv, d, bs, dtype, fp8, prefix_of=of, prefix=pre)
        order = np.random.default_rng(seed).permutation(len(lens)) if shuffle else np.arange(len(lens))
        p.lens, p.tables = p.lens[order], p.tables[order]
        p.k64, p.v64 = [p.k64[i] for i in order], [p.v64[i] for i in order]
        # Tables wide enough that the prefixes are read apart (the drawn ones, `narrow` columns,
        # mostly hold too little for that).
        self.narrow = p.tables.shape[1]
        block = 2 * n_kv * bs * d * (1 if fp8 else 2)
        wide = max(self.narrow, WORTH // (block * len(lens)) + 1)
        p.tables = np.pad(p.tables, ((0, 0), (0, wide - self.narrow)), constant_values=-1)
        self.group = np.array(gid, np.int32)[order]
        self.prefix = np.array([g[0] for g in groups], np.int32)
        g = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn(len(lens), n_q, d, generator=g).to(dtype).cuda()
        self.dtype, self.n_q = dtype, n_q
        self.tables, self.lens = p.dev()
        self.gd, self.pd = torch.from_numpy(self.group).cuda(), torch.from_numpy(self.prefix).cuda()
        size = max(pa.pa_decode_shared_workspace_size(len(lens), n_q, n_kv, d, bs, n * bs, len(groups))
                   for n in (wide, self.narrow))
        self.ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN partials

    def run(self, out_dtype=FF, out=None):
        out = torch.full(self.q.shape, float("nan"), dtype=out_dtype, device="cuda") if out is None else out
        pa.pa_decode_shared(out, self.q, self.p.kc, self.p.vc, self.tables, self.lens, self.gd, self.pd,
                            self.p.scale, self.p.bs, self.ws, **self.p.scales)
        return out

    def ref(self):
        q = self.q.double().cpu().numpy()
        return np.concatenate([attend64(q[s:s + 1], self.p.k64[s], self.p.v64[s], [n - 1], [0], [n - 1],
                                        self.p.scale) for s, n in enumerate(self.p.lens)])

    def test(self, error=0):
        out = self.run()
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == error
        ref = self.ref()
        check(out, ref, 2e-3)
        if not error:                                  # and with the drawn tables
            wide, self.tables = self.tables, self.tables[:, :self.narrow].contiguous()
            check(self.run(), ref, 2e-3)
            assert pa.pa_get_device_error() == 0
            self.tables = wide
        return out


FORMS = {   # (n_q, n_kv, d, bs, dtype, fp8)
    "bf16-g4": (8, 2, 128, 16, BF, False),
    "bf16-mha-d64-bs32": (3, 3, 64, 32, BF, False),
    "fp16-g3": (6, 2, 128, 32, FH, False),
    "fp16-g2-d64": (4, 2, 64, 16, FH, False),
    "fp8-g4": (8, 2, 128, 16, BF, True),
    "fp8-fp16-g2": (4, 2, 128, 32, FH, True),
    "fp8-g8-d64": (8, 1, 64, 16, BF, True),
    "bf16-g12": (12, 1, 64, 32, BF, False),
}
BATCHES = {
    "one-block": ([(32, [1, 17, 40])], []),
    "two-groups": ([(128, [5, 200, 33]), (992, [1, 1100, 64, 300])], [700, 1, 40]),
    "one-member": ([(160, [30]), (64, [3, 9])], [100]),
    "no-own-keys": ([(256, [50, 0, 0]), (32, [0, 0])], [32]),
    "long": ([(4096, [10, 1500, 1])], [20]),
    "many-members": ([(320, [1 + 3 * i for i in range(70)])], [64]),
    "no-groups": ([], [5, 300, 1200]),
}


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("form", FORMS)
def test_shared_decode(form, batch):
    Case(sorted(FORMS).index(form) * 10 + sorted(BATCHES).index(batch), *BATCHES[batch],
         *FORMS[form][:5], fp8=FORMS[form][5]).test()


@pytest.mark.parametrize("dtype,fp8,d", [(BF, False, 128), (FH, False, 64), (BF, True, 128), (FH, True, 64)])
@pytest.mark.parametrize("prefixes", [(384, 640, 1152, 1024), (256, 128, 2176, 16), (2048,)])
def test_few_rows_and_many_heads(prefixes, dtype, fp8, d):
    """Groups of a few rows whose blocks fill the GPU uncut: both row tiles hold the same rows
    and share the key tiles, an even or an odd number of them."""
    groups = [(p, [3, 40, 1][:2 + i % 2]) for i, p in enumerate(prefixes)]
    Case(88, groups, [70], 40, 40, d, 16, dtype, fp8=fp8).test()


@pytest.mark.parametrize("form", ["bf16-g4", "fp8-g4", "bf16-mha-d64-bs32"])
def test_many_groups_and_sequences(form):
    """Row tiles of several sizes, more sequences than a block has threads and than the
    partition prefix table holds, empty groups."""
    rng = np.random.default_rng(3)
    groups = [(32 * int(rng.integers(1, 8)), list(rng.integers(1, 60, int(rng.integers(1, 90)))))
              for _ in range(25)]
    c = Case(91, groups, list(rng.integers(1, 200, 120)), *FORMS[form][:5], fp8=FORMS[form][5])
    assert len(c.p.lens) > 1024
    c.gd = torch.where(c.gd >= 0, c.gd * 2 + 1, c.gd).contiguous()      # even groups have no member
    pre = np.full(2 * len(groups) + 3, 64, np.int32)
    pre[1:2 * len(groups):2] = c.prefix
    c.pd = torch.from_numpy(pre).cuda()
    size = pa.pa_decode_shared_workspace_size(len(c.p.lens), c.n_q, c.p.n_kv, c.p.d, c.p.bs, c.p.max_ctx,
                                              len(pre))
    c.ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    c.test()


@pytest.mark.parametrize("form", ["bf16-g4", "fp8-g4"])
def test_prefix_lengths_are_rounded_down_and_bounded(form):
    c = Case(92, [(128, [40, 7, 300]), (64, [9, 20])], [33], *FORMS[form][:5], fp8=FORMS[form][5])
    c.pd[0], c.pd[1] = 128 - 1, -5          # whole blocks below it; nothing
    c.test()
    c.pd[0] = 0
    c.test()


def test_members_shorter_than_the_prefix():
    """A prefix length beyond some members' context: they see their own keys only."""
    c = Case(93, [(256, [40, 0, 7]), (64, [9, 20])], [33], *FORMS["bf16-g4"][:5])
    n = np.array([200, 5, 97, 256], np.int64)
    who = np.flatnonzero(c.group == 0)[:3]
    for s, L in zip(who, n):
        c.p.lens[s] = min(L, c.p.lens[s])
        c.p.k64[s], c.p.v64[s] = c.p.k64[s][:c.p.lens[s]], c.p.v64[s][:c.p.lens[s]]
    c.lens = torch.from_numpy(c.p.lens).cuda()
    c.test()


@pytest.mark.parametrize("form", ["bf16-g4", "fp8-g4", "fp16-g3"])
def test_a_prefix_past_every_member(form):
    """Rows of shared blocks that no member has reached yet hold NaN and are not seen."""
    c = Case(100, [(256, [0, 0, 0]), (96, [4, 20])], [33], *FORMS[form][:5], fp8=FORMS[form][5])
    for s, L in zip(np.flatnonzero(c.group == 0), [200, 170, 9]):
        c.p.lens[s] = L
        c.p.k64[s], c.p.v64[s] = c.p.k64[s][:L], c.p.v64[s][:L]
    s = int(np.flatnonzero(c.group == 0)[0])
    at = np.arange(200, 256)
    b, o = c.p.tables[s, at // c.p.bs].astype(np.int64), at % c.p.bs
    if c.p.fp8:
        c.p.kc.view(torch.uint8)[b, :, o] = 0x7F
        c.p.vc.view(torch.uint8)[b, :, o // 16, :, o % 16] = 0x7F
    else:
        c.p.kc[b, :, o] = float("nan")
        c.p.vc[b, :, o] = float("nan")
    c.tables[c.gd == 0, -(-200 // c.p.bs):] = -1          # nor are blocks behind them read
    c.lens = torch.from_numpy(c.p.lens).cuda()
    c.test()


def test_groups_without_members():
    c = Case(101, [(64, [5, 20])], [300, 33], *FORMS["bf16-g4"][:5])
    c.gd.fill_(-3)
    c.test()


def test_a_group_out_of_range_is_flagged_and_shares_nothing():
    c = Case(94, [(64, [5, 20]), (96, [1, 2])], [33], *FORMS["bf16-g4"][:5])
    c.gd[c.gd == 1] = 2
    c.test(error=pa.PA_ERR_OUT_OF_RANGE)
    assert pa.pa_get_device_error() == 0


def test_a_bad_prefix_block_is_flagged():
    c = Case(95, [(64, [5, 20])], [], *FORMS["bf16-g4"][:5])
    c.tables[:, 1] = c.p.nb
    c.run()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == pa.PA_ERR_OUT_OF_RANGE


@pytest.mark.parametrize("form", ["bf16-g4", "fp8-g4"])
def test_a_call_with_small_tables_is_pa_decode(form):
    """Up to and including the limit bit for bit; one block more reads the prefixes apart."""
    n_q, n_kv, d, bs, _, fp8 = FORMS[form]
    c = Case(102, [(64, [5, 20, 33])], [40], *FORMS[form][:5], fp8=fp8)
    at_most = WORTH // (2 * n_kv * bs * d * (1 if fp8 else 2) * 4)
    assert c.tables.shape[1] == at_most + 1
    c.gd[c.gd == 0] = 7                                # flagged only where groups are read
    c.run()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == pa.PA_ERR_OUT_OF_RANGE
    c.tables = c.tables[:, :at_most].contiguous()
    plain = torch.empty(c.q.shape, device="cuda")
    ws = torch.empty(pa.pa_decode_workspace_size(4, n_q, n_kv, d, bs, at_most * bs), dtype=torch.uint8,
                     device="cuda")
    pa.pa_decode(plain, c.q, c.p.kc, c.p.vc, c.tables, c.lens, c.p.scale, bs, ws, **c.p.scales)
    assert torch.equal(c.run(), plain)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("out_dtype", [BF, FH])
def test_low_precision_output(out_dtype):
    c = Case(96, *BATCHES["two-groups"], *FORMS["bf16-g4"][:5])
    check(c.run(out_dtype), c.ref(), 2e-3, out_dtype)


def test_it_is_near_pa_decode_and_repeats_bit_for_bit():
    c = Case(97, *BATCHES["two-groups"], *FORMS["bf16-g4"][:5])
    plain = torch.empty(c.q.shape, device="cuda")
    ws = torch.empty(pa.pa_decode_workspace_size(len(c.p.lens), 8, 2, 128, 16, c.p.max_ctx),
                     dtype=torch.uint8, device="cuda")
    pa.pa_decode(plain, c.q, c.p.kc, c.p.vc, c.tables, c.lens, c.p.scale, 16, ws)
    a, b = c.run(), c.run()
    assert float((a - plain).abs().max()) <= 2e-3
    assert torch.equal(a, b)
    none = torch.full_like(c.gd, -1)
    c.gd, c.pd = none, c.pd[:0]
    assert torch.equal(c.run(), plain)


def test_replayed_graph_follows_new_groups_and_two_streams():
    a = Case(98, [(128, [50, 3, 70]), (64, [10, 90])], [40], *FORMS["bf16-g4"][:5])
    b = Case(99, *BATCHES["two-groups"], *FORMS["fp8-g4"][:5], fp8=True)
    ra, rb = a.ref(), b.ref()
    a.run(); b.run()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
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
    a.gd.copy_(torch.where(a.gd == 1, -1, a.gd))        # group 1 breaks up, group 0 shares less
    a.pd[0] = 64
    a.q.copy_(a.q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    check(out, a.ref(), 2e-3)
    assert pa.pa_get_device_error() == 0
