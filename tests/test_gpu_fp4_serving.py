"""The calls of 4-bit pools in one run, as a model's layers use them: rotary write by several axes, chunked prefill,
decode steps and rows read back; captured and replayed under other lengths and tables; on several streams at once.
Written rows are those of the format's steps bit for bit (the rotation in float32, every product and sum rounded by itself);
attention within fp4_ref's tolerance of the values that the bytes stand for."""
import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests import fp4_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
N_Q, N_KV, BS = 8, 2, 16
KS, VS = 0.07, 1 / 32
SCALES = dict(k_scale=KS, v_scale=VS)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a).astype(dtype)).cuda()


class Layer:
    """One layer's 4-bit pool behind block tables in random order, and what each sequence has in it"""

    def __init__(self, seed, seqs, d, width=40, fill=0xFF):
        self.rng, self.d, self.width = np.random.default_rng(seed), d, width
        nb = seqs * width + 5
        self.tables = self.rng.permutation(nb)[:seqs * width].reshape(seqs, width).astype(np.int32)
        self.kc = torch.full((nb, N_KV, BS, 9 * d // 16), fill, dtype=torch.uint8, device="cuda")
        self.vc = self.kc.clone()
        self.table = pa.pa_rope_table(4000, d)
        self.axis = pa.pa_rope_axes([d // 8, d // 8, d // 4], in_turn=True)
        self.k, self.v = ([np.zeros((0, N_KV, d)) for _ in range(seqs)] for _ in range(2))
        self.bytes = [[np.zeros((0, N_KV, 9 * d // 16), np.uint8) for _ in range(seqs)] for _ in range(2)]

    def draw(self, n):
        x = torch.from_numpy(self.rng.standard_normal((n, (N_Q + 2 * N_KV) * self.d))).to(BF)
        return x, self.rng.integers(0, 4000, (3, n)).astype(np.int32)

    def slots(self, s, n):
        at = len(self.k[s]) + np.arange(n)
        return self.tables[s][at // BS].astype(np.int64) * BS + at % BS

    def write(self, x, pos, slots):
        """the rotated queries; x, pos and slots on the device"""
        q, k, v = (t.unflatten(1, (-1, self.d)) for t in x.split([N_Q * self.d, N_KV * self.d, N_KV * self.d], 1))
        out = torch.empty(len(x), N_Q, self.d, dtype=BF, device="cuda")
        pa.pa_rope_axes_and_cache(out, q, k, v, pos, self.axis, self.table.cuda(), self.kc, self.vc, slots, **SCALES)
        return out

    def remember(self, s, x, pos):
        x = x.float().numpy().reshape(len(x), -1, self.d)
        k, v = x[:, N_Q:N_Q + N_KV], x[:, N_Q + N_KV:]
        half, t = self.d // 2, self.table.numpy()
        at = pos[self.axis].T
        c, sn = t[at, np.arange(half)][:, None], t[at, half + np.arange(half)][:, None]
        a, b = k[..., :half], k[..., half:]
        k = np.concatenate([a * c - b * sn, b * c + a * sn], -1)
        for rows, scale, values, raw in ((k, KS, self.k, self.bytes[0]), (v, VS, self.v, self.bytes[1])):
            y = ref.quantise(rows, scale)
            raw[s] = np.concatenate([raw[s], y])
            values[s] = np.concatenate([values[s], ref.values(y, scale)])

    def vmax(self):
        return max(np.abs(v).max() for v in self.v if v.size)

    def lens(self):
        return [len(k) for k in self.k]

    def check_pools(self):
        """every written byte, and the bytes of all other slots as they were"""
        for pool, raw in ((self.kc, self.bytes[0]), (self.vc, self.bytes[1])):
            want = np.full(pool.shape, 0xFF, np.uint8)
            for s, rows in enumerate(raw):
                at = np.arange(len(rows))
                want[self.tables[s][at // BS], :, at % BS] = rows
            assert np.array_equal(pool.cpu().numpy(), want)

    def attend(self, q, s, pos):
        return ref.attend(q.double().cpu().numpy(), self.k[s], self.v[s], pos, self.d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
def test_prompts_decode_steps_and_rows_read_back(d):
    m = Layer(d, 4, d)
    chunks = [[37, 150, 1, 64], [0, 100, 33, 16]]              # the second one of sequence 0 is empty
    for sizes in chunks:
        parts = [(m.draw(n) if n else None) for n in sizes]
        slots = np.concatenate([m.slots(s, n) for s, n in enumerate(sizes)])
        x = torch.cat([p[0] for p in parts if p])
        q = m.write(x.cuda(), dev(np.concatenate([p[1] for p in parts if p], 1)), dev(slots, np.int64))
        for s, p in enumerate(parts):
            if p:
                m.remember(s, *p)
        start = np.concatenate([[0], np.cumsum(sizes)])
        out = torch.empty(len(x), N_Q, d, device="cuda")
        pa.pa_prefill_chunk(out, q, m.kc, m.vc, dev(m.tables), dev(start), dev(m.lens()), max(sizes), d ** -0.5, BS, **SCALES)
        for s, n in enumerate(sizes):
            if n:
                rows = slice(start[s], start[s + 1])
                ref.check(out[rows], m.attend(q[rows], s, m.lens()[s] - n + np.arange(n)), ref.tolerance(m.vmax()), torch.float32)
    for rows in (1, 1, 3):                                       # two tokens each, then three drafts
        parts = [m.draw(rows) for _ in range(4)]
        slots = np.concatenate([m.slots(s, rows) for s in range(4)])
        q = m.write(torch.cat([p[0] for p in parts]).cuda(), dev(np.concatenate([p[1] for p in parts], 1)), dev(slots, np.int64))
        for s, p in enumerate(parts):
            m.remember(s, *p)
        q = q.view(4, rows, N_Q, d) if rows > 1 else q
        out = torch.empty(q.shape, device="cuda")
        ws = torch.empty(pa.pa_decode_verify_workspace_size(4, rows, N_Q, N_KV, d, BS, m.width * BS), dtype=torch.uint8,
                         device="cuda")
        f = pa.pa_decode if rows == 1 else pa.pa_decode_verify
        f(out, q, m.kc, m.vc, dev(m.tables), dev(m.lens()), d ** -0.5, BS, ws, **SCALES)
        for s in range(4):
            want = m.attend(q[s].view(rows, N_Q, d), s, m.lens()[s] - rows + np.arange(rows))
            ref.check(out[s].view(rows, N_Q, d), want, ref.tolerance(m.vmax()), torch.float32)
    m.check_pools()
    n = m.lens()[1]
    at = np.arange(n)[::-1]
    k, v = (torch.empty(n, N_KV, d, device="cuda") for _ in range(2))
    pa.pa_gather_cache(k, v, m.kc, m.vc, dev(m.tables[1][at // BS].astype(np.int64) * BS + at % BS, np.int64), **SCALES)
    assert np.array_equal(k.cpu().numpy(), m.k[1][at].astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), m.v[1][at].astype(np.float32))
    assert pa.pa_get_device_error() == 0


def step_of(m, x, pos, slots, tables, lens, rows, out, read, ws):
    """a decode step without a wait in between: write, attention, the written rows read back"""
    q = m.write(x, pos, slots)
    q = q.view(len(lens), rows, N_Q, m.d) if rows > 1 else q
    f = pa.pa_decode if rows == 1 else pa.pa_decode_verify
    f(out, q, m.kc, m.vc, tables, lens, m.d ** -0.5, BS, ws, **SCALES)
    pa.pa_gather_cache(read[0], read[1], m.kc, m.vc, slots, **SCALES)
    return q


@pytest.mark.parametrize("rows", [1, 3])
def test_replayed_graphs_follow_lengths_and_tables(rows):
    """two layers captured in graphs of their own with a workspace each, replayed in turn under new tokens, lengths and
    tables; one workspace too is shared by two graphs, whose replays come one after the other"""
    seqs, d = 5, 128
    layers = [Layer(40 + i, seqs, d) for i in range(2)]
    shared = torch.empty(pa.pa_decode_verify_workspace_size(seqs, rows, N_Q, N_KV, d, BS, 40 * BS), dtype=torch.uint8, device="cuda")
    state = []
    for m in layers:
        for s in range(seqs):                                     # 1 .. 400 tokens before
            x, pos = m.draw(int(m.rng.integers(1, 400)))
            m.write(x.cuda(), dev(pos), dev(m.slots(s, len(x)), np.int64))
            m.remember(s, x, pos)
        st = dict(x=torch.zeros(seqs * rows, (N_Q + 2 * N_KV) * d, dtype=BF, device="cuda"),
                  pos=torch.zeros(3, seqs * rows, dtype=torch.int32, device="cuda"),
                  slots=torch.full((seqs * rows,), -1, dtype=torch.int64, device="cuda"),
                  tables=dev(m.tables), lens=torch.full((seqs,), rows, dtype=torch.int32, device="cuda"), rows=rows,
                  out=torch.zeros((seqs, rows, N_Q, d) if rows > 1 else (seqs, N_Q, d), device="cuda"),
                  read=[torch.zeros(seqs * rows, N_KV, d, device="cuda") for _ in range(2)], ws=shared)
        host, m.table = m.table, m.table.cuda()                   # (no upload within the capture)
        step_of(m, **st)                                          # padding alone: the pool stays as it is
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st["q"] = step_of(m, **st)
        m.table = host
        state.append((g, st))
    for turn in range(3):
        for m, (g, st) in zip(layers, state):
            order = m.rng.permutation(seqs)                       # the batch's order changes from step to step
            parts = [m.draw(rows) for _ in order]
            st["x"].copy_(torch.cat([p[0] for p in parts]))
            st["pos"].copy_(dev(np.concatenate([p[1] for p in parts], 1)))
            st["slots"].copy_(dev(np.concatenate([m.slots(s, rows) for s in order]), np.int64))
            for s, p in zip(order, parts):
                m.remember(s, *p)
            st["tables"].copy_(dev(m.tables[order]))
            st["lens"].copy_(dev([m.lens()[s] for s in order]))
            st["order"] = order
        for g, _ in state:
            g.replay()
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == 0
        for m, (g, st) in zip(layers, state):
            for i, s in enumerate(st["order"]):
                want = m.attend(st["q"][i].view(rows, N_Q, d), s, m.lens()[s] - rows + np.arange(rows))
                ref.check(st["out"][i].view(rows, N_Q, d), want, ref.tolerance(m.vmax()), torch.float32)
                rs = slice(i * rows, (i + 1) * rows)
                assert np.array_equal(st["read"][0][rs].cpu().numpy(), m.k[s][-rows:].astype(np.float32))
                assert np.array_equal(st["read"][1][rs].cpu().numpy(), m.v[s][-rows:].astype(np.float32))
    for m in layers:
        m.check_pools()


def test_streams_of_their_own_at_once():
    """decode, several rows and prefill over three pools on three streams, a workspace each; results as on one stream"""
    pools = [ref.Pools(70 + i, lens, N_KV, d, BS) for i, (lens, d) in
             enumerate([([3000, 17, 900, 2100], 128), ([1500, 64, 5], 64), ([700, 1300], 128)])]
    qs = [ref.draw_q(1, (4, 32, 128), BF), ref.draw_q(2, (3, 4, 8, 64), BF), ref.draw_q(3, (350, 8, 128), BF)]
    start = dev([0, 300, 350])

    def call(i, ws):
        p, q = pools[i], qs[i]
        out = torch.empty(q.shape, device="cuda")
        if i == 2:
            pa.pa_prefill_chunk(out, q, p.kc, p.vc, p.tables, start, p.context, 300, 0.09, BS, **p.scales)
        else:
            f = pa.pa_decode if i == 0 else pa.pa_decode_verify
            f(out, q, p.kc, p.vc, p.tables, p.context, 0.1, BS, ws, **p.scales)
        return out

    size = max(pa.pa_decode_verify_workspace_size(4, 4, 32, N_KV, 128, BS, p.max_ctx) for p in pools)
    spaces = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in pools]
    alone = [call(i, spaces[i]) for i in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pools]
    outs = []
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs.append((i, call(i, spaces[i])))
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for i, o in outs:
        assert torch.equal(o, alone[i])


@pytest.mark.parametrize("rows,n_q,d,seqs,fewer", [(1, 8, 128, 4, False), (4, 8, 64, 4, False), (1, 8, 128, 60, True),
                                                   (4, 8, 64, 60, True)])
def test_workspaces_of_any_sufficient_size(rows, n_q, d, seqs, fewer):
    """the sizes that are taken, up to the one that the size function gives and more (fewer: with work for the whole GPU,
    a call takes less than that and uses fewer blocks); nothing behind them is written"""
    p = ref.Pools(9, [2000, rows + 2, 700, 1500] * (seqs // 4), N_KV, d, BS)
    q = ref.draw_q(5, (seqs, rows, n_q, d), BF)
    want = np.stack([ref.attend(q[s].double().cpu().numpy(), p.k[s], p.v[s], n - rows + np.arange(rows), 0.1)
                     for s, n in enumerate(p.lens)])
    full = pa.pa_decode_verify_workspace_size(seqs, rows, n_q, N_KV, d, BS, p.max_ctx)

    def call(n):
        out = torch.full(q.shape, 3.0, device="cuda")
        ws = torch.full((full + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        pa.pa_decode_verify(out, q, p.kc, p.vc, p.tables, p.context, 0.1, BS, ws[:n], **p.scales)
        torch.cuda.synchronize()
        assert (ws[n:] == 0x5A).all()                            # nothing behind the workspace is written
        return out

    taken = [n for n in range(0, full + 1, max(256, full // 64 // 256 * 256)) if n and _takes(call, n)] + [full, full + 4096]
    assert (len(taken) > 2) == fewer
    for n in taken:
        ref.check(call(n), want, ref.tolerance(p.vmax), torch.float32)
    with pytest.raises(pa.PAError):
        call(256)
    assert pa.pa_get_device_error() == 0


def _takes(call, n):
    try:
        call(n)
        return True
    except pa.PAError as e:
        assert e.status == pa.PA_ERR_WORKSPACE
        return False


def test_rows_past_4_gib():
    """pools of 4.7 GiB each, whose last blocks hold the sequences: write, prefill, decode, rows read back and a block copy"""
    m = Layer(5, 2, 128, width=12)
    nb = 550000
    m.kc, m.vc = (torch.full((nb, 8, BS, 72), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    m.tables = (nb - 1 - m.rng.permutation(24)).reshape(2, 12).astype(np.int32)
    n_kv, n_q, T = 8, 16, 180
    assert int(m.tables.min()) * 8 * BS * 72 > 2 ** 32
    qkv = torch.from_numpy(m.rng.standard_normal((2 * T, (n_q + 2 * n_kv) * 128))).to(BF).cuda()
    q, k, v = (t.unflatten(1, (-1, 128)) for t in qkv.split([n_q * 128, n_kv * 128, n_kv * 128], 1))
    pos = dev(m.rng.integers(0, 4000, (3, 2 * T)))
    at = np.arange(T)
    slots = dev(np.concatenate([t[at // BS].astype(np.int64) * BS + at % BS for t in m.tables]), np.int64)
    q_out = torch.empty(2 * T, n_q, 128, dtype=BF, device="cuda")
    pa.pa_rope_axes_and_cache(q_out, q, k, v, pos, m.axis, m.table.cuda(), m.kc, m.vc, slots, **SCALES)
    read = [torch.empty(2 * T, n_kv, 128, device="cuda") for _ in range(2)]
    pa.pa_gather_cache(read[0], read[1], m.kc, m.vc, slots, **SCALES)
    want_v = ref.values(ref.quantise(v.float().cpu().numpy(), VS), VS)
    assert np.array_equal(read[1].cpu().numpy(), want_v.astype(np.float32))
    rows = [r.double().cpu().numpy().reshape(2, T, n_kv, 128) for r in read]
    vmax = np.abs(rows[1]).max()
    out = torch.empty(2 * T, n_q, 128, device="cuda")
    pa.pa_prefill_chunk(out, q_out, m.kc, m.vc, dev(m.tables), dev([0, T, 2 * T]), dev([T, T]), T, 0.09, BS, **SCALES)
    ws = torch.empty(pa.pa_decode_workspace_size(2, n_q, n_kv, 128, BS, 12 * BS), dtype=torch.uint8, device="cuda")
    one = torch.empty(2, n_q, 128, device="cuda")
    last = q_out[[T - 1, 2 * T - 1]].contiguous()
    pa.pa_decode(one, last, m.kc, m.vc, dev(m.tables), dev([T, T]), 0.09, BS, ws, **SCALES)
    for s in range(2):
        x = q_out[s * T:(s + 1) * T].double().cpu().numpy()
        ref.check(out[s * T:(s + 1) * T], ref.attend(x, rows[0][s], rows[1][s], at, 0.09), ref.tolerance(vmax), torch.float32)
        ref.check(one[s:s + 1], ref.attend(x[-1:], rows[0][s], rows[1][s], at[-1:], 0.09), ref.tolerance(vmax), torch.float32)
    pa.pa_copy_blocks(m.kc, m.vc, dev([[int(m.tables[0, 3]), 1]]))
    torch.cuda.synchronize()
    assert torch.equal(m.kc[1], m.kc[int(m.tables[0, 3])]) and torch.equal(m.vc[1], m.vc[int(m.tables[0, 3])])
    assert (m.kc[2:1000] == 0xFF).all() and (m.kc[0] == 0xFF).all() and pa.pa_get_device_error() == 0
