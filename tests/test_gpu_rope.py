"""Rotary embedding fused with the cache write, against the rotation in fp64.

Tolerances: a rotated value is the rounding of x cos - y sin (or y cos + x sin),
computed in fp32 from the given fp32 cos and sin.  The fp32 part is off by at most
2 * 2^-24 * (|x| + |y|) (two products or one product and a fused add, each half a
step, |cos|, |sin| <= 1, and the sum's own rounding); the store by half a step of its dtype."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_25_gb300 import binding as pa

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


def rotate64(x, cs, rot, interleaved):
    """x [T][h][d] fp64, cs [T][rot] -> rotated, and |x| + |y| of each element's pair"""
    y, mag = x.copy(), np.abs(x)
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
           (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


def store_bound(ref, dtype, mag):
    eps = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype]
    tiny = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}[dtype]
    fp32 = 2 * 2.0 ** -24 * mag
    return (np.abs(ref) + fp32) * eps + tiny + fp32


class Case:
    def __init__(self, seed, T, n_q, n_kv, d, bs, dtype, rot, interleaved, slots, fused=True,
                 fp8=False, scale=1.0 / 64, max_pos=2000):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.__dict__.update(T=T, n_q=n_q, n_kv=n_kv, d=d, bs=bs, dtype=dtype, rot=rot,
                             interleaved=interleaved, fp8=fp8, scale=scale)
        self.nb = nb = T // bs + 6 if slots != "scattered" else T + 6
        if slots == "scattered":
            s = rng.permutation(nb * bs)[:T]
        else:      # consecutive tokens of one sequence from an offset, blocks in random order
            at = np.arange(T) + int(slots)
            s = rng.permutation(nb)[at // bs] * bs + at % bs
        self.slots = torch.from_numpy(s.astype(np.int64)).cuda()
        self.pos = torch.from_numpy(rng.integers(0, max_pos, T).astype(np.int32)).cuda()
        self.table = pa.pa_rope_table(max_pos, rot).cuda()
        if fused:
            qkv = torch.randn(T, (n_q + 2 * n_kv) * d, generator=g, device="cuda").to(dtype)
            q, k, v = qkv.split([n_q * d, n_kv * d, n_kv * d], 1)
            self.q, self.k, self.v = (x.unflatten(1, (-1, d)) for x in (q, k, v))
        else:
            self.q, self.k, self.v = (torch.randn(T, h, d, generator=g, device="cuda").to(dtype)
                                      for h in (n_q, n_kv, n_kv))
        self.q_out = torch.full((T, n_q, d), float("nan"), dtype=dtype, device="cuda")
        shape = (nb, n_kv, bs, d)
        if fp8:
            self.kc = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g).view(F8)
            self.vc = torch.randint(0, 256, (nb, n_kv, bs // 16, d, 16), dtype=torch.uint8,
                                    device="cuda", generator=g).view(F8)
        else:
            self.kc = torch.randn(shape, generator=g, device="cuda").to(dtype)
            self.vc = torch.randn(shape, generator=g, device="cuda").to(dtype)
        self.scales = dict(k_scale=scale, v_scale=scale) if fp8 else {}
        self.k0, self.v0 = self.bits(self.kc).clone(), self.bits(self.vc).clone()

    @staticmethod
    def bits(t):
        return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])

    def run(self, stream=None):
        pa.pa_rope_and_cache(self.q_out, self.q, self.k, self.v, self.pos, self.table, self.kc,
                             self.vc, self.slots, interleaved=self.interleaved, stream=stream,
                             **self.scales)

    def check(self, written=None, errors=0):
        """written: mask of the tokens that the call writes"""
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == errors
        w = np.ones(self.T, bool) if written is None else written
        cs = self.table.cpu().numpy().astype(np.float64)[np.clip(self.pos.cpu().numpy(), 0, len(self.table) - 1)]
        f64 = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
        ref, mag = rotate64(self.q64, cs, self.rot, self.interleaved)
        got = f64(self.q_out)
        assert np.isnan(got[~w]).all()
        assert (np.abs(got - ref)[w] <= store_bound(ref, self.dtype, mag)[w]).all()
        # the pools: token rows out, everything else as it was
        ref, mag = rotate64(f64(self.k), cs, self.rot, self.interleaved)
        s = self.slots.cpu().numpy()[w]
        b, o = s // self.bs, s % self.bs
        kc, vc = self.bits(self.kc).cpu().numpy(), self.bits(self.vc).cpu().numpy()
        k0, v0 = self.k0.cpu().numpy(), self.v0.cpu().numpy()
        if self.fp8:
            code = self.kc.float().cpu().numpy().astype(np.float64)[b, :, o] * self.scale
            ref, mag = ref[w], mag[w]
            # half an E4M3 step (2^-4 relative, at least half the smallest step, 2^-10 of the
            # scale), on top of the fp32 arithmetic (the division's rounding included)
            fp32 = 3 * 2.0 ** -24 * mag
            bound = np.maximum((np.abs(ref) + fp32) * 2.0 ** -4, self.scale * 2.0 ** -10) + fp32
            assert (np.abs(code - np.clip(ref, -448 * self.scale, 448 * self.scale)) <= bound).all()
            want_v = oracle.quantize_fp8(self.v.float().cpu()[w], self.scale)
            want_v = want_v.numpy() if isinstance(want_v, torch.Tensor) else want_v
            assert np.array_equal(vc[b, :, o // 16, :, o % 16], want_v.reshape(len(s), self.n_kv, self.d))
            vc[b, :, o // 16, :, o % 16] = v0[b, :, o // 16, :, o % 16]
        else:
            got = f64(self.kc)[b, :, o]
            assert (np.abs(got - ref[w]) <= store_bound(ref, self.dtype, mag)[w]).all()
            assert np.array_equal(vc[b, :, o], self.bits(self.v.contiguous()).cpu().numpy()[w])
            vc[b, :, o] = v0[b, :, o]
        kc[b, :, o] = k0[b, :, o]
        assert np.array_equal(kc, k0) and np.array_equal(vc, v0)

    def start(self):
        self.q64 = self.q.float().cpu().numpy().astype(np.float64)
        return self


BF, FH, FF = torch.bfloat16, torch.float16, torch.float32
CASES = [
    # seed, T, n_q, n_kv, d, bs, dtype, rot, interleaved, slots
    (1, 1, 32, 8, 128, 16, BF, 128, False, "scattered"),
    (2, 37, 32, 8, 128, 16, BF, 64, True, "scattered"),
    (3, 300, 8, 8, 64, 32, FH, 64, False, 5),
    (4, 65, 5, 1, 96, 16, FH, 96, True, 0),
    (5, 19, 4, 2, 256, 32, BF, 128, False, 31),
    (6, 50, 3, 3, 32, 16, FF, 16, False, "scattered"),
    (7, 33, 6, 2, 64, 16, FF, 64, True, 3),
    (8, 129, 1, 1, 32, 32, BF, 32, False, 1),
]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("case", CASES, ids=[f"r{c[0]}" for c in CASES])
def test_rotation_and_append(case, fused):
    c = Case(*case, fused=fused).start()
    c.run()
    c.check()


F8_CASES = [
    # seed, T, n_q, n_kv, d, bs, dtype, rot, interleaved, slots
    (11, 1, 32, 8, 128, 16, BF, 128, False, "scattered"),
    (12, 70, 32, 8, 128, 16, BF, 128, True, "scattered"),
    (13, 160, 8, 2, 64, 32, FH, 32, False, 0),       # whole 16-token pieces
    (14, 161, 10, 5, 64, 16, FF, 64, True, 4),       # aligned runs of 4, heads not a tile's multiple
    (15, 47, 6, 3, 128, 32, BF, 64, False, 7),       # odd offset: single bytes
]


@pytest.mark.parametrize("case", F8_CASES, ids=[f"f{c[0]}" for c in F8_CASES])
def test_rotation_and_append_fp8(case):
    c = Case(*case, fp8=True).start()
    c.run()
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_no_rotation_is_the_plain_cache_write(fp8):
    """cos 1, sin 0: the pools as pa_reshape_and_cache(_quant) leaves them, bit for bit."""
    c = Case(21, 90, 8, 4, 128, 16, BF, 128, False, 3, fused=False, fp8=fp8)
    c.table = torch.cat([torch.ones(2000, 64), torch.zeros(2000, 64)], 1).cuda()
    kc, vc = c.kc.clone(), c.vc.clone()
    c.run()
    if fp8:
        pa.pa_reshape_and_cache_quant(c.k, c.v, kc, vc, c.slots, **c.scales)
    else:
        pa.pa_reshape_and_cache(c.k, c.v, kc, vc, c.slots)
    torch.cuda.synchronize()
    assert torch.equal(c.bits(c.kc), c.bits(kc)) and torch.equal(c.bits(c.vc), c.bits(vc))
    assert torch.equal(c.q_out, c.q)


@pytest.mark.parametrize("scale", [0.013, 1.0, 0.25])
def test_fp8_other_scales(scale):
    """Scales with and without an exact reciprocal."""
    c = Case(28, 37, 8, 4, 64, 16, BF, 32, False, 3, fp8=True, scale=scale).start()
    c.run()
    c.check()


def test_fp8_saturates():
    c = Case(22, 20, 4, 2, 128, 16, BF, 128, False, 0, fp8=True, scale=1.0 / 1024).start()
    c.run()
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_padding_and_out_of_range_tokens_are_left_alone(fp8):
    c = Case(23, 40, 8, 2, 64, 16, BF, 64, False, "scattered", fp8=fp8).start()
    c.slots[3], c.slots[39] = -1, -7                  # padding
    c.pos[3] = -5                                      # its position is not looked at
    c.run()
    w = np.ones(40, bool)
    w[[3, 39]] = False
    c.check(w)
    c = Case(24, 40, 8, 2, 64, 16, BF, 64, False, "scattered", fp8=fp8).start()
    c.slots[5] = c.nb * c.bs                           # past the pool
    c.pos[6], c.pos[7] = 2000, -1                      # past the table, before it
    c.run()
    w = np.ones(40, bool)
    w[[5, 6, 7]] = False
    c.check(w, errors=pa.PA_ERR_OUT_OF_RANGE)


@pytest.mark.parametrize("interleaved", [False, True])
def test_q_in_place(interleaved):
    c = Case(25, 77, 8, 4, 128, 16, BF, 64, interleaved, "scattered").start()
    c.q_out = c.q
    c.run()
    c.check()


def test_q_out_may_be_a_slice():
    c = Case(30, 45, 8, 2, 64, 16, BF, 64, False, 1).start()
    wide = torch.full((45, 24, 64), float("nan"), dtype=BF, device="cuda")
    c.q_out = wide[:, 8:16]
    c.run()
    c.check()
    assert torch.isnan(wide[:, :8]).all() and torch.isnan(wide[:, 16:]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_more_tokens_than_the_grid_covers_at_once(fp8):
    c = Case(29, 3001, 8, 4, 128, 16, BF, 128, False, 9, fp8=fp8).start()
    c.slots[[0, 1700, 3000]] = -1
    c.run()
    w = np.ones(3001, bool)
    w[[0, 1700, 3000]] = False
    c.check(w)


def test_no_tokens():
    c = Case(26, 1, 8, 4, 64, 16, BF, 64, False, "scattered").start()
    pa.pa_rope_and_cache(c.q_out[:0], c.q[:0], c.k[:0], c.v[:0], c.pos[:0], c.table, c.kc, c.vc,
                         c.slots[:0])
    c.check(np.zeros(1, bool))


def test_stream_and_graph_replay():
    """Captured once, replayed over new contents of the same tensors."""
    c = Case(27, 60, 8, 4, 128, 32, BF, 128, False, 2).start()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run()
    torch.cuda.current_stream().wait_stream(s)
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.pos.copy_((c.pos * 7 + 3) % 2000)
    c.q.normal_()
    c.start()
    c.q_out.fill_(float("nan"))
    graph.replay()
    c.check()


def test_pool_beyond_32_bit_offsets():
    """The last block of a pool of more than 2^31 elements."""
    n_kv, d, bs, T = 8, 128, 16, 5
    nb = (1 << 31) // (n_kv * d * bs) + 10
    kc = torch.zeros(nb, n_kv, bs, d, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    q, k, v = (torch.randn(T, h, d, device="cuda").to(BF) for h in (4, n_kv, n_kv))
    slots = torch.arange(nb * bs - T, nb * bs, device="cuda")
    table = torch.cat([torch.ones(4, 64), torch.zeros(4, 64)], 1).cuda()
    pa.pa_rope_and_cache(torch.empty_like(q), q, k, v, torch.zeros(T, dtype=torch.int32, device="cuda"),
                         table, kc, vc, slots)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    assert torch.equal(kc[-1, :, -T:].transpose(0, 1), k)
    assert torch.equal(vc[-1, :, -T:].transpose(0, 1), v)
    assert not kc[:-1].any() and not vc[:-1].any()
