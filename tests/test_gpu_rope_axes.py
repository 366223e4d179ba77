"""Rotary write with several position axes, into every pool type.

q, and k of 16- and 32-bit pools, against the rotation in fp64 with test_gpu_rope's bounds; 4-bit rows
bit for bit against the rotation in float32 (every product and sum rounded by itself, as documented)
quantised by the format's steps."""
import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests import fp4_ref as ref
from tests.test_gpu_rope import store_bound

pytestmark = pytest.mark.gpu
ACT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


class Case:
    def __init__(self, seed, T, n_q, n_kv, d, bs, act, pool, rot, interleaved, axes, kind, scattered=True, max_pos=999):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(T=T, n_q=n_q, n_kv=n_kv, d=d, bs=bs, rot=rot, interleaved=interleaved, pool=pool,
                             dtype=ACT[act], act=act)
        nb = T + 3 if scattered else T // bs + 5
        at = np.arange(T) + 3
        self.slots = rng.permutation(nb * bs)[:T] if scattered else rng.permutation(nb)[at // bs] * bs + at % bs
        self.pos = rng.integers(0, max_pos, (axes, T)).astype(np.int32)
        half = rot // 2
        if kind == "sections":      # uneven runs
            cut = np.sort(rng.integers(0, half + 1, axes - 1))
            self.axis = np.searchsorted(cut, np.arange(half), side="right").astype(np.uint8)
        elif kind == "in turn":
            self.axis = (np.arange(half) % axes).astype(np.uint8)
        else:
            self.axis = rng.integers(0, axes, half).astype(np.uint8)
        self.table = pa.pa_rope_table(max_pos, rot)
        qkv = torch.randn(T, (n_q + 2 * n_kv) * d, generator=g).to(self.dtype)
        self.qkv = qkv.cuda()
        self.q, self.k, self.v = (x.unflatten(1, (-1, d)) for x in self.qkv.split([n_q * d, n_kv * d, n_kv * d], 1))
        self.q_out = torch.full((T, n_q, d), 77.0, dtype=self.dtype, device="cuda")
        self.scales = dict(k_scale=0.07, v_scale=1 / 32) if pool in ("fp4", "fp8") else {}
        if pool == "fp4":
            before = [torch.randint(0, 256, (nb, n_kv, bs, 9 * d // 16), dtype=torch.uint8, generator=g) for _ in range(2)]
        elif pool == "fp8":
            before = [torch.randint(0, 256, s, dtype=torch.uint8, generator=g).view(F8)
                      for s in ((nb, n_kv, bs, d), (nb, n_kv, bs // 16, d, 16))]
        else:
            before = [torch.randn(nb, n_kv, bs, d, generator=g).to(self.dtype) for _ in range(2)]
        self.before = before
        self.kc, self.vc = before[0].cuda(), before[1].cuda()
        self.given = torch.from_numpy(self.slots.copy()).cuda()
        self.given_pos = torch.from_numpy(self.pos.copy()).cuda()

    def run(self, **kw):
        pa.pa_rope_axes_and_cache(self.q_out, self.q, self.k, self.v, self.given_pos, self.axis, self.table.cuda(), self.kc,
                                  self.vc, self.given, interleaved=self.interleaved, **self.scales, **kw)

    def rotated(self, x, dtype):
        """x [T][h][d] rotated in dtype, every operation rounded by itself, and |x| + |y| of the pairs"""
        half = self.rot // 2
        t = self.table.numpy()
        at = np.clip(self.pos, 0, len(t) - 1)[self.axis].T        # [T][pairs]
        c, s = t[at, np.arange(half)][:, None].astype(dtype), t[at, half + np.arange(half)][:, None].astype(dtype)
        x = x.float().cpu().numpy().astype(dtype)
        y, mag = x.copy(), np.abs(x)
        a, b = (slice(0, self.rot, 2), slice(1, self.rot, 2)) if self.interleaved else \
               (slice(0, half), slice(half, self.rot))
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
        return y, mag

    def check(self, written=None, error=0):
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == error
        w = np.ones(self.T, bool) if written is None else written
        f64 = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
        want, mag = self.rotated(self.q, np.float64)
        got = f64(self.q_out)
        assert (got[~w] == 77).all()
        assert (np.abs(got - want)[w] <= store_bound(want, self.dtype, mag)[w]).all()
        at = self.slots[w]
        b, o = at // self.bs, at % self.bs
        if self.pool == "fp4":
            for pool, before, rows, s in ((self.kc, self.before[0], self.rotated(self.k, np.float32)[0], 0.07),
                                          (self.vc, self.before[1], self.v.float().cpu().numpy(), 1 / 32)):
                full = before.numpy().copy()
                full[b, :, o] = ref.quantise(rows, s)[w]
                assert np.array_equal(pool.cpu().numpy(), full)
            return
        want, mag = self.rotated(self.k, np.float64)
        if self.pool == "fp8":
            got = f64(self.kc)[b, :, o] * np.float32(0.07)
            fp32 = 3 * 2.0 ** -24 * mag[w]
            top = 448 * np.float64(np.float32(0.07))
            bound = np.maximum((np.abs(want[w]) + fp32) * 2.0 ** -4, 0.07 * 2.0 ** -10) + fp32
            assert (np.abs(got - np.clip(want[w], -top, top)) <= bound).all()
            got = f64(self.vc)[b, :, o // 16, :, o % 16] / 32
            v = f64(self.v)[w]
            assert (np.abs(got - np.clip(v, -14, 14)) <= np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -15)).all()
            return
        got = f64(self.kc)
        assert (np.abs(got[b, :, o] - want[w]) <= store_bound(want, self.dtype, mag)[w]).all()
        rest = np.ones(got.shape[0] * self.bs, bool)
        rest[at] = False
        rest = np.flatnonzero(rest)
        assert np.array_equal(got[rest // self.bs, :, rest % self.bs], f64(self.before[0])[rest // self.bs, :, rest % self.bs])
        full = f64(self.before[1])
        full[b, :, o] = f64(self.v)[w]
        assert np.array_equal(f64(self.vc), full)


@pytest.mark.parametrize("T,n_q,n_kv,d,bs,act,pool,rot,interleaved,axes,kind,scattered", [
    (1, 32, 8, 128, 16, "bf16", "fp4", 128, False, 3, "sections", True),
    (1, 4, 1, 64, 16, "fp16", "fp4", 16, False, 2, "in turn", True),
    (67, 4, 2, 64, 32, "bf16", "fp4", 48, False, 4, "random", False),
    (300, 8, 2, 128, 16, "fp16", "fp4", 112, True, 3, "in turn", False),
    (1025, 6, 6, 128, 16, "bf16", "fp4", 64, True, 1, "random", False),
    (50, 4, 4, 64, 16, "fp32", "fp4", 64, False, 3, "sections", True),
    (700, 16, 4, 128, 32, "bf16", "fp8", 128, False, 3, "in turn", False),
    (33, 8, 2, 64, 16, "fp16", "fp8", 32, True, 2, "sections", True),
    (513, 32, 8, 128, 16, "bf16", "bf16", 128, False, 3, "sections", True),
    (100, 5, 1, 96, 16, "fp16", "fp16", 96, False, 4, "random", False),
    (64, 4, 2, 256, 32, "fp32", "fp32", 256, True, 3, "random", True),
    (90, 4, 2, 32, 16, "fp32", "fp32", 16, False, 2, "in turn", True)])
def test_rotation_by_axes(T, n_q, n_kv, d, bs, act, pool, rot, interleaved, axes, kind, scattered):
    c = Case(T + d, T, n_q, n_kv, d, bs, act, pool, rot, interleaved, axes, kind, scattered)
    c.run()
    c.check()


@pytest.mark.parametrize("pool", ["fp4", "fp8", "bf16"])
def test_padding_and_bad_places(pool):
    c = Case(5, 40, 8, 2, 128, 16, "bf16", pool, 128, False, 3, "in turn")
    w = np.ones(40, bool)
    w[[0, 7, 9, 20, 39]] = False
    c.given[0], c.given[7], c.given[9] = -1, -(2 ** 33), c.kc.shape[0] * 16
    c.given_pos[1, 20], c.given_pos[2, 39] = -1, 999
    c.run()
    c.check(w, pa.PA_ERR_OUT_OF_RANGE)


@pytest.mark.parametrize("pool", ["fp4", "bf16"])
def test_equal_axes_are_the_rotary_write_of_one(pool):
    c = Case(8, 200, 8, 2, 128, 16, "bf16", pool, 128, False, 3, "in turn")
    c.given_pos[:] = c.given_pos[:1].clone()
    c.run()
    one = [c.before[0].cuda(), c.before[1].cuda(), torch.empty_like(c.q_out)]
    pa.pa_rope_and_cache(one[2], c.q, c.k, c.v, c.given_pos[0].contiguous(), c.table.cuda(), one[0], one[1], c.given,
                         **c.scales)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for a, b in ((c.kc, one[0]), (c.vc, one[1]), (c.q_out, one[2])):
        assert torch.equal(a, b)


def test_in_place_and_rows_of_positions_apart():
    c = Case(9, 77, 8, 2, 128, 16, "bf16", "fp4", 128, False, 3, "sections")
    want = Case(9, 77, 8, 2, 128, 16, "bf16", "fp4", 128, False, 3, "sections")
    want.run()
    big = torch.full((3, 200), -5, dtype=torch.int32, device="cuda")
    big[:, :77] = c.given_pos
    c.given_pos, c.q_out = big[:, :77], c.q
    c.run()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    assert torch.equal(c.q, want.q_out) and torch.equal(c.kc, want.kc) and torch.equal(c.vc, want.vc)


@pytest.mark.parametrize("T,n_q,n_kv,d,act,pool,rot,axes", [
    (6000, 8, 2, 128, "bf16", "fp4", 128, 3), (6000, 8, 2, 64, "fp16", "fp8", 32, 4), (2600, 14, 1, 128, "bf16", "bf16", 112, 2),
    (6100, 3, 3, 64, "bf16", "fp4", 64, 3), (2000, 14, 1, 64, "fp32", "fp32", 64, 4)])
def test_long_chunks_with_padding_and_bad_places(T, n_q, n_kv, d, act, pool, rot, axes):
    """more tokens than the grid covers at once; the last axis turns no pair, and its positions are checked like the others'"""
    c = Case(T, T, n_q, n_kv, d, 16, act, pool, rot, False, axes, "random", False)
    c.axis[c.axis == axes - 1] = 0
    w = np.ones(T, bool)
    rng = np.random.default_rng(T)
    bad = rng.permutation(T)[:60]
    w[bad] = False
    c.given[bad[:20]] = -1
    c.given[bad[20:30]] = c.kc.shape[0] * 16
    for i, t in enumerate(bad[30:]):
        c.given_pos[i % axes, t] = -1 if i % 2 else 999
    c.given_pos[0, bad[:10]] = 12345                       # padding: its positions do not matter
    c.run()
    c.check(w, pa.PA_ERR_OUT_OF_RANGE)


@pytest.mark.parametrize("n_q", [8, 3])
def test_padding_with_any_positions_is_no_error(n_q):
    c = Case(6, 50, n_q, 1, 128, 16, "bf16", "fp4", 128, False, 3, "in turn")
    w = np.ones(50, bool)
    w[10:30] = False
    c.given[10:30] = -1
    c.given_pos[:, 10:30] = -7
    c.run()
    c.check(w)
