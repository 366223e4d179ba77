"""4-bit pools: rows written, read back, copied.  Written rows are compared bit for bit with the format's
steps in NumPy; rows read back with the values of their bytes, rounded once."""
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


def slots_of(kind, T, bs, rng):
    """slots of T tokens and the pool's blocks: consecutive tokens of one sequence from an odd offset, or scattered"""
    nb = T // bs + 6 if kind == "chunk" else T + 6
    if kind == "chunk":
        at = np.arange(T) + 5
        return rng.permutation(nb)[at // bs] * bs + at % bs, nb
    return rng.permutation(nb * bs)[:T], nb


def rows_of(T, n_kv, d, dtype, seed, wild=True):
    x = torch.randn(T, n_kv, d, generator=torch.Generator().manual_seed(seed))
    if wild:      # large and tiny groups, exact ties, zeros, infinities, NaN
        scale = 2.0 ** torch.randint(-24, 16, (T, n_kv, d // 16, 1), generator=torch.Generator().manual_seed(seed + 1))
        x = (x.unflatten(2, (-1, 16)) * scale).flatten(2)
        x[0, 0, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6] * 2) / 16
        x[-1, -1, :16] = 0
        x[T // 2, 0, 3] = float("inf")
        x[T // 3, -1, 20] = float("-inf")
        x[T // 4, 0, d - 1] = float("nan")
    return x.to(dtype)


def bytes_of(x, scale):
    return ref.quantise(x.float().numpy(), scale)


@pytest.mark.parametrize("T,n_kv,d,bs,dtype,kind", [
    (1, 1, 64, 16, "bf16", "scattered"), (1, 8, 128, 16, "bf16", "chunk"), (16, 2, 128, 32, "fp16", "chunk"),
    (37, 3, 64, 16, "fp32", "chunk"), (255, 8, 128, 16, "bf16", "scattered"), (700, 10, 64, 32, "fp16", "scattered"),
    (1031, 4, 128, 32, "fp32", "chunk")])
def test_rows_are_written_bit_for_bit(T, n_kv, d, bs, dtype, kind):
    rng = np.random.default_rng(T)
    slots, nb = slots_of(kind, T, bs, rng)
    ks, vs = 0.07, 1.0 / 32
    k, v = rows_of(T, n_kv, d, ACT[dtype], T), rows_of(T, n_kv, d, ACT[dtype], T + 50)
    before = rng.integers(0, 256, (2, nb, n_kv, bs, 9 * d // 16), dtype=np.uint8)
    kc, vc = torch.from_numpy(before[0]).cuda(), torch.from_numpy(before[1]).cuda()
    given = slots.copy()
    skip = np.zeros(T, bool)
    if T > 20:      # padding, and a slot past the pool
        skip[[3, 11, T - 1]] = True
        given[3], given[11] = -1, -(2 ** 40)
        given[T - 1] = nb * bs
    pa.pa_reshape_and_cache_quant(k.cuda(), v.cuda(), kc, vc, torch.from_numpy(given).cuda(), ks, vs)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == (pa.PA_ERR_OUT_OF_RANGE if T > 20 else 0)
    for got, old, x, s in ((kc, before[0], k, ks), (vc, before[1], v, vs)):
        want = old.copy()
        at = slots[~skip]
        want[at // bs, :, at % bs] = bytes_of(x, s)[~skip]
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("scale", [1.0, 0.0371, 1 / 3, 7.7e-5, 3.3e8, 2.0 ** -55, 2.0 ** 52, 2.0 ** 54 * 1.3, 1.1e-17, 1e-25])
def test_borders_between_codes(scale):
    """elements that are a few units in the last place beside the quotients' borders, in both forms of the division
    (the divisors lie on both sides of 2^-60 and 2^60), and groups that saturate"""
    rng = np.random.default_rng(int(abs(np.log2(scale)) * 8))
    T, n_kv, d, bs = 500, 8, 128, 16
    s = rng.choice(ref.E4M3[1:127], (T, n_kv, d // 16, 1))
    r = (s.astype(np.float32) * np.float32(scale)).astype(np.float32)
    border = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 3.0], (T, n_kv, d // 16, 16))
    with np.errstate(all="ignore"):
        x = (r.astype(np.float64) * border * rng.choice([-1, 1], border.shape)).astype(np.float32)
        ulps = rng.integers(-3, 4, x.shape).astype(np.int32)
        x = (x.view(np.int32) + np.where(np.abs(x) > 1e-37, ulps, 0)).view(np.float32)
        x[..., 7] = (r[..., 0].astype(np.float64) * 6).astype(np.float32)          # the group's largest, which makes its scale
        x[::7, :, :, 3] *= np.float32(300)                                           # (and some that are far larger)
        x[::5, :, :, 2] = -0.0
    x = torch.from_numpy(np.ascontiguousarray(x.reshape(T, n_kv, d)))
    slots = np.arange(T)
    kc, vc = (torch.zeros(T // bs + 1, n_kv, bs, 9 * d // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    pa.pa_reshape_and_cache_quant(x.cuda(), (-x).cuda(), kc, vc, torch.from_numpy(slots).cuda(), scale, scale)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for got, y in ((kc, x), (vc, -x)):
        assert np.array_equal(got.cpu().numpy()[slots // bs, :, slots % bs], bytes_of(y, scale))


@pytest.mark.parametrize("scale", [1e-30, 2.0 ** -40, 1e30])
def test_extreme_scales(scale):
    x = torch.randn(40, 2, 64, generator=torch.Generator().manual_seed(1)) * torch.tensor(
        [1e-36, 1e-30, 1e-8, 1.0, 1e30]).repeat(8)[:, None, None]
    kc = torch.zeros(3, 2, 16, 36, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    pa.pa_reshape_and_cache_quant(x.cuda(), x.cuda(), kc, vc, torch.arange(40).cuda(), scale, scale)
    want = np.zeros((48, 2, 36), np.uint8)
    want[:40] = bytes_of(x, scale)
    assert pa.pa_get_device_error() == 0
    assert np.array_equal(kc.transpose(1, 2).flatten(0, 1).cpu().numpy(), want)
    assert np.array_equal(vc.cpu().numpy(), kc.cpu().numpy())


def to_dtype(x, dtype):
    """fp64 values rounded to float32, then to dtype"""
    with np.errstate(over="ignore"):
        return torch.from_numpy(x.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("T,n_kv,d,bs,out,kind", [
    (1, 8, 128, 16, "bf16", "scattered"), (17, 1, 64, 32, "fp32", "chunk"), (300, 8, 128, 16, "fp16", "scattered"),
    (1000, 3, 64, 16, "bf16", "chunk"), (5000, 10, 128, 32, "bf16", "chunk")])
@pytest.mark.parametrize("pool", ["fp4", "fp8", "bf16", "fp16", "fp32"])
def test_rows_are_read_back(T, n_kv, d, bs, out, kind, pool):
    rng = np.random.default_rng(T + d)
    slots, nb = slots_of(kind, T, bs, rng)
    if T > 2:
        slots[1] = slots[0]                          # the same row twice
    b, o = slots // bs, slots % bs
    scales = {"k_scale": 0.07, "v_scale": 1.0 / 32}
    raw = rng.integers(0, 256, (2, nb, n_kv, bs, 9 * d // 16), dtype=np.uint8)
    if pool == "fp4":
        raw[0, b[0], 0, o[0], d // 2] = 0x7F         # a NaN scale
        kc, vc = torch.from_numpy(raw[0]).cuda(), torch.from_numpy(raw[1]).cuda()
        k, v = (ref.values(raw[i][b, :, o], s) for i, s in enumerate(scales.values()))
    elif pool == "fp8":
        code = rng.integers(0, 256, (2, nb, n_kv, bs, d), dtype=np.uint8)
        vt = code[1].reshape(nb, n_kv, bs // 16, 16, d).swapaxes(3, 4)
        kc = torch.from_numpy(code[0]).cuda().view(torch.float8_e4m3fn)
        vc = torch.from_numpy(np.ascontiguousarray(vt)).cuda().view(torch.float8_e4m3fn)
        k, v = (ref.E4M3[code[i][b, :, o]] * np.float64(np.float32(s)) for i, s in enumerate(scales.values()))
    else:
        x = torch.randn(2, nb, n_kv, bs, d, generator=torch.Generator().manual_seed(T)).to(ACT[pool])
        kc, vc = x[0].cuda(), x[1].cuda()
        k, v = (x[i].double().numpy()[b, :, o] for i in range(2))
        scales = {}
    vc = vc.reshape(kc.shape) if pool != "fp8" else vc
    given = slots.copy()
    keep = np.zeros(T, bool)
    if T > 20:
        keep[[2, 9, T - 1]] = True
        given[2], given[9], given[T - 1] = -1, -7, nb * bs
    ko = torch.full((T, n_kv, d), 7.0, dtype=ACT[out], device="cuda")
    vo = ko.clone()
    pa.pa_gather_cache(ko, vo, kc, vc, torch.from_numpy(given).cuda(), **scales)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == (pa.PA_ERR_OUT_OF_RANGE if T > 20 else 0)
    for got, want in ((ko, k), (vo, v)):
        want = to_dtype(want, ACT[out])
        want[torch.from_numpy(keep)] = 7.0
        assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=1234.5), torch.nan_to_num(want.float(), nan=1234.5))


def test_no_tokens_is_no_work():
    pool = torch.zeros(2, 2, 16, 72, dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    pa.pa_gather_cache(none, none.clone(), pool, pool.clone(), slots, k_scale=1.0, v_scale=1.0)
    pa.pa_reshape_and_cache_quant(none, none, pool, pool.clone(), slots, 1.0, 1.0)
    assert pa.pa_get_device_error() == 0 and not pool.any()


@pytest.mark.parametrize("bs,d", [(16, 128), (32, 64)])
def test_blocks_are_copied_and_swapped(bs, d):
    rng = np.random.default_rng(bs)
    raw = rng.integers(0, 256, (2, 30, 3, bs, 9 * d // 16), dtype=np.uint8)
    kc, vc = torch.from_numpy(raw[0]).cuda(), torch.from_numpy(raw[1]).cuda()
    pairs = rng.permutation(30)[:20].reshape(10, 2).astype(np.int32)
    pa.pa_copy_blocks(kc, vc, torch.from_numpy(pairs).cuda())
    want = raw.copy()
    want[:, pairs[:, 1]] = raw[:, pairs[:, 0]]
    host = [torch.zeros(4, 3, bs, 9 * d // 16, dtype=torch.uint8).pin_memory() for _ in range(2)]
    out = np.array([[5, 3], [29, 0]], np.int32)
    pa.pa_swap_blocks(kc, vc, host[0], host[1], torch.from_numpy(out).cuda())
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for i, (dev, h) in enumerate(((kc, host[0]), (vc, host[1]))):
        assert np.array_equal(dev.cpu().numpy(), want[i])
        assert np.array_equal(h.numpy()[[3, 0]], want[i][[5, 29]]) and not h.numpy()[[1, 2]].any()
