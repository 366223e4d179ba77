"""CPU checks of the 4-bit pools' calls, the several-axes rotary write and the gather: what is refused before any
launch, and the host helper."""
import ctypes as C

import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from paged_kv_cache_25_gb300 import build

FP4, FP8, BF16, FP16, F32 = 4, 3, 2, 1, 0
INVALID, UNSUPPORTED = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    return pa.lib()


def desc(pool=FP4, nb=64, bs=16, n_kv=8, d=128, ks=0.5, vs=0.5, act=BF16):
    return pa._Desc(nb, bs, n_kv, d, pool, ks, vs, act)


BAD_POOLS = [(dict(d=32), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
             (dict(nb=0), INVALID), (dict(n_kv=0), INVALID), (dict(ks=0.0), INVALID), (dict(vs=-1.0), INVALID),
             (dict(ks=float("nan")), INVALID), (dict(vs=float("inf")), INVALID), (dict(ks=1e-31), UNSUPPORTED),
             (dict(vs=2e30), UNSUPPORTED), (dict(nb=1 << 24), UNSUPPORTED), (dict(pool=5), INVALID)]


def gather(T=3, out=BF16, ko=0x1000, vo=0x2000, kc=0x3000, vc=0x4000, slots=0x5000, **kw):
    return pa.lib().pa_gather_cache(ko, vo, out, kc, vc, slots, T, C.byref(desc(**kw)), None)


def write(T=3, dt=BF16, k=0x1000, v=0x2000, kc=0x3000, vc=0x4000, slots=0x5000, **kw):
    return pa.lib().pa_reshape_and_cache_quant(k, v, dt, kc, vc, slots, T, C.byref(desc(**kw)), None)


def rope(T=3, dt=BF16, rot=128, max_pos=100, axes=3, stride=3, axis=b"\0\1\2\0" * 16, q_out=0x1000, q=0x2000, k=0x3000,
         v=0x4000, pos=0x5000, cs=0x6000, kc=0x7000, vc=0x8000, slots=0x9000, n_q=32, q_s=4096, **kw):
    return pa.lib().pa_rope_axes_and_cache(q_out, q, k, v, dt, 4096, q_s, 1024, 1024, pos, stride, axes, axis, cs, max_pos,
                                           rot, 0, kc, vc, slots, T, n_q, C.byref(desc(**kw)), None)


def decode(rows=1, out=BF16, q=0x2000, kc=0x3000, tables=0x5000, lens=0x6000, seqs=2, n_q=32, scale=0.1, bs=16, ws=0x10000,
           ws_bytes=1 << 30, width=8, **kw):
    d = desc(bs=bs, **kw)
    if rows == 1:
        return pa.lib().pa_decode(0x1000, out, q, kc, 0x4000, C.byref(d), tables, width, lens, seqs, n_q, scale, bs, ws,
                                  ws_bytes, None)
    return pa.lib().pa_decode_verify(0x1000, out, q, kc, 0x4000, C.byref(d), tables, width, lens, seqs, rows, n_q, scale, bs,
                                     ws, ws_bytes, None)


def prefill(out=BF16, q=0x2000, start=0x5000, reqs=2, max_q=4, n_q=32, scale=0.1, **kw):
    return pa.lib().pa_prefill_chunk(0x1000, out, q, 0x3000, 0x4000, C.byref(desc(**kw)), 0x6000, 8, start, 0x7000, reqs, max_q,
                                     n_q, scale, 16, None, 0, None)


@pytest.mark.parametrize("call", [gather, write, rope, decode, prefill], ids=lambda f: f.__name__)
@pytest.mark.parametrize("bad,status", BAD_POOLS, ids=str)
def test_pools_that_are_refused(call, bad, status):
    assert call(**bad) == status and pa.lib().pa_last_error_message()


@pytest.mark.parametrize("call", [decode, prefill], ids=lambda f: f.__name__)
def test_attention_needs_an_activation_type(call):
    assert call(act=F32) == INVALID and call(act=-1) == INVALID


@pytest.mark.parametrize("bad,status", [
    (dict(out=FP8), INVALID), (dict(out=FP4), INVALID), (dict(out=9), INVALID), (dict(T=-1), INVALID), (dict(ko=None), INVALID),
    (dict(vo=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(slots=None), INVALID),
    (dict(ko=0x1008), INVALID), (dict(vc=0x4004), INVALID), (dict(slots=0x5004), INVALID),
    (dict(pool=FP8, d=96), UNSUPPORTED), (dict(n_kv=70000, nb=1), UNSUPPORTED)], ids=str)
def test_gather_refusals(bad, status):
    assert gather(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(dt=FP8), UNSUPPORTED), (dict(dt=7), UNSUPPORTED), (dict(T=-1), INVALID), (dict(k=None), INVALID),
    (dict(vc=None), INVALID), (dict(k=0x1004), INVALID), (dict(slots=0x5004), INVALID),
    (dict(dt=FP4), UNSUPPORTED)], ids=str)      # rows are quantised by the call: there are no ready codes
def test_write_refusals(bad, status):
    assert write(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(axes=0), INVALID), (dict(axes=5), INVALID), (dict(axes=-1), INVALID), (dict(axis=None), INVALID),
    (dict(axes=2), INVALID), (dict(stride=2), INVALID), (dict(stride=-3), INVALID), (dict(rot=8), INVALID),
    (dict(rot=144), INVALID), (dict(rot=24), INVALID), (dict(max_pos=0), INVALID), (dict(T=-1), INVALID),
    (dict(pos=None), INVALID), (dict(pos=0x5002), INVALID), (dict(q_out=None), INVALID), (dict(cs=0x6004), INVALID),
    (dict(dt=FP8), INVALID), (dict(dt=FP4), INVALID), (dict(n_q=0), INVALID), (dict(q_s=4095), INVALID),
    (dict(pool=FP16), UNSUPPORTED), (dict(T=1 << 23, stride=1 << 23), UNSUPPORTED)], ids=str)
def test_rope_axes_refusals(bad, status):
    assert rope(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INVALID), (dict(kc=0x3008), INVALID), (dict(n_q=12), INVALID), (dict(width=0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(ws=None), pa.PA_ERR_WORKSPACE), (dict(rows=17), INVALID),
    (dict(rows=4, q=None), INVALID), (dict(seqs=-1), INVALID), (dict(seqs=70000), UNSUPPORTED), (dict(out=FP4), INVALID)],
    ids=str)
def test_decode_refusals(bad, status):
    assert decode(**bad) == status


def test_nothing_to_do_needs_no_pointers():
    assert gather(T=0, ko=None, slots=None) == 0 and write(T=0, k=None) == 0 and rope(T=0, q=None) == 0
    assert decode(seqs=0, q=None) == 0 and prefill(reqs=0) == 0 and prefill(max_q=0) == 0


def test_calls_that_do_not_take_4_bit_pools():
    lib, d = pa.lib(), C.byref(desc())
    mod = C.byref(pa._ScoreMod(0.0, None, 0, None, None))
    assert lib.pa_reshape_and_cache(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 3, d, None) == UNSUPPORTED
    assert lib.pa_decode_no_alloc(0x1000, 2, 0x2000, 0x3000, 0x4000, d, 0x5000, 8, 0x6000, 2, 32, 0.1, 16, None) == UNSUPPORTED
    assert lib.pa_decode_scored(0x1000, 2, 0x2000, 0x3000, 0x4000, d, 0x5000, 8, 0x6000, 2, 1, 32, 0.1, 16, mod, 0x10000,
                                1 << 30, None) == UNSUPPORTED
    assert lib.pa_decode_shared(0x1000, 2, 0x2000, 0x3000, 0x4000, d, 0x5000, 8, 0x6000, 2, 32, 0.1, 16, 0x7000, 0x8000, 1,
                                0x10000, 1 << 30, None) == UNSUPPORTED
    assert lib.pa_prefill_scored(0x1000, 2, 0x2000, 0x3000, 0x4000, d, 0x5000, 8, 0x6000, 0x7000, 2, 4, 32, 0.1, 16, mod,
                                 None) == UNSUPPORTED


def test_axis_maps():
    assert pa.pa_rope_axes([2, 3, 1]).tolist() == [0, 0, 1, 1, 1, 2]
    assert pa.pa_rope_axes([2, 3, 1], in_turn=True).tolist() == [0, 1, 2, 0, 1, 1]
    assert pa.pa_rope_axes([4, 0]).tolist() == [0] * 4 and pa.pa_rope_axes([4, 0]).dtype == np.uint8
    for bad in ([], [1] * 5, [3, -1]):
        with pytest.raises(pa.PAError):
            pa.pa_rope_axes(bad)


def test_python_refusals():
    pool = torch.zeros(2, 2, 16, 72, dtype=torch.uint8)
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    kv = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    slots, table = torch.zeros(3, dtype=torch.int64), torch.zeros(9, 128)
    pos = torch.zeros(3, 3, dtype=torch.int32)

    def call(p=pos, axis=bytes(64), kc=pool):
        pa.pa_rope_axes_and_cache(q, q, kv, kv, p, axis, table, kc, kc, slots, k_scale=1.0, v_scale=1.0)

    for bad in (dict(p=pos[0]), dict(p=pos[:, :2]), dict(p=pos.t().contiguous().t()), dict(kc=pool[..., :71].contiguous()),
                dict(kc=torch.zeros(2, 2, 16, 36, dtype=torch.uint8)), {}):       # ({}: not on a GPU)
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(TypeError):
        call(p=pos.long())
    with pytest.raises(TypeError):
        call(axis=np.zeros(64, np.int64))
    out = torch.zeros(3, 2, 128)
    for bad in (dict(k=out[:, :1]), dict(k=out[..., :64]), dict(s=slots[:2]), {}):
        with pytest.raises(ValueError):
            pa.pa_gather_cache(bad.get("k", out), out, pool, pool, bad.get("s", slots), k_scale=1.0, v_scale=1.0)
    with pytest.raises(TypeError):
        pa.pa_gather_cache(out, out.half(), pool, pool, slots, k_scale=1.0, v_scale=1.0)
    lens, tables = torch.ones(3, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int32)
    for bad in (dict(q=q[..., :64].contiguous()), dict(q=q.float(), e=0), dict(lens=lens[:2]), {}):
        x = bad.get("q", q)
        with pytest.raises((ValueError, TypeError)):
            pa.pa_decode(torch.zeros_like(x), x, pool, pool, tables, bad.get("lens", lens), 1.0, 16, None, k_scale=1.0, v_scale=1.0)
    with pytest.raises(ValueError):
        pa._desc(torch.zeros(2, 2, 16, 70, dtype=torch.uint8), 1.0, 1.0, torch.bfloat16)
