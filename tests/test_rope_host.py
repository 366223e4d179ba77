"""CPU checks of the rotary cache write: the host table and the refusals, all
before any launch."""
import ctypes as C

import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from paged_kv_cache_25_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    return pa.lib()


@pytest.mark.parametrize("positions,rot,base", [(1, 16, 10000.0), (300, 64, 10000.0),
                                                (5000, 128, 500000.0)])
def test_table_is_the_cosines_and_sines_of_the_angles(positions, rot, base):
    t = pa.pa_rope_table(positions, rot, base).numpy().astype(np.float64)
    p = np.arange(positions)[:, None]
    a = p * base ** (-2.0 * np.arange(rot // 2) / rot)
    # one rounding to fp32 (2^-24 relative, values up to 1), plus the angle's own
    # rounding in fp64: |a| 2^-52, here below 1e-11
    tol = 2.0 ** -24 + 1e-11
    assert np.abs(t[:, :rot // 2] - np.cos(a)).max() <= tol
    assert np.abs(t[:, rot // 2:] - np.sin(a)).max() <= tol


def test_table_refusals():
    for args in [(0, 16, 1e4), (4, 15, 1e4), (4, 0, 1e4), (4, 16, 0.0), (4, 16, -1.0),
                 (4, 16, float("inf")), (4, 16, float("nan"))]:
        with pytest.raises(pa.PAError):
            pa.pa_rope_table(*args)


def _call(dt=2, pool=2, d=128, n_q=32, n_kv=8, rot=128, T=3, max_pos=100, q_out=0x1000, q=0x2000,
          k=0x3000, v=0x4000, pos=0x5000, cs=0x6000, kc=0x7000, vc=0x8000, slots=0x9000,
          qo_s=4096, q_s=4096, k_s=1024, v_s=1024, scale=0.5, nb=64):
    desc = pa._Desc(nb, 16, n_kv, d, pool, scale, scale, -1)
    return pa.lib().pa_rope_and_cache(q_out, q, k, v, dt, qo_s, q_s, k_s, v_s, pos, cs, max_pos,
                                      rot, 0, kc, vc, slots, T, n_q, C.byref(desc), None)


@pytest.mark.parametrize("bad", [
    dict(dt=3), dict(dt=9), dict(n_q=0), dict(rot=8), dict(rot=144), dict(rot=24), dict(max_pos=0),
    dict(T=-1), dict(q_out=None), dict(q=None), dict(k=None), dict(v=None), dict(pos=None),
    dict(cs=None), dict(kc=None), dict(vc=None), dict(slots=None), dict(q=0x2008),
    dict(slots=0x9004), dict(pos=0x5002), dict(cs=0x6008), dict(q_s=4095), dict(q_s=4097),
    dict(k_s=1020), dict(v_s=1028), dict(qo_s=8), dict(q_out=0x2000, qo_s=8192),
    dict(pool=3, scale=0.0), dict(pool=3, scale=float("nan")), dict(nb=0)],
    ids=lambda b: "-".join(f"{k}={v}" for k, v in b.items()))
def test_invalid_arguments_are_refused(bad):
    assert _call(**bad) == pa.PA_ERR_INVALID_ARG
    assert pa.lib().pa_last_error_message()


@pytest.mark.parametrize("bad", [
    dict(dt=1), dict(dt=0), dict(d=80, rot=16), dict(pool=3, d=96, rot=96),
    dict(T=1 << 30)], ids=lambda b: "-".join(f"{k}={v}" for k, v in b.items()))
def test_unsupported_arguments_are_refused(bad):
    assert _call(**bad) == pa.PA_ERR_UNSUPPORTED


def test_no_tokens_is_a_no_op():
    assert _call(T=0, q_out=None, q=None, k=None, v=None) == pa.PA_OK


def test_binding_checks_shapes_and_types():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    pos, slots = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    cs = torch.zeros(8, 64)
    ok = dict(q_out=q, q=q, k=k, v=k, positions=pos, cos_sin=cs, k_cache=kc, v_cache=kc,
              slot_mapping=slots)
    for change, err in [(dict(positions=pos.long()), TypeError), (dict(cos_sin=cs.double()), TypeError),
                        (dict(slot_mapping=slots.int()), TypeError), (dict(k=k.half()), TypeError),
                        (dict(q_out=q.float()), TypeError), (dict(positions=pos[:1]), ValueError),
                        (dict(k=k[:, :1]), ValueError), (dict(q_out=q[:1]), ValueError),
                        (dict(q=torch.zeros(2, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), ValueError)]:
        with pytest.raises(err):
            pa.pa_rope_and_cache(**{**ok, **change}, stream=0)
