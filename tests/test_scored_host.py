"""CPU checks of the scored calls: workspace rules and refusals before any launch."""
import ctypes as C

import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from paged_kv_cache_25_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    return pa.lib()


def _decode(mod=None, dt=2, d=128, nq=1, B=4, mb=16, ws=0x10000, ws_bytes=1 << 24, null_mod=False, **kw):
    desc = pa._Desc(64, 16, 8, d, dt, 1.0, 1.0, 2)
    m = pa._ScoreMod(*(mod or (0.0, None, 0, None, None)))
    a = dict(out=0x1000, q=0x2000, kc=0x3000, vc=0x4000, bt=0x5000, cl=0x6000, n_q=32, scale=0.1, bs=16)
    a.update(kw)
    return pa.lib().pa_decode_scored(a["out"], 0, a["q"], a["kc"], a["vc"], C.byref(desc), a["bt"], mb,
                                     a["cl"], B, nq, a["n_q"], a["scale"], a["bs"],
                                     None if null_mod else C.byref(m), ws, ws_bytes, None)


BAD_MODS = [(-1.0, None, 0, None, None), (float("nan"), None, 0, None, None),
            (float("inf"), None, 0, None, None), (0.0, None, -1, None, None),
            (0.0, 0x1002, 0, None, None), (0.0, None, 0, 0x1001, None),
            (0.0, None, 0, None, 0x1003)]


@pytest.mark.parametrize("mod", BAD_MODS + [(0.0, None, 0, None, 0x1000)])
def test_decode_refuses_bad_modifications(mod):
    assert _decode(mod) == pa.PA_ERR_INVALID_ARG
    assert pa.lib().pa_last_error_message()


def test_decode_refusals():
    assert _decode(null_mod=True) == pa.PA_ERR_INVALID_ARG
    assert _decode(nq=0) == pa.PA_ERR_INVALID_ARG
    assert _decode(nq=17) == pa.PA_ERR_INVALID_ARG
    assert _decode(nq=2, dt=0) == pa.PA_ERR_UNSUPPORTED
    assert _decode(nq=2, d=96) == pa.PA_ERR_UNSUPPORTED
    assert _decode((1e9, None, 0, None, None)) == pa.PA_ERR_UNSUPPORTED
    assert _decode(q=0x2008) == pa.PA_ERR_INVALID_ARG
    assert _decode(n_q=30) == pa.PA_ERR_INVALID_ARG
    assert _decode(scale=float("nan")) == pa.PA_ERR_INVALID_ARG
    assert _decode(ws=None, ws_bytes=0) == pa.PA_ERR_WORKSPACE
    assert _decode(B=0) == pa.PA_OK


def test_a_window_bounds_the_workspace():
    size = pa.pa_decode_scored_workspace_size
    assert size(256, 1, 32, 8, 128, 16, 65536) == pa.pa_decode_workspace_size(256, 32, 8, 128, 16, 65536)
    # 1024 + 15 tokens of the first block at most: one partition, no partials
    assert size(256, 1, 32, 8, 128, 16, 65536, 1024) == 256
    # 2999 + 15 tokens: three partitions
    w = size(256, 1, 32, 8, 128, 16, 65536, 2999)
    assert 256 + 256 * 32 * 3 * 130 * 4 <= w < size(256, 1, 32, 8, 128, 16, 65536) // 16
    assert size(256, 4, 32, 8, 128, 16, 4096) == pa.pa_decode_verify_workspace_size(256, 4, 32, 8, 128, 16, 4096)
    assert size(256, 1, 32, 8, 128, 16, 4096, -1) == 0
    assert size(0, 1, 32, 8, 128, 16, 4096, 0) == 0
    # enough for exactly what the call asks
    need = size(4, 1, 32, 8, 128, 16, 256, 100)
    assert _decode((0.0, None, 100, None, None), ws_bytes=need - 1) == pa.PA_ERR_WORKSPACE


def _prefill(mod=None, dt=2, d=128, reqs=2, max_q=16, null_mod=False, **kw):
    desc = pa._Desc(64, 16, 8, d, dt, 1.0, 1.0, 2)
    m = pa._ScoreMod(*(mod or (0.0, None, 0, None, None)))
    a = dict(out=0x1000, q=0x2000, kc=0x3000, vc=0x4000, bt=0x5000, qs=0x6000, cl=0x7000, n_q=32,
             scale=0.1, bs=16, mb=8)
    a.update(kw)
    return pa.lib().pa_prefill_scored(a["out"], 0, a["q"], a["kc"], a["vc"], C.byref(desc), a["bt"],
                                      a["mb"], a["qs"], a["cl"], reqs, max_q, a["n_q"], a["scale"],
                                      a["bs"], None if null_mod else C.byref(m), None)


@pytest.mark.parametrize("mod", BAD_MODS)
def test_prefill_refuses_bad_modifications(mod):
    assert _prefill(mod) == pa.PA_ERR_INVALID_ARG


def test_prefill_refusals():
    assert _prefill(null_mod=True) == pa.PA_ERR_INVALID_ARG
    assert _prefill(dt=0) == pa.PA_ERR_UNSUPPORTED
    assert _prefill(d=96) == pa.PA_ERR_UNSUPPORTED
    assert _prefill((1e-9, None, 0, None, None)) == pa.PA_ERR_UNSUPPORTED
    assert _prefill(q=None) == pa.PA_ERR_INVALID_ARG
    assert _prefill(n_q=30) == pa.PA_ERR_INVALID_ARG
    assert _prefill(reqs=0) == pa.PA_OK
    assert _prefill(max_q=0) == pa.PA_OK


def test_bindings_check_layouts_and_types():
    """The scored and shared-prefix bindings refuse what the library would misread."""
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    bt, cl = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    base = dict(out=q, q=q, k_cache=kc, v_cache=kc, block_tables=bt, context_lens=cl, scale=0.1,
                block_size=16)
    qs = torch.zeros(3, dtype=torch.int32)
    calls = [lambda **k: pa.pa_decode_scored(mod=pa.ScoreMod(), **{**base, **k}),
             lambda **k: pa.pa_decode_shared(group_of_seq=cl, prefix_lens=cl, **{**base, **k}),
             lambda **k: pa.pa_prefill_scored(mod=pa.ScoreMod(), query_start_loc=qs, max_query_len=1,
                                              **{**base, **k})]
    for call in calls:
        for change, err in [(dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
                            (dict(q=q.half()), TypeError), (dict(out=q[:1]), ValueError),
                            (dict(block_tables=bt.long()), TypeError),
                            (dict(context_lens=cl.long()), TypeError),
                            (dict(block_tables=bt.T.contiguous().T), ValueError),
                            (dict(block_tables=bt[:1]), ValueError),
                            (dict(v_cache=kc.half()), TypeError),
                            (dict(k_cache=kc[:, :, :, :32]), ValueError),
                            (dict(v_cache=kc[:4]), ValueError)]:
            with pytest.raises(err):
                call(**change)
    with pytest.raises(ValueError):
        pa.pa_prefill_scored(mod=pa.ScoreMod(), query_start_loc=qs[:2], max_query_len=1, **base)
    with pytest.raises(TypeError):
        pa.pa_decode_shared(group_of_seq=cl.long(), prefix_lens=cl, **base)
    with pytest.raises(ValueError):
        pa.pa_decode_shared(group_of_seq=cl[:1], prefix_lens=cl, **base)


def test_bindings_refuse_what_is_not_on_the_current_device():
    """Well-formed CPU tensors, and objects that are no tensors, never reach the library."""
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    kc = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    bt, cl = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    slots, cs = torch.zeros(2, dtype=torch.int64), torch.zeros(8, 64)
    qs = torch.zeros(3, dtype=torch.int32)
    base = dict(out=q, q=q, k_cache=kc, v_cache=kc, block_tables=bt, context_lens=cl, scale=0.1,
                block_size=16)
    calls = [lambda **k: pa.pa_decode_scored(mod=pa.ScoreMod(), **{**base, **k}),
             lambda **k: pa.pa_decode_shared(group_of_seq=cl, prefix_lens=cl, **{**base, **k}),
             lambda **k: pa.pa_prefill_scored(mod=pa.ScoreMod(), query_start_loc=qs, max_query_len=1,
                                              **{**base, **k}),
             lambda **k: pa.pa_rope_and_cache(**{**dict(
                 q_out=q, q=q, k=kv, v=kv, positions=cl, cos_sin=cs, k_cache=kc, v_cache=kc,
                 slot_mapping=slots), **k})]
    for call in calls:
        with pytest.raises(ValueError, match="current CUDA device"):
            call(stream=0)
        with pytest.raises(TypeError):
            call(stream=0, q=[0.0])
