"""Block copies and swaps of FP8 pools: they move codes, so the pool's scales and activation type are not asked for."""
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


@pytest.mark.parametrize("dtype,d", [(pa.PA_FP8_E4M3, 128), (pa.PA_FP4_E2M1, 64)])
@pytest.mark.parametrize("scales", [(0.0, 0.0, -1), (0.5, 0.25, pa.PA_BF16), (float("nan"), -1.0, pa.PA_F32)], ids=str)
def test_scales_are_not_asked_for(dtype, d, scales):
    desc = C.byref(pa._Desc(8, 16, 2, d, dtype, *scales))
    lib = pa.lib()
    assert lib.pa_copy_blocks(0x1000, 0x2000, desc, 0x3000, 0, None) == 0
    assert lib.pa_swap_blocks(0x1000, 0x2000, 8, 0x4000, 0x5000, 4, desc, 0x3000, 0, None) == 0
    assert lib.pa_copy_blocks(0x1000, 0x2000, desc, None, 1, None) == pa.PA_ERR_INVALID_ARG
    # the other calls do ask
    assert lib.pa_gather_cache(0x1000, 0x2000, 2, 0x3000, 0x4000, 0x5000, 1, C.byref(pa._Desc(8, 16, 2, d, dtype, 0.0, 0.0, -1)),
                               None) == pa.PA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("bs,d", [(16, 128), (32, 64)])
def test_blocks_are_copied_and_swapped(bs, d):
    assert pa.pa_get_device_error() == 0
    rng = np.random.default_rng(bs)
    raw = rng.integers(0, 256, (2, 30, 3, bs, d), dtype=np.uint8)
    kc = torch.from_numpy(raw[0]).cuda().view(torch.float8_e4m3fn)
    vc = torch.from_numpy(raw[1]).cuda().view(torch.float8_e4m3fn).view(30, 3, bs // 16, d, 16)      # (the layout of V)
    pairs = rng.permutation(30)[:20].reshape(10, 2).astype(np.int32)
    pa.pa_copy_blocks(kc, vc, torch.from_numpy(pairs).cuda())
    want = raw.copy()
    want[:, pairs[:, 1]] = raw[:, pairs[:, 0]]
    host = [torch.zeros(4, 3, bs, d, dtype=torch.uint8).pin_memory() for _ in range(2)]
    out = np.array([[5, 3], [29, 0]], np.int32)
    pa.pa_swap_blocks(kc, vc, host[0].view(torch.float8_e4m3fn), host[1].view(torch.float8_e4m3fn), torch.from_numpy(out).cuda())
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for i, (dev, h) in enumerate(((kc, host[0]), (vc, host[1]))):
        assert np.array_equal(dev.view(torch.uint8).cpu().numpy().reshape(want[i].shape), want[i])
        assert np.array_equal(h.numpy()[[3, 0]], want[i][[5, 29]]) and not h.numpy()[[1, 2]].any()
