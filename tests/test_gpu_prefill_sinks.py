"""Chunked prefill over fp16, bf16 and FP8 pools of one key far above a long flat rest, whose probabilities are each next to
nothing and together are not.

Tolerance: probabilities enter P V as one fp16 part over fp16 and FP8 pools, off by half a step, 2^-11 of themselves, or, below
the smallest normal number, by 2^-25 under a reference that lies 7 powers of two below the row's largest score: 2^-32.
(Over bf16 pools as two bf16 parts: 2^-16 of themselves.)  The sums round by 2^-23 of the output a key at worst.  All scores
are exact."""
import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
NATS = 17.4          # e^-17.4 = 2^-25.1 is nothing in fp16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("scored", [False, True], ids=["plain", "scored"])
@pytest.mark.parametrize("reqs,n_kv", [(1, 1), (20, 8)])
@pytest.mark.parametrize("pool,act,d", [("fp16", "fp16", 128), ("fp16", "fp16", 64), ("bf16", "bf16", 128), ("fp8", "bf16", 128),
                                        ("fp8", "fp16", 128), ("fp8", "bf16", 64)])
def test_a_long_flat_rest_below_one_key(pool, act, d, reqs, n_kv, scored):
    bs, blocks, chunk, token = 32, 4096, 3, 700
    n, scale = blocks * bs, NATS / 96
    kc = torch.zeros(blocks, n_kv, bs, d, dtype=torch.float32, device="cuda")
    vc = torch.ones_like(kc)
    kc[token // bs, :, token % bs, :16] = 6
    vc[token // bs, :, token % bs] = 0
    if pool == "fp8":          # V: [d][16 tokens] pieces
        vc = vc.reshape(blocks, n_kv, bs // 16, 16, d).transpose(3, 4).contiguous()
    kc, vc = kc.to(TYPES[pool]), vc.to(TYPES[pool])
    scales = dict(k_scale=1.0, v_scale=1.0) if pool == "fp8" else {}
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda").repeat(reqs, 1)
    lens = torch.full((reqs,), n, dtype=torch.int32, device="cuda")
    start = torch.arange(reqs + 1, dtype=torch.int32, device="cuda") * chunk
    q = torch.ones(reqs * chunk, 2 * n_kv, d, dtype=TYPES[act], device="cuda")
    out = torch.empty(q.shape, device="cuda")
    if scored:
        pa.pa_prefill_scored(out, q, kc, vc, tables, start, lens, chunk, pa.ScoreMod(window=n + 5), scale, bs, **scales)
    else:
        pa.pa_prefill_chunk(out, q, kc, vc, tables, start, lens, chunk, scale, bs, **scales)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    keys = np.tile(n - chunk + 1 + np.arange(chunk), reqs).astype(np.float64)
    w = (keys - 1) * np.exp(-96 * np.float64(np.float32(scale)))
    want = w / (1 + w)
    tol = want * (2.0 ** -11 + keys * 2.0 ** -23) + keys * 2.0 ** -32
    worst = np.abs(out.cpu().numpy().astype(np.float64) - want[:, None, None]).max((1, 2))
    assert (worst <= tol).all(), (worst.max(), (worst / tol).max())
