"""Plain fp64 attention with score modifications, and pools for the tests of the
scored and shared-prefix calls.  Expected values come from the drawn rows alone,
never from the CUDA path.

Tolerances.  For outputs in fp32 from 16-bit or FP8 pools with values of N(0, 1): a
probability enters P V with 11 (one fp16 part) or at least 16 bits, so an output moves by at
most 2^-12 max|v| (1.2e-3 for |v| <= 5) or 2^-17 max|v|; scores (fp32 sums of at most 128
exact products of magnitude summing to ~10) and the cap (score_mod.cuh: C 2^-22) are off by
less than 5e-5, which moves an output by 2 * 5e-5 * max|v| = 5e-4 at most: 2e-3 together.
For fp32 pools: 1e-5, and with a cap c or a bias (whose rounding is 2^-24 of its size; keys
that still weigh lie within 20 of the nearest) (c + 20) 2^-22 max|v| more.
A low-precision output adds half a step of its dtype."""
import numpy as np
import torch

import oracle
from paged_kv_cache_25_gb300 import binding as pa
from tests.helpers import half_ulp

F8 = torch.float8_e4m3fn


def tolerance(dtype, softcap=0.0, alibi=False):
    if dtype != torch.float32:
        return 2e-3
    return 1e-5 + ((softcap + 20) * 2.0 ** -22 * 5 if softcap or alibi else 0.0)


def slopes_of(n_q):
    return (2.0 ** (-8.0 * (np.arange(n_q) + 1) / n_q)).astype(np.float32)


def attend64(q, k, v, pos, lo, hi, scale, softcap=0.0, slopes=None):
    """q [rows][n_q][d], k, v [n][n_kv][d] fp64; row i at pos[i] sees keys lo[i]..hi[i]."""
    rows, n_q, _ = q.shape
    g = n_q // k.shape[1]
    out = np.zeros_like(q)
    j = np.arange(len(k))
    for i in range(rows):
        see = (j >= lo[i]) & (j <= hi[i])
        if not see.any():
            continue
        z = np.einsum("nkd,kgd->kgn", k[see], q[i].reshape(-1, g, q.shape[2])) * scale
        z = z.reshape(n_q, -1)
        if softcap:
            z = softcap * np.tanh(z / softcap)
        if slopes is not None:
            z = z - slopes.astype(np.float64)[:, None] * np.abs(j[see] - pos[i])
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out[i] = np.einsum("kgn,nkd->kgd", p.reshape(-1, g, p.shape[1]), v[see]).reshape(n_q, -1)
    return out


class Pools:
    """K/V rows of several sequences in NaN-filled pools behind block tables; sequences may
    share their leading blocks (prefix_of: for each sequence the one whose first `prefix[s]`
    tokens it shares, or -1; that one comes earlier)."""

    def __init__(self, seed, lens, n_kv, d, bs, dtype, fp8=False, scale=1.0 / 64, prefix_of=None,
                 prefix=None, max_blocks=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.bs, self.n_kv, self.d, self.dtype, self.fp8 = bs, n_kv, d, dtype, fp8
        self.lens = np.asarray(lens, np.int32)
        B = len(self.lens)
        need = -(-self.lens // bs)
        self.nb = nb = int(need.sum()) + 5
        order = rng.permutation(nb)
        mb = max_blocks or max(1, int(need.max()))
        self.tables = np.full((B, mb), -1, np.int32)
        shape = (nb, n_kv, bs, d)
        if fp8:
            self.kc = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(F8)
            self.vc = torch.full((nb, n_kv, bs // 16, d, 16), 0x7F, dtype=torch.uint8,
                                 device="cuda").view(F8)
            self.scales = dict(k_scale=scale, v_scale=scale)
        else:
            self.kc = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
            self.vc = torch.full_like(self.kc, float("nan"))
            self.scales = {}
        used, ks, vs, slots, raw_k, raw_v = 0, [], [], [], [], []
        for s, L in enumerate(self.lens):
            L = int(L)
            k = torch.randn(L, n_kv, d, generator=g).to(dtype)
            v = torch.randn(L, n_kv, d, generator=g).to(dtype)
            n0 = 0
            if prefix_of is not None and prefix_of[s] >= 0:
                f = prefix_of[s]
                n0 = min(int(prefix[s]), L)
                assert n0 % bs == 0 or n0 == L
                k[:n0], v[:n0] = raw_k[f][:n0], raw_v[f][:n0]
                self.tables[s, :-(-n0 // bs)] = self.tables[f, :-(-n0 // bs)]
            b0 = -(-n0 // bs)
            new = int(need[s]) - b0
            self.tables[s, b0:b0 + new] = order[used:used + new]
            used += new
            raw_k.append(k)
            raw_v.append(v)
            at = np.arange(n0, L)
            slots.append(self.tables[s, at // bs].astype(np.int64) * bs + at % bs)
            ks.append(k[at]); vs.append(v[at])
        k, v = torch.cat(ks).cuda(), torch.cat(vs).cuda()
        slots = torch.from_numpy(np.concatenate(slots)).cuda()
        if len(slots):
            write = pa.pa_reshape_and_cache_quant if fp8 else pa.pa_reshape_and_cache
            write(k, v, self.kc, self.vc, slots, **self.scales)
        stored = (lambda x: oracle.dequantize_fp8(oracle.quantize_fp8(x, scale), scale)) if fp8 else \
                 (lambda x: x.double().numpy())  # noqa: E731
        self.k64 = [np.asarray(stored(x), np.float64).reshape(x.shape) for x in raw_k]
        self.v64 = [np.asarray(stored(x), np.float64).reshape(x.shape) for x in raw_v]

    @property
    def scale(self):
        return float(np.float32(1.0 / np.sqrt(self.d)))

    @property
    def max_ctx(self):
        return self.tables.shape[1] * self.bs

    def dev(self):
        return torch.from_numpy(self.tables).cuda(), torch.from_numpy(self.lens).cuda()

    def spoil(self, s, first):
        """Keys of sequence s before `first` become NaN, and blocks that hold nothing else -1."""
        at = np.arange(min(int(first), int(self.lens[s])))
        b, o = self.tables[s, at // self.bs].astype(np.int64), at % self.bs
        if self.fp8:
            self.kc.view(torch.uint8)[b, :, o] = 0x7F
            self.vc.view(torch.uint8)[b, :, o // 16, :, o % 16] = 0x7F
        else:
            self.kc[b, :, o] = float("nan")
            self.vc[b, :, o] = float("nan")
        self.tables[s, :int(first) // self.bs] = -1


def check(got, ref, tol, dtype=torch.float32):
    """got within tol of ref, plus half a step where it is stored in fewer bits"""
    err = np.abs(got.detach().float().cpu().numpy().astype(np.float64) - ref)
    bound = tol + (half_ulp(ref, dtype) if dtype != torch.float32 else 0.0)
    assert np.isfinite(err).all()
    assert (err <= bound).all(), float((err - bound).max())
