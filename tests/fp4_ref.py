"""The 4-bit row format in NumPy, and 4-bit pools for the tests.  Expected values come from the drawn
rows and from tables of the two small formats, never from the CUDA path.

Tolerances of attention over 4-bit pools (fp32 outputs, |v| <= vmax in the pool): a pool's values are
exact in fp16 and so are queries (scaled by a power of two).  Scores are fp32 sums of at most
128 exact products whose magnitudes add up to ~20 (q, k of N(0, 1), scale d^-1/2): each of the
at most 136 additions rounds by 2^-24 of a partial sum of at most 20, less than 1.7e-4 in all at worst
and in practice a tenth of it; 5e-5 is counted, which moves an output by at most 2 * 5e-5 * vmax.
Exponentials are off by 2^-22.  A probability enters P V as one fp16 part: an output moves by at most
2^-12 vmax.  A low-precision output adds half a step of its dtype."""
import numpy as np
import torch

from tests.helpers import half_ulp

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def _e4m3():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, 2.0 ** (e - 7.0) * (1 + m / 8))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


E4M3 = _e4m3()


def nearest_code(x, table, top):
    """index of the entry of table[0..top] (ascending, from 0) nearest to x >= 0, ties to the even index"""
    t = table[:top + 1]
    hi = np.clip(np.searchsorted(t, x, side="left"), 1, top)
    lo = hi - 1
    mid = (t[lo] + t[hi]) / 2
    up = (x > mid) | ((x == mid) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantise(x, scale):
    """rows [..., d] (float32) -> bytes [..., 9 d / 16]: the documented steps, each rounded to float32"""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, 16)
    scale = np.float32(scale)
    with np.errstate(all="ignore"):
        a = np.abs(g).max(-1)                                     # (NaN if any is)
        nan = np.isnan(g).any(-1)
        t = (np.where(nan, 0, a) / (np.float32(6) * scale)).astype(np.float32)
        t = np.minimum(np.maximum(t, np.float32(2.0 ** -9)), np.float32(448))
        s = nearest_code(t.astype(np.float64), E4M3, 126)
        r = (E4M3[s].astype(np.float32) * scale).astype(np.float32)
        y = (g / r[..., None]).astype(np.float32)
        mag = np.where(np.isnan(y), 0, np.minimum(np.abs(y), 6)).astype(np.float64)
    code = nearest_code(mag, E2M1, 7) | (np.signbit(y).astype(np.int64) << 3)
    code = np.where(nan[..., None], 0, code)
    s = np.where(nan, 0x7F, s)
    code = code.reshape(*x.shape[:-1], -1)
    return np.concatenate([code[..., 0::2] | code[..., 1::2] << 4, s], -1).astype(np.uint8)


def values(rows, scale):
    """bytes [..., 9 d / 16] -> fp64 values [..., d]"""
    d = rows.shape[-1] // 9 * 16
    code = np.stack([rows[..., :d // 2] & 15, rows[..., :d // 2] >> 4], -1).reshape(*rows.shape[:-1], d)
    return E2M1[code] * np.repeat(E4M3[rows[..., d // 2:]], 16, -1) * np.float64(np.float32(scale))


def tolerance(vmax):
    return vmax * (2 * 5e-5 + 2.0 ** -20 + 2.0 ** -12)


class Pools:
    """4-bit K/V rows of several sequences, in pools whose other bytes are all ones (NaN scales),
    behind block tables in random order"""

    def __init__(self, seed, lens, n_kv, d, bs, k_scale=1.0 / 16, v_scale=1.0 / 32, spare=4, max_blocks=None):
        rng = np.random.default_rng(seed)
        self.lens, self.bs, self.n_kv, self.d = list(lens), bs, n_kv, d
        self.scales = dict(k_scale=k_scale, v_scale=v_scale)
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + spare
        width = max_blocks or max(max(need), 1)
        order = rng.permutation(nb)
        tables = np.full((len(lens), width), -1, np.int32)
        pools = np.full((2, nb, n_kv, bs, 9 * d // 16), 0xFF, np.uint8)
        self.k, self.v, at = [], [], 0
        for i, n in enumerate(lens):
            blocks = order[at:at + need[i]]
            at += need[i]
            tables[i, :need[i]] = blocks
            rows = rng.standard_normal((2, n, n_kv, d)).astype(np.float32)
            t = np.arange(n)
            for p, scale, out in ((0, k_scale, self.k), (1, v_scale, self.v)):
                q = quantise(rows[p], scale)
                pools[p][blocks[t // bs] if n else [], :, t % bs] = q
                out.append(values(q, scale))
        self.host_tables, self.host_pools = tables, pools
        self.tables = torch.from_numpy(tables).cuda()
        self.kc, self.vc = torch.from_numpy(pools[0]).cuda(), torch.from_numpy(pools[1]).cuda()
        self.context = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.max_ctx = width * bs
        self.vmax = max([np.abs(v).max() for v in self.v if v.size] + [0.0])


def draw_q(seed, shape, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def attend(q, k, v, pos, scale):
    """q [rows][n_q][d], k, v [n][n_kv][d] fp64: row i sees keys up to pos[i]"""
    g = q.shape[1] // k.shape[1]
    z = np.einsum("nkd,rkgd->rkgn", k, q.reshape(len(q), k.shape[1], g, -1)) * scale
    z = np.where(np.arange(len(k)) <= np.asarray(pos)[:, None, None, None], z, -np.inf)
    p = np.exp(z - z.max(-1, keepdims=True))
    return (np.einsum("rkgn,nkd->rkgd", p, v) / p.sum(-1, keepdims=True)).reshape(q.shape)


def check(got, want, tol, dtype):
    got = got.float().cpu().numpy().astype(np.float64)
    bound = tol + (half_ulp(want, dtype) if dtype != torch.float32 else 0)
    err = np.abs(got - want)
    assert np.isfinite(got).all() and (err <= bound).all(), (err.max(), np.max(err / bound))
