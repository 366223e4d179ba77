"""Cases that measure the 4-bit paged pool and the operators around it:

* ``rope``: rotary position embedding by several position axes (time, height, width), with k and v
  appended to the pool (pa_rope_axes_and_cache); rows of a 4-bit pool are read back as values in
  the same pass (pa_gather_cache);
* ``gather``: rows of a pool read back as values (pa_gather_cache);
* ``decode``: attention of one or several query rows a sequence over a 4-bit pool (pa_decode,
  pa_decode_verify);
* ``prefill``: chunked prefill over a 4-bit pool (pa_prefill_chunk).

A row of a 4-bit pool holds d / 2 bytes of E2M1 codes (element 2i in the low half of byte i) and d / 16
bytes of E4M3 scales, one for 16 elements; a value is code * scale * the pool's own scale.

``own`` says which side ``run`` computes: the plain form (elementary torch operations in fp32) or
the library's calls.  Pools, block tables and lengths are laid out as the library documents them.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "fp8": torch.float8_e4m3fn, "fp4": torch.uint8}
K_SCALE, V_SCALE = 1.0 / 16, 1.0 / 32   # 8- and 4-bit pools: the pool's own scales
MAX_POSITION = 32768                    # rows of the rotation table
ROPE_BASE = 500000.0


def _row_bytes(pool, d):
    return {"bf16": 2 * d, "fp16": 2 * d, "fp32": 4 * d, "fp8": d, "fp4": 9 * d // 16}[pool]


# ---------------------------------------------------------------- cases

def _rope(name, tokens, n_q, n_kv, d, bs, act, pool, rot, interleaved, axes, mixed, decode):
    return {"name": name, "op": "rope", "tokens": tokens, "n_q": n_q, "n_kv": n_kv, "d": d,
            "bs": bs, "act": act, "pool": pool, "rot": rot, "interleaved": interleaved,
            "axes": axes, "mixed": mixed, "decode": decode}


def _gather(name, tokens, n_kv, d, bs, act, pool, scattered):
    return {"name": name, "op": "gather", "tokens": tokens, "n_kv": n_kv, "d": d, "bs": bs,
            "act": act, "pool": pool, "scattered": scattered}


def _decode(name, batch, rows, lo, hi, n_q, n_kv, d, bs, act):
    return {"name": name, "op": "decode", "batch": batch, "rows": rows, "lo": lo, "hi": hi,
            "n_q": n_q, "n_kv": n_kv, "d": d, "bs": bs, "act": act, "pool": "fp4"}


def _prefill(name, reqs, chunk_lo, chunk_hi, ctx_lo, ctx_hi, n_q, n_kv, d, bs, act):
    return {"name": name, "op": "prefill", "batch": reqs, "chunk_lo": chunk_lo,
            "chunk_hi": chunk_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "n_q": n_q, "n_kv": n_kv,
            "d": d, "bs": bs, "act": act, "pool": "fp4"}


def listed():
    return [
        # one user's decode step after an image: one token, where only latency counts
        _rope("rope-1-fp4", 1, 32, 8, 128, 16, "bf16", "fp4", 128, False, 3, False, True),
        # a decode batch: one token of each of 256 sequences, slots all over the pool
        _rope("rope-256-fp4", 256, 32, 8, 128, 16, "bf16", "fp4", 128, False, 3, False, True),
        # an odd image (height and width mixed pair by pair), half of each head rotated, 16-bit pool
        _rope("rope-1023-fp16-d64", 1023, 8, 8, 64, 32, "fp16", "fp16", 32, True, 2, True, False),
        # the chunk of a long prompt with video
        _rope("rope-8192-fp4", 8192, 32, 8, 128, 16, "bf16", "fp4", 128, False, 3, True, False),
        # a short prompt's rows of an FP8 pool, handed on to another pool
        _gather("gather-300-fp8", 300, 8, 128, 16, "bf16", "fp8", True),
        # a long context's rows of a 4-bit pool
        _gather("gather-32768-fp4", 32768, 8, 128, 16, "bf16", "fp4", False),
        # one user's sequence (TinyLlama's heads)
        _decode("decode-1-fp4-d64", 1, 1, 1000, 1000, 32, 4, 64, 16, "bf16"),
        # the Llama-3-8B batch
        _decode("decode-256-fp4", 256, 1, 512, 4096, 32, 8, 128, 16, "bf16"),
        # eight users with long documents
        _decode("decode-8-fp4-long", 8, 1, 20000, 110001, 32, 8, 128, 32, "bf16"),
        # three drafted tokens checked in full multi-head attention (OPT-13B's heads)
        _decode("verify-40x4-fp4-fp16", 40, 4, 100, 2047, 40, 40, 128, 16, "fp16"),
        # the mixed step's four chunks
        _prefill("prefill-4x512-fp4", 4, 512, 512, 1024, 8192, 32, 8, 128, 32, "bf16"),
        # ragged chunks, some of whole prompts
        _prefill("prefill-5-fp4-fp16", 5, 33, 700, 0, 1500, 16, 4, 64, 16, "fp16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = [work(c) for c in listed()]
    while True:
        case = _draw(rng)
        w = work(case)
        if (all(w[k] <= max(t[k] for t in top) for k in ("bytes", "flops"))
                and case.get("batch", 1) * case.get("hi", 1) <= 1050000):
            return case


def _draw(rng):
    op = rng.choice(["rope", "gather", "decode", "prefill"])
    n_kv = rng.choice([1, 2, 4, 8, 10])
    n_q = n_kv * rng.choice([1, 2, 3, 4, 5, 8])
    d, bs = rng.choice([64, 128]), rng.choice([16, 32])
    act = rng.choice(["bf16", "fp16"])
    if op in ("rope", "gather"):
        pool = rng.choice(["fp4", "fp4", "fp8", act])
        if pool == act and rng.random() < 0.5:
            act = pool = rng.choice(["fp32", act])
            d = rng.choice([32, 64, 96, 128, 256])
        if op == "gather":
            case = _gather("", _log_int(rng, 1, 32768), n_kv, d, bs, act, pool, rng.random() < 0.5)
        else:
            case = _rope("", _log_int(rng, 1, 8192), n_q, n_kv, d, bs, act, pool,
                         rng.choice([d, d, d // 2]), rng.random() < 0.5, rng.randint(1, 4),
                         rng.random() < 0.5, rng.random() < 0.5)
    elif op == "decode":
        rows = rng.choice([1, 1, 1, 2, 4, 7, 16])
        lo = _log_int(rng, rows, 30000)
        case = _decode("", _log_int(rng, 1, 256), rows, lo, lo + _log_int(rng, 1, 60000), n_q, n_kv,
                       d, bs, act)
    else:
        lo, ctx = _log_int(rng, 1, 500), rng.choice([0, _log_int(rng, 1, 4000)])
        case = _prefill("", rng.randint(1, 8), lo, lo + _log_int(rng, 1, 1000), ctx,
                        ctx + _log_int(rng, 1, 4000), n_q, n_kv, d, bs, act)
    del case["name"]
    return case


# ---------------------------------------------------------------- sizes

def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]"""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def _lens(case):
    """context lengths before they are shuffled, and the query rows of each sequence"""
    n = case["batch"]
    if case["op"] == "prefill":
        chunk = _spread(case["chunk_lo"], case["chunk_hi"], n)
        return chunk + _spread(case["ctx_lo"], case["ctx_hi"], n), chunk
    return _spread(case["lo"], case["hi"], n), np.full(n, case["rows"], np.int64)


def _axis_of_pair(case):
    """Position axis of every rotated pair: in turn (mixed), or one run of pairs after another"""
    i = np.arange(case["rot"] // 2)
    axes = case["axes"]
    return (i % axes if case["mixed"] else i * axes // len(i)).astype(np.uint8)


def work(case):
    """Bytes: inputs, K/V rows and tables once, outputs once.  Operations: 2 for each product of q.k and
    of p.v, 3 for a rotated element, 2 for a value read back."""
    act = 4 if case["act"] == "fp32" else 2
    kv_row = 2 * case["n_kv"] * _row_bytes(case["pool"], case["d"])
    back = 2 * case["n_kv"] * case["d"]
    if case["op"] == "gather":
        t = case["tokens"]
        return {"bytes": t * (kv_row + back * act + 8), "flops": 2 * t * back}
    if case["op"] == "rope":
        t = case["tokens"]
        heads = case["n_q"] + case["n_kv"]
        read = t * (act * case["d"] * (heads + case["n_kv"]) + 4 * case["axes"] + 8 + 4 * case["rot"])
        write = t * (act * case["d"] * case["n_q"] + kv_row)
        if case["pool"] == "fp4":            # the rows as values
            write += t * back * act
        return {"bytes": read + write, "flops": 3 * t * heads * case["rot"]}
    lens, rows = _lens(case)
    # row i of a sequence sees all keys up to its own
    pairs = int((rows * lens - rows * (rows - 1) // 2).sum())
    kv, n_rows = int(lens.sum()), int(rows.sum())
    return {"bytes": kv * kv_row + 2 * n_rows * case["n_q"] * case["d"] * act + kv // case["bs"] * 4,
            "flops": 4 * pairs * case["n_q"] * case["d"]}


# ---------------------------------------------------------------- the 4-bit format

def _quantise(x, scale):
    """rows [..., d] (fp32) as bytes [..., 9 d / 16]; one rounding of every step to fp32"""
    x = x.unflatten(-1, (-1, 16))
    s = x.abs().amax(-1, keepdim=True) / (6 * scale)
    s = s.clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
    y = x / (s.float() * scale)
    m = y.abs()
    # to nearest even among 0, 0.5, 1, 1.5, 2, 3, 4, 6
    code = ((m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5)
            + (m > 5)) | (torch.signbit(y).byte() << 3)
    code = (code[..., 0::2] | code[..., 1::2] << 4).flatten(-2)
    return torch.cat([code, s.squeeze(-1).view(torch.uint8)], -1)


def _dequantise(rows, scale):
    """bytes [..., 9 d / 16] as values [..., d] (fp32)"""
    d = rows.shape[-1] * 16 // 9
    code = torch.stack([rows[..., :d // 2] & 15, rows[..., :d // 2] >> 4], -1).flatten(-2)
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=rows.device)[(code & 7).int()]
    value = torch.where(code >= 8, -value, value)
    s = rows[..., d // 2:].contiguous().view(torch.float8_e4m3fn).float()
    return ((value.unflatten(-1, (-1, 16)) * s[..., None]) * scale).flatten(-2)


# ---------------------------------------------------------------- inputs

def _pools(case, blocks, gen):
    """K and V pools with values in every slot (blocks that nobody owns hold old rows)"""
    shape = (blocks, case["n_kv"], case["bs"], case["d"])
    make = lambda s, t: torch.randn(s, generator=gen, device="cuda", dtype=t)  # noqa: E731
    if case["pool"] == "fp4":
        pools = []
        for scale in (K_SCALE, V_SCALE):
            pool = torch.empty((*shape[:3], 9 * case["d"] // 16), dtype=torch.uint8, device="cuda")
            for at in range(0, blocks, 4096):
                part = pool[at:at + 4096]
                part.copy_(_quantise(make((part.shape[0], *shape[1:]), torch.float32), scale))
            pools.append(pool)
        return pools
    if case["pool"] == "fp8":
        v_shape = (blocks, case["n_kv"], case["bs"] // 16, case["d"], 16)
        return [(make(s, torch.bfloat16) / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
                for s, scale in ((shape, K_SCALE), (v_shape, V_SCALE))]
    return [make(shape, DTYPES[case["pool"]]) for _ in range(2)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng([seed, 23])
    act, bs, d, n_kv = DTYPES[case["act"]], case["bs"], case["d"], case["n_kv"]
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)  # noqa: E731
    st = {"case": case, "scale": 1.0 / math.sqrt(d),
          "scales": ({"k_scale": K_SCALE, "v_scale": V_SCALE} if case["pool"] in ("fp4", "fp8")
                     else {})}
    if case["op"] in ("rope", "gather"):
        t = case["tokens"]
        apart = case.get("decode", case.get("scattered"))
        blocks = (t if apart else -(-t // bs)) + 8
        st["k_cache"], st["v_cache"] = _pools(case, blocks, gen)
        order = rng.permutation(blocks)
        at = np.arange(t)
        if apart:             # every token in a block of its own
            slots = order[at] * bs + rng.integers(0, bs, t)
        else:                 # consecutive tokens of one sequence
            slots = order[at // bs] * bs + at % bs
        st["slots"] = dev(slots, torch.int64)
        st["k_back"] = torch.empty((t, n_kv, d), device="cuda", dtype=act)
        st["v_back"] = torch.empty((t, n_kv, d), device="cuda", dtype=act)
        if case["op"] == "gather":
            return st
        n_q, rot, axes = case["n_q"], case["rot"], case["axes"]
        if case["decode"]:    # text after an image: the axes have gone on by different amounts
            pos = rng.integers(0, MAX_POSITION, (axes, t))
        else:                 # frames of an image grid: time, height, width and further axes
            grid = [at // 1024, at // 32 % 32, at % 32, at % 7][:axes]
            pos = np.stack(grid) + rng.integers(0, MAX_POSITION - 40)
        st["positions"] = dev(pos, torch.int32)
        st["axis_of_pair"] = _axis_of_pair(case)
        # one projection's output holds q, k and v side by side
        qkv = torch.randn((t, (n_q + 2 * n_kv) * d), generator=gen, device="cuda", dtype=act)
        st["q"] = qkv[:, :n_q * d].unflatten(1, (n_q, d))
        st["k"] = qkv[:, n_q * d:(n_q + n_kv) * d].unflatten(1, (n_kv, d))
        st["v"] = qkv[:, (n_q + n_kv) * d:].unflatten(1, (n_kv, d))
        angle = torch.arange(MAX_POSITION, device="cuda", dtype=torch.float64)[:, None] * (
            ROPE_BASE ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot))
        st["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        st["q_out"] = torch.empty((t, n_q, d), device="cuda", dtype=act)
        return st
    lens, rows = _lens(case)
    n = len(lens)
    shuffle = rng.permutation(n)
    lens, rows = lens[shuffle], rows[shuffle]
    max_blocks = -(-int(lens.max()) // bs)
    need = -(-lens // bs)
    blocks = int(need.sum() * 1.25) + 8
    order = rng.permutation(blocks)
    col = np.arange(max_blocks)[None]
    tables = np.where(col < need[:, None], order[np.minimum(np.cumsum(need)[:, None] - need[:, None]
                                                            + col, blocks - 1)], -1)
    st["k_cache"], st["v_cache"] = _pools(case, blocks, gen)
    st["tables"], st["lens"] = dev(tables, torch.int32), dev(lens, torch.int32)
    if case["op"] == "prefill":
        lead = (int(rows.sum()),)
        st["q_start"] = dev(np.concatenate([[0], np.cumsum(rows)]), torch.int32)
        st["max_q"] = int(rows.max())
    else:
        lead = (n,) if case["rows"] == 1 else (n, case["rows"])
    st["q"] = torch.randn((*lead, case["n_q"], d), generator=gen, device="cuda", dtype=act)
    st["out"] = torch.empty_like(st["q"])
    st["workspace"] = None
    if own and case["op"] == "decode":
        # the scratch that a serving loop keeps
        from paged_kv_cache_25_gb300 import binding as pa
        size = pa.pa_decode_verify_workspace_size(n, case["rows"], case["n_q"], n_kv, d, bs,
                                                  max_blocks * bs)
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    from paged_kv_cache_25_gb300 import binding as pa
    case = st["case"]
    if case["op"] == "gather":
        pa.pa_gather_cache(st["k_back"], st["v_back"], st["k_cache"], st["v_cache"], st["slots"],
                           **st["scales"])
        return {"k": st["k_back"], "v": st["v_back"]}
    if case["op"] == "rope":
        pa.pa_rope_axes_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["positions"],
                                  st["axis_of_pair"], st["table"], st["k_cache"], st["v_cache"],
                                  st["slots"], interleaved=case["interleaved"], **st["scales"])
        if case["pool"] != "fp4":
            return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
        pa.pa_gather_cache(st["k_back"], st["v_back"], st["k_cache"], st["v_cache"], st["slots"],
                           **st["scales"])
        return {"q": st["q_out"], "k": st["k_back"], "v": st["v_back"]}
    if case["op"] == "prefill":
        pa.pa_prefill_chunk(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"],
                            st["q_start"], st["lens"], st["max_q"], st["scale"], case["bs"],
                            **st["scales"])
    else:
        call = pa.pa_decode if case["rows"] == 1 else pa.pa_decode_verify
        call(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"],
             st["scale"], case["bs"], st["workspace"], **st["scales"])
    return st["out"]


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x = x.float()
    y, rest = x[..., :rot], x[..., rot:]
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y, rest], -1)


def _read_back(st):
    """the rows of the slots as values"""
    case, act = st["case"], st["k_back"].dtype
    kc, vc = st["k_cache"], st["v_cache"]
    block, at = st["slots"] // case["bs"], st["slots"] % case["bs"]
    if case["pool"] == "fp4":
        return {"k": _dequantise(kc[block, :, at], K_SCALE).to(act),
                "v": _dequantise(vc[block, :, at], V_SCALE).to(act)}
    if case["pool"] == "fp8":
        k = kc.view(torch.uint8)[block, :, at].view(torch.float8_e4m3fn).float()
        v = vc.view(torch.uint8)[block, :, at // 16, :, at % 16].view(torch.float8_e4m3fn).float()
        return {"k": (k * K_SCALE).to(act), "v": (v * V_SCALE).to(act)}
    return {"k": kc[block, :, at], "v": vc[block, :, at]}


def _plain_rope(st):
    case = st["case"]
    half = case["rot"] // 2
    # every pair's row of the table is the position of its axis
    axis = torch.from_numpy(st["axis_of_pair"].astype(np.int64)).cuda()
    pos = st["positions"].long()[axis].T                      # [tokens][pairs]
    pair = torch.arange(half, device="cuda")
    cos = st["table"][pos, pair][:, None]
    sin = st["table"][pos, half + pair][:, None]
    q = _rotate(st["q"], cos, sin, case["interleaved"]).to(st["q"].dtype)
    k, v = _rotate(st["k"], cos, sin, case["interleaved"]), st["v"].float()
    block, at = st["slots"] // case["bs"], st["slots"] % case["bs"]
    kc, vc = st["k_cache"], st["v_cache"]
    if case["pool"] == "fp4":
        kc[block, :, at] = _quantise(k, K_SCALE)
        vc[block, :, at] = _quantise(v, V_SCALE)
        return {"q": q, **_read_back(st)}
    if case["pool"] == "fp8":
        code = lambda x, s: (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        kc.view(torch.uint8)[block, :, at] = code(k, K_SCALE)
        vc.view(torch.uint8)[block, :, at // 16, :, at % 16] = code(v, V_SCALE)
    else:
        kc[block, :, at] = k.to(kc.dtype)
        vc[block, :, at] = v.to(vc.dtype)
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _attend(st, q, pos):
    """q [B][rows][n_q][d]; pos [B][rows]: a row's position, its last visible key"""
    n_kv = st["case"]["n_kv"]
    table = st["tables"].clamp(min=0).long()
    k, v = (_dequantise(st[name][table], s).transpose(1, 2).flatten(2, 3)
            for name, s in (("k_cache", K_SCALE), ("v_cache", V_SCALE)))
    b, rows, n_q, d = q.shape
    q = q.float().view(b, rows, n_kv, n_q // n_kv, d).permute(0, 2, 3, 1, 4).reshape(b, n_kv, -1, d)
    z = (q @ k.transpose(2, 3)).view(b, n_kv, n_q // n_kv, rows, -1) * st["scale"]
    key = torch.arange(k.shape[2], device=k.device)
    z = z.masked_fill((key > pos[..., None])[:, None, None], float("-inf"))
    z = torch.exp(z - z.amax(-1, keepdim=True))
    o = (z.flatten(2, 3) @ v).view(b, n_kv, -1, rows, d) / z.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(b, rows, n_q, d).to(st["q"].dtype)


def _plain(st):
    case = st["case"]
    if case["op"] == "rope":
        return _plain_rope(st)
    if case["op"] == "gather":
        return _read_back(st)
    lens = st["lens"].long()
    if case["op"] == "decode":
        rows = case["rows"]
        pos = lens[:, None] - rows + torch.arange(rows, device="cuda")
        return _attend(st, st["q"].view(len(lens), rows, case["n_q"], case["d"]), pos).view(st["q"].shape)
    start = st["q_start"].long()
    at = torch.arange(st["q"].shape[0], device="cuda")
    req = torch.searchsorted(start, at, right=True) - 1
    col = at - start[req]
    pos = (lens - start[1:] + start[:-1])[:, None] + torch.arange(st["max_q"], device="cuda")
    q = st["q"].new_zeros((len(lens), st["max_q"], *st["q"].shape[1:]))
    q[req, col] = st["q"]
    return _attend(st, q, pos)[req, col]


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_rows(pool, scale):
    """values of 4-bit rows [..., 9 d / 16] by the format's definition"""
    d = pool.shape[-1] // 9 * 16
    byte = pool.long()
    nib = torch.empty((*pool.shape[:-1], d), dtype=torch.int64, device=pool.device)
    nib[..., 0::2], nib[..., 1::2] = byte[..., :d // 2] % 16, byte[..., :d // 2] // 16
    e, m = nib % 8 // 2, (nib % 2).double()
    mag = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m))
    s = byte[..., d // 2:]
    se, sm = s % 128 // 8, (s % 8).double()
    sv = torch.where(se == 0, sm * 2.0 ** -9, torch.exp2(se.double() - 7) * (1 + sm / 8))
    return torch.where(nib > 7, -mag, mag) * sv.repeat_interleave(16, -1) * scale


def _exact_quantised(x, scale):
    """the values that the 4-bit format stores for rows [..., d], every step in 64 bits"""
    g = x.double().unflatten(-1, (-1, 16))
    a = (g.abs().amax(-1, keepdim=True) / (6 * scale)).clamp(2.0 ** -9, 448)
    step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6) - 3)
    s = (a / step).round() * step                         # (round: to even)
    y = g / (s * scale)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1))) - 1)
    y = ((y / step).round() * step).clamp(-6, 6)
    return (y * s * scale).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    bs = case["bs"]
    if case["op"] in ("rope", "gather"):
        slots = st["slots"].tolist()
        block = torch.tensor([x // bs for x in slots], device="cuda")
        at = torch.tensor([x % bs for x in slots], device="cuda")
    if case["op"] == "gather":
        kc, vc = st["k_cache"], st["v_cache"]
        if case["pool"] == "fp4":
            return {"k": _exact_rows(kc[block, :, at], K_SCALE),
                    "v": _exact_rows(vc[block, :, at], V_SCALE)}
        if case["pool"] == "fp8":
            return {"k": kc.double()[block, :, at] * K_SCALE,
                    "v": vc.double()[block, :, at // 16, :, at % 16] * V_SCALE}
        return {"k": kc.double()[block, :, at], "v": vc.double()[block, :, at]}
    if case["op"] == "rope":
        half = case["rot"] // 2
        i = torch.arange(half, device="cuda")
        lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        turn = torch.empty((case["tokens"], 1, half), dtype=torch.complex128, device="cuda")
        for p, a in enumerate(st["axis_of_pair"].tolist()):
            angle = st["table"].double()[st["positions"][a].long()]
            turn[:, 0, p] = torch.complex(angle[:, p], angle[:, half + p])
        out = {}
        for name in ("q", "k"):
            x = st[name].double().clone()
            w = torch.complex(x[..., lo], x[..., hi]) * turn
            x[..., lo], x[..., hi] = w.real, w.imag
            out[name] = x
        if case["pool"] == "fp4":
            return {"q": out["q"], "k": _exact_quantised(out["k"], K_SCALE),
                    "v": _exact_quantised(st["v"], V_SCALE)}
        kc, vc, v = st["k_cache"].double(), st["v_cache"].double(), st["v"].double()
        if case["pool"] == "fp8":
            kc[block, :, at] = (out["k"] / K_SCALE).clamp(-448, 448)
            vc[block, :, at // 16, :, at % 16] = (v / V_SCALE).clamp(-448, 448)
        else:
            kc[block, :, at], vc[block, :, at] = out["k"], v
        return {"q": out["q"], "k_cache": kc, "v_cache": vc}
    lens = st["lens"].tolist()
    rows = [case["rows"]] * len(lens) if case["op"] == "decode" else st["q_start"].diff().tolist()
    q = st["q"].double().reshape(-1, case["n_q"], case["d"])
    per = case["n_q"] // case["n_kv"]
    outs, begin = [], 0
    for s, n in enumerate(lens):
        token = torch.arange(n, device="cuda")
        where, o = st["tables"][s].long()[token // bs], token % bs
        x = q[begin:begin + rows[s]].transpose(0, 1)             # [n_q][rows][d]
        last = torch.arange(n - rows[s], n, device="cuda")
        got = []
        for h in range(case["n_kv"]):
            k = _exact_rows(st["k_cache"][where, h, o], K_SCALE)
            v = _exact_rows(st["v_cache"][where, h, o], V_SCALE)
            z = x[h * per:(h + 1) * per] @ k.T / math.sqrt(case["d"])
            z = torch.where(token[None] > last[:, None], -math.inf, z)
            got.append(torch.softmax(z, -1) @ v)
        outs.append(torch.cat(got).transpose(0, 1))              # [rows][n_q][d]
        begin += rows[s]
    return torch.cat(outs).view(st["q"].shape)
