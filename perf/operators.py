"""Cases that measure the serving operators around the paged K/V pool:

* ``rope``: rotary position embedding of q and k, with k and v appended to the pool
  (pa_rope_and_cache);
* ``shared``: decode of a batch in which groups of sequences share a prefix (pa_decode_shared);
* ``decode``: decode with score modifications: soft cap, linear distance bias, window, document
  mask; one or several query rows a sequence (pa_decode_scored);
* ``prefill``: chunked prefill with the same, and a prefix mask (pa_prefill_scored).

``own`` says which side ``run`` computes: the plain form (elementary torch operations in fp32) or
the library's calls.  Pools, block tables and lengths are laid out as the library documents them.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "fp8": torch.float8_e4m3fn}
KV_SCALE = 1.0 / 64          # FP8 pools: scale of K and of V
MAX_POSITION = 32768         # rows of the rotation table
ROPE_BASE = 500000.0


def _act(case):
    """dtype of q, of new rows and of the output (FP8 pools serve bf16 activations)"""
    return torch.bfloat16 if case["dtype"] == "fp8" else DTYPES[case["dtype"]]


def _bytes(case):
    return {"bf16": 2, "fp16": 2, "fp32": 4, "fp8": 1}[case["dtype"]]


# ---------------------------------------------------------------- cases

def _rope(name, tokens, n_q, n_kv, d, bs, dtype, rot, interleaved, decode):
    return {"name": name, "op": "rope", "tokens": tokens, "n_q": n_q, "n_kv": n_kv, "d": d,
            "bs": bs, "dtype": dtype, "rot": rot, "interleaved": interleaved, "decode": decode}


def _shared(name, batch, members, groups, prefix, lo, hi, n_q, n_kv, d, bs, dtype):
    return {"name": name, "op": "shared", "batch": batch, "members": members, "groups": groups,
            "prefix": prefix, "lo": lo, "hi": hi, "n_q": n_q, "n_kv": n_kv, "d": d, "bs": bs,
            "dtype": dtype}


def _decode(name, batch, nq, lo, hi, n_q, n_kv, d, bs, dtype, softcap, alibi, window, doc):
    return {"name": name, "op": "decode", "batch": batch, "nq": nq, "lo": lo, "hi": hi, "n_q": n_q,
            "n_kv": n_kv, "d": d, "bs": bs, "dtype": dtype, "softcap": softcap, "alibi": alibi,
            "window": window, "doc": doc, "prefix": 0}


def _prefill(name, reqs, chunk_lo, chunk_hi, ctx_lo, ctx_hi, n_q, n_kv, d, bs, dtype, softcap,
             alibi, window, doc, prefix):
    return {"name": name, "op": "prefill", "batch": reqs, "chunk_lo": chunk_lo,
            "chunk_hi": chunk_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "n_q": n_q, "n_kv": n_kv,
            "d": d, "bs": bs, "dtype": dtype, "softcap": softcap, "alibi": alibi,
            "window": window, "doc": doc, "prefix": prefix}


def listed():
    return [
        # one user's decode step: one token, where only latency counts
        _rope("rope-1-bf16", 1, 32, 8, 128, 16, "bf16", 128, False, True),
        # the FP8 decode batch: one token of each of 256 sequences, slots all over the pool
        _rope("rope-256-fp8", 256, 32, 8, 128, 16, "fp8", 128, False, True),
        # an odd chunk of a model that rotates adjacent pairs of half of each head
        _rope("rope-777-fp16-d64", 777, 8, 8, 64, 32, "fp16", 32, True, False),
        # a long prompt's chunk
        _rope("rope-8192-bf16", 8192, 32, 8, 128, 16, "bf16", 128, False, False),
        # four samples of one short prompt (TinyLlama's heads)
        _shared("shared-4-bf16-d64", 4, 4, 1, 512, 1, 64, 32, 4, 64, 16, "bf16"),
        # the mixed batch: a quarter of 192 sequences behind one 1024-token system prompt
        _shared("shared-192-bf16", 192, 48, 1, 1024, 16, 4096, 32, 8, 128, 32, "bf16"),
        # three prompts' samples, full multi-head attention (OPT-13B's heads)
        _shared("shared-48-fp16-mha", 48, 45, 3, 2000, 17, 1000, 40, 40, 128, 16, "fp16"),
        # a whole batch behind one long document, FP8 pool
        _shared("shared-128-fp8", 128, 128, 1, 8192, 16, 512, 32, 8, 128, 16, "fp8"),
        # a window layer with capped scores over the Llama-3-8B batch
        _decode("decode-256-bf16-cap-window", 256, 1, 512, 4096, 32, 8, 128, 16, "bf16", 50.0,
                False, 1024, 0),
        # a distance bias, full multi-head attention
        _decode("decode-32-fp16-bias", 32, 1, 100, 2047, 40, 40, 128, 16, "fp16", 0.0, True, 0, 0),
        # the mixed step's four chunks on a layer with capped scores
        _prefill("prefill-4x512-bf16-cap", 4, 512, 512, 1024, 8192, 32, 8, 128, 32, "bf16", 30.0,
                 False, 0, 0, 0),
        # ragged chunks of packed documents with a distance bias
        _prefill("prefill-5-fp16-bias-doc", 5, 33, 700, 0, 1500, 16, 4, 64, 16, "fp16", 0.0, True,
                 0, 300, 0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = [work(c) for c in listed()]
    while True:
        case = _draw(rng)
        w = work(case)
        if all(w[k] <= max(t[k] for t in top) for k in ("bytes", "flops")):
            return case


def _draw(rng):
    op = rng.choice(["rope", "shared", "decode", "prefill"])
    n_kv = rng.choice([1, 2, 4, 8, 10])
    n_q = n_kv * rng.choice([1, 2, 3, 4, 5, 8])
    d, bs = rng.choice([64, 128]), rng.choice([16, 32])
    dtype = rng.choice(["bf16", "fp16", "fp8"])
    if op == "rope":
        if rng.random() < 0.3:
            dtype = rng.choice(["fp32", "bf16"])
            d = rng.choice([32, 64, 96, 128, 256])
        rot = rng.choice([d, d, d // 2])
        case = _rope("", _log_int(rng, 1, 8192), n_q, n_kv, d, bs, dtype, rot,
                     rng.random() < 0.5, rng.random() < 0.5)
    elif op == "shared":
        batch = _log_int(rng, 1, 192)
        members = rng.randint(1, batch)
        lo = _log_int(rng, 1, 1000)
        case = _shared("", batch, members, rng.randint(1, min(4, members)),
                       _log_int(rng, 16, 8192), lo, lo + _log_int(rng, 1, 3000), n_q, n_kv, d, bs,
                       dtype)
    else:
        softcap = rng.choice([0.0, 20.0, 50.0])
        alibi = rng.random() < 0.4
        window = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        doc = rng.choice([0, 0, _log_int(rng, 20, 3000)])
        if op == "decode":
            if rng.random() < 0.2:
                dtype, d = "fp32", rng.choice([32, 64, 96, 128, 256])
            nq = 1 if dtype == "fp32" else rng.choice([1, 1, 2, 4, 7])
            lo = _log_int(rng, nq, 3000)
            case = _decode("", _log_int(rng, 1, 256), nq, lo, lo + _log_int(rng, 1, 6000), n_q,
                           n_kv, d, bs, dtype, softcap, alibi, window, doc)
        else:
            lo, ctx = _log_int(rng, 1, 500), rng.choice([0, _log_int(rng, 1, 4000)])
            case = _prefill("", rng.randint(1, 8), lo, lo + _log_int(rng, 1, 1000), ctx,
                            ctx + _log_int(rng, 1, 4000), n_q, n_kv, d, bs, dtype, softcap, alibi,
                            window, doc, rng.choice([0, _log_int(rng, 1, 2000)]))
    del case["name"]
    return case


# ---------------------------------------------------------------- sizes

def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]"""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def _lens(case):
    """context lengths before they are shuffled, and (prefill) the chunks'"""
    n = case["batch"]
    if case["op"] == "prefill":
        chunk = _spread(case["chunk_lo"], case["chunk_hi"], n)
        return chunk + _spread(case["ctx_lo"], case["ctx_hi"], n), chunk
    if case["op"] == "shared":
        # the first `members` sequences stand behind a prefix, and their lengths count from its end
        lens = _spread(case["lo"], case["hi"], n)[np.arange(n) * 7 % n if n % 7 else np.arange(n)]
        return lens + np.where(np.arange(n) < case["members"], _prefix_tokens(case), 0), None
    lens = _spread(case["lo"], case["hi"], n)
    return lens, np.full(n, case["nq"], np.int64)


def _prefix_tokens(case):
    """shared prefixes are whole blocks"""
    return max(1, case["prefix"] // case["bs"]) * case["bs"]


def _visible(case, lens, rows):
    """for every query row, in order: its sequence, its position, and its first and last visible key"""
    seq = np.repeat(np.arange(len(lens)), rows)
    start = np.cumsum(rows) - rows
    pos = np.repeat(lens - rows, rows) + np.arange(len(seq)) - np.repeat(start, rows)
    first = np.zeros(len(seq), np.int64)
    if case["window"]:
        first = np.maximum(first, pos - case["window"] + 1)
    if case["doc"]:
        first = np.maximum(first, pos // case["doc"] * case["doc"])
    last = np.maximum(pos, np.minimum(case["prefix"], lens[seq]) - 1)
    return seq, pos, first, last


def work(case):
    """Bytes: q, K/V rows that some query sees (a shared prefix once), output, tables.  Operations:
    2 for each product of q.k and of p.v."""
    act = 4 if case["dtype"] == "fp32" else 2
    kv_row = 2 * case["n_kv"] * case["d"] * _bytes(case)
    if case["op"] == "rope":
        t = case["tokens"]
        heads = case["n_q"] + case["n_kv"]
        return {"bytes": t * (act * case["d"] * (heads + case["n_kv"]) + act * case["d"] * case["n_q"]
                              + kv_row + 4 * case["rot"] + 12),
                "flops": t * heads * case["rot"] * 3}
    lens, rows = _lens(case)
    if case["op"] == "shared":
        pre = _prefix_tokens(case)
        kv = int(lens.sum()) - case["members"] * pre + case["groups"] * pre
        pairs, n_rows = int(lens.sum()), case["batch"]
    else:
        seq, _, first, last = _visible(case, lens, rows)
        lo = np.full(len(lens), 1 << 40)
        hi = np.zeros(len(lens), np.int64)
        np.minimum.at(lo, seq, first)
        np.maximum.at(hi, seq, last + 1)
        kv, n_rows = int((hi - lo).sum()), len(seq)
        pairs = int(np.maximum(0, last - first + 1).sum())
    return {"bytes": kv * kv_row + 2 * n_rows * case["n_q"] * case["d"] * act + kv // case["bs"] * 4,
            "flops": 4 * pairs * case["n_q"] * case["d"]}


# ---------------------------------------------------------------- inputs

def _pools(case, blocks, gen):
    """K and V pools with values in every slot (blocks that nobody owns hold old rows)"""
    shape = (blocks, case["n_kv"], case["bs"], case["d"])
    if case["dtype"] != "fp8":
        make = lambda: torch.randn(shape, generator=gen, device="cuda", dtype=DTYPES[case["dtype"]])  # noqa: E731
        return make(), make()
    make = lambda s: (torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16) / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    return make(shape), make((blocks, case["n_kv"], case["bs"] // 16, case["d"], 16))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng([seed, 17])
    act, bs = _act(case), case["bs"]
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)  # noqa: E731
    st = {"case": case, "scale": 1.0 / math.sqrt(case["d"]),
          "scales": {"k_scale": KV_SCALE, "v_scale": KV_SCALE} if case["dtype"] == "fp8" else {}}
    if case["op"] == "rope":
        t, d, n_q, n_kv, rot = (case[k] for k in ("tokens", "d", "n_q", "n_kv", "rot"))
        blocks = (t if case["decode"] else -(-t // bs)) + 8
        st["k_cache"], st["v_cache"] = _pools(case, blocks, gen)
        order = rng.permutation(blocks)
        at = np.arange(t)
        if case["decode"]:    # one token of each sequence, each in a block of its own
            slots, pos = order[at] * bs + rng.integers(0, bs, t), rng.integers(0, MAX_POSITION, t)
        else:                 # a chunk of one sequence
            slots, pos = order[at // bs] * bs + at % bs, at + rng.integers(0, MAX_POSITION - t + 1)
        st["slots"], st["positions"] = dev(slots, torch.int64), dev(pos, torch.int32)
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
    group = np.full(n, -1)
    shuffle = rng.permutation(n)
    if case["op"] == "shared":
        group[:case["members"]] = np.arange(case["members"]) % case["groups"]
        st["prefix"] = _prefix_tokens(case)
    lens, group = lens[shuffle], group[shuffle]
    rows = None if rows is None else rows[shuffle]
    max_blocks = -(-int(lens.max()) // bs)
    need = -(-lens // bs)
    blocks = int(need.sum() * 1.25) + 8
    order = rng.permutation(blocks)
    col = np.arange(max_blocks)[None]
    tables = np.where(col < need[:, None], order[np.minimum(np.cumsum(need)[:, None] - need[:, None]
                                                            + col, blocks - 1)], -1)
    for g in range(case.get("groups", 0)):
        who = np.flatnonzero(group == g)
        tables[who, :st["prefix"] // bs] = tables[who[0], :st["prefix"] // bs]
    st["k_cache"], st["v_cache"] = _pools(case, blocks, gen)
    st["tables"], st["lens"] = dev(tables, torch.int32), dev(lens, torch.int32)
    st["max_ctx"] = max_blocks * bs
    if case["op"] == "shared":
        st["group"] = dev(group, torch.int32)
        st["prefix_lens"] = torch.full((case["groups"],), st["prefix"], dtype=torch.int32, device="cuda")
        lead = (n,)
    else:
        _, _, first, _ = _visible({**case, "window": 0}, lens, rows)
        st["first_key"] = dev(first, torch.int32) if case["doc"] else None
        st["slopes"] = (2.0 ** (-8.0 * (torch.arange(case["n_q"], device="cuda") + 1) / case["n_q"])
                        if case["alibi"] else None)
        lead = (int(rows.sum()),)
        if case["op"] == "decode":
            lead = (n, case["nq"])
            st["first_key"] = None if st["first_key"] is None else st["first_key"].view(lead)
        else:
            st["q_start"] = dev(np.concatenate([[0], np.cumsum(rows)]), torch.int32)
            st["max_q"] = int(rows.max())
            st["prefix_lens"] = (torch.clamp(st["lens"], max=case["prefix"])
                                 if case["prefix"] else None)
    st["q"] = torch.randn((*lead, case["n_q"], case["d"]), generator=gen, device="cuda", dtype=act)
    st["out"] = torch.empty_like(st["q"])
    if own:
        # the scratch that a serving loop keeps
        from paged_kv_cache_25_gb300 import binding as pa
        size = {"shared": lambda: pa.pa_decode_shared_workspace_size(
                    n, case["n_q"], case["n_kv"], case["d"], bs, st["max_ctx"], case["groups"]),
                "decode": lambda: pa.pa_decode_scored_workspace_size(
                    n, case["nq"], case["n_q"], case["n_kv"], case["d"], bs, st["max_ctx"],
                    case["window"]),
                "prefill": lambda: 0}[case["op"]]()
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    from paged_kv_cache_25_gb300 import binding as pa
    case = st["case"]
    if case["op"] == "rope":
        pa.pa_rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["positions"], st["table"],
                             st["k_cache"], st["v_cache"], st["slots"],
                             interleaved=case["interleaved"], **st["scales"])
        return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if case["op"] == "shared":
        pa.pa_decode_shared(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"],
                            st["lens"], st["group"], st["prefix_lens"], st["scale"], case["bs"],
                            st["workspace"], **st["scales"])
        return st["out"]
    mod = pa.ScoreMod(softcap=case["softcap"], alibi_slopes=st["slopes"], window=case["window"],
                      first_key=st["first_key"], prefix_lens=st.get("prefix_lens"))
    if case["op"] == "decode":
        pa.pa_decode_scored(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"],
                            st["lens"], mod, st["scale"], case["bs"], st["workspace"],
                            **st["scales"])
    else:
        pa.pa_prefill_scored(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"],
                             st["q_start"], st["lens"], st["max_q"], mod, st["scale"], case["bs"],
                             **st["scales"])
    return st["out"]


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x = x.float()
    y, rest = x[..., :rot], x[..., rot:]
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y, rest], -1)


def _plain_rope(st):
    case = st["case"]
    cos, sin = st["table"][st["positions"].long()][:, None].chunk(2, -1)
    q = _rotate(st["q"], cos, sin, case["interleaved"]).to(st["q"].dtype)
    k, v = _rotate(st["k"], cos, sin, case["interleaved"]), st["v"].float()
    block, at = st["slots"] // case["bs"], st["slots"] % case["bs"]
    kc, vc = st["k_cache"], st["v_cache"]
    if case["dtype"] == "fp8":
        code = lambda x: (x / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        kc.view(torch.uint8)[block, :, at] = code(k)
        vc.view(torch.uint8)[block, :, at // 16, :, at % 16] = code(v)
    else:
        kc[block, :, at] = k.to(kc.dtype)
        vc[block, :, at] = v.to(vc.dtype)
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _rows(st):
    """K and V of every sequence in logical order, [B][n_kv][tokens][d], in fp32"""
    table = st["tables"].clamp(min=0).long()
    if st["case"]["dtype"] != "fp8":
        k, v = st["k_cache"][table], st["v_cache"][table]
        return k.float().transpose(1, 2).flatten(2, 3), v.float().transpose(1, 2).flatten(2, 3)
    k, v = (st[name].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * KV_SCALE
            for name in ("k_cache", "v_cache"))
    return k.transpose(1, 2).flatten(2, 3), v.permute(0, 2, 1, 3, 5, 4).flatten(2, 4)


def _attend(st, q, pos, first, last):
    """q [B][rows][n_q][d]; pos, first, last [B][rows]: a row's position and its visible keys"""
    case = st["case"]
    k, v = _rows(st)
    b, rows, n_q, d = q.shape
    n_kv = case["n_kv"]
    q = q.float().view(b, rows, n_kv, n_q // n_kv, d).permute(0, 2, 3, 1, 4).reshape(b, n_kv, -1, d)
    z = (q @ k.transpose(2, 3)).view(b, n_kv, n_q // n_kv, rows, -1) * st["scale"]
    if case.get("softcap"):
        z = case["softcap"] * torch.tanh(z / case["softcap"])
    key = torch.arange(k.shape[2], device=k.device)
    if st.get("slopes") is not None:
        far = (key - pos[..., None]).abs()[:, None, None]
        z = z - st["slopes"].float().view(n_kv, -1, 1, 1) * far
    seen = ((key >= first[..., None]) & (key <= last[..., None]))[:, None, None]
    z = z.masked_fill(~seen, float("-inf"))
    z = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e30))
    total = z.sum(-1, keepdim=True)
    o = (z.flatten(2, 3) @ v).view(b, n_kv, -1, rows, d) / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4).reshape(b, rows, n_q, d).to(st["q"].dtype)


def _plain(st):
    case = st["case"]
    if case["op"] == "rope":
        return _plain_rope(st)
    lens = st["lens"].long()
    if case["op"] == "shared":
        zero = torch.zeros_like(lens)[:, None]
        return _attend(st, st["q"][:, None], zero, zero, lens[:, None] - 1)[:, 0]
    if case["op"] == "decode":
        nq = case["nq"]
        pos = lens[:, None] - nq + torch.arange(nq, device="cuda")
        q, first = st["q"], st["first_key"]
    else:
        start = st["q_start"].long()
        at = torch.arange(st["q"].shape[0], device="cuda")
        req = torch.searchsorted(start, at, right=True) - 1
        col = at - start[req]
        pos = (lens - start[1:] + start[:-1])[:, None] + torch.arange(st["max_q"], device="cuda")
        q = st["q"].new_zeros((len(lens), st["max_q"], *st["q"].shape[1:]))
        q[req, col] = st["q"]
        first = st["first_key"]
        if first is not None:
            first = torch.zeros_like(pos).index_put((req, col), first.long())
    first = torch.zeros_like(pos) if first is None else first.long()
    if case["window"]:
        first = torch.maximum(first, pos - case["window"] + 1)
    last = pos
    if case["prefix"]:
        last = torch.maximum(pos, st["prefix_lens"].long()[:, None] - 1)
    o = _attend(st, q, pos, first, last)
    return o if case["op"] == "decode" else o[req, col]


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        half = case["rot"] // 2
        i = torch.arange(half, device="cuda")
        lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        angle = st["table"].double()[st["positions"].long()]
        turn = torch.complex(angle[:, :half], angle[:, half:])[:, None]
        out = {}
        for name in ("q", "k"):
            x = st[name].double().clone()
            w = torch.complex(x[..., lo], x[..., hi]) * turn
            x[..., lo], x[..., hi] = w.real, w.imag
            out[name] = x
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        unit = KV_SCALE if case["dtype"] == "fp8" else 1.0
        for t, slot in enumerate(st["slots"].tolist()):
            b, o = divmod(slot, case["bs"])
            kc[b, :, o] = (out["k"][t] / unit).clamp(-448, 448) if unit != 1.0 else out["k"][t]
            if unit != 1.0:
                vc[b, :, o // 16, :, o % 16] = (st["v"][t].double() / unit).clamp(-448, 448)
            else:
                vc[b, :, o] = st["v"][t].double()
        return {"q": out["q"], "k_cache": kc, "v_cache": vc}
    lens = st["lens"].tolist()
    rows = ([1] * len(lens) if case["op"] == "shared" else
            [case["nq"]] * len(lens) if case["op"] == "decode" else st["q_start"].diff().tolist())
    q = st["q"].double().reshape(-1, case["n_q"], case["d"])
    first = None if st.get("first_key") is None else st["first_key"].reshape(-1).tolist()
    per = case["n_q"] // case["n_kv"]
    outs, at = [], 0
    for s, n in enumerate(lens):
        token = torch.arange(n, device="cuda")
        block, o = st["tables"][s].long()[token // case["bs"]], token % case["bs"]
        if case["dtype"] == "fp8":                               # k and v: [n][n_kv][d]
            k = st["k_cache"].view(torch.uint8)[block, :, o].view(torch.float8_e4m3fn)
            v = st["v_cache"].view(torch.uint8)[block, :, o // 16, :, o % 16].view(torch.float8_e4m3fn)
            k, v = k.double() * KV_SCALE, v.double() * KV_SCALE
        else:
            k, v = st["k_cache"][block, :, o].double(), st["v_cache"][block, :, o].double()
        x = q[at:at + rows[s]].transpose(0, 1)                  # [n_q][rows][d]
        p = torch.arange(n - rows[s], n, device="cuda", dtype=torch.float64)
        low = torch.zeros_like(p)
        if first is not None:
            low = torch.tensor(first[at:at + rows[s]], device="cuda", dtype=torch.float64)
        if case.get("window"):
            low = torch.maximum(low, p - (case["window"] - 1))
        high = p.clamp(min=min(case["prefix"], n) - 1) if case["op"] == "prefill" else p
        dist = token.double()[None] - p[:, None]
        hide = (token.double()[None] < low[:, None]) | (token.double()[None] > high[:, None])
        got = []
        for h in range(case["n_q"]):
            z = x[h] @ k[:, h // per].T / math.sqrt(case["d"])
            if case.get("softcap"):
                z = torch.tanh(z / case["softcap"]) * case["softcap"]
            if st.get("slopes") is not None:
                z = z - float(st["slopes"][h]) * dist.abs()
            w = torch.where(hide, torch.zeros((), device="cuda", dtype=torch.float64),
                            torch.exp(z - torch.where(hide, -math.inf, z).amax(1, keepdim=True)))
            w = torch.where(hide.all(1, keepdim=True), 0.0, w)
            got.append((w @ v[:, h // per]) / w.sum(1, keepdim=True).clamp(min=1e-300))
        outs.append(torch.stack(got, 1))                         # [rows][n_q][d]
        at += rows[s]
    return torch.cat(outs).view(st["q"].shape)
