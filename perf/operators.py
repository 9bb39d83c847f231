"""The 4-bit operators of the library as measurable passes: the NVFP4 KV cache
(its writer, its reader and the attention over it) and the matrix-vector
product with NVFP4 weights.

Every case is one call of one operator.  ``own`` selects what ``run`` does:
False computes the operator's definition with elementary torch operations,
True calls the library.  Both start from the same inputs (``prepare``).

NVFP4 throughout: e2m1 codes, two per byte (element 2j in the low nibble), 16
consecutive elements share an e4m3 scale factor, one fp32 scale per tensor.
In the KV cache the scale factors of four neighbouring slots lie side by side:
[capacity / 4, Hkv, hd / 16, 4].
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = float(np.float32(1e-6))
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one flow step of a small action decoder: ten new tokens into a 1024-slot cache
        {"name": "write 10 tokens 8/1x256", "op": "write", "dt": "bf16", "m": 10, "Hq": 8, "Hkv": 1, "hd": 256,
         "norm": False, "cap": 1024, "slots": False},
        # a large prefill batch scattered over a 131072-slot pool
        {"name": "write 4096 tokens 32/8x128", "op": "write", "dt": "bf16", "m": 4096, "Hq": 32, "Hkv": 8, "hd": 128,
         "norm": True, "cap": 131072, "slots": True},
        # a short prefix handed back to a 16-bit consumer
        {"name": "read 181 slots 8x128", "op": "read", "dt": "f16", "n": 181, "Hkv": 8, "hd": 128, "cap": 256},
        # a long prefix handed back
        {"name": "read 16384 slots 8x128", "op": "read", "dt": "bf16", "n": 16384, "Hkv": 8, "hd": 128, "cap": 131072},
        # the action decoder's ten tokens, all seeing the prefix and one another
        {"name": "attend 10 over 978 8/1x256", "op": "attn", "dt": "bf16", "seqs": 1, "q": 10, "Hq": 8, "Hkv": 1,
         "hd": 256, "kv": 978, "causal": False, "window": 0, "page": 0, "ragged": False},
        # one token of one user at the end of a long context
        {"name": "attend 1 over 131072 32/8x128", "op": "attn", "dt": "bf16", "seqs": 1, "q": 1, "Hq": 32, "Hkv": 8,
         "hd": 128, "kv": 131072, "causal": True, "window": 0, "page": 0, "ragged": False},
        # a serving batch, one token each, paged, every length from a few slots to the longest
        {"name": "attend 64 paged seqs 16/8x128", "op": "attn", "dt": "f16", "seqs": 64, "q": 1, "Hq": 16, "Hkv": 8,
         "hd": 128, "kv": 8000, "causal": True, "window": 0, "page": 64, "ragged": True},
        # a chunk of a text prefill, causal behind what the cache already holds
        {"name": "attend 512 over 4608 16/8x128", "op": "attn", "dt": "bf16", "seqs": 1, "q": 512, "Hq": 16, "Hkv": 8,
         "hd": 128, "kv": 4608, "causal": True, "window": 0, "page": 0, "ragged": False},
        # the action decoder's QKV projection for one token
        {"name": "matvec 1x1024->2560", "op": "matvec", "dt": "bf16", "m": 1, "n": 2560, "k": 1024, "x": "16",
         "bias": False, "layout": "rows"},
        # a wide gate/up projection of one decoded token
        {"name": "matvec 1x4096->32768", "op": "matvec", "dt": "f16", "m": 1, "n": 32768, "k": 4096, "x": "16",
         "bias": False, "layout": "rows"},
        # the denoise step's gate/up projection on block-scaled FP8 rows
        {"name": "matvec 41x2048->16384 e4m3", "op": "matvec", "dt": "bf16", "m": 41, "n": 16384, "k": 2048,
         "x": "e4m3_block", "bias": False, "layout": "swizzled"},
        # the action decoder's down projection on the activation's NVFP4 rows, with a bias
        {"name": "matvec 10x4096->1024 nvfp4", "op": "matvec", "dt": "bf16", "m": 10, "n": 1024, "k": 4096, "x": "nvfp4",
         "bias": True, "layout": "rows"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["write", "read", "attn", "attn", "matvec", "matvec"])
    dt = rng.choice(["bf16", "f16"])
    hd = rng.choice([64, 80, 96, 128, 128, 192, 256])
    hkv = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    if op == "write":
        m = _log(rng, 1, 4096)
        return {"op": op, "dt": dt, "m": m, "Hq": hkv * group, "Hkv": hkv, "hd": hd, "norm": rng.random() < 0.7,
                "cap": m + _log(rng, 16, 65536), "slots": rng.random() < 0.5}
    if op == "read":
        n = _log(rng, 1, 16384)
        return {"op": op, "dt": dt, "n": n, "Hkv": hkv, "hd": hd, "cap": n + _log(rng, 16, 65536)}
    if op == "attn":
        kind = rng.choice(["batch", "batch", "chunk", "long"])
        c = {"op": op, "dt": dt, "seqs": 1, "q": 1, "Hq": hkv * group, "Hkv": hkv, "hd": hd, "kv": 0,
             "causal": rng.random() < 0.7, "window": rng.choice([0, 0, 512]), "page": rng.choice([0, 16, 64, 20]),
             "ragged": rng.random() < 0.7}
        if kind == "batch":
            c.update(seqs=_log(rng, 2, 64), q=rng.choice([1, 1, 1, 3, 8]), kv=_log(rng, 16, 8000),
                     page=rng.choice([16, 64, 20]))
        elif kind == "chunk":
            c.update(q=_log(rng, 2, 512), kv=_log(rng, 600, 4608))
        else:
            c.update(q=_log(rng, 1, 41), kv=_log(rng, 64, 131072))
        return c
    return {"op": op, "dt": dt, "m": _log(rng, 1, 64), "n": _log(rng, 100, 32768), "k": 16 * _log(rng, 4, 512),
            "x": rng.choice(["16", "16", "e4m3", "e4m3_block", "nvfp4"]), "bias": rng.random() < 0.3,
            "layout": rng.choice(["rows", "swizzled"])}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    """A case of the listed ranges, no dearer than the dearest listed case of its operator."""
    while True:
        case = _drawn(rng)
        if _cost(case) <= max(_cost(c) for c in listed() if c["op"] == case["op"]):
            return case


def _pairs(case):
    """(query, key) pairs of an attention case with every sequence at its longest."""
    q, kv = case["q"], case["kv"]
    seen = np.minimum(kv, kv - q + 1 + np.arange(q)) if case["causal"] else np.full(q, kv)
    seen = np.maximum(seen, 0)
    if case["window"]:
        seen = np.minimum(seen, case["window"])
    return int(seen.sum())


def work(case):
    op = case["op"]
    if op == "write":
        m, hq, hkv, hd = case["m"], case["Hq"], case["Hkv"], case["hd"]
        tables = 4 * hd + 4 + (4 if case["slots"] else 0)
        return {"bytes": m * ((hq + 2 * hkv) * hd * 2 + hq * hd * 2 + 2 * hkv * (hd // 2 + hd // 16) + tables),
                "flops": m * (hq + 2 * hkv) * hd * 6}
    if op == "read":
        n, hkv, hd = case["n"], case["Hkv"], case["hd"]
        return {"bytes": n * (2 * hkv * (hd // 2 + hd // 16) + 2 * hkv * hd * 2 + 4), "flops": n * hkv * hd * 4}
    if op == "attn":
        b, q, hq, hkv, hd = case["seqs"], case["q"], case["Hq"], case["Hkv"], case["hd"]
        half = 0.5 if case["ragged"] and b > 1 else 1.0  # ragged batches: lengths spread evenly up to the longest
        reach = min(case["kv"], case["window"] + q) if case["window"] else case["kv"]
        return {"bytes": b * (half * reach * 2 * hkv * (hd // 2 + hd // 16) + 2 * q * hq * hd * 2),
                "flops": b * half * 4.0 * hq * hd * _pairs(case)}
    m, n, k = case["m"], case["n"], case["k"]
    x_bits = {"16": 16, "e4m3": 8, "e4m3_block": 8.25, "nvfp4": 4.5}[case["x"]]
    return {"bytes": n * k * 4.5 / 8 + m * k * x_bits / 8 + m * n * 2 + (2 * n if case["bias"] else 0),
            "flops": 2.0 * m * n * k}


# --------------------------------------------------------- NVFP4 in torch --
def _e2m1_code(a, negative):
    """Nearest e2m1 code of magnitudes a (ties to the even code), with the sign in bit 3."""
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c + 8 * negative.to(torch.uint8)


def _quantise(y, gs):
    """fp32 y [..., 16 j] -> (codes [..., 8 j] uint8, scale factors [..., j] uint8), scaled by rounded reciprocals."""
    blocks = y.unflatten(-1, (-1, 16))
    rden = 1.0 / (6.0 * gs)
    sf = (blocks.abs().amax(-1) * rden).clamp(max=448.0).to(torch.float8_e4m3fn)
    eff = sf.float() * gs
    reff = torch.where(eff > 0, 1.0 / eff, torch.zeros_like(eff))
    scaled = blocks * reff.unsqueeze(-1)
    codes = _e2m1_code(scaled.abs(), torch.signbit(scaled)).flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), sf.view(torch.uint8)


def _e2m1_table(dtype):
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(v + [-x for x in v], dtype=dtype, device=DEV)


def _decode(codes, sf, gs, dtype=torch.float32):
    """codes [..., 8 j], sf [..., j] -> code * sf * gs [..., 16 j]."""
    pair = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = _e2m1_table(dtype)[pair.int()].unflatten(-1, (-1, 16))
    return (v * sf.view(torch.float8_e4m3fn).to(dtype).unsqueeze(-1) * gs.to(dtype)).flatten(-2)


def _sf_pack(sf):
    """[capacity, Hkv, hd/16] (capacity a multiple of 4) -> [capacity/4, Hkv, hd/16, 4]."""
    return sf.unflatten(0, (-1, 4)).permute(0, 2, 3, 1).contiguous()


def _sf_rows(sf4, slots):
    """The scale factors [..., Hkv, hd/16] of slots [...]."""
    return sf4[slots // 4, :, :, slots % 4]


def _swizzle(sf):
    """[N, K/16] -> the 128x4-swizzled bytes."""
    n, c = sf.shape
    pad = torch.zeros((-(-n // 128) * 128, -(-c // 4) * 4), dtype=torch.uint8, device=sf.device)
    pad[:n, :c] = sf
    return pad.view(-1, 4, 32, pad.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().flatten()


def _unswizzle(flat, n, c):
    t = flat.view(-(-n // 128), -(-c // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
    return t.reshape(-(-n // 128) * 128, -1)[:n, :c]


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


def _kv_scales(g):
    """Scales of a calibrated cache: largest magnitudes between 4.5 and 5.5 of N(0, 1) data."""
    return (4.5 + torch.rand(2, generator=g, device=DEV)) / 2688


def _cache(cap, hkv, hd, gs, g, used):
    """A quantised N(0, 1) tensor of `used` slots in a cache of cap slots; the other slots hold arbitrary bytes,
    scale factors that are NaN among them."""
    cap4 = -(-cap // 4) * 4
    codes = torch.randint(0, 256, (cap, hkv, hd // 2), generator=g, device=DEV, dtype=torch.uint8)
    sf = torch.full((cap4, hkv, hd // 16), 0x7F, device=DEV, dtype=torch.uint8)
    codes[:used], sf[:used] = _quantise(_randn((used, hkv, hd), g), gs)
    return codes, _sf_pack(sf)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    dt = DT.get(case["dt"])
    op = case["op"]
    if op in ("write", "read"):
        hkv, hd, cap = case["Hkv"], case["hd"], case["cap"]
        s["kv_scales"] = _kv_scales(g)
    if op == "write":
        m, hq = case["m"], case["Hq"]
        s["qkv"] = _randn((m, (hq + 2 * hkv) * hd), g).to(dt)
        s["qw"], s["kw"] = [(1 + 0.1 * _randn((hd,), g)).to(dt) if case["norm"] else None for _ in range(2)]
        ang = torch.outer(torch.arange(cap, dtype=torch.float64, device=DEV),
                          1e4 ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64, device=DEV) / hd))
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        where = torch.randperm(cap, generator=g, device=DEV)[:m].int()
        if case["slots"]:
            s["pos"], s["slots"] = torch.randint(0, cap, (m,), generator=g, device=DEV, dtype=torch.int32), where
        else:
            s["pos"], s["slots"] = where, None
        s["where"] = where
        s["k"] = torch.zeros((cap, hkv, hd // 2), dtype=torch.uint8, device=DEV)
        s["v"] = torch.zeros_like(s["k"])
        s["ksf"] = torch.zeros((-(-cap // 4), hkv, hd // 16, 4), dtype=torch.uint8, device=DEV)
        s["vsf"] = torch.zeros_like(s["ksf"])
        s["q_out"] = torch.empty((m, hq, hd), dtype=dt, device=DEV)
        s["k_out"], s["v_out"] = [torch.empty((m, hkv, hd), dtype=dt, device=DEV) for _ in range(2)]
    elif op == "read":
        n = case["n"]
        s["k"], s["ksf"] = _cache(cap, hkv, hd, s["kv_scales"][0], g, cap)
        s["v"], s["vsf"] = _cache(cap, hkv, hd, s["kv_scales"][1], g, cap)
        s["where"] = torch.randperm(cap, generator=g, device=DEV)[:n].int()
        s["k_out"], s["v_out"] = [torch.empty((n, hkv, hd), dtype=dt, device=DEV) for _ in range(2)]
    elif op == "attn":
        _prepare_attn(s, case, dt, g, seed)
    else:
        _prepare_matvec(s, case, dt, g)
    return s


def _prepare_attn(s, case, dt, g, seed):
    rng = np.random.RandomState(seed % (1 << 31))
    b, q, kv, page = case["seqs"], case["q"], case["kv"], case["page"]
    hq, hkv, hd = case["Hq"], case["Hkv"], case["hd"]
    s["kv_scales"] = _kv_scales(g)
    tokens = np.full(b, q)
    lens = np.full(b, kv)
    if case["ragged"]:
        if b > 1:
            # token counts and lengths spread evenly, the largest among them
            tokens = 1 + (q - 1) * (rng.permutation(b) + 1) // b
            lens = 1 + (kv - 1) * (rng.permutation(b) + 1) // b
        else:
            lens = rng.randint(max(1, kv // 2), kv + 1, b)
    indptr = np.concatenate(([0], np.cumsum(tokens)))
    m = int(indptr[-1])
    seq = np.repeat(np.arange(b), tokens)
    at = np.arange(m) - indptr[seq]
    seen = lens[seq] - (tokens[seq] - 1 - at) if case["causal"] else lens[seq]
    s["kv_len"] = torch.from_numpy(np.maximum(seen, 0).astype(np.int32)).to(DEV)
    s["indptr"] = torch.from_numpy(indptr.astype(np.int32)).to(DEV)
    s["max_q"] = int(tokens.max())
    s["tokens_of"] = torch.from_numpy(np.where(np.arange(s["max_q"])[None] < tokens[:, None],
                                               indptr[:-1, None] + np.arange(s["max_q"])[None], -1)).to(DEV)
    if page:
        need = -(-lens // page)
        wide = -(-kv // page)
        pool = int(need.sum()) + 3
        order = rng.permutation(pool)
        table = np.full((b, wide), -1, dtype=np.int32)
        first = np.concatenate(([0], np.cumsum(need)))
        used = np.arange(wide)[None] < need[:, None]
        table[used] = order[(first[:-1, None] + np.arange(wide)[None])[used]]
        s["table"] = torch.from_numpy(table).to(DEV)
        cap = pool * page
        written = cap
    else:
        s["table"] = None
        cap = kv + 37
        written = int(lens.max())
    s["k"], s["ksf"] = _cache(cap, hkv, hd, s["kv_scales"][0], g, written)
    s["v"], s["vsf"] = _cache(cap, hkv, hd, s["kv_scales"][1], g, written)
    # queries with a gain: scores spread enough for the softmax to favour some keys
    s["q"] = (2.0 * _randn((m, hq, hd), g)).to(dt)
    s["out"] = torch.empty((m, hq, hd), dtype=dt, device=DEV)
    s["scale"] = float(np.float32(1.0 / math.sqrt(hd)))
    if own:  # a serving program keeps the attention's workspace from step to step
        import memory_bound_non_b200 as frt
        s["workspace"] = frt.attn_nvfp4_workspace(s["q"], hkv, kv, n_seqs=b, max_q_len=s["max_q"])


def _prepare_matvec(s, case, dt, g):
    m, n, k = case["m"], case["n"], case["k"]
    w = _randn((n, k), g) / math.sqrt(k)
    s["w_scale"] = (w.abs().amax() / 2688).reshape(1)
    s["w"], sf = _quantise(w, s["w_scale"])
    s["wsf"] = _swizzle(sf) if case["layout"] == "swizzled" else sf
    del w
    x = _randn((m, k), g)
    loud = torch.randperm(k, generator=g, device=DEV)[:max(1, k // 100)]
    x[:, loud] *= 50.0  # a hundredth of the channels far above the rest
    s["xsf"] = s["x_scales"] = None
    if case["x"] == "16":
        s["x"] = x.to(dt)
    elif case["x"] == "e4m3":
        s["x_scales"] = (x.abs().amax() / 448).reshape(1)
        s["x"] = (x / s["x_scales"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    elif case["x"] == "e4m3_block":
        nb = -(-k // 128)
        pad = torch.zeros((m, nb * 128), device=DEV)
        pad[:, :k] = x
        pad = pad.view(m, nb, 128)
        s["x_scales"] = (pad.abs().amax(-1) / 448).contiguous()
        s["x"] = (pad / s["x_scales"].unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) \
            .flatten(1)[:, :k].contiguous()
    else:
        s["x_scales"] = (x.abs().amax() / 2688).reshape(1)
        s["x"], xsf = _quantise(x, s["x_scales"])
        s["xsf"] = _swizzle(xsf) if case["layout"] == "swizzled" else xsf
    s["bias"] = _randn((n,), g).to(dt) if case["bias"] else None
    s["y"] = torch.empty((m, n), dtype=dt, device=DEV)


# ------------------------------------------------------------------ plain --
def _rope(v, cos, sin):
    a, b = v.chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _head_norm(v, w):
    return v if w is None else v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS) * w.to(v.dtype)


def _plain_write(s):
    c = s["case"]
    m, hq, hkv, hd = c["m"], c["Hq"], c["Hkv"], c["hd"]
    heads = s["qkv"].view(m, hq + 2 * hkv, hd)
    cos, sin = s["cos"][s["pos"]].unsqueeze(1), s["sin"][s["pos"]].unsqueeze(1)
    q = _rope(_head_norm(heads[:, :hq].float(), s["qw"]), cos, sin).to(s["qkv"].dtype)
    # keys in 64 bits, rounded to 32: a code is decided next to a border
    k = _rope(_head_norm(heads[:, hq:hq + hkv].double(), s["kw"]), cos.double(), sin.double()).float()
    v = heads[:, hq + hkv:].float()
    where = s["where"].long()
    for name, y, gs in (("k", k, s["kv_scales"][0]), ("v", v, s["kv_scales"][1])):
        codes, sf = _quantise(y, gs)
        s[name][where] = codes
        s[name + "sf"][where // 4, :, :, where % 4] = sf
    return (q,) + _plain_read(s)


def _plain_read(s):
    where = s["where"].long()
    dt = s["k_out"].dtype
    return (_decode(s["k"][where], _sf_rows(s["ksf"], where), s["kv_scales"][0]).to(dt),
            _decode(s["v"][where], _sf_rows(s["vsf"], where), s["kv_scales"][1]).to(dt))


def _plain_attn(s):
    c = s["case"]
    b, hq, hkv, hd, page = c["seqs"], c["Hq"], c["Hkv"], c["hd"], c["page"]
    kv, tq = c["kv"], s["max_q"]
    at = torch.arange(kv, device=DEV)
    if page:
        slots = s["table"].long().clamp(min=0)[:, at // page] * page + at % page
    else:
        slots = at.expand(b, kv)
    tok = s["tokens_of"]
    length = torch.where(tok >= 0, s["kv_len"][tok.clamp(min=0)].long(), 0)        # [b, tq]
    seen = at < length.unsqueeze(-1)                                               # [b, tq, kv]
    if c["window"]:
        seen &= at >= (length - c["window"]).unsqueeze(-1)
    used = seen.any(1)[:, None, :, None]                                           # [b, 1, kv, 1]
    k = _decode(s["k"][slots], _sf_rows(s["ksf"], slots), s["kv_scales"][0]).transpose(1, 2)
    v = _decode(s["v"][slots], _sf_rows(s["vsf"], slots), s["kv_scales"][1]).transpose(1, 2)
    k, v = torch.where(used, k, 0), torch.where(used, v, 0)                        # [b, hkv, kv, hd]
    q = s["q"].float()[tok.clamp(min=0)].view(b, tq, hkv, hq // hkv, hd).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = (q @ k.transpose(-1, -2) * s["scale"]).unflatten(2, (tq, -1))          # [b, hkv, tq, group, kv]
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (tq, -1)) / torch.where(total > 0, total, 1)
    return o.permute(0, 2, 1, 3, 4).reshape(b, tq, hq, hd)[tok >= 0].to(s["q"].dtype)


def _plain_matvec(s):
    c = s["case"]
    n, k, m = c["n"], c["k"], c["m"]
    sf = _unswizzle(s["wsf"], n, k // 16) if c["layout"] == "swizzled" else s["wsf"]
    w = _decode(s["w"], sf, s["w_scale"])
    if c["x"] == "16":
        x = s["x"].float()
    elif c["x"] == "nvfp4":
        x = _decode(s["x"], _unswizzle(s["xsf"], m, k // 16) if c["layout"] == "swizzled" else s["xsf"], s["x_scales"])
    else:
        x = s["x"].view(torch.float8_e4m3fn).float()
        x = x * (s["x_scales"] if c["x"] == "e4m3" else s["x_scales"].repeat_interleave(128, 1)[:, :k])
    y = x @ w.t()
    return (y if s["bias"] is None else y + s["bias"].float()).to(s["y"].dtype)


# -------------------------------------------------------------------- run --
def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attn": _plain_attn, "matvec": _plain_matvec}[op](s)
    import memory_bound_non_b200 as frt
    if op == "write":
        frt.frt_qkv_norm_rope_nvfp4_kvcache(s["qkv"], s["qw"], s["kw"], s["cos"], s["sin"], s["pos"], s["q_out"],
                                            s["k"], s["ksf"], s["v"], s["vsf"], s["kv_scales"], c["Hq"], c["Hkv"],
                                            c["hd"], slots=s["slots"], eps=EPS)
    if op in ("write", "read"):
        frt.frt_nvfp4_kvcache_read(s["k"], s["ksf"], s["v"], s["vsf"], s["kv_scales"], s["where"], s["k_out"],
                                   s["v_out"])
        return (s["q_out"], s["k_out"], s["v_out"]) if op == "write" else (s["k_out"], s["v_out"])
    if op == "attn":
        frt.frt_attn_nvfp4_kvcache(s["q"], s["k"], s["ksf"], s["v"], s["vsf"], s["kv_scales"], s["kv_len"], s["out"],
                                   s["scale"], window=c["window"], q_indptr=s["indptr"], page_table=s["table"],
                                   page_size=c["page"], max_q_len=s["max_q"], max_kv_len=c["kv"],
                                   workspace=s["workspace"])
        return s["out"]
    frt.frt_matvec_nvfp4(s["x"], s["w"], s["wsf"], s["w_scale"], s["y"], bias=s["bias"], x_format=c["x"],
                         x_scales=s["x_scales"], x_sf=s["xsf"], sf_layout=c["layout"])
    return s["y"]


# ------------------------------------------------------------------ exact --
def _exact_values(codes, sf, gs):
    """The real numbers that NVFP4 codes stand for, in 64 bits."""
    lo, hi = (codes & 15).long(), (codes >> 4).long()
    c = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.int64, device=codes.device)
    c[..., 0::2], c[..., 1::2] = lo, hi
    e, f = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e == 0, 0.5 * f, torch.pow(2.0, (e - 1).double()) * (1 + 0.5 * f))
    t = sf.long()
    se, sm = (t >> 3) & 15, (t & 7).double()
    scale = torch.where(se == 0, sm * 2.0 ** -9, torch.pow(2.0, (se - 7).double()) * (1 + sm / 8))
    scale = torch.where((t & 127) == 127, torch.nan, scale) * torch.where(t >= 128, -1.0, 1.0)
    return torch.where(c >= 8, -mag, mag) * scale.repeat_interleave(16, -1) * gs.double()


def _exact_quantised(y, gs):
    """y in 64 bits -> the NVFP4 value of each element: nearest scale factor, then nearest code, of the quotients."""
    z = y.unflatten(-1, (-1, 16))
    want = (z.abs().amax(-1, keepdim=True) / (6 * gs.double())).clamp(max=448.0)
    step = torch.pow(2.0, torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
    sf = torch.round(want / step) * step
    eff = sf * gs.double()
    a = torch.where(eff > 0, z.abs() / torch.where(eff > 0, eff, 1), 0.0).clamp(max=6.0)
    st = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / st) * st * eff * torch.sign(z)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "write":
        m, hq, hkv, hd = c["m"], c["Hq"], c["Hkv"], c["hd"]
        x = s["qkv"].double().view(m, -1, hd)
        p = s["pos"].long()
        co, si = s["cos"].double()[p][:, None], s["sin"].double()[p][:, None]
        got = []
        for part, w in ((x[:, :hq], s["qw"]), (x[:, hq:hq + hkv], s["kw"])):
            if w is not None:
                part = part * (part.pow(2).sum(-1, keepdim=True) / hd + EPS).pow(-0.5) * w.double()
            first, second = part[..., :hd // 2], part[..., hd // 2:]
            got.append(torch.cat((first * co - second * si, second * co + first * si), -1))
        return (got[0], _exact_quantised(got[1], s["kv_scales"][0]),
                _exact_quantised(x[:, hq + hkv:], s["kv_scales"][1]))
    if op == "read":
        w = s["where"].long()
        return tuple(_exact_values(s[n][w], s[n + "sf"].permute(0, 3, 1, 2).flatten(0, 1)[w], s["kv_scales"][i])
                     for i, n in enumerate(("k", "v")))
    if op == "attn":
        return _exact_attn(s, c)
    w = _exact_values(s["w"], _unswizzle(s["wsf"], c["n"], c["k"] // 16) if c["layout"] == "swizzled" else s["wsf"],
                      s["w_scale"])
    if c["x"] == "16":
        x = s["x"].double()
    elif c["x"] == "nvfp4":
        sf = _unswizzle(s["xsf"], c["m"], c["k"] // 16) if c["layout"] == "swizzled" else s["xsf"]
        x = _exact_values(s["x"], sf, s["x_scales"])
    else:
        x = s["x"].view(torch.float8_e4m3fn).double()
        block = 128 if c["x"] == "e4m3_block" else c["k"]
        for i, k0 in enumerate(range(0, c["k"], block)):
            x[:, k0:k0 + block] *= s["x_scales"].double().view(-1, -(-c["k"] // block))[:, i:i + 1]
    y = torch.einsum("mk,nk->mn", x, w)
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_attn(s, c):
    hq, hkv, hd = c["Hq"], c["Hkv"], c["hd"]
    group, page = hq // hkv, c["page"]
    indptr, lens = s["indptr"].tolist(), s["kv_len"].long()
    sf_of = {n: s[n].permute(0, 3, 1, 2).flatten(0, 1) for n in ("ksf", "vsf")}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for i in range(c["seqs"]):
        t0, t1 = indptr[i], indptr[i + 1]
        n = int(lens[t0:t1].max())
        if n == 0:
            continue
        j = torch.arange(n, device=DEV)
        slot = s["table"][i].long()[j // page] * page + j % page if page else j
        k = _exact_values(s["k"][slot], sf_of["ksf"][slot], s["kv_scales"][0])
        v = _exact_values(s["v"][slot], sf_of["vsf"][slot], s["kv_scales"][1])
        q = s["q"][t0:t1].double()
        ln = lens[t0:t1, None]
        keep = (j < ln) & (j >= (ln - c["window"] if c["window"] else 0))
        for h in range(hkv):
            sc = torch.einsum("tgd,nd->gtn", q[:, h * group:(h + 1) * group], k[:, h]) * s["scale"]
            sc = sc.masked_fill(~keep, -math.inf)
            some = keep.any(-1)[None, :, None]
            p = torch.where(some, torch.softmax(torch.where(some, sc, 0.0), -1), 0.0)
            out[t0:t1, h * group:(h + 1) * group] = torch.einsum("gtn,nd->tgd", p, v[:, h])
    return out
