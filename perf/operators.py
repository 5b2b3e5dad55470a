"""Measured cases of the operators around a decoder layer's quantized matmuls: the residual addition with RMS norm
(bf16 or E4M3 output), the paged key-value cache (written and read back; bf16, E4M3 or Q4) and the attention of one new
token per sequence over that cache.

A case's "op" is one of
  norm       one w4a16_add_rmsnorm / w8a8_add_rmsnorm_quantize call
  cache      one kv_cache_write of new tokens, then one kv_cache_read of the context with them
  attention  one kv_cache_attention call

With ``own`` false, run() computes the plain form in elementary torch operations; with ``own`` true it calls the
library."""

import math

import torch

own = False

_DEV = "cuda"
_BF = torch.bfloat16
_E4M3_MAX = 448.0


def listed():
    return [
        # one token's hidden state between two layers: pure latency
        {"name": "norm_one_token", "op": "norm", "out": "bf16", "rows": 1, "d": 2816, "residual": True, "offset": 0.0},
        # a decode batch in front of FP8 experts
        {"name": "norm_batch_e4m3", "op": "norm", "out": "e4m3", "rows": 64, "d": 2816, "residual": True,
         "offset": 0.0},
        # a prompt in front of FP8 experts
        {"name": "norm_prompt_e4m3", "op": "norm", "out": "e4m3", "rows": 4096, "d": 2816, "residual": True,
         "offset": 0.0},
        # a packed prompt batch of odd length, first norm (no residual yet), weights stored around zero
        {"name": "norm_prompt_bf16", "op": "norm", "out": "bf16", "rows": 8191, "d": 4096, "residual": False,
         "offset": 1.0},
        # one new token for each of 64 sequences, some slots padded out
        {"name": "cache_decode_q4", "op": "cache", "format": "q4", "tokens": 64, "context": 0, "kv_heads": 8,
         "head_dim": 128, "page": 64, "padded": 3},
        # a prompt chunk and the context it attends to
        {"name": "cache_chunk_e4m3", "op": "cache", "format": "e4m3", "tokens": 4096, "context": 4096, "kv_heads": 8,
         "head_dim": 128, "page": 32, "padded": 0},
        # a long read-back, odd lengths, wide heads
        {"name": "cache_long_q4", "op": "cache", "format": "q4", "tokens": 2045, "context": 28675, "kv_heads": 4,
         "head_dim": 256, "page": 16, "padded": 5},
        # a single user's chat
        {"name": "attn_one_q4", "op": "attention", "format": "q4", "seqs": 1, "max_len": 1000, "ragged": False,
         "kv_heads": 8, "group": 4, "head_dim": 128, "page": 16, "window": 0},
        # a ragged serving batch
        {"name": "attn_ragged_e4m3", "op": "attention", "format": "e4m3", "seqs": 48, "max_len": 8000, "ragged": True,
         "kv_heads": 8, "group": 4, "head_dim": 128, "page": 32, "window": 0},
        # long documents over the 4-bit cache
        {"name": "attn_long_q4", "op": "attention", "format": "q4", "seqs": 16, "max_len": 32768, "ragged": False,
         "kv_heads": 8, "group": 8, "head_dim": 128, "page": 64, "window": 0},
        # long documents over the unquantized cache
        {"name": "attn_long_bf16", "op": "attention", "format": "bf16", "seqs": 8, "max_len": 32768, "ragged": False,
         "kv_heads": 8, "group": 4, "head_dim": 128, "page": 64, "window": 0},
        # sliding-window layers with wide heads
        {"name": "attn_window_bf16", "op": "attention", "format": "bf16", "seqs": 64, "max_len": 6000, "ragged": True,
         "kv_heads": 4, "group": 2, "head_dim": 256, "page": 16, "window": 1024},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "cache", "attention"])
    if op == "norm":
        d = 32 * _log_int(rng, 2, 256)
        return {"op": op, "out": rng.choice(["bf16", "e4m3"]), "rows": _log_int(rng, 1, min(16384, 40000000 // d)),
                "d": d, "residual": rng.random() < 0.7, "offset": rng.choice([0.0, 1.0])}
    form, dim = rng.choice(["bf16", "e4m3", "q4"]), rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "cache":
        heads = rng.choice([1, 2, 3, 4, 8])
        new = _log_int(rng, 1, 4096)
        most = 32000000 // (heads * dim) - new
        return {"op": op, "format": form, "tokens": new, "context": rng.choice([0, _log_int(rng, 1, max(1, most))]),
                "kv_heads": heads, "head_dim": dim, "page": page, "padded": rng.randint(0, new // 8)}
    heads, seqs = rng.choice([1, 2, 3, 4, 8]), _log_int(rng, 1, 64)
    most = min(65536, 250000000 // (heads * dim * seqs))
    return {"op": op, "format": form, "seqs": seqs, "max_len": _log_int(rng, 1, most), "ragged": rng.random() < 0.6,
            "kv_heads": heads, "group": rng.choice([1, 2, 3, 4, 6, 8, 16]), "head_dim": dim, "page": page,
            "window": rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])}


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """Sequence lengths of an attention case, longest last; a ragged batch spreads from an empty slot to max_len."""
    n, most = case["seqs"], case["max_len"]
    return [int(most * (i / (n - 1)) ** 2) if case["ragged"] and n > 1 else most for i in range(n)]


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=_DEV)


def _ratio(a, b):
    """a / b in 32 bits, correctly rounded (a quotient of 32-bit numbers taken in 64 bits rounds only once)."""
    return (a.double() / (b.double() if torch.is_tensor(b) else b)).float()


def _to_codes(x, form):
    """Rows [..., D] of 32-bit values -> (codes, scales) of a cache format: bf16 values and no scales, E4M3 values with
    a 32-bit scale a row, or integers with a bf16 scale for each 32 values."""
    if form == "bf16":
        return x.to(_BF), None
    if form == "e4m3":
        amax = x.abs().amax(-1, keepdim=True)
        s = torch.where(amax > 0, _ratio(amax, _E4M3_MAX), torch.ones_like(amax))
        return _ratio(x, s).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn), s[..., 0]
    x = x.unflatten(-1, (-1, 32))
    s = _ratio(x.abs().amax(-1, keepdim=True), 7.0).to(_BF)
    q = torch.where(s > 0, _ratio(x, s.float()), torch.zeros_like(x)).round().clamp(-8, 7)
    return q.to(torch.int8).flatten(-2), s[..., 0]


def _values(codes, scales, form):
    """The 32-bit values that codes and scales stand for."""
    v = codes.float()
    if form == "e4m3":
        return v * scales.float().unsqueeze(-1)
    if form == "q4":
        return (v.unflatten(-1, (-1, 32)) * scales.float().unsqueeze(-1)).flatten(-2)
    return v


def _bytes_of(t):
    return t.contiguous().view(torch.uint8).flatten(2)


def _block(codes, scales, form, is_v):
    """One K or V block of every (page, head) as the library lays it out: codes [pages, heads, page, D] -> bytes
    [pages, heads, block]."""
    pages, heads, page, dim = codes.shape
    groups = dim // 32
    unit = {"bf16": 1, "e4m3": 2, "q4": min(4, groups)}[form]
    c = (codes + 8).to(torch.uint8) if form == "q4" else codes.view(torch.uint8) if form == "e4m3" else codes
    if is_v:    # [tile, 4 c, 4 j, unit, part, 16 m, 2 b] -> [tile, unit, c, m, part, b, j]
        c = c.view(pages, heads, page // 16, 4, 4, groups // unit, unit, 16, 2).permute(0, 1, 2, 5, 3, 7, 6, 8, 4)
        if form == "q4":
            c = c[..., 0, :] | (c[..., 1, :] << 4)
    else:       # [tile, 16 r, unit, part, 4 c, 8 i] -> [tile, unit, c, r, part, i]
        c = c.view(pages, heads, page // 16, 16, groups // unit, unit, 4, 8).permute(0, 1, 2, 4, 6, 3, 5, 7)
        if form == "q4":
            c = c[..., [0, 4, 1, 5]] | (c[..., [2, 6, 3, 7]] << 4)
    out = [_bytes_of(c)]
    if form == "e4m3":
        out.append(_bytes_of(scales))
    elif form == "q4":      # [tile, 4 c, 4 j, group] -> [tile, c, group, j]
        out.append(_bytes_of(scales.view(pages, heads, page // 16, 4, 4, groups).transpose(-1, -2)))
    return torch.cat(out, 2)


def _cache(gen, case, pages):
    """A filled cache of `pages` pages: its codes and scales ([page, head, token, ...], K then V) and the packed buffer
    that the library's calls take."""
    form, heads, dim, page = case["format"], case["kv_heads"], case["head_dim"], case["page"]
    channel = torch.exp(0.5 * _normal(gen, heads, 1, dim))       # keys have channels of uneven size
    k = _to_codes((_normal(gen, pages, heads, page, dim) * channel).to(_BF).float(), form)
    v = _to_codes(_normal(gen, pages, heads, page, dim).to(_BF).float(), form)
    packed = torch.cat([_block(*k, form, False), _block(*v, form, True)], 2)
    return k, v, packed


def _formats(w4, form):
    return {"bf16": w4.W4_KV_BF16, "e4m3": w4.W4_KV_E4M3, "q4": w4.W4_KV_Q4}[form]


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        s["x"] = _normal(gen, rows, d).to(_BF)
        s["residual"] = (4.0 * _normal(gen, rows, d)).to(_BF) if case["residual"] else None
        s["weight"] = (1.0 - case["offset"] + 0.2 * _normal(gen, d)).to(_BF)
        s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["y"] = torch.empty(rows, d, dtype=_BF if case["out"] == "bf16" else torch.uint8, device=_DEV)
        s["scale"] = torch.empty(rows, dtype=torch.float32, device=_DEV)
        return s
    heads, dim, page = case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "cache":
        new, ctx = case["tokens"], case["context"]
        need = -(-(new + ctx) // page)
        pages = need + 2
        s["k"], s["v"], s["cache"] = _cache(gen, case, pages)
        # token i of the sequence sits in its page list's place i; a decode batch has one token in each of many pages
        table = torch.randperm(pages, generator=gen, device=_DEV)[:need]
        i = torch.arange(new + ctx, device=_DEV)
        slots = table[i // page] * page + i % page
        if ctx == 0 and new > 1:
            slots = torch.randperm(pages * page, generator=gen, device=_DEV)[:new]
        # a fused projection's output: q, k and v side by side
        qkv = _normal(gen, new, 4 * heads * dim).to(_BF)
        s["new_k"] = qkv[:, 2 * heads * dim:3 * heads * dim].view(new, heads, dim)
        s["new_v"] = qkv[:, 3 * heads * dim:].view(new, heads, dim)
        s["new_slots"] = slots[ctx:].clone()
        s["new_slots"][new - case["padded"]:] = -1
        s["slots"] = slots[:ctx + new - case["padded"]].clone()
        n = ctx + new - case["padded"]
        s["out_k"] = torch.empty(n, heads, dim, dtype=_BF, device=_DEV)
        s["out_v"] = torch.empty(n, heads, dim, dtype=_BF, device=_DEV)
        return s
    lens = _lengths(case)
    order = torch.randperm(case["seqs"], generator=gen, device=_DEV)
    width = max(1, -(-case["max_len"] // page))
    used = sum(-(-n // page) for n in lens)
    pages = used + 1
    s["k"], s["v"], s["cache"] = _cache(gen, case, pages)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=_DEV)[order]
    ids = torch.randperm(pages, generator=gen, device=_DEV).to(torch.int32)
    have = -(-s["lens"].long() // page)
    first = have.cumsum(0) - have
    col = torch.arange(width, device=_DEV)
    s["table"] = torch.where(col < have[:, None], ids[(first[:, None] + col).clamp(max=pages - 1)], 0).to(torch.int32)
    hq = heads * case["group"]
    qkv = _normal(gen, case["seqs"], (hq + 2 * heads) * dim).to(_BF)
    s["q"] = qkv[:, :hq * dim].view(case["seqs"], hq, dim)
    s["out"] = torch.empty(case["seqs"], hq, dim, dtype=_BF, device=_DEV)
    s["lse"] = torch.empty(case["seqs"], hq, dtype=torch.float32, device=_DEV)
    return s


# ------------------------------------------------------------- plain forms
def _plain_norm(s):
    case = s["case"]
    r = s["x"]
    if case["residual"]:
        r = (s["x"].float() + s["residual"].float()).to(_BF)
    # 64 bits: a row's values are small multiples of one another, so many quotients by the scale fall on or next to the
    # middle between two E4M3 values
    r64 = r.double()
    y = r64 * (case["offset"] + s["weight"].float()).double() / torch.sqrt(r64.square().mean(-1, keepdim=True) + 1e-6)
    out = {"sum": r} if case["residual"] else {}
    if case["out"] == "bf16":
        return dict(out, y=y.to(_BF))
    amax = y.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, (amax / _E4M3_MAX).float(), 1.0)
    q = (y / scale.double()).float().clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn)
    return dict(out, y=q, scale=scale[:, 0])


def _plain_cache(s):
    form, page = s["case"]["format"], s["case"]["page"]
    keep = s["new_slots"] >= 0
    at = s["new_slots"][keep]
    out = {}
    for name in ("k", "v"):
        codes, scales = s[name]
        c, f = _to_codes(s["new_" + name][keep].float(), form)
        # float8 has no indexed writes: moved as bytes
        bits = codes.view(torch.uint8) if form == "e4m3" else codes
        bits[at // page, :, at % page] = c.view(torch.uint8) if form == "e4m3" else c
        if scales is not None:
            scales[at // page, :, at % page] = f
        slots = s["slots"]
        c = bits[slots // page, :, slots % page]
        f = None if scales is None else scales[slots // page, :, slots % page]
        out[name] = _values(c.view(torch.float8_e4m3fn) if form == "e4m3" else c, f, form).to(_BF)
    return out


def _plain_attention(s):
    case = s["case"]
    form, heads, group, dim = case["format"], case["kv_heads"], case["group"], case["head_dim"]
    seqs, width = s["table"].shape

    def gather(codes, scales):      # [seqs, heads, width * page, D] of the sequences' pages
        at = s["table"].long()
        c = codes.view(torch.uint8)[at].view(codes.dtype) if form == "e4m3" else codes[at]
        v = _values(c, None if scales is None else scales[at], form)
        return v.transpose(1, 2).reshape(seqs, heads, -1, dim)

    i = torch.arange(width * case["page"], device=_DEV)
    n = s["lens"].long()[:, None]
    live = i < n
    if case["window"] > 0:
        live = live & (i >= n - case["window"])
    q = s["q"].float().view(seqs, heads, group, dim)
    score = torch.matmul(q, gather(*s["k"]).transpose(-1, -2).contiguous()) / math.sqrt(dim)
    score = score.masked_fill(~live[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = gather(*s["v"]).masked_fill(~live[:, None, :, None], 0.0)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + top
    return {"out": out.to(_BF).view(seqs, heads * group, dim), "lse": lse.view(seqs, heads * group)}


def _own_run(s):
    import int4_group_quantized_q4_amd as w4
    case = s["case"]
    if case["op"] == "norm":
        out = {"sum": s["sum"]} if case["residual"] else {}
        if case["out"] == "bf16":
            w4.w4a16_add_rmsnorm(s["x"], s["residual"], s["weight"], 1e-6, s["sum"], s["y"], case["offset"])
            return dict(out, y=s["y"])
        w4.w8a8_add_rmsnorm_quantize(s["x"], s["residual"], s["weight"], 1e-6, s["sum"], s["y"], s["scale"],
                                     case["offset"])
        return dict(out, y=s["y"].view(torch.float8_e4m3fn), scale=s["scale"])
    form = _formats(w4, case["format"])
    if case["op"] == "cache":
        w4.kv_cache_write(s["new_k"], s["new_v"], s["new_slots"], form, case["page"], s["cache"])
        w4.kv_cache_read(s["cache"], form, case["page"], s["slots"], s["out_k"], s["out_v"])
        return {"k": s["out_k"], "v": s["out_v"]}
    if "ws" not in s:       # kept between calls, as a serving loop does
        seqs, hq, dim = s["q"].shape
        need = w4.kv_cache_attention_workspace(seqs, hq, case["kv_heads"], dim, s["table"].shape[1], case["page"])
        s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device=_DEV)
    w4.kv_cache_attention(s["q"], s["cache"], form, case["page"], case["kv_heads"], s["table"], s["lens"],
                          1.0 / math.sqrt(case["head_dim"]), s["out"], case["window"], s["lse"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own_run(state)
    return {"norm": _plain_norm, "cache": _plain_cache, "attention": _plain_attention}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the work
def _row_bytes(case):
    """Bytes of one token's keys (or values) of one head in the cache."""
    d = case["head_dim"]
    return {"bf16": 2 * d, "e4m3": d + 4, "q4": d // 2 + d // 16}[case["format"]]


def work(case):
    if case["op"] == "norm":
        n, d = case["rows"], case["d"]
        b = 2 * n * d + 2 * d + (4 * n * d if case["residual"] else 0)
        return {"bytes": b + (2 * n * d if case["out"] == "bf16" else n * d + 4 * n), "flops": 6 * n * d}
    heads, d = case["kv_heads"], case["head_dim"]
    if case["op"] == "cache":
        new = case["tokens"] - case["padded"]
        held = case["context"] + new
        return {"bytes": 2 * heads * (new * (2 * d + _row_bytes(case)) + held * (2 * d + _row_bytes(case)))
                + 8 * (case["tokens"] + held), "flops": 4 * heads * d * (new + held)}
    lens = _lengths(case)
    seen = sum(min(n, case["window"]) if case["window"] > 0 else n for n in lens)
    hq = heads * case["group"]
    return {"bytes": 2 * heads * seen * _row_bytes(case) + case["seqs"] * hq * (4 * d + 4)
            + 4 * sum(-(-n // case["page"]) for n in lens), "flops": 4 * hq * d * seen}


# ------------------------------------------------ the definitions in 64 bits
def _e4m3_round(x):
    """64-bit values -> the nearest E4M3 values, ties to even: steps of 2^(e-3) in [2^e, 2^(e+1)), 2^-9 below 2^-6."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 1
    step = torch.ldexp(torch.ones_like(x), e - 3)
    return (torch.round(x / step) * step).clamp(-_E4M3_MAX, _E4M3_MAX)


def _exact_quantized(x, form):
    """What 64-bit rows [..., D] stand for once they went through a cache format."""
    if form == "bf16":
        return x
    if form == "e4m3":
        amax = x.abs().amax(-1, keepdim=True)
        s = (amax / _E4M3_MAX).float().double()
        s = torch.where(amax > 0, s, 1.0)
        return _e4m3_round((x / s).float().double()) * s
    g = x.reshape(*x.shape[:-1], -1, 32)
    s = (g.abs().amax(-1, keepdim=True) / 7.0).float().to(_BF).double()
    q = torch.round((g / s).float().double()).clamp(-8, 7)
    return torch.where(s > 0, q * s, 0.0).reshape(x.shape)


def _exact_held(codes, scales, form):
    c = codes.double()
    if form == "e4m3":
        return c * scales.double()[..., None]
    if form == "q4":
        return c * scales.double().repeat_interleave(32, -1)
    return c


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        r = s["x"].double()
        out = {}
        if case["residual"]:
            r = (r + s["residual"].double()).float().to(_BF).double()
            out["sum"] = r
        w = (case["offset"] + s["weight"].double()).float().double()
        y = r * torch.rsqrt((r * r).sum(1) / case["d"] + 1e-6)[:, None] * w
        if case["out"] == "bf16":
            return dict(out, y=y)
        scale = (y.abs().amax(1) / _E4M3_MAX).float().double()
        scale = torch.where(scale > 0, scale, 1.0)
        return dict(out, y=_e4m3_round((y / scale[:, None]).float().double()), scale=scale)     # quotients of 32 bits
    form, page = case["format"], case["page"]
    if case["op"] == "cache":
        out, ctx, n = {}, case["context"], case["context"] + case["tokens"] - case["padded"]
        for name in ("k", "v"):
            old = s["slots"][:ctx]
            c, f = s[name]
            before = _exact_held(c[old // page, :, old % page] if form != "e4m3" else
                                 c.view(torch.uint8)[old // page, :, old % page].view(torch.float8_e4m3fn),
                                 None if f is None else f[old // page, :, old % page], form)
            out[name] = torch.cat([before, _exact_quantized(s["new_" + name][:n - ctx].double(), form)])
        return out
    heads, group, dim = case["kv_heads"], case["group"], case["head_dim"]
    outs, lses = [], []
    for i, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] > 0 else 0
        if n == 0:
            outs.append(torch.zeros(heads * group, dim, dtype=torch.float64, device=_DEV))
            lses.append(torch.full((heads * group,), -math.inf, dtype=torch.float64, device=_DEV))
            continue
        at = s["table"][i, :-(-n // page)].long()

        def rows(codes, scales):    # [heads, n - lo, D]
            c = codes.view(torch.uint8)[at].view(codes.dtype) if form == "e4m3" else codes[at]
            v = _exact_held(c, None if scales is None else scales[at], form)
            return v.permute(1, 0, 2, 3).reshape(heads, -1, dim)[:, lo:n]

        k, v = rows(*s["k"]), rows(*s["v"])
        q = s["q"][i].double().view(heads, group, dim)
        w = torch.stack([(k[h] @ q[h].T).T for h in range(heads)]) * dim ** -0.5
        lse = torch.logsumexp(w, -1)
        outs.append(torch.stack([torch.softmax(w[h], -1) @ v[h] for h in range(heads)]).view(heads * group, dim))
        lses.append(lse.view(-1))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
