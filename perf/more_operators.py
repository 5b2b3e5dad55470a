"""Measured cases of the operators of a serving step around the projections, the cache and the attention: the plan of
the step's rows over the paged cache, low-rank adapters beside a projection, rotary positions, and the draw of the next
tokens from the logits.

A case's "op" is one of
  plan    one kv_cache_plan call: pages given out and taken back, slots and positions of the step's rows
  rope    one w4a16_rope call on q and k
  lora    one w4a16_lora_add call on a projection's output
  sample  one w4a16_sample call

With ``own`` false, run() computes the plain form in elementary torch operations; with ``own`` true it calls the
library."""

import math

import torch

own = False

_DEV = "cuda"
_BF = torch.bfloat16


def listed():
    return [
        # a decode step's bookkeeping: one new token for each of 64 sequences, pure latency
        {"name": "plan_decode", "op": "plan", "seqs": 64, "max_len": 32000, "page": 64, "prompts": 0, "chunk": 0,
         "ended": 2},
        # a mixed step: most sequences decode, some bring prompt chunks of odd lengths, some have ended
        {"name": "plan_mixed", "op": "plan", "seqs": 500, "max_len": 16000, "page": 16, "prompts": 30, "chunk": 1000,
         "ended": 40},
        # one chat's token
        {"name": "rope_one", "op": "rope", "rows": 1, "q_heads": 32, "k_heads": 8, "head_dim": 128, "rotary": 128,
         "layout": "half", "max_pos": 32768, "prompt": False, "scale": 1.0},
        # a decode batch at far positions, amplitudes scaled for a long context
        {"name": "rope_decode", "op": "rope", "rows": 64, "q_heads": 32, "k_heads": 8, "head_dim": 128, "rotary": 128,
         "layout": "half", "max_pos": 1000000, "prompt": False, "scale": 1.1},
        # a packed prompt batch of odd length, adjacent pairs in half of a wide head
        {"name": "rope_prompt", "op": "rope", "rows": 8191, "q_heads": 16, "k_heads": 4, "head_dim": 256, "rotary": 128,
         "layout": "interleaved", "max_pos": 131072, "prompt": True, "scale": 1.0},
        # one request with an adapter
        {"name": "lora_one", "op": "lora", "rows": 1, "K": 2816, "N": 4096, "rank": 16, "adapters": 4, "prompt": False},
        # a decode batch whose requests hold many adapters, some none
        {"name": "lora_decode", "op": "lora", "rows": 64, "K": 4096, "N": 14336, "rank": 16, "adapters": 48,
         "prompt": False},
        # prompts of several requests, one after another
        {"name": "lora_prompt", "op": "lora", "rows": 4090, "K": 4096, "N": 14336, "rank": 64, "adapters": 7,
         "prompt": True},
        # one chat's token with the usual filters
        {"name": "sample_one", "op": "sample", "rows": 1, "vocab": 131072, "dtype": "bf16", "filters": "usual",
         "masked": 0.0},
        # a serving batch in which every request has its own settings, greedy ones and masked vocabularies among them
        {"name": "sample_mixed", "op": "sample", "rows": 64, "vocab": 131072, "dtype": "f32", "filters": "mixed",
         "masked": 0.2},
        # a batch of a small odd vocabulary
        {"name": "sample_small", "op": "sample", "rows": 48, "vocab": 50021, "dtype": "f32", "filters": "mixed",
         "masked": 0.0},
        # rollouts: the whole distribution, many rows
        {"name": "sample_whole", "op": "sample", "rows": 256, "vocab": 131072, "dtype": "f32", "filters": "none",
         "masked": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "lora", "sample"])
    if op == "plan":
        seqs, page = _log_int(rng, 1, 2000), rng.choice([16, 32, 64, 128])
        prompts = rng.choice([0, rng.randint(0, seqs // 4)])
        return {"op": op, "seqs": seqs, "max_len": _log_int(rng, 1, 32000), "page": page, "prompts": prompts,
                "chunk": _log_int(rng, 1, 20000 // max(1, prompts)), "ended": rng.randint(0, seqs // 4)}
    if op == "rope":
        dim = rng.choice([64, 80, 128, 256])
        heads = rng.choice([1, 2, 3, 4, 8])
        q = heads * rng.choice([1, 2, 3, 4, 6, 8])
        rows = _log_int(rng, 1, min(16384, 40000000 // ((q + heads) * dim)))
        return {"op": op, "rows": rows, "q_heads": q, "k_heads": rng.choice([heads, heads, 0]), "head_dim": dim,
                "rotary": rng.choice([dim, 16 * rng.randint(1, dim // 16)]),
                "layout": rng.choice(["half", "interleaved"]),
                "max_pos": _log_int(rng, rows, 1000000), "prompt": rng.random() < 0.5,
                "scale": rng.choice([1.0, rng.uniform(1.0, 1.5)])}
    if op == "lora":
        K, N, rank = 32 * _log_int(rng, 2, 448), 16 * _log_int(rng, 2, 896), 8 * rng.choice([1, 2, 2, 3, 4, 8, 16])
        rows = _log_int(rng, 1, max(1, min(8192, 120000000 // (K + 2 * N), 4000000000 // (rank * (K + N)))))
        most = max(1, min(100, 200000000 // (rank * (K + N))))
        return {"op": op, "rows": rows, "K": K, "N": N, "rank": rank, "adapters": _log_int(rng, 1, most),
                "prompt": rng.random() < 0.5 if rows > 16 else False}
    vocab = _log_int(rng, 100, 262144)
    return {"op": op, "rows": _log_int(rng, 1, min(512, 32000000 // vocab)), "vocab": vocab,
            "dtype": rng.choice(["bf16", "f32"]), "filters": rng.choice(["usual", "mixed", "mixed", "none"]),
            "masked": rng.choice([0.0, 0.0, rng.uniform(0.0, 0.9)])}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=_DEV)


def _plan_sizes(case):
    """(tokens held, new tokens) of each sequence: the first ones bring prompt chunks (some of them a first chunk, with
    nothing held yet), the last ones have ended (-1); a sequence between them brings one token."""
    n, most = case["seqs"], case["max_len"]
    held = [int(most * ((7919 * i + 13) % 1009) / 1009) for i in range(n)]
    new = [1] * n
    for i in range(case["prompts"]):
        new[i] = max(1, case["chunk"] - (37 * i) % max(1, case["chunk"] // 2))
        if i % 2 == 0:
            held[i] = 0
    for i in range(case["ended"]):
        new[n - 1 - i] = -1
    return held, new


def _prepare_plan(s, gen):
    case, page = s["case"], s["case"]["page"]
    held, new = _plan_sizes(case)
    n = case["seqs"]
    order = torch.randperm(n, generator=gen, device=_DEV)
    lens = torch.tensor(held, device=_DEV)[order]
    s["lens"] = lens.to(torch.int32)
    s["new"] = torch.tensor(new, device=_DEV)[order].to(torch.int32)
    width = max(-(-(h + max(0, t)) // page) for h, t in zip(held, new)) + 1
    used = sum(-(-h // page) for h in held)
    spare = sum(-(-(h + max(0, t)) // page) for h, t in zip(held, new)) - used + 7
    pages = used + spare
    ids = torch.randperm(pages, generator=gen, device=_DEV).to(torch.int32)
    have = -(-lens // page)
    first = have.cumsum(0) - have
    col = torch.arange(width, device=_DEV)
    s["table"] = torch.where(col < have[:, None], ids[(first[:, None] + col).clamp(max=pages - 1)], 0).to(torch.int32)
    s["free"] = torch.zeros(pages, dtype=torch.int32, device=_DEV)
    s["free"][:spare] = ids[used:]
    s["free_count"] = torch.tensor([spare], dtype=torch.int32, device=_DEV)
    rows = sum(max(0, t) for t in new) + 5      # a step's buffers are a little longer than its rows
    s["lens_out"] = torch.empty(n, dtype=torch.int32, device=_DEV)
    s["free_count_out"] = torch.empty(1, dtype=torch.int32, device=_DEV)
    s["offsets"] = torch.empty(n + 1, dtype=torch.int32, device=_DEV)
    s["slots"] = torch.empty(rows, dtype=torch.int64, device=_DEV)
    s["positions"] = torch.empty(rows, dtype=torch.int32, device=_DEV)
    s["row_seqs"] = torch.empty(rows, dtype=torch.int32, device=_DEV)


def _prepare_rope(s, gen):
    case = s["case"]
    rows, dim, hq, hk = case["rows"], case["head_dim"], case["q_heads"], case["k_heads"]
    # a fused projection's output: q, k and v side by side
    qkv = _normal(gen, rows, (hq + 2 * hk) * dim).to(_BF)
    s["q"] = qkv[:, :hq * dim].view(rows, hq, dim)
    s["k"] = qkv[:, hq * dim:(hq + hk) * dim].view(rows, hk, dim) if hk else None
    if case["prompt"]:      # chunks of four requests, each with its own start
        piece = -(-rows // 4)
        start = torch.randint(0, max(1, case["max_pos"] - piece), (4,), generator=gen, device=_DEV)
        i = torch.arange(rows, device=_DEV)
        s["positions"] = (start[i // piece] + i % piece).to(torch.int32)
    else:
        s["positions"] = torch.randint(0, case["max_pos"], (rows,), generator=gen, device=_DEV).to(torch.int32)
    pair = torch.arange(case["rotary"] // 2, dtype=torch.float64, device=_DEV)
    s["inv_freq"] = (10000.0 ** (-2.0 * pair / case["rotary"])).float()
    s["q_out"] = torch.empty(rows, hq, dim, dtype=_BF, device=_DEV)
    s["k_out"] = torch.empty(rows, hk, dim, dtype=_BF, device=_DEV) if hk else None


def _prepare_lora(s, gen):
    case = s["case"]
    rows, K, N, R, n = case["rows"], case["K"], case["N"], case["rank"], case["adapters"]
    s["x"] = _normal(gen, rows, K).to(_BF)
    s["a"] = (_normal(gen, n, R, K) / math.sqrt(K)).to(_BF)
    s["b"] = (0.1 * _normal(gen, n, N, R)).to(_BF)
    s["scaling"] = torch.rand(n, generator=gen, device=_DEV) * 1.5 + 0.5
    if case["prompt"]:      # uneven requests one after another; id n means a request without an adapter
        pieces = min(rows, n + 1)
        cuts = torch.sort(torch.randperm(rows, generator=gen, device=_DEV)[:pieces - 1])[0]
        which = torch.randperm(n + 1, generator=gen, device=_DEV)
        ids = which[torch.searchsorted(cuts, torch.arange(rows, device=_DEV), right=True)]
    else:
        ids = torch.randint(0, n, (rows,), generator=gen, device=_DEV)
        bare = torch.rand(rows, generator=gen, device=_DEV) < 0.1
        ids = torch.where(bare & (rows > 1), n, ids)
    s["ids"] = torch.where(ids == n, -1, ids).to(torch.int32)
    s["y"] = _normal(gen, rows, N).to(_BF)
    s["out"] = torch.empty(rows, N, dtype=_BF, device=_DEV)


def _prepare_sample(s, gen):
    case = s["case"]
    rows, V = case["rows"], case["vocab"]
    # a bulk of unlikely tokens and a head that falls off by a power of the rank, each row its own
    z = 2.0 * _normal(gen, rows, V)
    head = min(2000, V)
    power = 1.2 + 1.8 * torch.rand(rows, 1, generator=gen, device=_DEV)
    rank = torch.arange(1, head + 1, device=_DEV, dtype=torch.float32)
    top = 18.0 - power * torch.log(rank) + 0.3 * _normal(gen, rows, head)
    at = torch.randperm(V, generator=gen, device=_DEV)[:head]
    at = (at + torch.randint(0, V, (rows, 1), generator=gen, device=_DEV)) % V
    z.scatter_(1, at, torch.maximum(top, z.gather(1, at)))
    if case["masked"] > 0:      # a grammar that forbids tokens
        z[torch.rand(rows, V, generator=gen, device=_DEV) < case["masked"]] = -math.inf
        z[:, V // 3] = 15.0     # and always allows one
    s["logits"] = z.to(_BF) if case["dtype"] == "bf16" else z
    s["uniforms"] = torch.rand(rows, generator=gen, device=_DEV)
    full = lambda v, t: torch.full((rows,), v, dtype=t, device=_DEV)
    pick = lambda values, t: torch.tensor(values, dtype=t, device=_DEV)[
        torch.randint(0, len(values), (rows,), generator=gen, device=_DEV)]
    s["temperature"] = s["top_k"] = s["top_p"] = s["min_p"] = None
    if case["filters"] == "usual":
        s["temperature"], s["top_k"] = full(0.8, torch.float32), full(50, torch.int32)
        s["top_p"] = full(0.95, torch.float32)
    elif case["filters"] == "mixed":
        s["temperature"] = pick([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.2], torch.float32)
        s["top_k"] = pick([0, 0, 1, 20, 50, 100, 1000], torch.int32)
        s["top_p"] = pick([1.0, 1.0, 0.5, 0.8, 0.9, 0.95, 0.99], torch.float32)
        s["min_p"] = pick([0.0, 0.0, 0.0, 0.02, 0.1], torch.float32)
    s["tokens"] = torch.empty(rows, dtype=torch.int32, device=_DEV)
    s["logprobs"] = torch.empty(rows, dtype=torch.float32, device=_DEV)


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    {"plan": _prepare_plan, "rope": _prepare_rope, "lora": _prepare_lora, "sample": _prepare_sample}[case["op"]](s, gen)
    return s


# ------------------------------------------------------------- plain forms
def _plain_plan(s):
    page = s["case"]["page"]
    table, free, rows = s["table"], s["free"], s["slots"].shape[0]
    n, width = table.shape
    lens, new = s["lens"].long(), s["new"].long()
    ended = new < 0
    have = (lens + page - 1) // page
    # pages of ended sequences go back onto the stack, in the order of the sequences
    back = torch.where(ended, have, 0)
    at = back.cumsum(0) - back
    col = torch.arange(width, device=_DEV)
    seq, c = torch.nonzero(col < back[:, None], as_tuple=True)
    free[s["free_count"].long() + at[seq] + c] = table[seq, c]
    count = s["free_count"].long() + back.sum()
    # sequences whose pages or rows do not suffice get nothing
    rows_of = new.clamp(min=0)
    total = torch.where(ended, 0, lens + rows_of)
    want = torch.where(ended, 0, (total + page - 1) // page - have)
    ok = ~ended & (want.cumsum(0) <= count) & (rows_of.cumsum(0) <= rows)
    rows_of, want = torch.where(ok, rows_of, 0), torch.where(ok, want, 0)
    first = want.cumsum(0) - want
    j = torch.arange(int(want.max()), device=_DEV)
    seq, c = torch.nonzero(j < want[:, None], as_tuple=True)
    table[seq, have[seq] + c] = free[count - 1 - first[seq] - c]
    lens_out = torch.where(ended, 0, torch.where(ok, total, lens))
    offsets = torch.zeros(n + 1, dtype=torch.int64, device=_DEV)
    offsets[1:] = rows_of.cumsum(0)
    i = torch.arange(rows, device=_DEV)
    seq = torch.searchsorted(offsets[1:].contiguous(), i, right=True)
    live = seq < n
    seq = seq.clamp(max=n - 1)
    pos = torch.where(live, lens[seq] + i - offsets[seq], 0)
    slots = torch.where(live, table[seq, pos // page].long() * page + pos % page, -1)
    return {"lens": lens_out.to(torch.int32), "table": table, "free": free, "offsets": offsets.to(torch.int32),
            "free_count": (count - want.sum()).to(torch.int32), "slots": slots, "positions": pos.to(torch.int32),
            "row_seqs": torch.where(live, seq, -1).to(torch.int32)}


def _plain_rope(s):
    case = s["case"]
    r = case["rotary"]
    # 64 bits: the angle of a far position keeps 32-bit accuracy only if it is reduced in more than 32 bits
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos = (torch.cos(angle).float() * case["scale"])[:, None]
    sin = (torch.sin(angle).float() * case["scale"])[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name]
        if x is None:
            continue
        x = x.float()
        if case["layout"] == "half":
            a, b = x[..., :r // 2], x[..., r // 2:r]
        else:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = [a * cos - b * sin, b * cos + a * sin]
        turned = torch.cat(turned, -1) if case["layout"] == "half" else torch.stack(turned, -1).flatten(-2)
        out[name] = torch.cat([turned, x[..., r:]], -1).to(_BF)
    return out


def _plain_lora(s):
    ids, y = s["ids"].long(), s["y"].float()
    if ids.shape[0] <= 64:      # few rows: every row's own factors side by side
        at = ids.clamp(min=0)
        h = torch.matmul(s["a"][at].float(), s["x"].float().unsqueeze(-1))
        d = torch.matmul(s["b"][at].float(), h)[..., 0] * s["scaling"][at][:, None]
        return {"y": torch.where(ids[:, None] >= 0, y + d, y).to(_BF)}
    for i in ids.unique().tolist():
        if i >= 0:
            rows = torch.nonzero(ids == i)[:, 0]
            h = torch.matmul(s["x"][rows].float(), s["a"][i].float().t())
            y[rows] += torch.matmul(h, s["b"][i].float().t()) * s["scaling"][i]
    return {"y": y.to(_BF)}


def _plain_sample(s):
    rows, V = s["logits"].shape
    z = s["logits"].float()
    if s["temperature"] is None and s["top_k"] is None and s["top_p"] is None and s["min_p"] is None:
        top, order = z, None        # the whole distribution needs no order
    else:
        top, order = torch.sort(z, dim=-1, descending=True, stable=True)
    # 64 bits: a draw lies next to a border between two tokens
    t = torch.ones(rows, device=_DEV) if s["temperature"] is None else s["temperature"]
    greedy = t <= 0
    w = torch.exp((top.double() - top.amax(-1, keepdim=True).double()) / torch.where(greedy, 1.0, t).double()[:, None])
    rank = torch.arange(V, device=_DEV)
    k = torch.full((rows,), V, device=_DEV) if s["top_k"] is None else s["top_k"].long()
    k = torch.where(greedy, 1, torch.where(k <= 0, V, k))
    w = torch.where((rank < k[:, None]) | (order is None), w, 0.0)
    if s["top_p"] is not None:
        total = w.cumsum(-1)
        inside = total - w < s["top_p"].double()[:, None] * total[:, -1:]
        w = torch.where(inside | (s["top_p"] >= 1)[:, None] | (rank == 0), w, 0.0)
    if s["min_p"] is not None:
        w = torch.where(w >= s["min_p"].double()[:, None], w, 0.0)
    if order is not None:
        w = torch.zeros_like(w).scatter_(1, order, w)
    total = w.cumsum(-1)
    past = total > s["uniforms"].double()[:, None] * total[:, -1:]
    last = torch.where(w > 0, rank, 0).amax(-1)
    token = torch.minimum(torch.where(past, rank, V).amin(-1), last)
    p = w.gather(1, token[:, None])[:, 0] / total[:, -1]
    return {"tokens": token.to(torch.int32), "logprobs": torch.log(p).float()}


def _own_run(s):
    import int4_group_quantized_q4_amd as w4
    case = s["case"]
    if case["op"] == "plan":
        w4.kv_cache_plan(s["lens"], s["new"], s["table"], case["page"], s["free"], s["free_count"], s["lens_out"],
                         s["free_count_out"], s["offsets"], s["slots"], s["positions"], s["row_seqs"])
        return {"lens": s["lens_out"], "table": s["table"], "free": s["free"], "offsets": s["offsets"],
                "free_count": s["free_count_out"], "slots": s["slots"], "positions": s["positions"],
                "row_seqs": s["row_seqs"]}
    if case["op"] == "rope":
        w4.w4a16_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], s["k_out"],
                      w4.W4_ROPE_HALF if case["layout"] == "half" else w4.W4_ROPE_INTERLEAVED, case["scale"])
        return {"q": s["q_out"]} if s["k"] is None else {"q": s["q_out"], "k": s["k_out"]}
    if case["op"] == "lora":
        if "ws" not in s:       # kept between calls, as a serving loop does
            need = w4.w4a16_lora_workspace(case["rows"], case["K"], case["N"], case["adapters"], case["rank"])
            s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device=_DEV)
        w4.w4a16_lora_add(s["x"], s["ids"], s["a"], s["b"], s["scaling"], s["y"], s["out"], s["ws"])
        return {"y": s["out"]}
    if "ws" not in s:
        need = w4.w4a16_sample_workspace(case["rows"], case["vocab"])
        s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device=_DEV)
    w4.w4a16_sample(s["logits"], s["uniforms"], s["tokens"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                    s["logprobs"], s["ws"])
    return {"tokens": s["tokens"], "logprobs": s["logprobs"]}


def run(state):
    if own:
        return _own_run(state)
    return {"plan": _plain_plan, "rope": _plain_rope, "lora": _plain_lora,
            "sample": _plain_sample}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the work
def work(case):
    if case["op"] == "plan":
        held, new = _plan_sizes(case)
        page = case["page"]
        pages = sum(-(-h // page) if t < 0 else -(-(h + t) // page) - -(-h // page) for h, t in zip(held, new))
        rows = sum(max(0, t) for t in new)
        return {"bytes": 16 * case["seqs"] + 8 * pages + 16 * rows, "flops": 4 * case["seqs"] + 8 * rows}
    if case["op"] == "rope":
        n = case["rows"] * (case["q_heads"] + case["k_heads"])
        return {"bytes": 4 * n * case["head_dim"] + 4 * case["rows"] + 2 * case["rotary"],
                "flops": 3 * n * case["rotary"]}
    if case["op"] == "lora":
        rows, K, N, R = case["rows"], case["K"], case["N"], case["rank"]
        # rows without an adapter are about one in ten, or one request in the prompt
        live = rows if rows == 1 else rows * case["adapters"] / (case["adapters"] + 1) if case["prompt"] else 0.9 * rows
        used = case["adapters"] * (1 - (1 - 1 / case["adapters"]) ** live)
        if case["prompt"]:
            used = min(case["adapters"], rows)
        return {"bytes": int(2 * live * K + 4 * rows * N + 2 * used * R * (K + N) + 4 * rows),
                "flops": int(2 * live * R * (K + N))}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 28 * case["rows"], "flops": 4 * n}


# ------------------------------------------------ the definitions in 64 bits
def _exact_plan(s):
    page = s["case"]["page"]
    lens, new, count = s["lens"].tolist(), s["new"].tolist(), s["free_count"].item()
    table, free, most = s["table"].cpu(), s["free"].tolist(), s["slots"].shape[0]
    for i, t in enumerate(new):
        if t < 0:
            for c in range(-(-lens[i] // page)):
                free[count] = table[i, c].item()
                count += 1
    out_lens, offsets, slots, positions, seqs = [], [0], [], [], []
    top, asked_pages, asked_rows = count, 0, 0
    for i, t in enumerate(new):
        if t < 0:
            out_lens.append(0)
            offsets.append(len(slots))
            continue
        have, need = -(-lens[i] // page), -(-(lens[i] + t) // page)
        asked_pages += need - have
        asked_rows += t
        fits = asked_pages <= top and asked_rows <= most
        if fits:
            for c in range(have, need):
                count -= 1
                table[i, c] = free[count]
            pages = table[i].tolist() if t else []
            for p in range(lens[i], lens[i] + t):
                slots.append(pages[p // page] * page + p % page)
                positions.append(p)
                seqs.append(i)
        out_lens.append(lens[i] + t if fits else lens[i])
        offsets.append(len(slots))
    pad = most - len(slots)
    put = lambda v, like: torch.tensor(v, dtype=like.dtype, device=_DEV)
    return {"lens": put(out_lens, s["lens"]), "table": table.to(_DEV), "free": put(free, s["free"]),
            "offsets": put(offsets, s["offsets"]), "free_count": put([count], s["free_count"]),
            "slots": put(slots + [-1] * pad, s["slots"]), "positions": put(positions + [0] * pad, s["positions"]),
            "row_seqs": put(seqs + [-1] * pad, s["row_seqs"])}


def _exact_rope(s):
    case, half = s["case"], s["case"]["rotary"] // 2
    # a pair as a complex number, turned by e^(i angle)
    angle = s["positions"].double().unsqueeze(1) * s["inv_freq"].double().unsqueeze(0)
    turn = torch.polar(torch.full_like(angle, case["scale"]), angle).unsqueeze(1)
    out = {}
    for name in ("q", "k"):
        if s[name] is None:
            continue
        x = s[name].double()
        lo = torch.arange(half, device=_DEV) * (1 if case["layout"] == "half" else 2)
        hi = lo + (half if case["layout"] == "half" else 1)
        z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * turn
        y = x.clone()
        y[..., lo] = z.real
        y[..., hi] = z.imag
        out[name] = y
    return out


def _exact_lora(s):
    y = s["y"].double()
    for i in range(s["a"].shape[0]):
        mine = s["ids"] == i
        if bool(mine.any()):
            h = s["x"][mine].double() @ s["a"][i].double().T
            y[mine] += s["scaling"][i].double() * (h @ s["b"][i].double().T)
    return {"y": y}


def _exact_sample(s):
    rows, V = s["logits"].shape
    tokens, logprobs = [], []
    value = lambda name, i, default: default if s[name] is None else s[name][i].item()
    for i in range(rows):
        z = s["logits"][i].double()
        t, k = value("temperature", i, 1.0), value("top_k", i, 0)
        ids = torch.argsort(-z, stable=True)
        if t <= 0:
            ids = ids[:1]
        elif 0 < k < V:
            ids = ids[:k]
        lp = torch.log_softmax(z[ids] / (t if t > 0 else 1.0), 0)
        p = value("top_p", i, 1.0)
        if p < 1:
            upto = torch.cumsum(torch.exp(lp), 0)
            keep = 1 + int((upto < p).sum())
            ids, lp = ids[:keep], lp[:keep]
        few = value("min_p", i, 0.0)
        if few > 0:
            keep = int((torch.exp(lp - lp[0]) >= few).sum())
            ids, lp = ids[:keep], lp[:keep]
        lp = lp - torch.logsumexp(lp, 0)
        ids, at = torch.sort(ids)
        lp = lp[at]
        upto = torch.cumsum(torch.exp(lp), 0)
        j = min(int((upto <= s["uniforms"][i].double() * upto[-1]).sum()), len(ids) - 1)
        tokens.append(ids[j])
        logprobs.append(lp[j])
    return {"tokens": torch.stack(tokens).to(torch.int32), "logprobs": torch.stack(logprobs)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rope": _exact_rope, "lora": _exact_lora, "sample": _exact_sample}[case["op"]](s)
