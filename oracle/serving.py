"""Oracle of a serving step's operators: the plan of its rows over the paged
cache, rotary positions, low-rank adapters beside a projection, and the draw of
a token from its logits (test infrastructure only).

The pages do not describe these; include/w4a16.h has the definitions, which are
followed here step by step in Python integers and fp64.  Pinned by
tests/test_oracle_serving.py.
"""

import numpy as np

from .bf16 import bf16_bits_to_f64


def plan(lens, new, table, page, free, count, max_rows):
    """One step; table [seqs, width] and free are changed in place.  Returns a
    dict of the call's outputs, `counters` (what it adds) among them."""
    width = table.shape[1]
    count = min(max(int(count), 0), len(free))
    lens, new = [int(n) for n in lens], [int(n) for n in new]
    ceil = lambda n: -(-n // page)
    bad = [n < 0 or n + max(t, 0) > width * page for n, t in zip(lens, new)]
    lost = 0
    for i, (n, t) in enumerate(zip(lens, new)):
        if t < 0 and not bad[i]:
            for c in range(ceil(n)):
                if count < len(free):
                    free[count] = table[i, c]
                    count += 1
                else:
                    lost += 1
    out = {"lens": [], "offsets": [0], "slots": [], "positions": [], "row_seqs": []}
    top, pages, rows, short = count, 0, 0, 0
    for i, (n, t) in enumerate(zip(lens, new)):
        if bad[i] or t < 0:
            out["lens"].append(n if bad[i] else 0)
            out["offsets"].append(len(out["slots"]))
            continue
        pages += ceil(n + t) - ceil(n)
        rows += t
        if pages <= top and rows <= max_rows:
            for c in range(ceil(n), ceil(n + t)):
                count -= 1
                table[i, c] = free[count]
            for p in range(n, n + t):
                out["slots"].append(int(table[i, p // page]) * page + p % page)
                out["positions"].append(p)
                out["row_seqs"].append(i)
            out["lens"].append(n + t)
        else:
            short += t > 0
            out["lens"].append(n)
        out["offsets"].append(len(out["slots"]))
    pad = max_rows - len(out["slots"])
    out["slots"] += [-1] * pad
    out["positions"] += [0] * pad
    out["row_seqs"] += [-1] * pad
    return dict({k: np.array(v, dtype=np.int64) for k, v in out.items()}, count=count,
                counters=(sum(bad) + lost, short))


def rope(x, positions, inv_freq, interleaved=False, scale=1.0):
    """x float64 [rows, heads, dim] -> float64, turned.  Angles are taken modulo a
    turn in extended precision where the platform has it."""
    half = len(inv_freq)
    wide = np.longdouble
    t = np.asarray(positions, dtype=wide)[:, None] * np.asarray(inv_freq, dtype=np.float32).astype(wide)[None, :]
    turn = wide("6.283185307179586476925286766559005768")
    t = t - np.rint(t / turn) * turn
    c = (np.cos(t) * np.float32(scale)).astype(np.float64)[:, None]
    s = (np.sin(t) * np.float32(scale)).astype(np.float64)[:, None]
    y = np.array(x, dtype=np.float64)
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y


def lora_add(x_bits, ids, a_bits, b_bits, scaling, y_bits):
    """(out float64 [rows, N], bound): out before its rounding, and what fp32 sums
    of any order may be off: K and rank additions of terms |x a| and |h b|."""
    x, y = bf16_bits_to_f64(x_bits), bf16_bits_to_f64(y_bits)
    a, b = bf16_bits_to_f64(a_bits), bf16_bits_to_f64(b_bits)
    adapters, rank, K = a.shape
    out, bound = y.copy(), np.zeros_like(y)
    for i in range(adapters):
        rows = np.nonzero(np.asarray(ids) == i)[0]
        if len(rows) == 0:
            continue
        s = np.float64(1.0 if scaling is None else np.float32(scaling[i]))
        h = x[rows] @ a[i].T
        out[rows] += s * (h @ b[i].T)
        off = (K + 2) * 2.0 ** -24 * (np.abs(x[rows]) @ np.abs(a[i]).T)
        bound[rows] = abs(s) * ((off + (rank + 4) * 2.0 ** -24 * np.abs(h)) @ np.abs(b[i]).T) + 2.0 ** -23 * (
            np.abs(y[rows]) + np.abs(out[rows]))
    return out, bound


def sample(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, uniform=0.0):
    """(token, log probability, ids kept) of one row of float64 logits."""
    z = np.asarray(z, dtype=np.float64)
    if np.isnan(z).any() or z.max() == -np.inf:
        return -1, np.nan, []
    order = np.lexsort((np.arange(len(z)), -z))
    temperature, top_p, min_p, uniform = (float(np.float32(v)) for v in (temperature, top_p, min_p, uniform))
    if not temperature > 0:
        return int(order[0]), 0.0, [int(order[0])]
    m = z[order[0]]
    with np.errstate(all="ignore"):
        d = z - m
        w = np.where(z == m, 1.0, np.where(d == -np.inf, 0.0, np.exp(d / temperature)))
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        sums = np.cumsum(w[order])
        order = order[:1 + int(np.sum(sums < max(top_p, 0.0) * sums[-1]))]
    if min_p > 0:
        order = order[w[order] >= min(min_p, 1.0)]
    kept = np.sort(order)
    sums = np.cumsum(w[kept])
    uniform = min(max(uniform, 0.0), 1.0) if uniform == uniform else 0.0
    past = np.nonzero(sums > uniform * sums[-1])[0]
    at = past[0] if len(past) else np.nonzero(w[kept] > 0)[0][-1]
    return int(kept[at]), float(np.log(w[kept[at]] / sums[-1])), [int(i) for i in kept]
