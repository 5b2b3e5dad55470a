"""Host-side encoder/decoder of the key-value cache's page layout, written from
its description in include/w4a16.h (test infrastructure; independent of the
HIP code that reads and writes the layout on the GPU)."""

import numpy as np

FORMATS = ("bf16", "e4m3", "q4")


def block_bytes(form, page, D):
    return {"bf16": page * D * 2, "e4m3": page * (D + 4), "q4": page * (D // 2 + D // 16)}[form]


def page_bytes(form, page, heads, D):
    return heads * 2 * block_bytes(form, page, D)


def _code_index(form, page, D, is_v):
    """Byte offset in a block (and nibble shift for Q4) of the code of (token, dimension): [page, D]."""
    NG = D // 32
    U = {"bf16": 1, "e4m3": 2, "q4": min(4, NG)}[form]
    group_bytes = {"bf16": 16, "e4m3": 8, "q4": 4}[form]
    unit_lane = U * group_bytes
    tok = np.arange(page)[:, None]
    d = np.arange(D)[None, :]
    t, r = tok // 16, tok % 16
    g = d // 32
    unit = t * (NG // U) + g // U
    if is_v:
        a, j = r // 4, r % 4
        m, b = (d % 32) // 2, d % 2
        lane = 16 * a + m
        inner = {"bf16": (4 * b + j) * 2, "e4m3": 4 * b + j, "q4": j + 0 * b}[form]
        shift = 4 * b + 0 * r
    else:
        c, i = (d % 32) // 8, d % 8
        lane = 16 * c + r
        bit = 4 * (i // 2) + 16 * (i % 2)
        inner = {"bf16": 2 * i, "e4m3": i, "q4": bit // 8}[form]
        shift = bit % 8 + 0 * r
    off = (unit * 64 + lane) * unit_lane + (g % U) * group_bytes + inner
    return np.broadcast_to(off, (page, D)), np.broadcast_to(shift, (page, D)).astype(np.uint8)


def _scale_index(form, page, D):
    """Element index of the scale of (token[, group]) in the block's scale array."""
    tok = np.arange(page)
    if form == "e4m3":
        return tok
    NG = D // 32
    t, a, j = (tok // 16)[:, None], (tok % 16 // 4)[:, None], (tok % 4)[:, None]
    return ((t * 4 + a) * NG + np.arange(NG)[None, :]) * 4 + j


def decode_block(raw, form, page, D, is_v):
    """One block's bytes -> (codes [page, D], scales): as oracle.decode.cache_rows lays them out."""
    raw = np.asarray(raw, dtype=np.uint8)
    off, shift = _code_index(form, page, D, is_v)
    n = {"bf16": page * D * 2, "e4m3": page * D, "q4": page * D // 2}[form]
    if form == "bf16":
        return raw[off].astype(np.uint16) | (raw[off + 1].astype(np.uint16) << 8), None
    if form == "e4m3":
        return raw[off], raw[n:].view(np.float32)[_scale_index(form, page, D)]
    codes = (((raw[off] >> shift) & 0xF).astype(np.int16) - 8).astype(np.int8)
    return codes, raw[n:].view(np.uint16)[_scale_index(form, page, D)]


def encode_block(codes, scales, form, D, is_v):
    """codes [page, D] and scales -> the block's bytes."""
    page = codes.shape[0]
    out = np.zeros(block_bytes(form, page, D), dtype=np.uint8)
    off, shift = _code_index(form, page, D, is_v)
    n = {"bf16": page * D * 2, "e4m3": page * D, "q4": page * D // 2}[form]
    if form == "bf16":
        out[off] = codes & 0xFF
        out[off + 1] = codes >> 8
    elif form == "e4m3":
        out[off] = codes
        out[n:].view(np.float32)[_scale_index(form, page, D)] = scales
    else:
        np.bitwise_or.at(out, off, ((codes.astype(np.int16) + 8).astype(np.uint8) << shift).astype(np.uint8))
        out[n:].view(np.uint16)[_scale_index(form, page, D)] = scales
    return out


def decode_cache(raw, form, pages, page, heads, D):
    """Cache bytes -> {"k": (codes [pages, heads, page, D], scales), "v": ...}."""
    raw = np.asarray(raw, dtype=np.uint8).reshape(pages, heads, 2, block_bytes(form, page, D))
    out = {}
    for which, name in ((0, "k"), (1, "v")):
        got = [[decode_block(raw[p, h, which], form, page, D, which == 1) for h in range(heads)] for p in range(pages)]
        codes = np.array([[b[0] for b in row] for row in got])
        scales = None if form == "bf16" else np.array([[b[1] for b in row] for row in got])
        out[name] = (codes, scales)
    return out


def encode_cache(k, v, form):
    """(codes, scales) of k and v, [pages, heads, page, ...] -> cache bytes [pages, page bytes]."""
    pages, heads, page, D = k[0].shape
    out = np.zeros((pages, heads, 2, block_bytes(form, page, D)), dtype=np.uint8)
    for which, (codes, scales) in ((0, k), (1, v)):
        for p in range(pages):
            for h in range(heads):
                out[p, h, which] = encode_block(codes[p, h], None if scales is None else scales[p, h], form, D,
                                                which == 1)
    return out.reshape(pages, -1)
