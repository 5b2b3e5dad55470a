"""Oracle of what a decoder layer runs between the quantized matmuls: the
residual addition with RMS norm, the key-value cache's formats, and the
attention of one new token over cached rows (test infrastructure only).

[VG] "2. What you can quantize" names the KV cache beside weights and
activations; the pages fix neither encoding nor scales.  Readings taken:

  * norm: r = bf16(fl32(x + residual)); y = r * fl32(offset + w) /
    sqrt(mean(r^2) + eps) in fp64; bf16 form: y rounded; E4M3 form: scale =
    fl32(max|y| / 448) (1 where that is 0), codes E4M3(clamp(fl32(y / scale),
    +-448)); a row with a NaN or infinite y: scale NaN, codes 0.
  * cache rows: E4M3 per (token, head) row as fp8.quantize_rows; Q4 per group
    of 32: s = bf16(fl32(amax / 7)), codes clamp(rint(fl32(x / s)), -8, 7), 0
    where s is 0 (textbook_quantize with m = 7 and the step kept in bf16, the
    precision the library stores its group scales in); NaN or infinity in a
    row / group: scale NaN, codes 0.
  * attention: fp64 softmax over the attended rows, as code * scale unrounded.

Pinned by tests/test_oracle_decode.py.
"""

import numpy as np

from .bf16 import bf16_bits_to_f32, bf16_bits_to_f64, bf16_from_f32, bf16_from_f64
from .fp8 import E4M3_MAX, e4m3_decode, e4m3_encode

Q4_STEPS = 7


def add_rmsnorm(x_bits, residual_bits, weight_bits, eps, offset=0.0):
    """(r uint16 [rows, d], y float64 [rows, d])."""
    x = bf16_bits_to_f32(x_bits)
    with np.errstate(all="ignore"):
        r_bits = np.asarray(x_bits, dtype=np.uint16)
        if residual_bits is not None:
            r_bits = bf16_from_f32((x + bf16_bits_to_f32(residual_bits)).astype(np.float32))
        r = bf16_bits_to_f64(r_bits)
        w = (np.float32(offset) + bf16_bits_to_f32(weight_bits)).astype(np.float32).astype(np.float64)
        y = r * w / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + np.float64(np.float32(eps)))
    return r_bits, y


def quantize_f64_rows(y):
    """E4M3 codes uint8 and float32 scales of float64 rows."""
    y = np.asarray(y, dtype=np.float64)
    ok = np.all(np.isfinite(y), axis=1)
    safe = np.where(ok[:, None], y, 0.0)
    s = (np.max(np.abs(safe), axis=1) / E4M3_MAX).astype(np.float32)
    s = np.where(s > 0, s, np.float32(1.0))
    q = np.clip((safe / s[:, None].astype(np.float64)).astype(np.float32), -E4M3_MAX, E4M3_MAX)
    codes = e4m3_encode(q)
    codes = np.where(ok[:, None], codes, 0).astype(np.uint8)
    return codes, np.where(ok, s, np.float32(np.nan)).astype(np.float32)


def q4_rows(x_bits):
    """bf16 rows [..., D] -> (codes int8 [..., D], scale bits uint16 [..., D/32])."""
    x = bf16_bits_to_f32(np.asarray(x_bits, dtype=np.uint16))
    g = x.reshape(*x.shape[:-1], -1, 32)
    ok = np.all(np.isfinite(g), axis=-1)
    safe = np.where(ok[..., None], g, np.float32(0))
    s_bits = bf16_from_f32((np.max(np.abs(safe), axis=-1) / np.float32(Q4_STEPS)).astype(np.float32))
    s = bf16_bits_to_f32(s_bits)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = (safe / s[..., None]).astype(np.float32)
    q = np.where(s[..., None] > 0, np.clip(np.rint(r), -8, 7), 0).astype(np.int8)
    return q.reshape(x.shape), np.where(ok, s_bits, np.uint16(0x7FC0)).astype(np.uint16)


def cache_rows(x_bits, form):
    """bf16 rows [..., D] -> (codes, scales): ("bf16") the bits and None; ("e4m3") uint8 codes and float32 scales
    [...]; ("q4") int8 codes and uint16 scale bits [..., D/32]."""
    x_bits = np.asarray(x_bits, dtype=np.uint16)
    if form == "bf16":
        return x_bits, None
    if form == "q4":
        return q4_rows(x_bits)
    x = bf16_bits_to_f32(x_bits)
    ok = np.all(np.isfinite(x), axis=-1)
    safe = np.where(ok[..., None], x, np.float32(0))
    amax = np.max(np.abs(safe), axis=-1)
    s = np.where(amax > 0, amax / np.float32(E4M3_MAX), np.float32(1)).astype(np.float32)
    r = np.clip((safe / s[..., None]).astype(np.float32), -E4M3_MAX, E4M3_MAX)
    return e4m3_encode(r), np.where(ok, s, np.float32(np.nan)).astype(np.float32)


def row_values(codes, scales, form):
    """What codes and scales stand for, float64 (exact)."""
    if form == "bf16":
        return bf16_bits_to_f64(codes)
    if form == "e4m3":
        return e4m3_decode(codes) * np.asarray(scales, dtype=np.float64)[..., None]
    s = bf16_bits_to_f64(scales)
    return (np.asarray(codes, dtype=np.float64).reshape(*s.shape, 32) * s[..., None]).reshape(np.shape(codes))


def attention(q_bits, k, v, scale):
    """One sequence: q_bits uint16 [heads, D]; k, v float64 [n, kv_heads, D] (the attended rows).
    Returns (out float64 [heads, D], lse float64 [heads], p float64 [heads, n], s float64 [heads, n])."""
    q = bf16_bits_to_f64(q_bits)
    heads, D = q.shape
    n, kv_heads, _ = k.shape
    G = heads // kv_heads
    s = np.zeros((heads, n))
    for h in range(heads):
        s[h] = np.float64(np.float32(scale)) * (k[:, h // G] @ q[h])
    if n == 0:
        return np.zeros((heads, D)), np.full(heads, -np.inf), s, s
    m = np.max(s, axis=1, keepdims=True)
    e = np.exp(s - m)
    p = e / np.sum(e, axis=1, keepdims=True)
    out = np.stack([p[h] @ v[:, h // G] for h in range(heads)])
    return out, np.log(np.sum(e, axis=1)) + m[:, 0], p, s
