"""Pins of oracle/decode.py (norm, cache formats, one-token attention) and of
the cache layout's host decoder, on the CPU."""

import numpy as np
import pytest
import torch

import kv_layout
import oracle
from oracle import decode, fp8
from oracle.bf16 import bf16_bits_to_f64, bf16_from_f64


def rnd(seed, *shape):
    return bf16_from_f64(np.random.default_rng(seed).standard_normal(shape))


def test_norm_against_torch_float64():
    x, e, w = rnd(1, 7, 96), rnd(2, 7, 96), rnd(3, 96)
    t = lambda b: torch.from_numpy(bf16_bits_to_f64(b))
    r, y = decode.add_rmsnorm(x, e, w, 1e-5, 1.0)
    rt = (t(x).float() + t(e).float()).to(torch.bfloat16).double()
    assert np.array_equal(bf16_bits_to_f64(r), rt.numpy())
    wt = (1.0 + t(w).float()).double()
    want = torch.nn.functional.rms_norm(rt, (96,), None, float(np.float32(1e-5))) * wt
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-14)


def test_norm_closed_forms():
    """A constant row c with unit weights has y = c / sqrt(c^2 + eps); a row of
    zeros is zero, with scale 1; without a residual r is x."""
    x = np.repeat(bf16_from_f64(np.array([[3.0], [-0.5], [0.0]])), 32, axis=1)
    one = bf16_from_f64(np.ones(32))
    r, y = decode.add_rmsnorm(x, None, one, 0.25)
    assert np.array_equal(r, x)
    np.testing.assert_allclose(y[:, 0], [3 / np.sqrt(9.25), -0.5 / np.sqrt(0.5), 0.0], rtol=1e-15)
    q, s = decode.quantize_f64_rows(y)
    assert s[2] == 1.0 and not q[2].any()
    assert (q[0] == 0x7E).all() and (q[1] == 0xFE).all()      # +-448: every element is the row's amax


def test_norm_poison_rows():
    x = rnd(4, 3, 64)
    x[0, 5], x[1, 9] = 0x7F80, 0x7FC0                        # infinity, NaN
    q, s = decode.quantize_f64_rows(decode.add_rmsnorm(x, None, rnd(5, 64), 1e-6)[1])
    assert np.isnan(s[:2]).all() and not q[:2].any() and np.isfinite(s[2])


def test_cache_formats_agree_with_the_librarys_quantizers():
    x = rnd(6, 5, 3, 64)
    c, s = decode.cache_rows(x, "e4m3")
    cr, sr = fp8.quantize_rows(x.reshape(15, 64))
    assert np.array_equal(c.reshape(15, 64), cr) and np.array_equal(s.reshape(15), sr)
    c, s = decode.cache_rows(x, "q4")
    g = oracle.bf16_bits_to_f32(x).reshape(-1, 32)
    _, step = oracle.textbook_quantize(g, 7)
    assert np.array_equal(s.reshape(-1), oracle.bf16_from_f32(step[:, 0]))
    v = decode.row_values(c, s, "q4").reshape(-1, 32)
    sf = bf16_bits_to_f64(s.reshape(-1))[:, None]
    assert (np.abs(v - g) <= sf * 0.5 + 2.0 ** -8 * 7 * sf).all()   # half a step, plus what the step's rounding moves


def test_cache_special_groups():
    x = np.zeros((1, 64), dtype=np.uint16)
    c, s = decode.cache_rows(x, "q4")
    assert not c.any() and not s.any()
    x[0, 3] = 0x7F80
    c, s = decode.cache_rows(x, "q4")
    assert s[0, 0] == 0x7FC0 and s[0, 1] == 0 and not c.any()
    c, s = decode.cache_rows(x, "e4m3")
    assert np.isnan(s[0]) and not c.any()


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout_roundtrip(form, D):
    """Every code has a place of its own and the decoder finds it again."""
    pages, heads, page = 2, 2, 32
    kc = decode.cache_rows(rnd(7, pages, heads, page, D), form)
    vc = decode.cache_rows(rnd(8, pages, heads, page, D), form)
    raw = kv_layout.encode_cache(kc, vc, form)
    assert raw.shape == (pages, kv_layout.page_bytes(form, page, heads, D))
    got = kv_layout.decode_cache(raw, form, pages, page, heads, D)
    for want, have in ((kc, got["k"]), (vc, got["v"])):
        assert np.array_equal(want[0], have[0])
        assert form == "bf16" or np.array_equal(want[1], have[1])


def test_layout_documented_offsets():
    """Single codes by hand.  head_dim 128, Q4, page 32: token 21 (t 1, r 5 = 4*1 + 1).
    K dimension 75 = 32*2 + 11 (g 2, c 1, i 3): unit 1, lane 21, part 2, code 3 at bit 4*1 + 16 = 20.
    V dimension 75 (m 5, b 1): unit 1, lane 16*1 + 5, part 2, byte 1, high nibble."""
    codes = np.full((32, 128), -8, dtype=np.int8)
    codes[21, 75] = 3
    s = np.zeros((32, 4), dtype=np.uint16)
    s[21, 2] = 0x3F80
    k = kv_layout.encode_block(codes, s, "q4", 128, False)
    v = kv_layout.encode_block(codes, s, "q4", 128, True)
    at = 2048 + ((1 * 4 + 1) * 4 + 2) * 4 * 2 + 1 * 2
    assert list(np.nonzero(k)[0]) == [(64 + 21) * 16 + 8 + 2, at, at + 1] and k[(64 + 21) * 16 + 10] == 0xB0
    assert list(np.nonzero(v)[0]) == [(64 + 21) * 16 + 8 + 1, at, at + 1] and v[(64 + 21) * 16 + 9] == 0xB0


def test_attention_against_torch():
    rng = np.random.default_rng(9)
    heads, kv, D, n = 6, 2, 64, 37
    q, k, v = rnd(10, heads, D), rng.standard_normal((n, kv, D)), rng.standard_normal((n, kv, D))
    out, lse, p, s = decode.attention(q, k, v, 0.125)
    kt = torch.from_numpy(k).repeat_interleave(3, 1).permute(1, 0, 2)
    vt = torch.from_numpy(v).repeat_interleave(3, 1).permute(1, 0, 2)
    qt = torch.from_numpy(bf16_bits_to_f64(q))[:, None]
    want = torch.nn.functional.scaled_dot_product_attention(qt, kt, vt, scale=0.125)[:, 0]
    np.testing.assert_allclose(out, want.numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse, torch.logsumexp((qt * 0.125) @ kt.transpose(1, 2), -1)[:, 0].numpy(), rtol=1e-13)
    out, lse, _, _ = decode.attention(q, k[:0], v[:0], 0.125)
    assert not out.any() and np.isneginf(lse).all()
