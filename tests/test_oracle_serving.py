"""Pins of oracle/serving.py: hand-computed plans, rotations against complex
numbers and torch, adapters against torch, draws against brute force."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from oracle import serving


def test_plan_by_hand():
    table = np.array([[5, 6, 0], [7, 0, 0], [2, 3, 0], [0, 0, 0]])
    free = np.array([11, 12, 13, 99, 99, 99])
    # 20 tokens + 13: one page more; 16 + 1: one more; an ended one gives 2, 3 back; a prompt of 16
    out = serving.plan([20, 16, 32, 0], [13, 1, -1, 16], table, 16, free, 3, 32)
    assert free.tolist() == [11, 12, 13, 2, 3, 99] and out["count"] == 2
    assert table.tolist() == [[5, 6, 3], [7, 2, 0], [2, 3, 0], [13, 0, 0]]
    assert out["lens"].tolist() == [33, 17, 0, 16]
    assert out["offsets"].tolist() == [0, 13, 14, 14, 30]
    assert out["slots"].tolist() == ([6 * 16 + p for p in range(4, 16)] + [3 * 16] + [2 * 16]
                                     + [13 * 16 + p for p in range(16)] + [-1, -1])
    assert out["positions"].tolist() == list(range(20, 33)) + [16] + list(range(16)) + [0, 0]
    assert out["row_seqs"].tolist() == [0] * 13 + [1] + [3] * 16 + [-1, -1]
    assert out["counters"] == (0, 0)


def test_plan_cut_and_bad_ones():
    free = np.array([4, 5])
    # the second sequence asks for more pages than there are; the third would fit, but comes behind it
    table = np.zeros((5, 2), dtype=np.int64)
    out = serving.plan([0, 0, 3, 40, -1], [16, 32, 1, 0, 2], table, 16, free, 2, 100)
    assert out["lens"].tolist() == [16, 0, 3, 40, -1] and out["offsets"].tolist() == [0, 16, 16, 16, 16, 16]
    assert out["count"] == 1 and out["counters"] == (2, 2)      # 40 > 2 pages and a negative length; two cut
    out = serving.plan([0, 0], [3, 3], np.zeros((2, 1), dtype=np.int64), 16, np.array([1, 2]), 2, 5)
    assert out["lens"].tolist() == [3, 0] and out["counters"] == (0, 1)         # rows run out
    free = np.array([8, 9])
    out = serving.plan([48], [-1], np.array([[1, 2, 3]]), 16, free, 1, 0)
    assert free.tolist() == [8, 1] and out["count"] == 2 and out["counters"] == (2, 0)      # two pages lost


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_rotation(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 48))
    f = (10000.0 ** (-np.arange(16) / 16)).astype(np.float32)
    p = [0, 1, 77, 12345, -3]
    y = serving.rope(x, p, f, interleaved, 1.5)
    lo = np.arange(16) * (2 if interleaved else 1)
    hi = lo + (1 if interleaved else 16)
    z = (x[..., lo] + 1j * x[..., hi]) * 1.5 * np.exp(1j * np.outer(p, f.astype(np.float64)))[:, None]
    assert np.allclose(y[..., lo], z.real, atol=1e-11) and np.allclose(y[..., hi], z.imag, atol=1e-11)
    assert np.array_equal(y[..., 32:], x[..., 32:])
    assert np.allclose(serving.rope(y, [-v for v in p], f, interleaved, 1.0)[..., :32], 1.5 * x[..., :32], atol=1e-11)


def test_rope_frequencies():
    f, s = w4.rope_frequencies(64, 500000.0)
    j = np.arange(32)
    assert f.dtype == torch.float32 and s == 1.0
    assert np.array_equal(f.numpy(), (500000.0 ** (-2.0 * j / 64)).astype(np.float32))
    lin, s = w4.rope_frequencies(64, 500000.0, "linear", 8.0)
    assert s == 1.0 and np.allclose(lin.numpy(), f.numpy() / 8.0, rtol=2 ** -23, atol=0)
    base, _ = w4.rope_frequencies(64, 500000.0, "base", 8.0)
    assert base[0] == 1.0 and np.isclose(float(base[-1]), float(f[-1]) / 8.0, rtol=1e-6)
    bands, s = w4.rope_frequencies(64, 500000.0, "bands", 8.0, trained=4096)
    turns = 4096 * f.numpy().astype(np.float64) / (2 * np.pi)
    assert np.isclose(s, 1 + 0.1 * np.log(8.0))
    assert np.array_equal(bands.numpy()[turns > 40], f.numpy()[turns > 40])
    assert np.allclose(bands.numpy()[turns < 0.6], f.numpy()[turns < 0.6] / 8.0, rtol=2 ** -23, atol=0)
    part = f.numpy() / bands.numpy()
    assert (np.diff(part) >= -1e-6).all() and part.min() >= 1 and part.max() <= 8 + 1e-5
    for bad in (dict(rotary_dim=63), dict(rotary_dim=0), dict(rotary_dim=64, factor=0.5),
                dict(rotary_dim=64, scaling="bands"), dict(rotary_dim=64, scaling="other"),
                dict(rotary_dim=2, scaling="base", factor=2.0),
                dict(rotary_dim=64, scaling="bands", trained=4096, fast=1.0, slow=1.0)):
        with pytest.raises(ValueError):
            w4.rope_frequencies(**bad)


def test_lora_add_against_torch():
    rng = np.random.default_rng(2)
    bits = lambda *s: oracle.bf16_from_f64(rng.standard_normal(s))
    x, a, b, y = bits(6, 64), bits(3, 8, 64), bits(3, 32, 8), bits(6, 32)
    ids, scaling = [2, -1, 0, 2, 3, 0], np.array([0.5, 9.0, 2.0], dtype=np.float32)
    out, bound = serving.lora_add(x, ids, a, b, scaling, y)
    d = lambda v: torch.from_numpy(oracle.bf16_bits_to_f64(v))
    for t, i in enumerate(ids):
        want = d(y)[t]
        if 0 <= i < 3:
            want = want + float(scaling[i]) * (d(b)[i] @ (d(a)[i] @ d(x)[t]))
            # at most K + rank + 8 roundings of 2^-24 of the sum of all terms' sizes
            size = abs(float(scaling[i])) * (d(b)[i].abs() @ (d(a)[i].abs() @ d(x)[t].abs())) + d(y)[t].abs()
            assert (bound[t] > 0).all() and (bound[t] <= (64 + 8 + 8) * 2.0 ** -24 * 2 * size.numpy()).all()
        assert np.allclose(out[t], want.numpy(), rtol=1e-13, atol=1e-13)


def test_sample_by_hand():
    ln = np.log
    z = [ln(1.0), ln(4.0), ln(2.0), ln(4.0), -np.inf, ln(0.5)]       # weights 1 4 2 4 0 .5 over 4
    draw = lambda **kw: serving.sample(z, **kw)
    assert draw(uniform=0.0)[0] == 0 and draw(uniform=0.999)[0] == 5
    assert [draw(uniform=u / 11.5)[0] for u in (0.9, 1.1, 4.9, 5.1, 6.9, 7.1, 10.9, 11.1)] == [0, 1, 1, 2, 2, 3, 3, 5]
    assert draw(temperature=0.0, uniform=0.9) == (1, 0.0, [1])
    assert draw(temperature=float("nan"))[0] == 1
    assert draw(top_k=1)[2] == [1] and draw(top_k=3)[2] == [1, 2, 3] and draw(top_k=100)[2] == [0, 1, 2, 3, 4, 5]
    assert draw(top_p=0.34)[2] == [1] and draw(top_p=0.36)[2] == [1, 3] and draw(top_p=0.0)[2] == [1]
    assert draw(top_k=3, top_p=0.79)[2] == [1, 3] and draw(top_k=3, top_p=0.81)[2] == [1, 2, 3]
    assert draw(min_p=0.2)[2] == [0, 1, 2, 3] and draw(min_p=0.3)[2] == [1, 2, 3] and draw(min_p=5.0)[2] == [1, 3]
    token, lp, kept = draw(temperature=0.5, uniform=0.5)             # squares: 1 16 4 16 0 .25
    assert kept == [0, 1, 2, 3, 4, 5] and token == 2 and np.isclose(lp, ln(4 / 37.25))
    assert serving.sample([np.nan, 1.0])[0] == -1 and serving.sample([-np.inf] * 3)[0] == -1
    assert serving.sample([0.0, np.inf, -np.inf, np.inf], uniform=0.6)[::2] == (3, [0, 1, 2, 3])
    assert serving.sample([0.0, -0.0, 0.0], top_k=2)[2] == [0, 1]


def test_sample_distribution():
    rng = np.random.default_rng(3)
    z = rng.standard_normal(7)
    p = torch.softmax(torch.from_numpy(z) / 0.7, 0).numpy()
    grid = (np.arange(20000) + 0.5) / 20000
    got = np.bincount([serving.sample(z, 0.7, uniform=u)[0] for u in grid], minlength=7) / len(grid)
    assert np.abs(got - p).max() < 1e-4
