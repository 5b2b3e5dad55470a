"""GPU parity of w4a16_rope against oracle/serving.py.

Tolerance.  cos and sin are good to 4 fp32 roundings (the angle's own, the
function's two, the scale's), the two products and their sum to 2 more: with
half a step 2^-24 each, at most 6 * 2^-24 * scale * (|a| + |b|), taken as 2^-21;
the rounding to bf16 adds 2^-8 of the value (2^-134 below the normal range).  An
angle t keeps max(1, t) 2^-52 beyond that."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from oracle import serving
from gpu_util import bf16_dev, bits_host, dev, say

pytestmark = pytest.mark.gpu


def rnd(rng, *shape):
    return oracle.bf16_from_f64(rng.standard_normal(shape))


def check(got, x_bits, positions, freq, layout, scale):
    x = oracle.bf16_bits_to_f64(x_bits)
    want = serving.rope(x, positions, freq, layout == w4.W4_ROPE_INTERLEAVED, scale)
    r = 2 * len(freq)
    size = np.abs(x)
    if layout == w4.W4_ROPE_INTERLEAVED:
        pair = size[..., 0:r:2] + size[..., 1:r:2]
        pair = np.repeat(pair, 2, -1)
    else:
        pair = np.tile(size[..., :r // 2] + size[..., r // 2:r], 2)
    angle = np.abs(np.outer(np.asarray(positions, dtype=np.float64), freq.astype(np.float64)))
    angle = np.maximum(1, angle) * 2.0 ** -52
    angle = (np.repeat(angle, 2, -1) if layout == w4.W4_ROPE_INTERLEAVED else np.tile(angle, 2))[:, None]
    y = oracle.bf16_bits_to_f64(bits_host(got))
    bound = np.abs(want[..., :r]) * 2.0 ** -8 + (2.0 ** -21 + angle) * abs(scale) * pair * (1 + 2.0 ** -8) + 2.0 ** -134
    assert (np.abs(y[..., :r] - want[..., :r]) <= bound).all()
    assert np.array_equal(bits_host(got)[..., r:], x_bits[..., r:])       # the dimensions behind stay as they are


CASES = [  # rows, q heads, k heads, dim, rotary
    (1, 1, 1, 16, 16), (1, 32, 8, 128, 128), (2, 3, 0, 64, 32), (3, 5, 5, 80, 16), (7, 4, 1, 80, 80),
    (64, 32, 8, 128, 128), (5, 1, 1, 512, 512), (33, 16, 4, 256, 128), (300, 2, 1, 64, 48), (1000, 1, 1, 16, 16),
    (70, 64, 64, 256, 256), (9, 17, 3, 96, 96), (2049, 8, 2, 128, 64)]


@pytest.mark.parametrize("rows,hq,hk,dim,rot", CASES)
@pytest.mark.parametrize("layout", [w4.W4_ROPE_HALF, w4.W4_ROPE_INTERLEAVED])
def test_rope(rows, hq, hk, dim, rot, layout):
    say("[rope] rows=%d heads=%d+%d dim=%d rotary=%d layout=%d" % (rows, hq, hk, dim, rot, layout))
    rng = np.random.default_rng(rows * 1009 + dim + rot)
    q, k = rnd(rng, rows, hq, dim), rnd(rng, rows, hk, dim)
    p = rng.integers(0, 200000, rows)
    f = (10000.0 ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32)
    scale = 1.0 if rows % 2 else 1.25
    pd, fd = torch.tensor(p, dtype=torch.int32, device=dev()), torch.from_numpy(f).to(dev())
    qo, ko = w4.rope(bf16_dev(q), bf16_dev(k) if hk else None, pd, fd, layout, scale)
    # slices of a wider buffer, turned in place
    wide = rnd(rng, rows, (hq + hk + 1) * dim)
    wide[:, 8:8 + hq * dim] = q.reshape(rows, -1)
    wide[:, 8 + hq * dim:8 + (hq + hk) * dim] = k.reshape(rows, -1)
    w = bf16_dev(wide)
    qs, ks = w[:, 8:8 + hq * dim].view(rows, hq, dim), w[:, 8 + hq * dim:8 + (hq + hk) * dim].view(rows, hk, dim)
    w4.w4a16_rope(qs, ks if hk else None, pd, fd, qs, ks if hk else None, layout, scale)
    torch.cuda.synchronize()
    check(qo, q, p, f, layout, scale)
    if hk:
        check(ko, k, p, f, layout, scale)
        assert np.array_equal(bits_host(ks), bits_host(ko))
    assert np.array_equal(bits_host(qs), bits_host(qo))
    after = bits_host(w)
    assert np.array_equal(after[:, :8], wide[:, :8]) and np.array_equal(after[:, 8 + (hq + hk) * dim:],
                                                                        wide[:, 8 + (hq + hk) * dim:])


@pytest.mark.parametrize("layout", [w4.W4_ROPE_HALF, w4.W4_ROPE_INTERLEAVED])
def test_far_negative_and_zero_positions(layout):
    rng = np.random.default_rng(3)
    p = [0, 1, -1, 5, 2 ** 20, 2 ** 24 + 1, -2 ** 24 - 1, 2 ** 31 - 1, -2 ** 31, 999999999]
    x = rnd(rng, len(p), 2, 64)
    f = np.concatenate([[1.0, 0.0, 3.0e-7, 100.0], 500000.0 ** (-2.0 * np.arange(28) / 64)]).astype(np.float32)
    y, _ = w4.rope(bf16_dev(x), None, torch.tensor(p, dtype=torch.int32, device=dev()), torch.from_numpy(f).to(dev()),
                   layout)
    torch.cuda.synchronize()
    check(y, x, p, f, layout, 1.0)
    assert np.array_equal(bits_host(y)[0], x[0])          # no turn


def test_quarter_turns():
    """Angles next to quarter turns, where sine or cosine nearly vanish: their relative accuracy shows where the other
    product is zero."""
    f = np.zeros(8, dtype=np.float32)
    f[:] = [np.pi / 2, np.pi, 1.5 * np.pi, 2 * np.pi, np.pi / 4, 0.75 * np.pi, 7.0, 355.0 / 113.0]
    p = np.arange(0, 4096)
    rng = np.random.default_rng(4)
    x = np.zeros((len(p), 1, 16), dtype=np.uint16)
    x[:, 0, :8] = oracle.bf16_from_f64(np.exp(rng.uniform(-1, 1, (len(p), 8))))
    y, _ = w4.rope(bf16_dev(x), None, torch.tensor(p, dtype=torch.int32, device=dev()), torch.from_numpy(f).to(dev()))
    torch.cuda.synchronize()
    got = oracle.bf16_bits_to_f64(bits_host(y))
    want = serving.rope(oracle.bf16_bits_to_f64(x), p, f)
    # each output is one product: 2^-8 of it from the bf16 rounding, 2^-21 from cos or sin, and the angle's own error
    # (t 2^-52, at most 2^18) times |a|
    a = np.tile(np.abs(oracle.bf16_bits_to_f64(x[..., :8])), 2)
    assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -20) + a * 2.0 ** -34).all()


def test_special_values():
    """NaN and infinities stay with their pairs; rows and heads beside them do not change."""
    rng = np.random.default_rng(5)
    x = rnd(rng, 4, 3, 64)
    f = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    p = torch.tensor([3, 10, 500, 7], dtype=torch.int32, device=dev())
    fd = torch.from_numpy(f).to(dev())
    good, _ = w4.rope(bf16_dev(x), None, p, fd)
    bad = x.copy()
    bad[1, 2, 5], bad[2, 0, 40], bad[3, 1, 0] = 0x7FC0, 0x7F80, 0xFF80
    got, _ = w4.rope(bf16_dev(bad), None, p, fd)
    torch.cuda.synchronize()
    g, h = oracle.bf16_bits_to_f64(bits_host(got)), oracle.bf16_bits_to_f64(bits_host(good))
    touched = np.zeros(g.shape, dtype=bool)
    for r, n, j in ((1, 2, 5), (2, 0, 8), (3, 1, 0)):
        touched[r, n, j] = touched[r, n, j + 32] = True
    assert not np.isfinite(g[touched]).any() and np.array_equal(g[~touched], h[~touched])


def test_inverse_turn_scales_back():
    """Turning by -p after p gives the row back up to two roundings."""
    rng = np.random.default_rng(6)
    x = rnd(rng, 50, 4, 128)
    p = torch.tensor(rng.integers(0, 100000, 50), dtype=torch.int32, device=dev())
    f, s = w4.rope_frequencies(128, 10000.0, "bands", 4.0, trained=8192)
    f = f.to(dev())
    y, _ = w4.rope(bf16_dev(x), None, p, f, scale=s)
    z, _ = w4.rope(y, None, -p, f, scale=1.0 / s)
    torch.cuda.synchronize()
    a, b = oracle.bf16_bits_to_f64(x), oracle.bf16_bits_to_f64(bits_host(z))
    size = np.tile(np.abs(a[..., :64]) + np.abs(a[..., 64:]), 2)
    assert (np.abs(a - b) <= size * (2 * 2.0 ** -8 + 2.0 ** -8 * 2.0 ** -8 + 2.0 ** -19)).all()


def test_graph_and_stream():
    rng = np.random.default_rng(7)
    x = bf16_dev(rnd(rng, 40, 6, 64))
    p = torch.zeros(40, dtype=torch.int32, device=dev())
    f = w4.rope_frequencies(64)[0].to(dev())
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4a16_rope(x, None, p, f, out, None)
    for i in range(4):
        p.add_(1000 + i)
        x.mul_(-1)
        g.replay()
        want, _ = w4.rope(x, None, p, f)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
