"""GPU parity of the residual addition with RMS norm (bf16 and E4M3 output)
against oracle/decode.py.

Tolerances.  The kernel's sums and products are 64-bit, so y carries a few
2^-52; the bf16 form rounds to fp32 and then to bf16: at most half a bf16 step
plus half an fp32 step, relative 2^-8 + 2^-24 of the value (2^-134 + 2^-150
below the normal range).  The E4M3 form's quotient is rounded to fp32 and then
to a code, on both sides: equal codes and scales unless a quotient's 64-bit
error crosses an fp32 rounding border (chance about 2^-27 an element), so they
are compared exactly."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from oracle import decode
from gpu_util import bf16_dev, bits_host, dev, say

pytestmark = pytest.mark.gpu


def rnd(rng, *shape, sigma=1.0):
    return oracle.bf16_from_f64(sigma * rng.standard_normal(shape))


def check_bf16(y, want):
    got = oracle.bf16_bits_to_f64(bits_host(y))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    bound = np.abs(want[ok]) * (2.0 ** -8 + 2.0 ** -24) + 2.0 ** -134 + 2.0 ** -150
    assert (np.abs(got[ok] - want[ok]) <= bound).all()


SIZES = [(1, 32), (1, 2816), (3, 2048), (64, 2816), (5, 2080), (7, 4096), (2, 8192), (33, 8224), (2, 20000), (301, 96)]


@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("residual,offset", [(True, 0.0), (False, 1.0)])
def test_norm(rows, d, residual, offset):
    say("[norm] rows=%d d=%d residual=%s" % (rows, d, residual))
    rng = np.random.default_rng(rows * 10007 + d)
    x, w = rnd(rng, rows, d), rnd(rng, d, sigma=0.3)
    e = rnd(rng, rows, d, sigma=4.0) if residual else None
    r, y = decode.add_rmsnorm(x, e, w, 1e-5, offset)
    xd, wd, ed = bf16_dev(x), bf16_dev(w), None if e is None else bf16_dev(e)
    got, sum_ = w4.add_rmsnorm(xd, ed, wd, 1e-5, offset)
    q, s, sum2 = w4.add_rmsnorm_quantize(xd, ed, wd, 1e-5, offset)
    torch.cuda.synchronize()
    check_bf16(got, y)
    qr, sr = decode.quantize_f64_rows(y)
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)
    assert np.array_equal(bits_host(sum_), r) and np.array_equal(bits_host(sum2), r)
    assert np.array_equal(bits_host(xd), x)        # inputs stay


def test_norm_quantize_matches_quantize_rows_where_y_is_bf16():
    """With weights 1 and rows of +-c the norm is +-1 exactly (eps 0, c a power
    of two): the fused codes are w8a8_quantize_rows' of those bf16 rows."""
    rng = np.random.default_rng(5)
    y = np.where(rng.random((9, 128)) < 0.5, -1.0, 1.0)
    x = oracle.bf16_from_f64(y * 2.0 ** rng.integers(-20, 20, (9, 1)))
    q, s, _ = w4.add_rmsnorm_quantize(bf16_dev(x), None, bf16_dev(oracle.bf16_from_f64(np.ones(128))), 0.0)
    q2 = torch.empty_like(q)
    s2 = torch.empty_like(s)
    w4.w8a8_quantize_rows(bf16_dev(oracle.bf16_from_f64(y)), q2, s2)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_norm_special_rows():
    """Zeros, the smallest and largest magnitudes, a sum that overflows bf16, infinities and NaN; other rows of the
    call are not touched by them."""
    rng = np.random.default_rng(6)
    x, e, w = rnd(rng, 9, 96), rnd(rng, 9, 96), rnd(rng, 96)
    x[0], e[0] = 0, 0
    x[1], e[1] = 1, 0x8000                          # the smallest subnormal, minus zero
    x[2], e[2] = 0x7F7F, 0                          # the largest finite value
    x[3, 7], e[3, 7] = 0x7F7F, 0x7F7F               # overflows to infinity
    x[4, 95] = 0x7FC1
    x[5, 0] = 0xFF80
    x[6, 1], e[6, 1] = 0x7F80, 0xFF80               # inf - inf
    for eps in (1e-6, 0.0):
        r, y = decode.add_rmsnorm(x, e, w, eps)
        got, sum_ = w4.add_rmsnorm(bf16_dev(x), bf16_dev(e), bf16_dev(w), eps)
        q, s, _ = w4.add_rmsnorm_quantize(bf16_dev(x), bf16_dev(e), bf16_dev(w), eps)
        torch.cuda.synchronize()
        rf = oracle.bf16_bits_to_f64
        np.testing.assert_array_equal(rf(bits_host(sum_)), rf(r))
        check_bf16(got, y)
        qr, sr = decode.quantize_f64_rows(y)
        np.testing.assert_array_equal(s.cpu().numpy(), sr)
        assert np.array_equal(q.cpu().numpy(), qr)


@pytest.mark.parametrize("d", [2816, 20000])
def test_norm_in_place(d):
    """y over x, sum over the residual; and y over the residual, sum over x."""
    rng = np.random.default_rng(d)
    x, e, w = rnd(rng, 6, d), rnd(rng, 6, d), rnd(rng, d)
    r, y = decode.add_rmsnorm(x, e, w, 1e-6)
    wd = bf16_dev(w)
    a, b = bf16_dev(x), bf16_dev(e)
    w4.w4a16_add_rmsnorm(a, b, wd, 1e-6, b, a)
    check_bf16(a, y)
    assert np.array_equal(bits_host(b), r)
    a, b = bf16_dev(x), bf16_dev(e)
    w4.w4a16_add_rmsnorm(a, b, wd, 1e-6, a, b)
    check_bf16(b, y)
    assert np.array_equal(bits_host(a), r)
    a, b = bf16_dev(x), bf16_dev(e)
    w4.w4a16_add_rmsnorm(a, b, wd, 1e-6, None, a)      # the sum is not kept
    check_bf16(a, y)
    assert np.array_equal(bits_host(b), e)


def test_norm_stream_and_graph():
    """On a stream of its own and replayed from a graph after the inputs changed."""
    rng = np.random.default_rng(8)
    w = bf16_dev(rnd(rng, 2816))
    x = torch.empty(17, 2816, dtype=torch.bfloat16, device=dev())
    e, y, r = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    q, s = torch.empty(17, 2816, dtype=torch.uint8, device=dev()), torch.empty(17, device=dev())
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    x.zero_(), e.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        w4.w4a16_add_rmsnorm(x, e, w, 1e-6, r, y)
        w4.w8a8_add_rmsnorm_quantize(x, e, w, 1e-6, None, q, s)
    for _ in range(3):
        xb, eb = rnd(rng, 17, 2816), rnd(rng, 17, 2816)
        x.copy_(bf16_dev(xb)), e.copy_(bf16_dev(eb))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        rr, yr = decode.add_rmsnorm(xb, eb, bits_host(w), 1e-6)
        check_bf16(y, yr)
        assert np.array_equal(bits_host(r), rr)
        qr, sr = decode.quantize_f64_rows(yr)
        assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)


def test_norm_leaves_neighbours():
    rng = np.random.default_rng(11)
    buf = torch.full((8, 96), 7.0, dtype=torch.bfloat16, device=dev())
    x = bf16_dev(rnd(rng, 5, 96))
    w4.w4a16_add_rmsnorm(x, None, bf16_dev(rnd(rng, 96)), 1e-6, None, buf[1:6])
    torch.cuda.synchronize()
    assert (buf[0] == 7).all() and (buf[6:] == 7).all()


def test_norm_largest():
    """The longest row, and more rows than one launch takes (2^22): the rows around the border and at the end."""
    rng = np.random.default_rng(41)
    d = 1 << 20
    x, w = rnd(rng, 1, d), rnd(rng, d, sigma=0.3)
    _, y = decode.add_rmsnorm(x, None, w, 1e-5, 0.0)
    got, _ = w4.add_rmsnorm(bf16_dev(x), None, bf16_dev(w), 1e-5)
    q, s, _ = w4.add_rmsnorm_quantize(bf16_dev(x), None, bf16_dev(w), 1e-5)
    check_bf16(got, y)
    qr, sr = decode.quantize_f64_rows(y)
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)
    rows, d = (1 << 22) + 5, 32
    block = rnd(rng, 4096, d)
    xd = bf16_dev(block).repeat(-(-rows // 4096), 1)[:rows].contiguous()
    w = rnd(rng, d, sigma=0.3)
    _, y = decode.add_rmsnorm(block, None, w, 1e-5, 0.0)
    got, _ = w4.add_rmsnorm(xd, None, bf16_dev(w), 1e-5)
    q, s, _ = w4.add_rmsnorm_quantize(xd, None, bf16_dev(w), 1e-5)
    qr, sr = decode.quantize_f64_rows(y)
    for at in (0, (1 << 22) - 3, (1 << 22) + 1):
        part = slice(at, min(at + 5, rows))
        pick = np.arange(part.start, part.stop) % 4096
        check_bf16(got[part], y[pick])
        assert np.array_equal(s[part].cpu().numpy(), sr[pick]) and np.array_equal(q[part].cpu().numpy(), qr[pick])
