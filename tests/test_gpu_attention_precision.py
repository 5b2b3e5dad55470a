"""The attention's arithmetic, where the output's own rounding does not hide it.

Two positions whose values nearly cancel: an output far below A = sum_t p_t
|v_t| is rounded by far less than A's last bits, so what is left of the
difference to 64 bits is the kernel's.  Relative to A, with s the scores, S =
scale * sum |q_i| |k_i| (at most 2^-6 here), n = 2:
  score      D + 8 fp32 roundings: (D + 8) 2^-23 S;
  p          the exponent (two roundings of the score's size, one of up to 8,
             the distance to the running reference) and the exponential:
             2^-22 |s| + 8 ln 2 2^-24 + 2^-22;
  p times V's scale  2^-24;
  products   three terms for each of n positions, a rounding (or a truncation:
             twice as much) for each, and the accumulator's and its rescaling's:
             (3 n + 3) 2^-23;
relative to the output: the sum l has p's errors and 20 roundings, the division
two, and the output half a bf16 step, 2^-8."""

import numpy as np
import pytest

import int4_group_quantized_q4_amd as w4  # noqa: F401
import kv_layout
import oracle
from oracle import decode
from gpu_util import bits_host, say, to_dev
from test_gpu_attention import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,group", [(64, 2), (128, 1), (128, 6), (256, 2)])
def test_cancelling_values(form, D, group):
    say("[attn precision] %s D=%d" % (form, D))
    s = Setup(form, [2] * 192, 2, group, D, 16, seed=D + group)
    s.scale = 2.0 ** -14
    got = oracle.bf16_bits_to_f64(bits_host(s.run()[0]))
    small = 0
    for i in range(len(s.lens)):
        (k, km), (v, vm) = s.rows(i, 0)
        ref, _, p, sc = decode.attention(s.q[i], k, v, s.scale)
        qa = np.abs(oracle.bf16_bits_to_f64(s.q[i]))
        for h in range(s.heads):
            S = s.scale * np.max(km[:, h // group] @ qa[h])
            assert S < 2.0 ** -6
            ep = (D + 8) * 2.0 ** -23 * S + 2.0 ** -22 * np.max(np.abs(sc[h])) + (8 * np.log(2) + 4) * 2.0 ** -24
            A = p[h] @ vm[:, h // group]
            rel = ep + 2.0 ** -24 + 9 * 2.0 ** -23
            bound = (2.0 ** -8 + ep + 22 * 2.0 ** -24) * np.abs(ref[h]) + rel * A
            err = np.abs(got[i, h] - ref[h])
            assert (err <= bound).all(), (i, h, np.max(err / bound), np.max(err / A))
            small += np.sum(np.abs(ref[h]) < 2.0 ** -11 * A)
    assert small >= 8       # outputs whose own rounding is below 2^-19 of A


def _put(s, which, edit):
    """Replace the codes and scales of the cache's K (0) or V (1)."""
    codes, scales = (s.k, s.v)[which]
    codes, scales = codes.copy(), scales.copy()
    edit(codes, scales)
    if which:
        s.v = (codes, scales)
    else:
        s.k = (codes, scales)
    s.cache = to_dev(kv_layout.encode_cache(s.k, s.v, "q4"))


@pytest.mark.parametrize("D,group", [(64, 1), (64, 16), (128, 4), (128, 8), (128, 16), (256, 4), (256, 5), (256, 9)])
def test_q4_zeros_beside_a_large_scale(D, group):
    """A group whose scale one large value set: its other codes are 0, and what the other position has in their places
    comes out as it is.  Equal scores (scale 0) and scales 2^18 and 1: sums of codes -8 .. 7 times them, with the 8 that
    is added to a code and taken off again, are integers below 2^23, so every step is exact."""
    s = Setup("q4", [2] * 12, 2, group, D, 16, seed=D + group)
    s.scale = 0.0
    rng = np.random.default_rng(D)

    def edit(codes, scales):
        p = s.table[:, 0]
        codes[p, :, 0] = 0
        codes[p, :, 0, ::32] = 7
        codes[p, :, 1] = rng.integers(-8, 8, codes[p, :, 1].shape)
        scales[p, :, 0] = oracle.bf16_from_f64(np.float64(2.0 ** 18))
        scales[p, :, 1] = oracle.bf16_from_f64(np.float64(1.0))

    _put(s, 1, edit)
    got = bits_host(s.run()[0])
    for i in range(len(s.lens)):
        v = s.rows(i, 0)[1][0]
        want = oracle.bf16_from_f64((v[0] + v[1]) / 2.0)
        assert np.array_equal(got[i], np.repeat(want, group, axis=0)), i


@pytest.mark.parametrize("D,group", [(64, 1), (64, 16), (128, 4), (128, 8), (128, 16), (256, 4), (256, 5), (256, 9)])
def test_q4_zeros_beside_a_large_query(D, group):
    """The same for the scores: large elements of q meet codes 0.  q is a multiple of 2^-7 (2^12 where the code is 0),
    the scales are 1: the sums, with the codes' 8, are multiples of 2^-7 below 2^17, exact in fp32.  One position, so
    lse is its score, up to the roundings of the score in base 2, of the reference 8 above it and of the way back."""
    s = Setup("q4", [1] * 12, 2, group, D, 16, seed=D + group)
    s.scale = 0.25
    rng = np.random.default_rng(D)
    q = rng.integers(-128, 129, s.q.shape) * 2.0 ** -7
    q[..., ::32] = 2.0 ** 12
    s.q = oracle.bf16_from_f64(q)

    def edit(codes, scales):
        p = s.table[:, 0]
        codes[p, :, 0] = rng.integers(-8, 8, codes[p, :, 0].shape)
        codes[p, :, 0, ::32] = 0
        scales[p, :, 0] = oracle.bf16_from_f64(np.float64(1.0))

    _put(s, 0, edit)
    lse = s.run()[1].cpu().numpy().astype(np.float64)
    for i in range(len(s.lens)):
        (k, _), (v, _) = s.rows(i, 0)
        _, want, _, _ = decode.attention(s.q[i], k, v, s.scale)
        assert (np.abs(lse[i] - want) <= 2.0 ** -22 * (np.abs(want) + 8.0)).all(), (i, np.max(np.abs(lse[i] - want)))


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_values_after_a_growing_maximum(form, D):
    """Values near the stated limit (n |v| < 2^126), met by a wave whose scores first grow by less than 2^8: the
    probabilities enter relative to a reference that is never below the maximum, so the sums stay finite."""
    n = 300     # 40 sequences: enough rows for workgroups of 8 waves, whose first wave takes chunks 0 and 8
    s = Setup(form, [n] * 40, 2, 2, D, 16, seed=D, junk=False, share=True)
    s.scale = 1.0
    q = np.zeros(s.q.shape)
    q[..., 0] = 1.0
    s.q = oracle.bf16_from_f64(q)
    pos = np.arange(n)
    k = np.zeros((s.pages, 2, 16, D))
    k[s.table[0, pos // 16], :, pos % 16, 0] = np.where(pos < 256, 0.0, 5.25)[:, None]     # 2^7.57
    v = 2.0 ** 117 * (0.5 + 0.5 * s.rng.random((s.pages, 2, 16, D)))
    s.k, s.v = (decode.cache_rows(oracle.bf16_from_f64(x), form) for x in (k, v))
    s.cache = to_dev(kv_layout.encode_cache(s.k, s.v, form))
    out, lse = s.run()
    assert np.isfinite(oracle.bf16_bits_to_f64(bits_host(out))).all()
    s.check(out, lse, only=[0, 39])
