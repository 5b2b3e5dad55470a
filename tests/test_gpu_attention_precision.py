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
