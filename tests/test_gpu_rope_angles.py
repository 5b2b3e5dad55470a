"""Rotary angles of more than 53 bits: positions and frequencies whose product, rounded to 64-bit floating point, is off
by 2^-10 and more, chosen next to quarter turns, where the sine or the cosine shows all of it."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from gpu_util import bits_host, dev

pytestmark = pytest.mark.gpu

PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
PAIRS = [(2117742597, "0x1.8c3f5ep+13"), (1727764425, "0x1.9fb244p+13"), (1383189122, "0x1.cae3cap+13"),
         (-1080076179, "0x1.51cccep+13"), (1453471878, "0x1.ace12ap+12"), (-1189909973, "0x1.974f7ep+13"),
         (1647089734, "0x1.8ffb02p+13"), (1372200919, "0x1.30fdcep+13")]


@pytest.mark.parametrize("layout", [w4.W4_ROPE_HALF, w4.W4_ROPE_INTERLEAVED])
def test_angles_of_more_than_53_bits(layout):
    freq = np.array([float.fromhex(f) for _, f in PAIRS], dtype=np.float32)
    positions = [p for p, _ in PAIRS]
    x = torch.zeros(len(PAIRS), 1, 16, dtype=torch.bfloat16, device=dev())
    x[..., slice(0, 8) if layout == w4.W4_ROPE_HALF else slice(0, 16, 2)] = 1.0       # (1, 0) -> (cos, sin)
    y, _ = w4.rope(x, None, torch.tensor(positions, dtype=torch.int32, device=dev()), torch.from_numpy(freq).to(dev()),
                   layout)
    torch.cuda.synchronize()
    got = oracle.bf16_bits_to_f64(bits_host(y))[:, 0]
    for i, p in enumerate(positions):
        angle = p * Fraction(float(freq[i]))
        assert abs(Fraction(p * float(freq[i])) - angle) >= Fraction(1, 1024)
        quarters = round(angle / (PI / 2))
        rest = float(angle - quarters * (PI / 2))
        assert abs(rest) < 0.003
        c, s = math.cos(rest), math.sin(rest)
        c, s = [(c, s), (-s, c), (-c, -s), (s, -c)][quarters % 4]
        at = (i, i + 8) if layout == w4.W4_ROPE_HALF else (2 * i, 2 * i + 1)
        for have, want in ((got[i, at[0]], c), (got[i, at[1]], s)):
            # half a bf16 step, and what fp32 sines and cosines and their arguments are off
            assert abs(have - want) <= abs(want) * (2.0 ** -8 + 2.0 ** -20), (i, have, want)
