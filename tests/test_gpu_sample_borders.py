"""Draws and cuts whose number lies next to the border between two tokens, nearer than 64-bit weights of less care
would resolve.  The side is that of the definition in 50 digits, and every case is farther from its border than the
errors that w4a16.h allows the weights can move it."""

from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
from gpu_util import dev

pytestmark = pytest.mark.gpu
getcontext().prec = 50


def call(z, u, temperature=None, top_k=None, top_p=None):
    """Tokens of the rows z (float32 numpy), each with the settings given."""
    n = len(z)
    full = lambda v, t: None if v is None else torch.full((n,), v, dtype=t, device=dev())
    tokens, _ = w4.sample(torch.from_numpy(z).to(dev()), torch.tensor(u, dtype=torch.float32, device=dev()),
                          full(temperature, torch.float32), full(top_k, torch.int32), full(top_p, torch.float32))
    torch.cuda.synchronize()
    return tokens.tolist()


def two_logits(V, first, z):
    """Rows of V logits: z at `first`, 0 behind it at V - 1, the others at -infinity."""
    out = np.full((1, V), -np.inf, dtype=np.float32)
    out[0, first], out[0, V - 1] = z, 0.0
    return out


# z, temperature, number: w = exp(z / temperature) is about 2^-1/2, where powers of 2 by a series are at their worst
@pytest.mark.parametrize("V,first,top_k", [(2, 0, None), (3, 0, 2), (40000, 5, None), (40000, 17000, 2)])
@pytest.mark.parametrize("z,t,u", [("-0x1.8fa824p-2", "0x1.2a30e0p+0", "0x1.ab0428p-2"),
                                   ("-0x1.6eb5fcp-2", "0x1.0b0776p+0", "0x1.a8f64ep-2"),
                                   ("-0x1.498a80p-2", "0x1.e825dcp-1", "0x1.aa6680p-2")])
def test_a_number_next_to_a_border(V, first, top_k, z, t, u):
    z, t, u = (float.fromhex(v) for v in (z, t, u))
    w = (Decimal(z) / Decimal(t)).exp()
    # w is off by 2^-50 at most, and moves the difference by (1 - u) of that, 0.6 of 2^-50; roundings of the sum 1 + w
    # and of its product with u add 2^-52
    assert 2.0 ** -50 < w - Decimal(u) * (w + 1) < 2.0 ** -48
    assert call(two_logits(V, first, z), [u], t, top_k) == [first]


def test_a_top_p_next_to_a_border():
    """1 / (1 + w) is just short of top_p: both stay, and a number behind it draws the one at the end."""
    z, t, p = (float.fromhex(v) for v in ("-0x1.d89a94p-2", "0x1.56f91cp+0", "0x1.2ba9f0p-1"))
    w = (Decimal(z) / Decimal(t)).exp()
    assert 2.0 ** -50 < Decimal(p) * (w + 1) - 1 < 2.0 ** -49       # moved by 0.6 of 2^-50 and 2^-52, as above
    for V in (3, 1500, 40000):
        zs = np.full((1, V), -np.inf, dtype=np.float32)
        zs[0, 0], zs[0, V - 1] = 0.0, z
        assert call(zs, [0.9], t, None, p) == [V - 1], V


# (z, top_p, whether both stay): w = exp(z) beside 1
@pytest.mark.parametrize("V", [5000, 131072])
@pytest.mark.parametrize("z,p,both", [("-0x1.cdbfb2p-1", "0x1.6c3378p-1", True),
                                      ("-0x1.348b70p-3", "0x1.133f66p-1", False),
                                      ("-0x1.359688p-2", "0x1.26680ap-1", False)])
def test_a_cut_next_to_a_border_among_few_allowed_tokens(V, z, p, both):
    """Fewer allowed tokens than top_k: the cut is as fine as elsewhere."""
    z, p = float.fromhex(z), float.fromhex(p)
    over = Decimal(p) * (Decimal(z).exp() + 1) - 1
    assert 2.0 ** -47 < abs(over) < 2.0 ** -46 and (over > 0) == both      # moved by 2^-50 and 2^-52 at most
    zs = np.full((1, V), -np.inf, dtype=np.float32)
    zs[0, 0], zs[0, V - 1] = 0.0, z
    for k in (50, 2000):
        assert call(zs, [0.9], None, k, p) == [V - 1 if both else 0], k


@pytest.mark.parametrize("z", ["-0x1.b9ed74p+2", "-0x1.bf1844p+2", "-0x1.bb9980p+2", "-0x1.bda182p+2"])
def test_numbers_next_to_borders_in_a_long_nucleus(z):
    """16000 equal weights of some 2^-10, which lie halfway between multiples of 2^-43, behind the largest one: rounded
    to these they move the draw by 2^-30 in all, a millionth of a token.  The nucleus ends among 300 lower ones."""
    many, few, V, z = 16000, 300, 16384, float.fromhex(z)
    wide = np.longdouble
    exp = lambda v: wide(str(Decimal(v).exp()))
    w, low = exp(z), exp(-9.0)
    total = 1 + many * w + few * low
    p = np.float32(1 - 149.5 * low / total)
    kept = (p * total - 1 - many * w) / low                 # lower tokens that the nucleus takes: the next whole number
    assert 0.01 < kept - np.floor(kept) < 0.99
    total = 1 + many * w + np.ceil(kept) * low
    i = np.arange(many)
    sums = 1 + i * w                                        # of the ids up to i
    u = (sums / total).astype(np.float32)
    over = u * total - sums
    # each weight is off by 2^-49 at most, all of them by 2^-35
    rows = np.nonzero((np.abs(over) > 2.0 ** -33.5) & (np.abs(over) < 2.0 ** -30.5) & (i > 6000))[0]
    assert len(rows) >= 5
    zs = np.full((len(rows), V), -np.inf, dtype=np.float32)
    zs[:, 0], zs[:, 1:1 + many], zs[:, 1 + many:1 + many + few] = 0.0, z, -9.0
    assert call(zs, u[rows], None, None, float(p)) == [int(r) + (1 if over[r] > 0 else 0) for r in rows]
