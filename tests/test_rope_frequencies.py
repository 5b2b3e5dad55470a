"""rope_frequencies refuses what would make its table or scale infinite, zero or complex."""

import math

import pytest

import int4_group_quantized_q4_amd as w4


@pytest.mark.parametrize("bad", [dict(base=0.0), dict(base=-10.0), dict(base=math.inf), dict(base=math.nan),
                                 dict(scaling="linear", factor=math.inf), dict(scaling="base", factor=math.nan),
                                 dict(scaling="bands", factor=math.inf, trained=4096),
                                 dict(scaling="bands", factor=2.0, trained=0),
                                 dict(scaling="bands", factor=2.0, trained=-5),
                                 dict(scaling="bands", factor=2.0, trained=4096, base=1.0),
                                 dict(scaling="bands", factor=2.0, trained=4096, base=0.5)])
def test_refusals(bad):
    with pytest.raises(ValueError, match="base|factor"):
        w4.rope_frequencies(64, **bad)


def test_a_base_of_one_turns_all_pairs_alike():
    f, scale = w4.rope_frequencies(64, 1.0)
    assert (f == 1.0).all() and scale == 1.0
