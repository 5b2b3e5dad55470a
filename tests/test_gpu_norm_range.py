"""The norm where weights or elements lie far from 1: a row's usual two fp32
terms hold only while no product of an element and the row's factor is small
beside its weight.  Tolerances as in test_gpu_norm.py: half a bf16 step and
half an fp32 step, 2^-8 + 2^-24 of the value; the values here stay above
2^-117, where the two terms are whole."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from oracle import decode
from gpu_util import bf16_dev, bits_host

pytestmark = pytest.mark.gpu


def check(got, want):
    """Infinities with their signs and NaN where the formula has them, other values within the roundings."""
    got = oracle.bf16_bits_to_f64(bits_host(got))
    want = np.where(np.abs(want) >= 2.0 ** 128 * (1 - 2.0 ** -9), np.copysign(np.inf, want), want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    ok = np.isfinite(want)
    err = np.abs(got[ok] - want[ok]) / np.maximum(np.abs(want[ok]), 2.0 ** -117)
    assert np.max(err) <= 2.0 ** -8 + 2.0 ** -24, np.max(err)


def run(x, w, offset):
    _, y = decode.add_rmsnorm(x, None, w, 1e-6, offset)
    got, _ = w4.add_rmsnorm(bf16_dev(x), None, bf16_dev(w), 1e-6, offset)
    q, s, _ = w4.add_rmsnorm_quantize(bf16_dev(x), None, bf16_dev(w), 1e-6, offset)
    torch.cuda.synchronize()
    check(got, y)
    qr, sr = decode.quantize_f64_rows(y)
    np.testing.assert_array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(q.cpu().numpy(), qr)


@pytest.mark.parametrize("d", [96, 800, 2816, 20000])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_infinite_weights(d, offset):
    """Infinite (and NaN) weights, beside finite ones and beside zero elements."""
    rng = np.random.default_rng(d)
    x = oracle.bf16_from_f64(rng.standard_normal((5, d)))
    w = oracle.bf16_from_f64(0.3 * rng.standard_normal(d))
    w[rng.permutation(d)[:40]] = 0x7F80
    w[rng.permutation(d)[:40]] = 0xFF80
    w[5] = 0x7FC0
    x[3, ::7] = 0
    run(x, w, offset)


@pytest.mark.parametrize("d", [96, 2816, 20000])
@pytest.mark.parametrize("offset", [0.0, 1.0, 2.0 ** 100, 3e38])
def test_large_weights(d, offset):
    """Weights up to the largest finite values: products that overflow are infinite, others are right."""
    rng = np.random.default_rng(d + 1)
    x = oracle.bf16_from_f64(rng.standard_normal((4, d)) * 2.0 ** rng.integers(-4, 4, (4, 1)))
    w = oracle.bf16_from_f64(rng.standard_normal(d) * 2.0 ** rng.integers(0, 127, d))
    run(x, w, offset)


@pytest.mark.parametrize("d", [96, 800, 2816, 20000])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_small_elements_with_large_weights(d, offset):
    """Rows with elements 2^140 below the largest whose weights bring them back into the normal range."""
    rng = np.random.default_rng(d + 2)
    x = rng.standard_normal((6, d))
    w = rng.standard_normal(d)
    w[::3] *= 2.0 ** rng.integers(55, 90, w[::3].size)
    x[:, ::3] *= 2.0 ** rng.integers(-115, -95, x[:, ::3].shape)
    x[:, 1] = 2.0 ** 38
    run(oracle.bf16_from_f64(x), oracle.bf16_from_f64(w), offset)


@pytest.mark.parametrize("d", [96, 2816])
def test_codes_of_small_elements_with_large_weights(d):
    """E4M3 codes down to the smallest of elements 2^64 and more below the row's largest."""
    rng = np.random.default_rng(d + 3)
    x, w = rng.standard_normal((6, d)), 1.0 + rng.random(d)
    x[:, 1::2] *= 2.0 ** -64 * 2.0 ** rng.integers(-14, 1, x[:, 1::2].shape)
    w[::2] *= 2.0 ** 60
    w[1::2] *= 2.0 ** 120
    run(oracle.bf16_from_f64(x), oracle.bf16_from_f64(w), 0.0)
