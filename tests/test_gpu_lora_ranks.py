"""w4a16_lora_add at the ranks around the second product's change of form (four groups of rows up to rank 168, two
above), with sums that are exact in any order."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from oracle import serving
from gpu_util import bf16_dev, bits_host, dev, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rank", [152, 160, 168, 176, 248, 256])
@pytest.mark.parametrize("rows", [100, 129, 300, 700])
def test_ranks_around_the_forms(rows, rank):
    say("[lora] rows=%d rank=%d" % (rows, rank))
    rng = np.random.default_rng(rows + rank)
    K, N, n = 512, 336, 3
    whole = lambda lo, hi, *s: oracle.bf16_from_f64(rng.integers(lo, hi + 1, s))
    x, a = whole(0, 8, rows, K), whole(0, 4, n, rank, K)         # h <= 2^14
    b = oracle.bf16_from_f64(np.where(rng.random((n, N, rank)) < 8 / rank, rng.integers(-8, 9, (n, N, rank)), 0))
    y = whole(-100, 100, rows, N)
    ids = rng.integers(-1, n, rows)
    h = oracle.bf16_bits_to_f64(x) @ oracle.bf16_bits_to_f64(a).reshape(n * rank, K).T
    assert 2 ** 11 < h.max() and h.max() * np.abs(oracle.bf16_bits_to_f64(b)).sum(-1).max() < 2 ** 24
    want, _ = serving.lora_add(x, ids, a, b, None, y)
    ws = torch.full((w4.w4a16_lora_workspace(rows, K, N, n, rank),), 255, dtype=torch.uint8, device=dev())
    out = torch.empty(rows, N, dtype=torch.bfloat16, device=dev())
    w4.w4a16_lora_add(bf16_dev(x), torch.tensor(ids, dtype=torch.int32, device=dev()), bf16_dev(a), bf16_dev(b), None,
                      bf16_dev(y), out, ws)
    torch.cuda.synchronize()
    assert np.array_equal(bits_host(out), oracle.bf16_from_f64(want))
