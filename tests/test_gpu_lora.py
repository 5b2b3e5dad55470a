"""GPU parity of w4a16_lora_add against oracle/serving.py.

Tolerance: half a bf16 step of the value (2^-8 of it), and what K and rank fp32
additions in any order may be off (the oracle's bound).  Cases with small whole
numbers have exact sums in any order and are compared exactly."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from oracle import serving
from gpu_util import bf16_dev, bits_host, dev, say

pytestmark = pytest.mark.gpu


def rnd(rng, *shape, sigma=1.0):
    return oracle.bf16_from_f64(sigma * rng.standard_normal(shape))


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev())


def check(got, x, ids, a, b, scaling, y):
    want, bound = serving.lora_add(x, ids, a, b, scaling, y)
    g = oracle.bf16_bits_to_f64(bits_host(got))
    assert (np.abs(g - want) <= np.abs(want) * 2.0 ** -8 + bound * (1 + 2.0 ** -8) + 2.0 ** -134).all()
    bare = (np.asarray(ids) < 0) | (np.asarray(ids) >= len(a))
    assert np.array_equal(bits_host(got)[bare], y[bare])      # rows without an adapter come out bit for bit


CASES = [  # rows, K, N, rank, adapters, order
    (1, 32, 16, 8, 1, "random"), (1, 2816, 4096, 16, 4, "random"), (2, 64, 48, 8, 3, "random"),
    (15, 96, 1040, 24, 5, "random"), (16, 256, 512, 16, 1, "random"), (17, 4096, 256, 32, 40, "random"),
    (64, 704, 2816, 16, 64, "random"), (65, 2816, 1408, 64, 7, "random"), (100, 1024, 336, 40, 300, "random"),
    (200, 512, 1024, 128, 3, "random"), (256, 2048, 512, 8, 30, "random"), (300, 320, 272, 256, 4, "random"),
    (130, 1024, 512, 16, 5, "runs"), (700, 512, 784, 16, 9, "runs"), (1025, 256, 512, 64, 6, "runs"),
    (2500, 160, 144, 24, 12, "runs"), (1500, 128, 256, 16, 50, "random"), (3000, 96, 80, 8, 1000, "random")]


@pytest.mark.parametrize("rows,K,N,rank,adapters,order", CASES)
def test_lora(rows, K, N, rank, adapters, order):
    say("[lora] rows=%d K=%d N=%d rank=%d adapters=%d %s" % (rows, K, N, rank, adapters, order))
    rng = np.random.default_rng(rows * 31 + K + rank)
    x, a, b = rnd(rng, rows, K), rnd(rng, adapters, rank, K, sigma=K ** -0.5), rnd(rng, adapters, N, rank)
    y = rnd(rng, rows, N)
    scaling = rng.uniform(0.1, 2.0, adapters).astype(np.float32)
    ids = rng.integers(-1, adapters + 1, rows)
    if order == "runs":
        ids = np.repeat(rng.integers(-1, adapters, 8), -(-rows // 8))[:rows]
    if rows > 3:
        ids[1], ids[2] = -2 ** 31, 2 ** 31 - 1
    xd, ad, bd, yd, idd, sd = (bf16_dev(x), bf16_dev(a), bf16_dev(b), bf16_dev(y), i32(ids),
                               torch.from_numpy(scaling).to(dev()))
    out = w4.lora_add(xd, idd, ad, bd, sd, yd)
    plain = w4.lora_add(xd, idd, ad, bd, None, yd)
    # strided rows, in place, over a workspace of NaN bits
    wide = torch.zeros(rows, N + 24, dtype=torch.bfloat16, device=dev())
    wide[:, 8:8 + N] = yd
    wx = torch.zeros(rows, K + 16, dtype=torch.bfloat16, device=dev())
    wx[:, 16:] = xd
    ws = torch.full((w4.w4a16_lora_workspace(rows, K, N, adapters, rank),), 255, dtype=torch.uint8, device=dev())
    w4.w4a16_lora_add(wx[:, 16:], idd, ad, bd, sd, wide[:, 8:8 + N], wide[:, 8:8 + N], ws)
    torch.cuda.synchronize()
    check(out, x, ids, a, b, scaling, y)
    check(plain, x, ids, a, b, None, y)
    assert torch.equal(wide[:, 8:8 + N], out)
    assert not wide[:, :8].any() and not wide[:, 8 + N:].any()
    assert np.array_equal(bits_host(yd), y) and np.array_equal(bits_host(xd), x)


@pytest.mark.parametrize("rows,rank", [(1, 8), (5, 16), (40, 24), (40, 64), (600, 16), (600, 64), (600, 136)])
def test_exact_sums(rows, rank):
    """Small whole numbers: h of some 15 bits (more than a bf16 holds), outer sums below 2^24, so every fp32 sum is
    exact and out is the exact value rounded once."""
    rng = np.random.default_rng(rows + rank)
    K, N, n = 4096, 48, 3
    whole = lambda lo, hi, *s: oracle.bf16_from_f64(rng.integers(lo, hi + 1, s))
    x, a = whole(0, 8, rows, K), whole(0, 4, n, rank, K)         # h <= 2^17
    b = oracle.bf16_from_f64(np.where(rng.random((n, N, rank)) < 8 / rank, rng.integers(-8, 9, (n, N, rank)), 0))
    y = whole(-100, 100, rows, N)
    ids = np.sort(rng.integers(0, n, rows))
    want, _ = serving.lora_add(x, ids, a, b, None, y)
    h = oracle.bf16_bits_to_f64(x) @ oracle.bf16_bits_to_f64(a).reshape(n * rank, K).T
    assert 2 ** 14 < h.max() and h.max() * np.abs(oracle.bf16_bits_to_f64(b)).sum(-1).max() < 2 ** 24
    got = w4.lora_add(bf16_dev(x), i32(ids), bf16_dev(a), bf16_dev(b), None, bf16_dev(y))
    torch.cuda.synchronize()
    assert np.array_equal(bits_host(got), oracle.bf16_from_f64(want))


@pytest.mark.parametrize("rows", [3, 70, 700])
def test_cancelling_outputs(rows):
    """Outer sums whose terms cancel to a few units, from h of some 17 bits: nothing of h may be lost."""
    rng = np.random.default_rng(rows)
    K, N, rank = 4096, 32, 16
    x = oracle.bf16_from_f64(rng.integers(0, 9, (rows, K)))
    half = rng.integers(0, 9, (rank // 2, K))
    other = half.copy()
    other[:, 0] += 1                     # the second half of a differs from the first by one element
    a = oracle.bf16_from_f64(np.concatenate([half, other]))[None]
    b = np.ones((1, N, rank))
    b[..., rank // 2:] = -1              # and is taken off again
    y = np.zeros((rows, N), dtype=np.uint16)
    got = w4.lora_add(bf16_dev(x), i32(np.zeros(rows)), bf16_dev(a), bf16_dev(oracle.bf16_from_f64(b)), None,
                      bf16_dev(y))
    torch.cuda.synchronize()
    want = -oracle.bf16_bits_to_f64(x)[:, :1] * (rank // 2)
    assert np.array_equal(oracle.bf16_bits_to_f64(bits_host(got)), np.broadcast_to(want, (rows, N)))


@pytest.mark.parametrize("rows", [20, 300, 1200])
def test_rows_do_not_touch_one_another(rows):
    """NaN and infinities in one row's x or y, or in one adapter, stay with the rows that use them; rows of an unused
    adapter's NaN do not see it."""
    rng = np.random.default_rng(rows)
    K, N, rank, n = 128, 96, 16, 6
    x, a, b, y = rnd(rng, rows, K), rnd(rng, n, rank, K), rnd(rng, n, N, rank), rnd(rng, rows, N)
    ids = rng.integers(-1, n - 2, rows)
    clean = w4.lora_add(bf16_dev(x), i32(ids), bf16_dev(a), bf16_dev(b), None, bf16_dev(y))
    a[n - 1], b[n - 2] = 0x7FC0, 0x7F80      # adapters that no row has
    a[1, 3, 7] = 0x7FC0                       # one that some have
    x[7, 5], x[11] = 0x7F80, 0x7FC0
    y[13, 4] = 0xFF80
    ids[13] = -1
    got = w4.lora_add(bf16_dev(x), i32(ids), bf16_dev(a), bf16_dev(b), None, bf16_dev(y))
    torch.cuda.synchronize()
    g, c = bits_host(got), bits_host(clean)
    used = ids == 1
    special = np.isin(np.arange(rows), [7, 11, 13]) | used
    assert np.array_equal(g[~special], c[~special])
    assert np.isnan(oracle.bf16_bits_to_f64(g[used])).all()
    for t in (7, 11):
        if ids[t] >= 0:
            assert not np.isfinite(oracle.bf16_bits_to_f64(g[t])).any()
        else:
            assert np.array_equal(g[t], y[t])
    assert np.array_equal(g[13], y[13])


def test_infinite_inner_sums_keep_their_sign():
    """An inner sum that is infinite makes the outputs with a weight on it infinite, not NaN."""
    x = np.zeros((4, 64), dtype=np.uint16)
    x[1, 0], x[2, 0], x[3, 0] = 0x7F80, 0xFF80, oracle.bf16_from_f64(np.array([2.0]))[0]
    a = np.zeros((1, 8, 64), dtype=np.uint16)
    a[0, 0, 0] = oracle.bf16_from_f64(np.array([1.0]))[0]
    b = oracle.bf16_from_f64(np.ones((1, 16, 8)))
    a[0, :, 1:] = 0
    a[0, 1:, 0] = oracle.bf16_from_f64(np.array([0.5]))[0]
    y = np.zeros((4, 16), dtype=np.uint16)
    got = w4.lora_add(bf16_dev(x), i32(np.zeros(4)), bf16_dev(a), bf16_dev(b), None, bf16_dev(y))
    torch.cuda.synchronize()
    g = oracle.bf16_bits_to_f64(bits_host(got))
    assert (g[0] == 0).all() and (g[1] == np.inf).all() and (g[2] == -np.inf).all() and (g[3] == 2.0 + 7.0).all()


def test_no_adapters_at_all():
    y = rnd(np.random.default_rng(1), 5, 32)
    x = torch.zeros(5, 64, dtype=torch.bfloat16, device=dev())
    none = torch.zeros(0, 8, 64, dtype=torch.bfloat16, device=dev())
    got = w4.lora_add(x, i32([0, 1, -1, 5, 0]), none, torch.zeros(0, 32, 8, dtype=torch.bfloat16, device=dev()), None,
                      bf16_dev(y))
    torch.cuda.synchronize()
    assert np.array_equal(bits_host(got), y)


@pytest.mark.parametrize("rows", [1, 48, 900])
def test_graph_replays_with_other_ids(rows):
    rng = np.random.default_rng(rows)
    K, N, rank, n = 512, 272, 16, 9
    x, a, b = bf16_dev(rnd(rng, rows, K)), bf16_dev(rnd(rng, n, rank, K)), bf16_dev(rnd(rng, n, N, rank))
    y, ids = bf16_dev(rnd(rng, rows, N)), i32(rng.integers(-1, n, rows))
    scaling = torch.rand(n, device=dev())
    out = torch.empty_like(y)
    ws = torch.empty(max(16, w4.w4a16_lora_workspace(rows, K, N, n, rank)), dtype=torch.uint8, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4a16_lora_add(x, ids, a, b, scaling, y, out, ws)
    for i in range(5):
        ids.copy_(i32(rng.integers(-1, n, rows)))
        x.mul_(-0.5)
        ws.fill_(255)
        g.replay()
        want = w4.lora_add(x, ids, a, b, scaling, y)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("rows", [64, 200, 700])
@pytest.mark.parametrize("rank", [16, 64])
def test_a_row_does_not_depend_on_its_place(rows, rank):
    """In calls of the same size a row's result is the same bit for bit, whatever adapters the others have and wherever
    the row stands; and so it is from run to run."""
    rng = np.random.default_rng(rows + rank)
    K, N, n = 1024, 320, 5
    x, a, b, y = rnd(rng, rows, K), rnd(rng, n, rank, K), rnd(rng, n, N, rank), rnd(rng, rows, N)
    ad, bd = bf16_dev(a), bf16_dev(b)
    ids = rng.integers(0, n, rows)
    first = bits_host(w4.lora_add(bf16_dev(x), i32(ids), ad, bd, None, bf16_dev(y)))
    torch.cuda.synchronize()
    again = bits_host(w4.lora_add(bf16_dev(x), i32(ids), ad, bd, None, bf16_dev(y)))
    assert np.array_equal(first, again)
    order = rng.permutation(rows)
    moved = bits_host(w4.lora_add(bf16_dev(x[order]), i32(ids[order]), ad, bd, None, bf16_dev(y[order])))
    assert np.array_equal(moved, first[order])
    other = np.where(np.arange(rows) % 3 == 0, ids, rng.integers(-1, n, rows))
    mixed = bits_host(w4.lora_add(bf16_dev(x), i32(other), ad, bd, None, bf16_dev(y)))
    assert np.array_equal(mixed[::3], first[::3])


def test_two_streams_at_once():
    """Calls that overlap in time, each with a workspace of its own, as they are one after another."""
    rng = np.random.default_rng(3)
    K, N, n, rank = 2048, 2048, 6, 32
    a, b = bf16_dev(rnd(rng, n, rank, K)), bf16_dev(rnd(rng, n, N, rank))
    sets = []
    for rows in (600, 40):
        x, y, ids = bf16_dev(rnd(rng, rows, K)), bf16_dev(rnd(rng, rows, N)), i32(rng.integers(-1, n, rows))
        ws = torch.empty(w4.w4a16_lora_workspace(rows, K, N, n, rank), dtype=torch.uint8, device=dev())
        want = w4.lora_add(x, ids, a, b, None, y)
        sets.append((x, ids, y, torch.zeros_like(y), ws, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for x, ids, y, out, ws, _, s in sets:
            with torch.cuda.stream(s):
                w4.w4a16_lora_add(x, ids, a, b, None, y, out, ws)
    torch.cuda.synchronize()
    for *_, out, _, want, _ in sets:
        assert torch.equal(out, want)


@pytest.mark.parametrize("rows", [15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 193, 257])
@pytest.mark.parametrize("adapters", [1, 3])
def test_rows_around_the_tiles(rows, adapters):
    rng = np.random.default_rng(rows * 10 + adapters)
    K, N, rank = 96, 80, 16
    x, y, a, b = rnd(rng, rows, K), rnd(rng, rows, N), rnd(rng, adapters, rank, K), rnd(rng, adapters, N, rank)
    s = rng.uniform(0.5, 2, adapters).astype(np.float32)
    for ids in (np.zeros(rows, int), rng.integers(0, adapters, rows), np.arange(rows) * adapters // rows):
        got = w4.lora_add(bf16_dev(x), i32(ids), bf16_dev(a), bf16_dev(b), torch.tensor(s, device=dev()), bf16_dev(y))
        check(got, x, ids, a, b, s, y)
