"""The largest sizes that the serving step's calls take: the most rows, adapters, columns and sequences, and rows past
one launch's workgroups."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from oracle import serving
from gpu_util import bf16_dev, bits_host, dev, say

pytestmark = pytest.mark.gpu


def test_draw_of_the_most_rows():
    rng = np.random.default_rng(1)
    rows, V = 65535, 7
    z = rng.standard_normal((rows, V)).astype(np.float32)
    u = rng.random(rows).astype(np.float32)
    k, p = rng.integers(0, 9, rows), rng.choice([0.5, 0.9, 1.0], rows).astype(np.float32)
    d = lambda v, t: torch.tensor(v, dtype=t, device=dev())
    tokens, lp = w4.sample(d(z, torch.float32), d(u, torch.float32), None, d(k, torch.int32), d(p, torch.float32))
    torch.cuda.synchronize()
    tokens, lp = tokens.cpu().numpy(), lp.cpu().numpy()
    for i in list(range(0, rows, 97)) + [rows - 2, rows - 1]:
        token, want, _ = serving.sample(z[i], 1.0, int(k[i]), p[i], 0.0, u[i])
        assert tokens[i] == token and abs(lp[i] - want) <= abs(want) * 2.0 ** -24 + 2.0 ** -40, i


def exact_lora(x, ids, a, b, y):
    """out of small whole numbers, whose sums are exact; rows by adapter."""
    x, a, b, want = (oracle.bf16_bits_to_f64(v) for v in (x, a, b, y))
    order = np.argsort(ids, kind="stable")
    for rows in np.split(order, np.nonzero(np.diff(ids[order]))[0] + 1):
        if 0 <= ids[rows[0]] < len(a):
            want[rows] += (x[rows] @ a[ids[rows[0]]].T) @ b[ids[rows[0]]].T
    assert np.abs(want).max() < 2 ** 24
    return oracle.bf16_from_f64(want)


@pytest.mark.parametrize("rows,K,N,rank,adapters", [(1 << 20, 32, 16, 8, 4096), (1, 1 << 20, 16, 8, 1),
                                                    (2, 32, 1 << 20, 8, 2), (150, 64, 1 << 20, 16, 3),
                                                    (128, 32, 16, 256, 4096), (65537, 64, 48, 24, 5)])
def test_adapters_at_the_limits(rows, K, N, rank, adapters):
    say("[lora] rows=%d K=%d N=%d rank=%d adapters=%d" % (rows, K, N, rank, adapters))
    rng = np.random.default_rng(rows + N)
    whole = lambda lo, hi, *s: oracle.bf16_from_f64(rng.integers(lo, hi + 1, s))
    x, y = whole(-1, 1, rows, K), whole(-9, 9, rows, N)
    a, b = whole(-1, 1, adapters, rank, K), whole(-1, 1, adapters, N, rank)
    ids = rng.integers(-1, adapters + 1, rows) if rows > 2 else np.zeros(rows, dtype=np.int64)
    got = w4.lora_add(bf16_dev(x), torch.tensor(ids, dtype=torch.int32, device=dev()), bf16_dev(a), bf16_dev(b), None,
                      bf16_dev(y))
    torch.cuda.synchronize()
    assert np.array_equal(bits_host(got), exact_lora(x, ids, a, b, y))


@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("power", [0, -60, -110, -117])
def test_small_inner_sums_keep_24_bits(rows, power):
    """Pairs of inner sums, whole numbers of 24 bits times 2^(power - 16), that differ by one unit, the outer sum being
    the units alone."""
    rng = np.random.default_rng(rows)
    K, N, rank = 32, 16, 16
    x, a, b = np.zeros((rows, K)), np.zeros((1, rank, K)), np.zeros((1, N, rank))
    x[:, :3] = 1.0, 2.0 ** -8, 2.0 ** -16
    for r in range(0, rank, 2):
        digits = np.array([rng.integers(128, 256), rng.integers(0, 256), rng.integers(0, 255)])
        a[0, r, :3], a[0, r + 1, :3] = digits * 2.0 ** power, (digits + [0, 0, 1]) * 2.0 ** power
        b[0, :, r], b[0, :, r + 1] = -2.0 ** -power, 2.0 ** -power
    bits = lambda v: bf16_dev(oracle.bf16_from_f64(v))
    got = w4.lora_add(bits(x), torch.zeros(rows, dtype=torch.int32, device=dev()), bits(a), bits(b), None,
                      bits(np.zeros((rows, N))))
    torch.cuda.synchronize()
    assert (oracle.bf16_bits_to_f64(bits_host(got)) == rank / 2 * 2.0 ** -16).all()


def test_rows_past_one_launch_are_turned():
    """2^23 workgroups and three more, a row each of 8 KB, in place (64 GiB)."""
    rows, heads, dim = (1 << 23) + 3, 16, 256
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of free memory")
    look = [0, 1, 4099, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, rows - 1]
    q = torch.empty(rows, heads, dim, dtype=torch.bfloat16, device=dev())
    try:
        rng = np.random.default_rng(2)
        x = oracle.bf16_from_f64(rng.standard_normal((len(look), heads, dim)))
        q[look] = bf16_dev(x)
        p = torch.arange(rows, dtype=torch.int32, device=dev())
        freq, _ = w4.rope_frequencies(dim)
        w4.w4a16_rope(q, None, p, freq.to(dev()), q, None)
        want, _ = w4.rope(bf16_dev(x), None, p[look].contiguous(), freq.to(dev()))
        torch.cuda.synchronize()
        assert torch.equal(q[look], want)
    finally:
        del q
        torch.cuda.empty_cache()


def test_plan_of_the_most_sequences_and_rows():
    rng = np.random.default_rng(3)
    seqs, page, width, max_rows = 65535, 16, 3, 1 << 26
    lens = rng.integers(0, 33, seqs)
    new = np.where(rng.random(seqs) < 0.1, -1, rng.integers(0, 15, seqs))
    have = -(-lens // page)
    pages = int(have.sum()) + seqs
    ids = rng.permutation(pages)
    table = np.zeros((seqs, width), dtype=np.int64)
    at = 0
    for i in range(seqs):
        table[i, :have[i]] = ids[at:at + have[i]]
        at += have[i]
    free = np.zeros(pages, dtype=np.int64)
    free[:pages - at] = ids[at:]
    d = lambda v: torch.tensor(v, dtype=torch.int32, device=dev())
    dl, dt, df, dc = d(lens), d(table), d(free), d([pages - at])
    slots, positions, row_seqs, offsets = w4.kv_plan(dl, d(new), dt, page, df, dc, max_rows)
    torch.cuda.synchronize()
    rows = int(np.maximum(new, 0).sum())
    want = serving.plan(lens, new, table, page, free, pages - at, rows)
    for got, name in ((slots, "slots"), (positions, "positions"), (row_seqs, "row_seqs")):
        assert np.array_equal(got[:rows].cpu().numpy(), want[name]), name
    assert bool((slots[rows:] == -1).all()) and not positions[rows:].any() and bool((row_seqs[rows:] == -1).all())
    assert np.array_equal(offsets.cpu().numpy(), want["offsets"]) and np.array_equal(dl.cpu().numpy(), want["lens"])
    assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(df.cpu().numpy(), free)
    assert dc.item() == want["count"]
