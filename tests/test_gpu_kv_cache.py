"""GPU parity of writing into and reading from the paged key-value cache
against oracle/decode.py, through the independent layout decoder.  Codes and
scales are integer decisions taken from single IEEE fp32 divisions on both
sides and compared bit for bit; so are the values read back (fp32 exact for
Q4, one rounding for E4M3; bf16 one more)."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import kv_layout
import oracle
from oracle import decode
from gpu_util import bf16_dev, bits_host, dev, say, to_dev

pytestmark = pytest.mark.gpu
FMT = {"bf16": w4.W4_KV_BF16, "e4m3": w4.W4_KV_E4M3, "q4": w4.W4_KV_Q4}


def rnd(rng, *shape, sigma=1.0):
    return oracle.bf16_from_f64(sigma * rng.standard_normal(shape))


def empty_cache(form, pages, page, heads, D, fill=0xA5):
    return torch.full((pages, kv_layout.page_bytes(form, page, heads, D)), fill, dtype=torch.uint8, device=dev())


def place(cache_codes, slots, page):
    """codes [pages, heads, page, ...] -> the slots' rows [tokens, heads, ...]"""
    return cache_codes[slots // page, :, slots % page]


def check_written(cache, before, form, pages, page, heads, D, slots, k, v):
    """Written rows hold the oracle's codes; every other code and scale is as it was."""
    got = kv_layout.decode_cache(cache.cpu().numpy(), form, pages, page, heads, D)
    old = kv_layout.decode_cache(before, form, pages, page, heads, D)
    live = (slots >= 0) & (slots < pages * page)
    for name, x in (("k", k), ("v", v)):
        c, s = decode.cache_rows(x[live], form)
        want_c, want_s = old[name]
        want_c = want_c.copy()
        want_c[slots[live] // page, :, slots[live] % page] = c
        assert np.array_equal(got[name][0], want_c)
        if form != "bf16":
            want_s = want_s.copy()
            want_s[slots[live] // page, :, slots[live] % page] = s
            bits = np.uint32 if form == "e4m3" else np.uint16
            nan = np.isnan(want_s) if form == "e4m3" else np.zeros(want_s.shape, bool)
            assert np.array_equal(got[name][1].view(bits)[~nan], want_s.view(bits)[~nan])
            assert not nan.any() or np.isnan(got[name][1][nan]).all()


CASES = [(1, 1, 64, 16), (7, 3, 64, 16), (64, 8, 128, 64), (33, 2, 256, 32), (200, 5, 128, 16), (129, 1, 256, 128)]


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("tokens,heads,D,page", CASES)
def test_write_and_read(form, tokens, heads, D, page):
    say("[kv] %s tokens=%d heads=%d D=%d page=%d" % (form, tokens, heads, D, page))
    rng = np.random.default_rng(tokens + D)
    pages = -(-tokens // page) + 3
    k, v = rnd(rng, tokens, heads, D), rnd(rng, tokens, heads, D, sigma=3.0)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if tokens > 5:
        slots[3] = -1
        slots[4] = pages * page + 5               # past the cache: skipped and counted
        slots[5] = -(1 << 40)
    cache = empty_cache(form, pages, page, heads, D)
    before = cache.cpu().numpy().copy()
    counters = torch.zeros(2, dtype=torch.int64, device=dev())
    w4.kv_cache_write(bf16_dev(k), bf16_dev(v), to_dev(slots), FMT[form], page, cache, counters)
    torch.cuda.synchronize()
    check_written(cache, before, form, pages, page, heads, D, slots, k, v)
    assert counters.tolist() == [1 if tokens > 5 else 0, 0]
    # read back, in another order and with repeats
    order = rng.integers(0, tokens, tokens + 9)
    live = (slots >= 0) & (slots < pages * page)
    for dt in (torch.bfloat16, torch.float32):
        ko = torch.full((tokens + 9, heads, D), 5.0, dtype=dt, device=dev())
        vo = ko.clone()
        w4.kv_cache_read(cache, FMT[form], page, to_dev(slots[order]), ko, vo, counters)
        torch.cuda.synchronize()
        for got, x in ((ko, k), (vo, v)):
            want = decode.row_values(*decode.cache_rows(x, form), form)[order]
            want[~live[order]] = 5.0
            if dt == torch.float32:
                assert np.array_equal(got.cpu().numpy(), want.astype(np.float32))
            else:
                assert np.array_equal(bits_host(got), oracle.bf16_from_f32(want.astype(np.float32)))


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("first", [0, 5, 16])
def test_prompt_into_consecutive_slots(form, first):
    """A prompt: consecutive positions, starting inside a tile or at one, through shuffled pages; heads of one fused
    projection's output (strided rows)."""
    rng = np.random.default_rng(first)
    page, heads, D, tokens = 32, 2, 128, 150
    pages = 7
    table = rng.permutation(pages)
    pos = first + np.arange(tokens)
    slots = (table[pos // page] * page + pos % page).astype(np.int64)
    qkv = rnd(rng, tokens, 6 * D)
    d = bf16_dev(qkv)
    kd, vd = d[:, 2 * D:4 * D].unflatten(1, (heads, D)), d[:, 4 * D:].unflatten(1, (heads, D))
    k, v = qkv[:, 2 * D:4 * D].reshape(tokens, heads, D), qkv[:, 4 * D:].reshape(tokens, heads, D)
    cache = empty_cache(form, pages, page, heads, D)
    before = cache.cpu().numpy().copy()
    w4.kv_cache_write(kd, vd, to_dev(slots), FMT[form], page, cache)
    torch.cuda.synchronize()
    check_written(cache, before, form, pages, page, heads, D, slots, k, v)
    out = torch.full((tokens, 6 * D), 9.0, dtype=torch.bfloat16, device=dev())
    w4.kv_cache_read(cache, FMT[form], page, to_dev(slots), out[:, :2 * D].unflatten(1, (heads, D)),
                     out[:, 3 * D:5 * D].unflatten(1, (heads, D)))
    torch.cuda.synchronize()
    got = bits_host(out).reshape(tokens, 6, D)
    for at, x in ((0, k), (3, v)):
        want = decode.row_values(*decode.cache_rows(x, form), form)
        assert np.array_equal(got[:, at:at + 2], oracle.bf16_from_f32(want.astype(np.float32)))
    nine = oracle.bf16_from_f64(np.array([9.0]))[0]
    assert (got[:, 2] == nine).all() and (got[:, 5] == nine).all()


@pytest.mark.parametrize("form", kv_layout.FORMATS)
def test_special_rows(form):
    """Zeros, subnormals, the largest value, ties between codes, infinities and NaN, each in a row of its own; poisoned
    rows and groups are counted and read back as NaN (E4M3, Q4)."""
    page, heads, D, pages = 16, 1, 64, 2
    rng = np.random.default_rng(3)
    k = rnd(rng, 12, heads, D)
    k[0] = 0
    k[1] = 0x8000
    k[2] = 1
    k[3] = rng.integers(0, 0x80, (heads, D))                     # subnormals
    k[4, 0, 0] = 0x7F7F
    grid = np.concatenate([np.arange(-7, 8), np.arange(-6.5, 7.5)])   # Q4 levels and the ties between them, step 1
    k[5, 0, :29] = oracle.bf16_from_f64(grid)
    k[5, 0, 29:32] = 0
    k[6, 0, 3] = 0x7F80
    k[7, 0, 40] = 0xFFC3
    k[8, 0, :2] = (0x7F80, 0xFF80)
    v = k[::-1].copy()
    slots = np.arange(12, dtype=np.int64) + 3
    cache = empty_cache(form, pages, page, heads, D)
    before = cache.cpu().numpy().copy()
    counters = torch.zeros(2, dtype=torch.int64, device=dev())
    w4.kv_cache_write(bf16_dev(k), bf16_dev(v), to_dev(slots), FMT[form], page, cache, counters)
    ko = torch.empty(12, heads, D, device=dev())
    vo = torch.empty_like(ko)
    w4.kv_cache_read(cache, FMT[form], page, to_dev(slots), ko, vo)
    torch.cuda.synchronize()
    check_written(cache, before, form, pages, page, heads, D, slots, k, v)
    want = decode.row_values(*decode.cache_rows(k, form), form).astype(np.float32)
    np.testing.assert_array_equal(ko.cpu().numpy(), want)
    np.testing.assert_array_equal(vo.cpu().numpy(), want[::-1])
    assert counters.tolist() == [0, 0 if form == "bf16" else 6]


@pytest.mark.parametrize("form", kv_layout.FORMATS)
def test_graph_replay(form):
    """A captured write and read, replayed with new rows and new slots."""
    rng = np.random.default_rng(12)
    page, heads, D, pages, tokens = 16, 2, 128, 6, 19
    k = torch.zeros(tokens, heads, D, dtype=torch.bfloat16, device=dev())
    v, ko, vo = torch.zeros_like(k), torch.zeros_like(k), torch.zeros_like(k)
    slots = torch.full((tokens,), -1, dtype=torch.int64, device=dev())
    cache = empty_cache(form, pages, page, heads, D)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        w4.kv_cache_write(k, v, slots, FMT[form], page, cache)
        w4.kv_cache_read(cache, FMT[form], page, slots, ko, vo)
    for _ in range(3):
        kb, vb = rnd(rng, tokens, heads, D), rnd(rng, tokens, heads, D)
        k.copy_(bf16_dev(kb)), v.copy_(bf16_dev(vb))
        slots.copy_(to_dev(rng.permutation(pages * page)[:tokens].astype(np.int64)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for got, x in ((ko, kb), (vo, vb)):
            want = decode.row_values(*decode.cache_rows(x, form), form)
            assert np.array_equal(bits_host(got), oracle.bf16_from_f32(want.astype(np.float32)))


@pytest.mark.parametrize("form", kv_layout.FORMATS)
def test_rows_of_one_buffer(form):
    """k and v as slices of one buffer, written from it and read back into it: the values between them stay."""
    tokens, heads, D, page = 37, 2, 64, 16
    rng = np.random.default_rng(77)
    k, v = rnd(rng, tokens, heads, D), rnd(rng, tokens, heads, D)
    qkv = torch.full((tokens, 5 * heads * D), 3.0, dtype=torch.bfloat16, device=dev())
    view = lambda i: qkv[:, i * heads * D:(i + 1) * heads * D].unflatten(1, (heads, D))
    view(1).copy_(bf16_dev(k))
    view(3).copy_(bf16_dev(v))
    cache = empty_cache(form, 4, page, heads, D)
    slots = to_dev(rng.permutation(4 * page)[:tokens].astype(np.int64))
    w4.kv_cache_write(view(1), view(3), slots, FMT[form], page, cache)
    w4.kv_cache_read(cache, FMT[form], page, slots, view(4), view(2))
    torch.cuda.synchronize()
    want = [oracle.bf16_from_f32(decode.row_values(*decode.cache_rows(x, form), form).astype(np.float32))
            for x in (k, v)]
    assert np.array_equal(bits_host(view(4).contiguous()), want[0])
    assert np.array_equal(bits_host(view(2).contiguous()), want[1])
    assert np.array_equal(bits_host(view(1).contiguous()), k) and np.array_equal(bits_host(view(3).contiguous()), v)
    assert (view(0) == 3).all()


@pytest.mark.parametrize("form", kv_layout.FORMATS)
def test_most_heads(form):
    """1024 heads: written, read back, and nothing else changed."""
    tokens, heads, D, page, pages = 21, 1024, 64, 16, 3
    rng = np.random.default_rng(78)
    k, v = rnd(rng, tokens, heads, D), rnd(rng, tokens, heads, D)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    cache = empty_cache(form, pages, page, heads, D)
    before = cache.cpu().numpy().copy()
    w4.kv_cache_write(bf16_dev(k), bf16_dev(v), to_dev(slots), FMT[form], page, cache)
    ko = torch.zeros(tokens, heads, D, device=dev())
    vo = torch.zeros_like(ko)
    w4.kv_cache_read(cache, FMT[form], page, to_dev(slots), ko, vo)
    torch.cuda.synchronize()
    check_written(cache, before, form, pages, page, heads, D, slots, k, v)
    for got, x in ((ko, k), (vo, v)):
        want = decode.row_values(*decode.cache_rows(x, form), form)
        assert np.array_equal(got.cpu().numpy(), want.astype(np.float32))


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("heads,D", [(1, 64), (3, 128), (2, 256)])
def test_many_tokens_as_pieces(form, heads, D):
    """A long list in one call, and in pieces of odd sizes on two streams at once (neighbouring tokens of a tile from
    both): the same bytes in the cache, and the same rows read."""
    page, tokens = 64, 50021
    pages = -(-tokens // page)
    g = torch.Generator(device="cuda").manual_seed(D)
    k = torch.randn(tokens, heads, D, generator=g, device=dev(), dtype=torch.bfloat16)
    v = torch.randn(tokens, heads, D, generator=g, device=dev(), dtype=torch.bfloat16)
    slots = torch.arange(tokens, device=dev(), dtype=torch.int64)
    mixed = slots.view(-1)[torch.randperm(tokens, generator=g, device=dev())].contiguous()
    one, two = empty_cache(form, pages, page, heads, D), empty_cache(form, pages, page, heads, D)
    w4.kv_cache_write(k, v, slots, FMT[form], page, one)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    at, i = 0, 0
    while at < tokens:
        n = min((1, 3, 61, 997, 12001)[i % 5], tokens - at)
        part = slice(at, at + n)
        w4.kv_cache_write(k[part], v[part], slots[part], FMT[form], page, two, stream=streams[i % 2])
        at, i = at + n, i + 1
    torch.cuda.synchronize()
    assert torch.equal(one, two)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    w4.kv_cache_read(one, FMT[form], page, slots, ko, vo)
    km, vm = torch.zeros_like(k), torch.zeros_like(v)
    w4.kv_cache_read(one, FMT[form], page, mixed, km, vm)
    torch.cuda.synchronize()
    assert torch.equal(km, ko[mixed]) and torch.equal(vm, vo[mixed])
    if form == "bf16":
        assert torch.equal(ko, k) and torch.equal(vo, v)
