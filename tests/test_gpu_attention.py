"""GPU parity of the one-token attention over the paged cache against
oracle/decode.py.

Tolerances, from the operations' roundings (all terms relative to what is
summed): with A = sum_t p_t |v'_t| (v' the value the matrix core multiplies:
144 |s| at most for Q4, whose codes enter as 136 + q) and S = scale * sum
|q_i| |k'_i|,
  score     D + 8 fp32 additions and multiplications: (D + 8) 2^-23 S;
  p         e^score: the score's error, 2^-22 of |score| (the base-2 exponent is
            rounded to fp32 twice) and 2^-22 for the exponential; the running
            maximum cancels;
  p . v     p * s in two bf16 terms (2^-16), n + 40 fp32 additions (chunks,
            waves, splits): 2^-16 + (n + 40) 2^-23, over A;
  division  the sum l has the same relative errors as p;
  out       half a bf16 step, 2^-8.
lse = m + log l: l's relative error plus 2^-22 (|lse| + |m|)."""

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


class Setup:
    """A cache of random rows and a batch over it.  Pages of different sequences are distinct unless share is set;
    junk: every row outside the sequences' positions, and its scale, is NaN (all ones) bytes."""

    def __init__(self, form, lens, kv_heads, group, D, page, seed=0, width=None, junk=True, share=False, window=0):
        rng = self.rng = np.random.default_rng(seed)
        self.form, self.page, self.kv_heads, self.group, self.D = form, page, kv_heads, group, D
        self.heads = kv_heads * group
        self.lens = np.asarray(lens, dtype=np.int32)
        seqs = len(lens)
        need = [-(-max(0, int(n)) // page) for n in lens]
        self.width = max(1, max(need)) if width is None else width
        used = max(1, max(need)) if share else max(1, sum(need))
        self.pages = used + 2
        ids = rng.permutation(self.pages)
        self.table = np.full((seqs, self.width), 1 << 20, dtype=np.int32)      # entries past a sequence: outside
        at = 0
        for i, n in enumerate(need):
            at = 0 if share else at
            self.table[i, :n] = ids[at:at + n]
            at += n
        k, v = rnd(rng, self.pages, kv_heads, page, D), rnd(rng, self.pages, kv_heads, page, D, sigma=2.0)
        self.k, self.v = decode.cache_rows(k, form), decode.cache_rows(v, form)
        if junk:
            seen = np.zeros((self.pages, page), dtype=bool)
            for i, n in enumerate(self.lens):
                pos = np.arange(max(0, int(n) - window) if window else 0, max(0, int(n)))
                seen[self.table[i, pos // page], pos % page] = True
            for codes, scales in (self.k, self.v):
                fill = {"bf16": 0xFFFF, "e4m3": 0xFF, "q4": -1}[form]
                codes[np.broadcast_to(~seen[:, None, :], codes.shape[:3])] = fill
                if scales is not None:
                    scales[np.broadcast_to(~seen[:, None, :], scales.shape[:3])] = np.nan if form == "e4m3" else 0xFFFF
        self.cache = to_dev(kv_layout.encode_cache(self.k, self.v, form))
        self.q = rnd(rng, seqs, self.heads, D)
        self.scale = 1.0 / np.sqrt(D)

    def rows(self, i, window):
        n = max(0, int(self.lens[i]))
        pos = np.arange(max(0, n - window) if window > 0 else 0, n)
        p, o = self.table[i, pos // self.page], pos % self.page
        out = []
        for codes, scales in (self.k, self.v):
            s = None if scales is None else scales[p, :, o]
            val = decode.row_values(codes[p, :, o], s, self.form)
            mag = np.abs(val)
            if self.form == "q4":
                mag = np.repeat(oracle.bf16_bits_to_f64(s), 32, axis=-1) * 144.0
            out.append((val, mag))
        return out

    def run(self, window=0, table=None, lens=None, **kw):
        out, lse = w4.kv_attention(bf16_dev(self.q), self.cache, FMT[self.form], self.page, self.kv_heads,
                                   to_dev(self.table if table is None else table),
                                   to_dev(self.lens if lens is None else lens), self.scale, window, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, window=0, only=None):
        o = oracle.bf16_bits_to_f64(bits_host(out))
        l = lse.cpu().numpy().astype(np.float64)
        for i in range(len(self.lens)) if only is None else only:
            (k, km), (v, vm) = self.rows(i, window)
            ref, rlse, p, s = decode.attention(self.q[i], k, v, self.scale)
            n = k.shape[0]
            if n == 0:
                assert not o[i].any() and np.isneginf(l[i]).all()
                continue
            qa = np.abs(oracle.bf16_bits_to_f64(self.q[i]))
            for h in range(self.heads):
                S = abs(self.scale) * (km[:, h // self.group] @ qa[h])
                ep = np.max((self.D + 8) * 2.0 ** -23 * S + 2.0 ** -22 * np.abs(s[h])) + 2.0 ** -22
                el = ep + (n + 40) * 2.0 ** -23
                A = p[h] @ vm[:, h // self.group]
                bound = 2.0 ** -8 * np.abs(ref[h]) + (el + ep + 2.0 ** -16 + (n + 40) * 2.0 ** -23) * A * 1.01
                assert (np.abs(o[i, h] - ref[h]) <= bound).all(), (i, h, np.max(np.abs(o[i, h] - ref[h]) / bound))
                lb = 1.01 * el + 2.0 ** -22 * (abs(rlse[h]) + np.max(np.abs(s[h])) + 1)
                assert abs(l[i, h] - rlse[h]) <= lb, (i, h, l[i, h], rlse[h], lb)


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 100, 127, 128, 129, 0, 300, 5]


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_lengths(form, D, page):
    say("[attn] %s D=%d page=%d" % (form, D, page))
    s = Setup(form, LENS, 2, 3, D, page, seed=D + page)
    s.check(*s.run())


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (3, 1), (2, 16), (1, 17), (2, 40), (5, 6)])
def test_head_layouts(form, kv_heads, group):
    say("[attn] %s kv=%d group=%d" % (form, kv_heads, group))
    s = Setup(form, [77, 1, 260], kv_heads, group, 128, 32, seed=group)
    s.check(*s.run())


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("group", [1, 4, 5, 8, 9, 16])
def test_q4_head_replicas(D, group):
    """The heads a kv head has decide how many matrix columns hold copies of them."""
    s = Setup("q4", [90, 33, 0, 400], 2, group, D, 16, seed=D + group)
    s.check(*s.run())


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("seqs,kv_heads,width",
                         [(150, 1, 40), (150, 1, 400), (300, 2, 40), (300, 2, 400), (70, 4, 400)])
def test_many_sequences(form, seqs, kv_heads, width):
    """Batches counted in several rounds of 64 lengths, batches that are not split at all, short and long tables."""
    rng = np.random.default_rng(seqs)
    lens = np.minimum((rng.random(seqs) ** 4 * 700).astype(int), 640)
    lens[[0, 63, 64, seqs - 1]] = [640, 0, 1, 333]
    s = Setup(form, lens, kv_heads, 1, 64, 16, seed=seqs + width, width=width, share=True, junk=False)
    s.check(*s.run())


def test_largest_pages():
    """Pages of 65536 tokens and a table of 2^30 positions (the lengths' sum no longer counted in 32 bits)."""
    s = Setup("e4m3", [70, 66000, 0, 65537], 1, 2, 64, 65536, seed=14, width=16384, share=True, junk=False)
    s.check(*s.run())
    s.check(*s.run(1000), 1000)


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("window", [1, 15, 16, 33, 100, 4096, 2 ** 31 - 1])
def test_windows(form, window):
    s = Setup(form, LENS, 1, 4, 64, 16, seed=window, window=window)
    s.check(*s.run(window), window)


@pytest.mark.parametrize("form", kv_layout.FORMATS)
def test_long_and_ragged(form):
    """Splits of the length (many for the long sequence, one for the short), shared pages."""
    s = Setup(form, [5000, 3, 1300, 0, 4999, 640], 2, 4, 128, 64, seed=4, share=True, junk=False)
    s.check(*s.run())


@pytest.mark.parametrize("form", kv_layout.FORMATS)
def test_wide_table_and_repeatability(form):
    """A table far wider than the lengths (other split sizes), and the same bits from a second call."""
    s = Setup(form, [200, 7, 900], 2, 8, 128, 16, seed=5, width=3000)
    a = s.run()
    s.check(*a)
    b = s.run()
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("form", kv_layout.FORMATS)
def test_bad_pages_and_lengths(form):
    """Table entries outside the cache count as absent positions and are counted; lengths outside the table are cut.
    Every access stays inside the cache and the table by the kernel's own checks."""
    page, n = 16, 100
    s = Setup(form, [n, n, n, n, n], 2, 2, 64, page, seed=6, junk=False)
    table = s.table.copy()
    table[0, 2] = -1
    table[1, :] = s.pages                       # nothing left
    table[2, 6] = np.iinfo(np.int32).max        # the last, partial page
    table[3, 0] = np.iinfo(np.int32).min
    lens = s.lens.copy()
    lens[4] = 1 << 30                           # cut to the table: 112 positions
    counters = torch.zeros(1 + 1, dtype=torch.int64, device=dev())
    out = torch.empty(5, s.heads, 64, dtype=torch.bfloat16, device=dev())
    lse = torch.empty(5, s.heads, device=dev())
    ws = torch.empty(max(16, w4.kv_cache_attention_workspace(5, s.heads, 2, 64, s.width, page)), dtype=torch.uint8,
                     device=dev())
    w4.kv_cache_attention(bf16_dev(s.q), s.cache, FMT[form], page, 2, to_dev(table), to_dev(lens), s.scale, out, 0, lse,
                          ws, counters)
    torch.cuda.synchronize()
    assert counters[0].item() == 1 + 7 + 1 + 1
    assert not out[1].any() and torch.isneginf(lse[1]).all()
    for i, drop in ((0, 2), (2, 6), (3, 0)):    # the oracle over the remaining positions
        pos = np.array([t for t in range(n) if t // page != drop])
        p, o = s.table[i, pos // page], pos % page
        kv = [decode.row_values(c[p, :, o], None if f is None else f[p, :, o], form) for c, f in (s.k, s.v)]
        ref, rl, _, _ = decode.attention(s.q[i], kv[0], kv[1], s.scale)
        got = oracle.bf16_bits_to_f64(bits_host(out[i]))
        # 2^-8 of the value, and 1e-4 of the values' size (sigma 2) for the sums: far above their roundings
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-3).all()
        np.testing.assert_allclose(lse[i].cpu().numpy(), rl, atol=1e-4)
    s.lens[4] = s.width * page
    s.check(out, lse, only=[4])


@pytest.mark.parametrize("form", kv_layout.FORMATS)
def test_poisoned_rows_pass_on(form):
    """A NaN in an attended row reaches the outputs of its kv head, and no other's."""
    s = Setup(form, [70, 70], 2, 2, 64, 16, seed=7)
    clean, _ = s.run()
    p, o = s.table[1, 40 // 16], 40 % 16
    for which in (0, 1):
        k, v = [(c.copy(), None if f is None else f.copy()) for c, f in (s.k, s.v)]
        c, f = (k, v)[which]
        if form == "bf16":
            c[p, 1, o, 3] = 0x7FC0
        elif form == "e4m3":
            c[p, 1, o], f[p, 1, o] = 0, np.nan
        else:
            c[p, 1, o, :32], f[p, 1, o, 0] = 0, 0x7FC0
        keep = s.cache
        s.cache = to_dev(kv_layout.encode_cache(k, v, form))
        out, lse = s.run()
        s.cache = keep
        assert torch.equal(out[0].view(torch.int16), clean[0].view(torch.int16))
        assert torch.equal(out[1, :2].view(torch.int16), clean[1, :2].view(torch.int16))
        nan = torch.isnan(out[1, 2:].float())
        if which == 0:
            assert nan.all() and torch.isnan(lse[1, 2:]).all()
        elif form == "bf16":
            assert nan[:, 3].all() and nan.sum() == 2
        elif form == "e4m3":
            assert nan.all()
        else:
            assert nan[:, :32].all() and not nan[:, 32:].any()
        assert which == 0 or torch.isfinite(lse).all()


def test_q4_scales_far_apart():
    """V scales that grow, shrink and vanish by many powers of two along a sequence and inside a chunk, up to
    rows that outweigh all others by 2^60."""
    for seed, draw in enumerate((lambda r, n: r.integers(-3, 4, n), lambda r, n: r.integers(-20, 20, n),
                                 lambda r, n: np.arange(n) // 8 - 20, lambda r, n: 20 - np.arange(n) // 4,
                                 lambda r, n: np.where(r.random(n) < 0.02, 60, r.integers(-60, 0, n)))):
        s = Setup("q4", [600, 33], 1, 4, 64, 16, seed=20 + seed)
        rng = np.random.default_rng(seed)
        codes, scales = s.v
        f = oracle.bf16_bits_to_f64(scales).copy()
        f[np.isnan(f)] = 1.0
        for i, n in enumerate(s.lens):
            pos = np.arange(n)
            f[s.table[i, pos // 16], 0, pos % 16] *= 2.0 ** draw(rng, int(n))[:, None]
            zero = pos[rng.random(int(n)) < 0.1]
            f[s.table[i, zero // 16], 0, zero % 16] = 0.0
            codes[s.table[i, zero // 16], 0, zero % 16] = 0
        s.v = (codes, oracle.bf16_from_f64(f))
        s.cache = to_dev(kv_layout.encode_cache(s.k, s.v, "q4"))
        s.check(*s.run())


def test_large_scores():
    """Scores of several hundred: only the largest position counts, and nothing overflows."""
    s = Setup("bf16", [200], 1, 4, 64, 16, seed=8)
    s.scale = 40.0
    s.check(*s.run())


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 3.0])
def test_scales(form, scale):
    """Any finite scale: zero averages the values, a negative one turns the order round."""
    s = Setup(form, [45, 170, 1], 2, 3, 64, 16, seed=15)
    s.scale = scale
    s.check(*s.run())


def test_infinite_scores():
    """K rows of -inf give the position no weight; a sequence that has only such positions counts as empty."""
    s = Setup("bf16", [40, 20], 1, 1, 64, 16, seed=9)
    q = np.abs(oracle.bf16_bits_to_f64(s.q)) + 0.5
    s.q = oracle.bf16_from_f64(q)
    for i, pos in ((0, [0, 17, 39]), (1, range(20))):
        for t in pos:
            s.k[0][s.table[i, t // 16], 0, t % 16] = 0xFF80
    s.cache = to_dev(kv_layout.encode_cache(s.k, s.v, "bf16"))
    out, lse = s.run()
    keep = np.array([t for t in range(40) if t not in (0, 17, 39)])
    p, o = s.table[0, keep // 16], keep % 16
    ref, rl, _, _ = decode.attention(s.q[0], oracle.bf16_bits_to_f64(s.k[0][p, :, o]),
                                     oracle.bf16_bits_to_f64(s.v[0][p, :, o]), s.scale)
    assert (np.abs(oracle.bf16_bits_to_f64(bits_host(out[0])) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-3).all()
    np.testing.assert_allclose(lse[0].cpu().numpy(), rl, atol=1e-4)
    assert not out[1].any() and torch.isneginf(lse[1]).all()


def test_strided_queries_streams_and_graphs():
    """q as a slice of a fused projection; two captured graphs with workspaces of their own on two streams, replayed
    together with new lengths, against the eager calls."""
    a = Setup("q4", [700, 33, 1500], 2, 4, 128, 32, seed=10, share=True, junk=False)
    b = Setup("e4m3", [90, 2000], 1, 8, 128, 16, seed=11, share=True, junk=False)
    jobs = []
    for s in (a, b):
        qkv = torch.zeros(len(s.lens), (s.heads + 2) * s.D, dtype=torch.bfloat16, device=dev())
        qkv[:, s.D:(s.heads + 1) * s.D] = bf16_dev(s.q).flatten(1)
        n = len(s.lens)
        need = w4.kv_cache_attention_workspace(n, s.heads, s.kv_heads, s.D, s.width, s.page)
        assert need > 0
        job = dict(q=qkv[:, s.D:(s.heads + 1) * s.D].unflatten(1, (s.heads, s.D)), lens=to_dev(s.lens),
                   table=to_dev(s.table), out=torch.zeros(n, s.heads, s.D, dtype=torch.bfloat16, device=dev()),
                   lse=torch.zeros(n, s.heads, device=dev()), ws=torch.empty(need, dtype=torch.uint8, device=dev()),
                   stream=torch.cuda.Stream(), graph=torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(job["graph"], stream=job["stream"]):
            w4.kv_cache_attention(job["q"], s.cache, FMT[s.form], s.page, s.kv_heads, job["table"], job["lens"],
                                  s.scale, job["out"], 0, job["lse"], job["ws"])
        jobs.append(job)
    for step in range(3):
        for s, job in zip((a, b), jobs):
            s.lens = np.maximum(s.lens - 31 * step, 0).astype(np.int32)
            job["lens"].copy_(to_dev(s.lens))
        torch.cuda.synchronize()
        for _ in range(4):
            for job in jobs:
                with torch.cuda.stream(job["stream"]):
                    job["graph"].replay()
        torch.cuda.synchronize()
        for s, job in zip((a, b), jobs):
            s.check(job["out"], job["lse"])
            eager = s.run()
            assert torch.equal(eager[0].view(torch.int16), job["out"].view(torch.int16))
            assert torch.equal(eager[1], job["lse"])


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: pages at its far end are written, read and attended to."""
    page, heads, D = 64, 8, 128
    per = w4.kv_cache_page_bytes(w4.W4_KV_BF16, page, heads, D)
    pages = (1 << 32) // per + 40
    cache = torch.empty(pages, per, dtype=torch.uint8, device=dev())
    rng = np.random.default_rng(13)
    n = 150
    table = np.array([[pages - 1, pages - 7, 3]], dtype=np.int32)
    pos = np.arange(n)
    slots = (table[0, pos // page].astype(np.int64) * page + pos % page)
    k, v = rnd(rng, n, heads, D), rnd(rng, n, heads, D)
    w4.kv_cache_write(bf16_dev(k), bf16_dev(v), to_dev(slots), w4.W4_KV_BF16, page, cache)
    ko = torch.empty(n, heads, D, dtype=torch.bfloat16, device=dev())
    vo = torch.empty_like(ko)
    w4.kv_cache_read(cache, w4.W4_KV_BF16, page, to_dev(slots), ko, vo)
    q = rnd(rng, 1, heads, D)
    out, lse = w4.kv_attention(bf16_dev(q), cache, w4.W4_KV_BF16, page, heads, to_dev(table),
                               to_dev(np.array([n], dtype=np.int32)), D ** -0.5)
    torch.cuda.synchronize()
    assert np.array_equal(bits_host(ko), k) and np.array_equal(bits_host(vo), v)
    ref, rl, _, _ = decode.attention(q[0], oracle.bf16_bits_to_f64(k), oracle.bf16_bits_to_f64(v), D ** -0.5)
    assert (np.abs(oracle.bf16_bits_to_f64(bits_host(out[0])) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-4).all()
    np.testing.assert_allclose(lse[0].cpu().numpy(), rl, atol=1e-5)


@pytest.mark.parametrize("form", kv_layout.FORMATS)
def test_rows_behind_the_batch_stay(form):
    """Outputs, lse and workspace of exactly the stated size: nothing past them is written, split or not."""
    for lens in ([40, 0, 70], [3000, 1, 900]):
        s = Setup(form, lens, 2, 5, 128, 16, seed=31, junk=False)
        n, need = len(lens), w4.kv_cache_attention_workspace(len(lens), s.heads, 2, 128, s.width, 16)
        out = torch.full((n + 2, s.heads, 128), 7.0, dtype=torch.bfloat16, device=dev())
        lse = torch.full((n + 2, s.heads), 7.0, device=dev())
        ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device=dev())
        w4.kv_cache_attention(bf16_dev(s.q), s.cache, FMT[form], 16, 2, to_dev(s.table), to_dev(s.lens), s.scale,
                              out[:n], 0, lse[:n], ws[:need] if need else None)
        torch.cuda.synchronize()
        assert (out[n:] == 7).all() and (lse[n:] == 7).all() and (ws[need:] == 0x5A).all()
        s.check(out[:n], lse[:n])


def test_helpers_on_another_stream():
    """The allocating helpers on a stream that is not the current one, as a torch stream and as a raw handle: what they
    allocate belongs to that stream, so work that the current stream does meanwhile in memory of the same sizes does not
    reach it."""
    s = Setup("q4", [1500, 33], 2, 4, 128, 32, seed=32, share=True, junk=False)
    want, wl = s.run()
    x = bf16_dev(rnd(s.rng, 4, 2816))
    w = bf16_dev(rnd(s.rng, 2816))
    wy, _ = w4.add_rmsnorm(x, x, w, 1e-6)
    wq, ws, _ = w4.add_rmsnorm_quantize(x, x, w, 1e-6)
    args = (bf16_dev(s.q), s.cache, FMT["q4"], 32, 2, to_dev(s.table), to_dev(s.lens), s.scale)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        busy = torch.zeros(1 << 26, device=dev())
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                busy.add_(1.0)      # the calls below start after this
        out, lse = w4.kv_attention(*args, stream=stream)
        y, r = w4.add_rmsnorm(x, x, w, 1e-6, stream=stream)
        q, sc, r2 = w4.add_rmsnorm_quantize(x, x, w, 1e-6, stream=stream)
        need = w4.kv_cache_attention_workspace(2, 8, 2, 128, s.width, 32)
        other = [torch.full((n,), 0xA5, dtype=torch.uint8, device=dev())
                 for n in (need, out.nbytes, lse.nbytes, y.nbytes)]
        torch.cuda.synchronize()
        assert all((o == 0xA5).all() for o in other)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wl)
        assert torch.equal(y.view(torch.int16), wy.view(torch.int16)) and torch.equal(q, wq) and torch.equal(sc, ws)
        assert torch.equal(r.view(torch.int16), r2.view(torch.int16))


@pytest.mark.parametrize("form", kv_layout.FORMATS)
@pytest.mark.parametrize("kv_heads,group", [(1024, 1), (300, 3), (1024, 16)])
def test_most_heads(form, kv_heads, group):
    """Up to the 1024 kv heads and 16384 query heads of the limits."""
    s = Setup(form, [33, 5], kv_heads, group, 64, 16, seed=33)
    s.check(*s.run())
