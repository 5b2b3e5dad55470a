"""GPU parity of w4a16_sample against oracle/serving.py: tokens exactly (both sides
weigh and add in 64 bits), log probabilities to half an fp32 step and 2^-40 of
their sums."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from oracle import serving
from gpu_util import bf16_dev, dev, say

pytestmark = pytest.mark.gpu


def run(z, temperature=None, top_k=None, top_p=None, min_p=None, uniform=None, dtype="f32", stride=0):
    """z: float64 rows that dtype holds exactly; settings: a value or one a row."""
    rows, V = z.shape
    d = bf16_dev(oracle.bf16_from_f64(z)) if dtype == "bf16" else torch.tensor(z, dtype=torch.float32, device=dev())
    if stride:
        wide = torch.full((rows, V + stride), float("nan"), dtype=d.dtype, device=dev())
        wide[:, 1:1 + V] = d
        d = wide[:, 1:1 + V]
    f = lambda v, t: None if v is None else torch.tensor(np.broadcast_to(v, rows).copy(), dtype=t, device=dev())
    u = np.zeros(rows) if uniform is None else np.broadcast_to(uniform, rows)
    tokens, lp = w4.sample(d, f(u, torch.float32), f(temperature, torch.float32), f(top_k, torch.int32),
                           f(top_p, torch.float32), f(min_p, torch.float32))
    torch.cuda.synchronize()
    at = lambda v, i, default: default if v is None else np.broadcast_to(v, rows)[i]
    for i in range(rows):
        token, want, kept = serving.sample(z[i], at(temperature, i, 1.0), int(at(top_k, i, 0)), at(top_p, i, 1.0),
                                           at(min_p, i, 0.0), u[i])
        got = lp[i].item()
        assert tokens[i].item() == token, (i, tokens[i].item(), token, len(kept))
        close = abs(got - want) <= abs(want) * 2.0 ** -24 + 2.0 ** -40
        assert close or (np.isnan(got) and np.isnan(want)), (i, got, want)
    return tokens.cpu().numpy(), lp.cpu().numpy()


def logits(rng, rows, V, dtype, sigma=2.0, peak=18.0):
    z = sigma * rng.standard_normal((rows, V))
    head = min(V, 500)
    for i in range(rows):
        ids = rng.permutation(V)[:head]
        z[i, ids] = np.maximum(z[i, ids], peak - rng.uniform(1.2, 3) * np.log(np.arange(1, head + 1)))
    if dtype == "bf16":
        return oracle.bf16_bits_to_f64(oracle.bf16_from_f64(z))
    return z.astype(np.float32).astype(np.float64)


SIZES = [(1, 1), (3, 2), (5, 63), (2, 64), (4, 65), (7, 1000), (3, 2047), (2, 4097), (64, 8192), (5, 32771),
         (2, 131072), (3, 200003), (1, 1 << 20)]


@pytest.mark.parametrize("rows,V", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mixed_settings(rows, V, dtype):
    say("[sample] rows=%d vocab=%d %s" % (rows, V, dtype))
    rng = np.random.default_rng(V + rows)
    z = logits(rng, rows, V, dtype)
    pick = lambda *v: rng.choice(v, rows)
    for trial in range(3):
        run(z, pick(0.0, 0.7, 1.0, 1.3), pick(0, 1, 20, 50, 300, 5000), pick(1.0, 0.5, 0.9, 0.95, 0.999),
            pick(0.0, 0.0, 0.01, 0.1), rng.random(rows).astype(np.float32), dtype, stride=trial * 3)
    run(z, uniform=rng.random(rows).astype(np.float32), dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_flat_distributions(dtype):
    """Nuclei of thousands of tokens, and top_k past any candidate list."""
    rng = np.random.default_rng(1)
    z = logits(rng, 6, 50000, dtype, sigma=1.0, peak=3.0)
    u = rng.random(6).astype(np.float32)
    run(z, top_p=[0.1, 0.5, 0.9, 0.99, 0.9999, 0.999999], uniform=u, dtype=dtype)
    run(z, top_k=[100, 1000, 3000, 10000, 49999, 50000], uniform=u, dtype=dtype)
    run(z, min_p=[1e-6, 1e-4, 1e-3, 0.01, 0.1, 0.5], uniform=u, dtype=dtype)
    run(z, temperature=[5.0, 50.0, 1e4, 3.0, 2.0, 1e30], top_k=20000, top_p=0.9, min_p=1e-5, uniform=u, dtype=dtype)


@pytest.mark.parametrize("V", [1, 5, 64, 1000, 40000])
def test_ties(V):
    """All logits equal, and a few values only: order and draw go by the id alone, sums of equal weights are exact."""
    n = 9
    u = (np.arange(n) / n).astype(np.float32)
    z = np.full((n, V), 3.25)
    run(z, uniform=u)
    run(z, top_k=max(1, V // 2), uniform=u)
    run(z, top_p=0.5, uniform=u)
    run(z, top_p=0.25, top_k=max(1, V // 4 * 2), uniform=u, dtype="bf16")
    run(z, min_p=1.0, uniform=u)
    rng = np.random.default_rng(V)
    z = rng.choice([0.0, -1.0, -2.0, 1.0, -0.0], (n, V))
    for kw in (dict(top_k=max(1, V // 3)), dict(top_p=0.3), dict(top_p=0.9, top_k=max(1, V // 2)), dict(min_p=0.2),
               dict(temperature=0.0)):
        run(z, uniform=u, **kw)


def test_masks_and_special_values():
    rng = np.random.default_rng(2)
    V, inf = 3000, np.inf
    z = logits(rng, 12, V, "f32")
    z[0, :] = -inf
    z[1, :] = -inf
    z[1, 1234] = -5.0                       # one token allowed
    z[2, 17] = np.nan
    z[3, 17] = -np.nan
    z[4, [5, 900, 2999]] = inf
    z[5, :] = -3.0e38                       # the type's lowest values, and one above
    z[5, 77] = -2.0e38
    z[6] = np.where(rng.random(V) < 0.99, -inf, z[6])
    z[7, :] = inf
    z[8, :2990] = -np.finfo(np.float32).max
    z[9] = 1e-42 * rng.integers(0, 5, V)    # subnormal logits
    z[9] = z[9].astype(np.float32)
    z[10, 100] = np.finfo(np.float32).max
    z[11] = np.where(np.arange(V) == 2998, 0.0, -inf)
    u = rng.random(12).astype(np.float32)
    run(z, uniform=u)
    run(z, 0.7, 50, 0.9, 0.05, u)
    run(z, 0.0, uniform=u)
    run(z, 1.0, 2000, uniform=u)
    run(z, 3.0, top_p=0.99, uniform=u)
    run(z, float("inf"), uniform=u)
    run(z, float("inf"), top_p=0.5, uniform=u)


def test_special_settings():
    rng = np.random.default_rng(3)
    z = logits(rng, 8, 5000, "f32")
    nan, inf = float("nan"), float("inf")
    u = rng.random(8).astype(np.float32)
    run(z, temperature=[0.0, -1.0, nan, 1e-30, 1e-45, 1e30, inf, 0.01], uniform=u)
    run(z, top_k=[0, -1, -2 ** 31, 2 ** 31 - 1, 5000, 4999, 1, 2], uniform=u)
    run(z, top_p=[0.0, -1.0, nan, 2.0, inf, 1e-30, 1.0, -inf], uniform=u)
    run(z, min_p=[0.0, -1.0, nan, 2.0, inf, 1e-30, 1.0, -inf], uniform=u)
    below = np.nextafter(np.float32(1), np.float32(0))
    for kw in (dict(), dict(top_k=7), dict(top_p=0.8)):
        run(z, uniform=np.array([0.0, -1.0, nan, 1.0, 5.0, below, inf, -inf], dtype=np.float32), **kw)


@pytest.mark.parametrize("kw", [dict(), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.01), dict(temperature=1.5)])
def test_draws_follow_the_distribution(kw):
    """Evenly spaced numbers meet each token as often as its share says, up to one at each of its two borders."""
    rng = np.random.default_rng(4)
    n, V = 4096, 300
    one = logits(rng, 1, V, "f32", peak=6.0)
    z = np.broadcast_to(one, (n, V)).copy()
    tokens, _ = run(z, uniform=((np.arange(n) + 0.5) / n).astype(np.float32), **kw)
    t = kw.get("temperature", 1.0)
    _, _, kept = serving.sample(one[0], t, kw.get("top_k", 0), kw.get("top_p", 1.0), kw.get("min_p", 0.0))
    w = np.exp((one[0][kept] - one[0].max()) / t)
    share = np.zeros(V)
    share[kept] = w / w.sum()
    assert (np.abs(np.bincount(tokens, minlength=V) - n * share) <= 1.0 + 1e-3).all()


def test_rows_behind_and_strides():
    rng = np.random.default_rng(5)
    z = torch.tensor(logits(rng, 6, 999, "f32"), dtype=torch.float32, device=dev())
    u = torch.rand(6, device=dev())
    tokens = torch.full((6,), -9, dtype=torch.int32, device=dev())
    lp = torch.full((6,), 9.0, device=dev())
    ws = torch.full((max(16, w4.w4a16_sample_workspace(3, 999)),), 255, dtype=torch.uint8, device=dev())
    w4.w4a16_sample(z[::2], u[:3], tokens, logprobs=lp, ws=ws)
    want, wlp = w4.sample(z[::2].contiguous(), u[:3])
    w4.w4a16_sample(z[:2], u, tokens[4:], ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(tokens[:3], want) and torch.equal(lp[:3], wlp)
    assert tokens[3].item() == -9 and (lp[3:] == 9).all()


@pytest.mark.parametrize("rows,V", [(1, 20000), (50, 3001)])
def test_graph_replays(rows, V):
    rng = np.random.default_rng(6)
    z = torch.tensor(logits(rng, rows, V, "f32"), dtype=torch.float32, device=dev())
    u = torch.rand(rows, device=dev())
    k = torch.full((rows,), 30, dtype=torch.int32, device=dev())
    p = torch.full((rows,), 0.9, device=dev())
    tokens, lp = torch.empty(rows, dtype=torch.int32, device=dev()), torch.empty(rows, device=dev())
    ws = torch.empty(max(16, w4.w4a16_sample_workspace(rows, V)), dtype=torch.uint8, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4a16_sample(z, u, tokens, None, k, p, None, lp, ws)
    for i in range(6):
        u.uniform_()
        k.fill_([30, 0, 2000, 1, 5, 100][i])
        p.fill_([0.9, 1.0, 0.99, 0.5, 0.999, 0.7][i])
        ws.fill_(255)
        g.replay()
        want, wlp = w4.sample(z, u, None, k, p)
        torch.cuda.synchronize()
        assert torch.equal(tokens, want) and torch.equal(lp, wlp)


@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 8, 9, 15, 17, 1023, 1025, 2048, 2049, 2060, 4500, 16384, 16385, 17000,
                               32768])
def test_vocabularies_around_the_pieces(V):
    rng = np.random.default_rng(V)
    for dtype in ("f32", "bf16"):
        z = logits(rng, 12, V, dtype, sigma=1.0, peak=6.0)
        u = rng.random(12).astype(np.float32)
        run(z, uniform=u, dtype=dtype, stride=1)
        run(z, top_k=rng.integers(1, V + 2, 12), uniform=u, dtype=dtype, stride=3)
        run(z, top_p=rng.uniform(0, 1, 12).astype(np.float32), uniform=u, dtype=dtype, stride=7)
        run(z, min_p=np.exp(rng.uniform(-8, 0, 12)).astype(np.float32), uniform=u, dtype=dtype)


@pytest.mark.parametrize("where", ["spread", "together"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cuts_of_every_length(where, dtype):
    """top_k, top_p and min_p that keep from one token to most of them, the likely ones spread over the vocabulary or
    next to one another: whichever way the row is cut."""
    rng = np.random.default_rng(7)
    V, n = 40000, 24
    z = logits(rng, n, V, dtype, sigma=1.5, peak=10.0)
    if where == "together":
        z = np.sort(z, axis=1)[:, ::-1].copy()
        z = np.concatenate([z[:, 300:20300], z[:, :300], z[:, 20300:]], 1)
    u = rng.random(n).astype(np.float32)
    ks = [1, 2, 16, 17, 50, 63, 64, 65, 66, 100, 191, 192, 193, 256, 500, 1000, 1500, 2000, 2048, 2049, 5000, 20000,
          39999, 40000]
    ps = 1 - np.exp(np.linspace(np.log(0.9), np.log(1e-7), n))
    ms = np.exp(np.linspace(-0.01, -20, n))
    run(z, top_k=ks, uniform=u, dtype=dtype)
    run(z, top_p=ps.astype(np.float32), uniform=u, dtype=dtype)
    run(z, min_p=ms.astype(np.float32), uniform=u, dtype=dtype)
    run(z, 1.7, ks, ps[::-1].astype(np.float32), None, u, dtype)
    run(z, 0.6, ks[::-1], ps.astype(np.float32), ms.astype(np.float32), u, dtype)
    run(z, 2.5, None, ps.astype(np.float32), ms[::-1].astype(np.float32), u, dtype)


def test_masked_beside_filters():
    """Most of the vocabulary at -infinity, or at the type's lowest value: fewer logits than top_k, chunks without any."""
    rng = np.random.default_rng(8)
    V = 70000
    z = logits(rng, 9, V, "f32")
    for i, share in enumerate([0.5, 0.9, 0.99, 0.999, 0.9999, 0.99999]):
        z[i, rng.random(V) < share] = -np.inf
        z[i, 69999 - i] = 1.0
    z[6, 16384:] = -np.inf
    z[7, :65536] = -np.inf
    z[8, 100:] = -np.finfo(np.float32).max
    u = rng.random(9).astype(np.float32)
    for kw in (dict(), dict(top_k=50), dict(top_k=1000), dict(top_p=0.95), dict(top_p=0.9999, temperature=2.0),
               dict(min_p=0.001), dict(top_k=3000, top_p=0.99, min_p=1e-6)):
        run(z, uniform=u, **kw)


def test_the_same_from_run_to_run():
    """Sums do not depend on the order in which workgroups and atomics finish: tokens and log probabilities are equal
    bit for bit, in rows cut in every way."""
    rng = np.random.default_rng(9)
    z = torch.tensor(logits(rng, 40, 60000, "f32", sigma=1.5, peak=9.0), dtype=torch.float32, device=dev())
    pick = lambda values, t: torch.tensor(rng.choice(values, 40), dtype=t, device=dev())
    k, p = pick([0, 0, 40, 70, 1000, 9000], torch.int32), pick([1.0, 0.9, 0.99, 0.9999], torch.float32)
    m, u = pick([0.0, 0.0, 1e-3], torch.float32), torch.rand(40, device=dev())
    tokens, lp = w4.sample(z, u, None, k, p, m)
    for _ in range(5):
        again, lp2 = w4.sample(z, u, None, k, p, m)
        torch.cuda.synchronize()
        assert torch.equal(tokens, again) and torch.equal(lp, lp2)


@pytest.mark.parametrize("V", [2048, 70000])
def test_many_candidates_alike(V):
    """Hundreds of equal logits around the cuts, and nearly equal ones beside a far larger one: candidates that share a
    bin of the order."""
    rng = np.random.default_rng(V)
    z = np.full((6, V), -4.0)
    for i, n in enumerate([200, 256, 257, 300, 900, 1500]):
        z[i, rng.permutation(V)[:n]] = 2.0
        z[i, rng.permutation(V)[:40]] = 2.5
    u = rng.random(6).astype(np.float32)
    for k in (30, 100, 290, 700, 1300):
        run(z, top_k=k, uniform=u)
        run(z, 0.7, k, 0.8, None, u)
    run(z, top_p=0.5, uniform=u)
    run(z, top_p=0.5, min_p=0.7, uniform=u)
    z = (rng.standard_normal((6, V)) * 1e-3).astype(np.float32).astype(np.float64)
    z[:, V // 2] = 30.0
    for k in (60, 500, 1000):
        run(z, top_k=k, uniform=u)
        run(z, 40.0, k, 0.9, None, u)


def test_weights_far_below_the_largest():
    """Positive weights under 2^-53 of the largest one are kept and counted like others, and drawn by numbers at the
    end."""
    V = 40000
    rng = np.random.default_rng(3)
    z = np.full((4, V), -300.0)
    at = rng.permutation(V)[:600]
    z[:, at] = -60.0 - np.sort(rng.random(600)).astype(np.float32)
    z[:, 20000] = 0.0
    u = np.array([0.0, 0.5, 1.0 - 2.0 ** -24, 1.0])
    for k in (100, 400, 601):
        run(z, top_k=k, uniform=u)
        run(z, 0.5, k, uniform=u)
    run(z, top_p=1.0 - 2.0 ** -24, uniform=u)
    run(z, min_p=1e-30, uniform=u)


@pytest.mark.parametrize("rows", [1, 3, 20, 100, 300])
def test_long_nuclei_in_every_number_of_rows(rows):
    """Rows that the candidates do not decide, among others that they do, however many workgroups share them; one
    workspace for all calls, in a graph beside eager calls of other rows."""
    rng = np.random.default_rng(rows)
    V = 40000
    z = logits(rng, rows, V, "f32", sigma=1.0, peak=7.0)
    u = rng.random(rows).astype(np.float32)
    p = np.where(np.arange(rows) % 3 == 0, 0.99, 0.5).astype(np.float32)
    k = np.where(np.arange(rows) % 5 == 2, 9000, 0)
    tokens, lp = run(z, 1.5, k, p, None, u)
    d = lambda v, t: torch.tensor(np.ascontiguousarray(v), dtype=t, device=dev())
    ws = torch.empty(w4.w4a16_sample_workspace(rows, V), dtype=torch.uint8, device=dev())
    out, out_lp = torch.empty(rows, dtype=torch.int32, device=dev()), torch.empty(rows, device=dev())
    args = [d(z, torch.float32), d(u, torch.float32), out, torch.full((rows,), 1.5, device=dev()), d(k, torch.int32),
            d(p, torch.float32), None, out_lp, ws]
    other = list(args)
    other[0], other[2] = torch.flip(args[0], [0]).contiguous(), torch.empty_like(out)
    w4.w4a16_sample(*args)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        w4.w4a16_sample(*args)
    for _ in range(3):
        out.fill_(-7)
        w4.w4a16_sample(*other)
        g.replay()
        torch.cuda.synchronize()
        assert (out.cpu().numpy() == tokens).all() and (out_lp.cpu().numpy() == lp).all()


def test_two_streams_at_once():
    """Calls that overlap in time, each with its own workspace: long nuclei among their rows, whose histograms several
    workgroups join."""
    rng = np.random.default_rng(17)
    rows, V = 12, 40000
    u = rng.random(rows).astype(np.float32)
    p = np.where(np.arange(rows) % 2 == 0, 0.99, 0.6).astype(np.float32)
    calls = []
    for sigma in (1.0, 1.3):
        z = logits(rng, rows, V, "f32", sigma=sigma, peak=7.0)
        tokens, lp = run(z, 1.5, None, p, None, u)
        d = lambda v: torch.tensor(v, dtype=torch.float32, device=dev())
        out, out_lp = torch.empty(rows, dtype=torch.int32, device=dev()), torch.empty(rows, device=dev())
        ws = torch.empty(w4.w4a16_sample_workspace(rows, V), dtype=torch.uint8, device=dev())
        calls.append((tokens, lp, [d(z), d(u), out, d(np.full(rows, 1.5)), None, d(p), None, out_lp, ws]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for (_, _, args), s in zip(calls, streams):
            w4.w4a16_sample(*args, stream=s)
    torch.cuda.synchronize()
    for tokens, lp, args in calls:
        assert (args[2].cpu().numpy() == tokens).all() and (args[7].cpu().numpy() == lp).all()
