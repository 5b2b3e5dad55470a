"""GPU parity of kv_cache_plan against oracle/serving.py: whole numbers, compared
exactly."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
from oracle import serving
from gpu_util import dev, say

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev())


class State:
    """The same cache state on the host (for the oracle) and on the device."""

    def __init__(self, rng, lens, width, page, spare, capacity=None):
        self.page, self.width = page, width
        n = len(lens)
        have = [0 if v < 0 or v > width * page else -(-v // page) for v in lens]
        capacity = sum(have) + spare + 3 if capacity is None else capacity
        ids = rng.permutation(sum(have) + spare)
        self.lens = np.array(lens, dtype=np.int64)
        self.table = rng.integers(1000, 2000, (n, width))         # columns that hold nothing
        self.free = rng.integers(3000, 4000, capacity)
        at = 0
        for i in range(n):
            self.table[i, :have[i]] = ids[at:at + have[i]]
            at += have[i]
        self.free[:spare] = ids[at:]
        self.count = spare
        self.d_lens, self.d_table = i32(self.lens), i32(self.table)
        self.d_free, self.d_count = i32(self.free), i32([spare])

    def step(self, new, max_rows, in_place=True, row_seqs=True, counters=True):
        n = len(self.lens)
        out = dict(lens=self.d_lens if in_place else torch.full_like(self.d_lens, -7),
                   count=self.d_count if in_place else torch.full_like(self.d_count, -7),
                   offsets=torch.full((n + 1,), -7, dtype=torch.int32, device=dev()),
                   slots=torch.full((max_rows,), -7, dtype=torch.int64, device=dev()),
                   positions=torch.full((max_rows,), -7, dtype=torch.int32, device=dev()),
                   row_seqs=torch.full((max_rows,), -7, dtype=torch.int32, device=dev()) if row_seqs else None)
        cnt = torch.tensor([100, 200], dtype=torch.int64, device=dev()) if counters else None
        w4.kv_cache_plan(self.d_lens, i32(new), self.d_table, self.page, self.d_free, self.d_count, out["lens"],
                         out["count"], out["offsets"], out["slots"], out["positions"], out["row_seqs"], cnt)
        torch.cuda.synchronize()
        want = serving.plan(self.lens, new, self.table, self.page, self.free, self.count, max_rows)
        for name in ("lens", "offsets", "slots", "positions", "row_seqs"):
            if out[name] is not None:
                assert np.array_equal(out[name].cpu().numpy(), want[name]), name
        assert out["count"].item() == want["count"]
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert np.array_equal(self.d_free.cpu().numpy(), self.free)
        if counters:
            assert (cnt.cpu().numpy() - [100, 200]).tolist() == list(want["counters"])
        if in_place:
            self.lens, self.count = want["lens"], want["count"]
        return want


@pytest.mark.parametrize("seqs", [1, 2, 63, 64, 65, 500, 1023, 1024, 1025, 2500])
@pytest.mark.parametrize("kind", ["decode", "mixed"])
def test_plan(seqs, kind):
    say("[plan] %d sequences, %s" % (seqs, kind))
    rng = np.random.default_rng(seqs)
    page, width = (16, 40) if kind == "mixed" else (64, 9)
    lens = rng.integers(0, 300, seqs)
    new = np.ones(seqs, dtype=np.int64)
    if kind == "mixed":
        new = np.where(rng.random(seqs) < 0.1, rng.integers(0, 300, seqs), new)
        new[rng.random(seqs) < 0.1] = -1
    s = State(rng, lens, width, page, spare=3 + int(np.maximum(new, 0).sum() // page + seqs))
    s.step(new, int(np.maximum(new, 0).sum()) + 9, in_place=False)
    s.step(new, int(np.maximum(new, 0).sum()) + 9, in_place=False, row_seqs=False, counters=False)   # again, same state
    s.step(new, int(np.maximum(new, 0).sum()), in_place=True)


@pytest.mark.parametrize("page", [16, 128, 65536])
def test_pages_and_rows_run_out(page):
    rng = np.random.default_rng(page)
    lens = rng.integers(0, 4 * page, 200)
    new = rng.integers(0, min(3 * page, 700), 200)
    new[rng.random(200) < 0.05] = -2 ** 31
    for spare in (0, 1, 40, 1000):
        for max_rows in (0, 1, 500, 20000):
            s = State(rng, lens, 8, page, spare)
            want = s.step(new, max_rows)
            assert want["counters"][1] > 0 or max_rows == 20000 or spare == 1000


def test_bad_lengths_and_stack():
    rng = np.random.default_rng(9)
    big = 2 ** 31 - 1
    lens = [-1, 65, big, 64, 10, 10, 0, 64, -big - 1, 33]
    new = [1, 1, 1, 1, big, -1, 0, 0, -1, -1]
    s = State(rng, lens, 4, 16, 12)
    want = s.step(new, 50)
    assert want["counters"][0] == 6
    # a stack without room for what comes back, and counts outside of it
    s = State(rng, [64, 64, 30], 4, 16, 6, capacity=8)
    want = s.step([-1, -1, 40], 64)
    assert want["counters"][0] == 6 + 1         # six pages lost; the third sequence is longer than its table
    for count in (-5, 10 ** 9):
        s = State(rng, [5, 5], 4, 16, 6)
        s.count = count
        s.d_count.fill_(count)
        s.step([30, -1], 64)
    # no free pages, no table, nothing at all
    State(rng, [5, 16], 1, 16, 0, capacity=0).step([11, 1], 64)
    State(rng, [0, 0, 3], 0, 16, 4).step([0, 1, -1], 8)
    State(rng, [], 4, 16, 4).step([], 8)


def test_long_prompts_and_ends():
    """Thousands of pages for one sequence, and as many given back."""
    rng = np.random.default_rng(10)
    s = State(rng, [100000, 3, 0, 77777], 16384, 16, 9000)
    s.step([-1, 30000, 60001, -1], 90003)
    s.step([5, -1, 1, 100], 107)


def test_serving_trace():
    """Forty steps of one cache: arrivals, chunks, decoding, ends, shortages; the pages in tables and on the stack stay
    a permutation of all."""
    rng = np.random.default_rng(11)
    page, pages = 16, 400
    s = State(rng, np.zeros(70, dtype=np.int64), 30, page, pages)
    for step in range(40):
        new = np.where(s.lens > 0, 1, 0)
        new[rng.random(70) < 0.1] = rng.integers(1, 120)
        new[(rng.random(70) < 0.06) & (s.lens > 0)] = -1
        new = np.where(s.lens + new > 30 * page, -1, new)
        s.step(new, 900)
        held = [p for i in range(70) for p in s.table[i, :-(-int(s.lens[i]) // page)]]
        assert sorted(held + list(s.free[:s.count])) == list(range(pages))


def test_other_stream_and_graph():
    rng = np.random.default_rng(12)
    s = State(rng, rng.integers(0, 200, 90), 20, 16, 500)
    new = i32(np.ones(90))
    seq = [torch.zeros(91, dtype=torch.int32, device=dev()), torch.zeros(96, dtype=torch.int64, device=dev()),
           torch.zeros(96, dtype=torch.int32, device=dev()), torch.zeros(96, dtype=torch.int32, device=dev())]
    call = lambda: w4.kv_cache_plan(s.d_lens, new, s.d_table, 16, s.d_free, s.d_count, s.d_lens, s.d_count, seq[0],
                                    seq[1], seq[2], seq[3])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        call()
    step = 0
    while True:
        want = serving.plan(s.lens, np.ones(90), s.table, 16, s.free, s.count, 96)
        for got, name in zip([s.d_lens] + seq, ("lens", "offsets", "slots", "positions", "row_seqs")):
            assert np.array_equal(got.cpu().numpy(), want[name]), (step, name)
        assert np.array_equal(s.d_table.cpu().numpy(), s.table)
        s.lens, s.count = want["lens"], want["count"]
        step += 1
        if step == 20:
            break
        graph.replay()
        torch.cuda.synchronize()
