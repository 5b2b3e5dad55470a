"""Decode steps of one attention layer and a sampled token, as a server runs them: the plan, a quantized projection with
its adapters, rotary positions, cache write, attention over the cache, logits, the draw -- eagerly against the oracle's
steps, and from one captured graph that is replayed as the sequences grow."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from oracle import decode, serving
from gpu_util import bf16_dev, bits_host, dev, linear_weights, to_dev

pytestmark = pytest.mark.gpu

SEQS, D, HQ, HK, DIM, PAGE, VOCAB = 9, 256, 4, 2, 64, 16, 1024
WIDTH, PAGES = 4, 24


class Step:
    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        n_qkv = (HQ + 2 * HK) * DIM
        self.embed = oracle.bf16_from_f64(rng.standard_normal((VOCAB, D)))
        self.w = [linear_weights(rng, n, D) for n in (n_qkv, VOCAB)]
        self.wd = [(to_dev(p), bf16_dev(s)) for p, s, _, _ in self.w]
        self.wo = linear_weights(rng, D, HQ * DIM)
        self.wod = (to_dev(self.wo[0]), bf16_dev(self.wo[1]))
        self.a = oracle.bf16_from_f64(rng.standard_normal((3, 8, D)) / 16)
        self.b = oracle.bf16_from_f64(rng.standard_normal((3, n_qkv, 8)))
        self.ids = rng.integers(-1, 3, SEQS).astype(np.int32)
        self.scaling = rng.uniform(0.5, 2, 3).astype(np.float32)
        self.freq, _ = w4.rope_frequencies(DIM)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev())
        self.lens, self.table, self.count, self.new = i32(SEQS), i32(SEQS, WIDTH), i32(1), i32(SEQS)
        self.free = torch.tensor(rng.permutation(PAGES), dtype=torch.int32, device=dev())
        self.count.fill_(PAGES)
        self.offsets, self.slots = i32(SEQS + 1), torch.zeros(SEQS, dtype=torch.int64, device=dev())
        self.positions = i32(SEQS)
        self.cache = w4.kv_cache(PAGES, w4.W4_KV_BF16, PAGE, HK, DIM)
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev())
        self.x, self.base, self.qkv, self.att = bf(SEQS, D), bf(SEQS, n_qkv), bf(SEQS, n_qkv), bf(SEQS, HQ, DIM)
        self.q, self.kk, self.h, self.z = bf(SEQS, HQ, DIM), bf(SEQS, HK, DIM), bf(SEQS, D), bf(SEQS, VOCAB)
        self.tokens, self.u = torch.tensor(rng.integers(0, VOCAB, SEQS), dtype=torch.int32, device=dev()), torch.zeros(
            SEQS, device=dev())
        self.logprobs = torch.zeros(SEQS, device=dev())
        self.k = torch.full((SEQS,), 50, dtype=torch.int32, device=dev())
        self.p = torch.full((SEQS,), 0.9, device=dev())
        self.embed_d, self.a_d, self.b_d = bf16_dev(self.embed), bf16_dev(self.a), bf16_dev(self.b)
        self.ids_d, self.scaling_d, self.freq_d = to_dev(self.ids), to_dev(self.scaling), self.freq.to(dev())
        self.scale_t = torch.full((SEQS,), 40.0, device=dev())
        need = max(w4.w4a16_linear_workspace(SEQS, D, n_qkv), w4.w4a16_linear_workspace(SEQS, D, VOCAB),
                   w4.w4a16_linear_workspace(SEQS, HQ * DIM, D),
                   w4.w4a16_lora_workspace(SEQS, D, n_qkv, 3, 8), w4.w4a16_sample_workspace(SEQS, VOCAB),
                   w4.kv_cache_attention_workspace(SEQS, HQ, HK, DIM, WIDTH, PAGE), 16)
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev())

    def run(self):
        w4.kv_cache_plan(self.lens, self.new, self.table, PAGE, self.free, self.count, self.lens, self.count,
                         self.offsets, self.slots, self.positions)
        torch.index_select(self.embed_d, 0, self.tokens, out=self.x)
        w4.w4a16_linear(self.x, *self.wd[0], self.qkv.shape[1], self.base, self.ws)
        w4.w4a16_lora_add(self.x, self.ids_d, self.a_d, self.b_d, self.scaling_d, self.base, self.qkv, self.ws)
        q = self.qkv[:, :HQ * DIM].view(SEQS, HQ, DIM)
        k = self.qkv[:, HQ * DIM:(HQ + HK) * DIM].view(SEQS, HK, DIM)
        v = self.qkv[:, (HQ + HK) * DIM:].view(SEQS, HK, DIM)
        w4.w4a16_rope(q, k, self.positions, self.freq_d, self.q, self.kk)
        w4.kv_cache_write(self.kk, v, self.slots, w4.W4_KV_BF16, PAGE, self.cache)
        w4.kv_cache_attention(self.q, self.cache, w4.W4_KV_BF16, PAGE, HK, self.table, self.lens, DIM ** -0.5, self.att,
                              ws=self.ws)
        w4.w4a16_linear(self.att.view(SEQS, HQ * DIM), *self.wod, D, self.h, self.ws)
        w4.w4a16_linear(self.h, *self.wd[1], VOCAB, self.z, self.ws)
        w4.w4a16_sample(self.z, self.u, self.tokens, self.scale_t, self.k, self.p, None, self.logprobs, self.ws)


def close(got_bits, want):
    ok, mx, rms = oracle.within_tolerance(oracle.bf16_bits_to_f64(got_bits), want)
    assert ok, (mx, rms)


def test_steps_against_the_oracle():
    """Every stage is checked against the oracle's, fed the stage's own input from the device."""
    s = Step(1)
    rng = np.random.default_rng(2)
    held = [([], []) for _ in range(SEQS)]
    lens, table, free, count = np.zeros(SEQS, int), s.table.cpu().numpy().copy(), s.free.cpu().numpy().copy(), PAGES
    for step in range(20):
        s.new.fill_(1)
        s.u.copy_(torch.tensor(rng.random(SEQS), dtype=torch.float32))
        before = s.tokens.cpu().numpy().copy()
        s.run()
        torch.cuda.synchronize()
        want = serving.plan(lens, [1] * SEQS, table, PAGE, free, count, SEQS)
        lens, count = want["lens"], want["count"]
        assert np.array_equal(s.slots.cpu().numpy(), want["slots"]) and np.array_equal(s.lens.cpu().numpy(), lens)
        assert np.array_equal(s.table.cpu().numpy(), table)
        x = s.embed[before]
        assert np.array_equal(bits_host(s.x), x)
        close(bits_host(s.base), oracle.bf16_bits_to_f64(oracle.linear(x, s.w[0][2], s.w[0][3])))
        close(bits_host(s.qkv), serving.lora_add(x, s.ids, s.a, s.b, s.scaling, bits_host(s.base))[0])
        heads = oracle.bf16_bits_to_f64(bits_host(s.qkv)).reshape(SEQS, HQ + 2 * HK, DIM)
        turned = serving.rope(heads[:, :HQ + HK], want["positions"], s.freq.numpy())
        close(bits_host(s.q), turned[:, :HQ])
        close(bits_host(s.kk), turned[:, HQ:])
        got = np.concatenate([bits_host(s.q), bits_host(s.kk), bits_host(s.qkv).reshape(SEQS, -1, DIM)[:, HQ + HK:]], 1)
        out = []
        for i in range(SEQS):
            held[i][0].append(oracle.bf16_bits_to_f64(got[i, HQ:HQ + HK]))
            held[i][1].append(oracle.bf16_bits_to_f64(got[i, HQ + HK:]))
            out.append(decode.attention(got[i, :HQ], np.stack(held[i][0]), np.stack(held[i][1]), DIM ** -0.5)[0])
        close(bits_host(s.att), np.stack(out))
        h = oracle.linear(bits_host(s.att).reshape(SEQS, -1), s.wo[2], s.wo[3])
        close(bits_host(s.h), oracle.bf16_bits_to_f64(h))
        z = oracle.bf16_bits_to_f64(bits_host(s.z))
        for i in range(SEQS):
            token, lp, _ = serving.sample(z[i], 40.0, 50, 0.9, 0.0, s.u[i].item())
            assert s.tokens[i].item() == token and abs(s.logprobs[i].item() - lp) <= abs(lp) * 2.0 ** -24 + 2.0 ** -40


def test_captured_steps_equal_eager_ones():
    eager, other = Step(3), Step(3)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        other.run()
    rng = np.random.default_rng(4)
    for step in range(30):
        new = rng.choice([1, 1, 1, 0, -1], SEQS)
        u = rng.random(SEQS)
        for s in (eager, other):
            s.new.copy_(torch.tensor(new, dtype=torch.int32))
            s.u.copy_(torch.tensor(u, dtype=torch.float32))
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("lens", "table", "free", "count", "slots", "positions", "qkv", "cache", "att", "z", "tokens",
                     "logprobs"):
            assert torch.equal(getattr(eager, name).view(torch.uint8) if getattr(eager, name).dtype == torch.bfloat16
                               else getattr(eager, name),
                               getattr(other, name).view(torch.uint8) if getattr(other, name).dtype == torch.bfloat16
                               else getattr(other, name)), (step, name)
