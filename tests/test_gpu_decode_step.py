"""The calls of a decoder layer together, as a decode step makes them: norm,
W4A16 qkv projection, cache write, attention, W4A16 output projection, norm
with the residual, MoE layer (W4A16 and FP8) -- every stage against the oracle
fed the GPU's own input to it -- over several steps, eagerly and from a
captured graph."""

import numpy as np
import pytest
import torch

import gen
import int4_group_quantized_q4_amd as w4
import kv_layout
import oracle
from oracle import decode, fp8
from gpu_util import bf16_dev, bits_host, dev, expert_weights, linear_weights, say, to_dev

pytestmark = pytest.mark.gpu
FMT = {"bf16": w4.W4_KV_BF16, "e4m3": w4.W4_KV_E4M3, "q4": w4.W4_KV_Q4}
T, d, heads, kv_heads, D, page = 5, 256, 8, 2, 64, 16
E, k, I = 8, 2, 128


class Layer:
    def __init__(self, form):
        rng = gen.rng_for(960, FMT[form])
        self.form = form
        N = (heads + 2 * kv_heads) * D
        self.wqkv, self.wo = linear_weights(rng, N, d), linear_weights(rng, d, heads * D)
        self.w1, self.w2 = expert_weights(rng, E, 2 * I, d), expert_weights(rng, E, d, I)
        self.n1, self.n2 = gen.bf16_normal(rng, d), gen.bf16_normal(rng, d)
        self.steps = 4
        self.pages = T * 3 + 1
        self.table = rng.permutation(self.pages)[:T * 3].reshape(T, 3).astype(np.int32)
        self.start = np.array([0, 14, 15, 31, 40])       # lengths before the first step
        self.x0 = [gen.bf16_normal(rng, (T, d)) for _ in range(self.steps)]
        self.logits = [gen.router_logits(rng, T, E) for _ in range(self.steps)]
        self.q1 = gen.fp8_codes(rng, (E, 2 * I, d)), gen.fp8_scales(rng, (E, 2 * I))
        self.past = [gen.bf16_normal(rng, (int(n), 2, kv_heads, D)) for n in self.start]
        b = {}
        b["cache"] = w4.kv_cache(self.pages, FMT[form], page, kv_heads, D)
        for name, shape, dt in (("x", (T, d), torch.bfloat16), ("h", (T, d), torch.bfloat16),
                                ("qkv", (T, N), torch.bfloat16),
                                ("att", (T, heads, D), torch.bfloat16), ("proj", (T, d), torch.bfloat16),
                                ("res", (T, d), torch.bfloat16), ("h2", (T, d), torch.bfloat16),
                                ("y", (T, d), torch.bfloat16),
                                ("q8", (T, d), torch.uint8), ("s8", (T,), torch.float32),
                                ("gmm", (T, 2 * I), torch.float32),
                                ("logits", (T, E), torch.float32), ("lse", (T, heads), torch.float32)):
            b[name] = torch.zeros(shape, dtype=dt, device=dev())
        b["lens"] = torch.zeros(T, dtype=torch.int32, device=dev())
        b["slots"] = torch.zeros(T, dtype=torch.int64, device=dev())
        b["table"] = to_dev(self.table)
        need = max(w4.w4a16_linear_workspace(T, d, N), w4.w4a16_linear_workspace(T, heads * D, d),
                   w4.kv_cache_attention_workspace(T, heads, kv_heads, D, 3, page),
                   w4.w4a16_moe_layer_workspace(T, E, k, d, I), 16)
        b["ws"] = torch.zeros(need, dtype=torch.uint8, device=dev())
        self.b = b
        self.weights = {n: [to_dev(w[0]), bf16_dev(w[1])] for n, w in
                        (("qkv", self.wqkv), ("o", self.wo), ("w1", self.w1), ("w2", self.w2))}
        self.weights["n1"], self.weights["n2"] = bf16_dev(self.n1), bf16_dev(self.n2)
        self.weights["q1"] = [to_dev(self.q1[0][0].reshape(-1)), to_dev(self.q1[1][0].reshape(-1))]

    def fill(self):
        for i, past in enumerate(self.past):
            n = past.shape[0]
            pos = np.arange(n)
            slots = self.table[i, pos // page].astype(np.int64) * page + pos % page
            if n:
                p = bf16_dev(past)
                w4.kv_cache_write(p[:, 0], p[:, 1], to_dev(slots), FMT[self.form], page, self.b["cache"])

    def load(self, step):
        pos = self.start + step
        self.b["x"].copy_(bf16_dev(self.x0[step]))
        self.b["logits"].copy_(to_dev(self.logits[step]))
        self.b["lens"].copy_(to_dev((pos + 1).astype(np.int32)))
        self.b["slots"].copy_(to_dev(self.table[np.arange(T), pos // page].astype(np.int64) * page + pos % page))

    def run(self):
        b, w = self.b, self.weights
        w4.w4a16_add_rmsnorm(b["x"], None, w["n1"], 1e-6, None, b["h"])
        w4.w4a16_linear(b["h"], w["qkv"][0], w["qkv"][1], b["qkv"].shape[1], b["qkv"], b["ws"])
        qkv = b["qkv"].unflatten(1, (heads + 2 * kv_heads, D))
        w4.kv_cache_write(qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:], b["slots"], FMT[self.form], page,
                          b["cache"])
        w4.kv_cache_attention(qkv[:, :heads], b["cache"], FMT[self.form], page, kv_heads, b["table"], b["lens"],
                              D ** -0.5, b["att"], 0, b["lse"], b["ws"])
        w4.w4a16_linear(b["att"].flatten(1), w["o"][0], w["o"][1], d, b["proj"], b["ws"])
        w4.w4a16_add_rmsnorm(b["proj"], b["x"], w["n2"], 1e-6, b["res"], b["h2"])
        w4.w4a16_moe_layer(b["h2"], b["logits"], k, I, w["w1"][0], w["w1"][1], w["w2"][0], w["w2"][1],
                           w4.W4_EPI_GEGLU_TANH, b["y"], b["ws"])
        w4.w8a8_add_rmsnorm_quantize(b["proj"], b["x"], w["n2"], 1e-6, None, b["q8"], b["s8"])
        w4.w8a8_moe_gmm(b["q8"], b["s8"], None, None, 1, T, d, 2 * I, w["q1"][0], w["q1"][1], w4.W4_EPI_NONE, b["gmm"],
                        w4.W4_OUT_F32)

    def outputs(self):
        torch.cuda.synchronize()
        return {n: self.b[n].clone() for n in ("h", "qkv", "att", "proj", "res", "h2", "y", "q8", "s8", "gmm", "lse")}

    def check(self, step, o, rows):
        """rows: per sequence, the bf16 k and v rows written so far."""
        f64 = lambda t: oracle.bf16_bits_to_f64(bits_host(t))

        def close(got, want):
            ok, mx, rms = oracle.within_tolerance(got, want)
            assert ok, (mx, rms)

        x = self.x0[step]
        _, y = decode.add_rmsnorm(x, None, self.n1, 1e-6)
        assert (np.abs(f64(o["h"]) - y) <= np.abs(y) * (2.0 ** -8 + 2.0 ** -24)).all()
        close(f64(o["qkv"]), oracle.bf16_bits_to_f64(oracle.linear(bits_host(o["h"]), self.wqkv[2], self.wqkv[3])))
        qkv = bits_host(o["qkv"]).reshape(T, heads + 2 * kv_heads, D)
        for i in range(T):
            rows[i].append(np.stack([qkv[i, heads:heads + kv_heads], qkv[i, heads + kv_heads:]]))
            kv = np.stack(rows[i])
            kk, vv = [decode.row_values(*decode.cache_rows(kv[:, j], self.form), self.form) for j in (0, 1)]
            ref, lse, _, _ = decode.attention(qkv[i, :heads], kk, vv, D ** -0.5)
            close(f64(o["att"][i]), ref)
            np.testing.assert_allclose(o["lse"][i].cpu().numpy(), lse, atol=1e-3, rtol=1e-4)
        close(f64(o["proj"]), oracle.bf16_bits_to_f64(oracle.linear(bits_host(o["att"]).reshape(T, -1), self.wo[2],
                                                                    self.wo[3])))
        r, y = decode.add_rmsnorm(bits_host(o["proj"]), x, self.n2, 1e-6)
        assert np.array_equal(bits_host(o["res"]), r)
        assert (np.abs(f64(o["h2"]) - y) <= np.abs(y) * (2.0 ** -8 + 2.0 ** -24)).all()
        q8, s8 = decode.quantize_f64_rows(y)
        assert np.array_equal(o["q8"].cpu().numpy(), q8) and np.array_equal(o["s8"].cpu().numpy(), s8)
        close(o["gmm"].cpu().numpy().astype(np.float64), fp8.linear(q8, s8, self.q1[0][0], self.q1[1][0]))
        m = oracle.moe_layer(bits_host(o["h2"]), self.logits[step], self.w1[2], self.w1[3], self.w2[2], self.w2[3], k=k)
        close(f64(o["y"]), oracle.bf16_bits_to_f64(m["y"]))


@pytest.mark.parametrize("form", kv_layout.FORMATS)
def test_decode_steps(form):
    say("[decode step] %s" % form)
    layer = Layer(form)
    layer.fill()
    rows = [list(p) for p in layer.past]
    eager = []
    for step in range(layer.steps):
        layer.load(step)
        layer.run()
        eager.append(layer.outputs())
        layer.check(step, eager[-1], rows)
    cache = layer.b["cache"].clone()
    # the same steps from a captured graph, twice over, on the same buffers
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.run()
    for _ in range(2):
        layer.b["cache"].zero_()
        layer.fill()
        for step in range(layer.steps):
            layer.load(step)
            torch.cuda.synchronize()
            g.replay()
            got = layer.outputs()
            for n, t in eager[step].items():
                a, b = (v.view(torch.int16) if v.dtype == torch.bfloat16 else v for v in (t, got[n]))
                assert torch.equal(a, b), (step, n)
        assert torch.equal(layer.b["cache"], cache)
