"""Long attention cases and a bound on the kernel's error that lies far below
the outputs (test infrastructure; numpy only).

The bound, with e = 2^-24 (a rounding's largest relative error), p the
softmax's weights, A' = sum_t p_t |v'_t|, where v' is what the sums hold: |v|,
or for Q4 (|code| + 16) times the scale, as codes enter as 8 + code and the 8 is
taken off.  Roundings are independent, so errors add as the root of the sum of
squares:
  score t    D + 8 sums and products, at most S_t = scale * sum |q_i| |k'_i| each
             (and twice that where the matrix core should truncate):
             2 e sqrt(D + 8) S_t; base 2: e (2 max |s| + 8); exponential 2 e;
             p times V's scale e
  p . v      those, over sqrt(sum_t (p_t v_t)^2)
  sums       three terms a position, 3 n additions: 2 e sqrt(3 n) A'; from 1000
             positions in four waves or more, each of which holds a quarter
  joins      30 more, of waves and items
  division   the sum of p likewise: relative to the output
  output     half a bf16 step, 2^-8
Four times the sum of all but the last: no case is near it unless something is
wrong."""

import numpy as np

import kv_layout
import oracle
from oracle import decode

E = 2.0 ** -24


class Case:
    """Long sequences over few distinct pages: the tables name them at random, again and again."""

    def __init__(self, form, D, kv_heads, group, lens, page=16, distinct=24, width=None, window=0, seed=0):
        rng = np.random.default_rng(seed)
        self.form, self.D, self.kv_heads, self.group, self.page, self.window = form, D, kv_heads, group, page, window
        self.heads, self.pages = kv_heads * group, distinct
        self.lens = np.asarray(lens, dtype=np.int32)
        self.width = -(-int(self.lens.max()) // page) if width is None else width
        self.table = rng.integers(0, distinct, (len(lens), self.width)).astype(np.int32)
        k, v = (oracle.bf16_from_f64(sigma * rng.standard_normal((distinct, kv_heads, page, D))) for sigma in (1, 2))
        self.k, self.v = decode.cache_rows(k, form), decode.cache_rows(v, form)
        self.q = oracle.bf16_from_f64(rng.standard_normal((len(lens), self.heads, D)))
        self.scale = D ** -0.5

    def cache(self):
        return kv_layout.encode_cache(self.k, self.v, self.form)

    def rows(self, i, kv_head):
        """(values, magnitudes in the sums) of K and V of sequence i's attended positions, [n, D] each."""
        n = int(self.lens[i])
        pos = np.arange(max(0, n - self.window) if self.window else 0, n)
        p, o = self.table[i, pos // self.page], pos % self.page
        out = []
        for codes, scales in (self.k, self.v):
            c, s = codes[p, kv_head, o], None if scales is None else scales[p, kv_head, o]
            val = decode.row_values(c, s, self.form)
            mag = np.abs(val)
            if self.form == "q4":
                mag = (np.abs(c.astype(np.float64)) + 16.0) * np.repeat(oracle.bf16_bits_to_f64(s), 32, axis=-1)
            out.append((val, mag))
        return out

    def reference(self, i, head):
        """(out [D], lse, bound of out [D], bound of lse, p, v) of sequence i, query head `head`."""
        (k, km), (v, vm) = self.rows(i, head // self.group)
        q = oracle.bf16_bits_to_f64(self.q[i, head])
        scale = np.float64(np.float32(self.scale))
        s = scale * (k @ q)
        m = np.max(s)
        p = np.exp(s - m)
        lse = m + np.log(np.sum(p))
        p = p / np.sum(p)
        out = p @ v
        n, top = len(s), np.max(np.abs(s))
        d = E * (2 * np.sqrt(self.D + 8) * scale * (km @ np.abs(q)) + 2 * top + 8 + 2 + 1)
        waves = 4 if n >= 1000 else 1
        rel = np.sqrt(np.sum((p * d) ** 2)) + 2 * E * np.sqrt(n + 30) / waves + 2 * E
        num = np.sqrt(((p * d)[:, None] ** 2 * v ** 2).sum(0)) + 2 * E * np.sqrt(3 * n + 30) * (p @ vm) / waves
        bound = 2.0 ** -8 * np.abs(out) + 4 * (num + rel * np.abs(out))
        return out, lse, bound, 4 * rel + 4 * E * (abs(lse) + top + 8), p, v


# name: form, D, query heads a kv head; for Q4 with 4, 2 and 1 replicas of the heads
FORMS = [("bf16", 64, 2), ("bf16", 128, 2), ("bf16", 256, 2), ("e4m3", 64, 2), ("e4m3", 128, 2), ("e4m3", 256, 2),
         ("q4", 64, 2), ("q4", 64, 9), ("q4", 128, 4), ("q4", 128, 8), ("q4", 128, 16), ("q4", 256, 4), ("q4", 256, 8),
         ("q4", 256, 16)]

# rows (sequences x kv heads) from which a call with tables of up to 4096 tokens is not split
ENOUGH = {("bf16", 64): 171, ("bf16", 128): 171, ("bf16", 256): 171, ("e4m3", 64): 512, ("e4m3", 128): 512,
          ("e4m3", 256): 171, ("q4", 64): 683, ("q4", 128): 512, ("q4", 256): 342}


def whole(form, D, group, window=0):
    """Sequences that one workgroup takes whole: up to 256 pages and 32 chunks a wave, lengths around the 64 pages that
    a wave holds the ids of."""
    seqs = -(-ENOUGH[form, D] // 8)
    if window:
        lens = [8000, 7777, window, window + 1, window + 15, 4096, 1500, 1]
    else:
        lens = [4096, 4095, 1024, 1025, 1023, 2049, 1040, 3000]
    lens = (lens + [40 + 7 * i for i in range(seqs)])[:seqs]
    return Case(form, D, 8, group, lens, width=-(-max(lens) // 16), window=window, seed=D + group + window)


def split(form, D, group):
    """A long sequence whose items span over 64 pages and 9 chunks a wave or more."""
    return Case(form, D, 64, group, [20000, 37, 9001], seed=D + group)


def short(form, D, group, page=16):
    """Rows of one to a few chunks, and some that are split at the smallest share."""
    return Case(form, D, 2, group, [1, 2, 15, 16, 17, 31, 33, 63, 100, 127, 129, 300, 600, 1300, 5000], page=page,
                seed=D + group + page)
