"""The counters of the cache and attention calls are written, so they may lie in
no other argument (host-side checks, no GPU)."""

import pytest

import int4_group_quantized_q4_amd as w4
from int4_group_quantized_q4_amd import _lib

FAKE = 0x100000   # 16-byte aligned, never dereferenced


def at(i):
    return FAKE + (i << 32)


# 4 tokens of 2 x 128, 4 pages of 16 tokens
ROWS = 4 * 256 * 2
PAGE = {0: 2 * 2 * 16 * 256, 1: 2 * 2 * 16 * 132, 2: 2 * 2 * 16 * 72}


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_counters_of_write_and_read(fmt):
    lib = _lib.lib()
    assert lib.kv_cache_page_bytes(fmt, 16, 2, 128) == PAGE[fmt]
    inside = [at(0), at(0) + ROWS - 8, at(0) - 8, at(1) + 512, at(1) + ROWS - 8, at(2), at(2) + 24, at(2) - 8, at(3),
              at(3) - 8, at(3) + 4 * PAGE[fmt] - 8]
    for c in inside:
        assert lib.kv_cache_write(at(0), at(1), 4, 256, 256, at(2), fmt, at(3), 4, 16, 2, 128, c, None) == w4.W4_ERR_ARG
    for out, size in ((w4.W4_OUT_BF16, 1), (w4.W4_OUT_F32, 2)):
        for c in inside + [at(0) + size * ROWS - 8, at(1) + size * ROWS - 8]:
            assert lib.kv_cache_read(at(3), fmt, 4, 16, 2, 128, at(2), 4, at(0), at(1), 256, 256, out, c,
                                     None) == w4.W4_ERR_ARG


def test_counters_of_attention():
    lib = _lib.lib()
    q, cache, table, lens, out, lse, ws = (at(i) for i in range(7))
    need = lib.kv_cache_attention_workspace(4, 8, 2, 128, 1024, 16)
    assert need > 0
    for c in (q, q + 4 * 2048 - 8, cache, cache + 4 * PAGE[1] - 8, table, table + 4 * 1024 * 4 - 8, lens,
              lens + 8, out, out + 4 * 2048 - 8, lse, lse + 4 * 8 * 4 - 8, ws, ws + need - 8):
        assert lib.kv_cache_attention(q, 4, 1024, 8, cache, 1, 4, 16, 2, 128, table, 1024, lens, 0.1, 0, out, lse, c, ws,
                                      need, None) == w4.W4_ERR_ARG
