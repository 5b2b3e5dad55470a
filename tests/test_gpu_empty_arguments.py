"""An empty argument overlaps nothing, wherever its pointer lies: a cache without pages, a block table without
columns."""

import pytest
import torch

import int4_group_quantized_q4_amd as w4
from int4_group_quantized_q4_amd import _lib
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [w4.W4_KV_BF16, w4.W4_KV_E4M3, w4.W4_KV_Q4])
def test_a_cache_without_pages_takes_no_token(fmt):
    tokens, heads, dim = 3, 2, 64
    k = torch.randn(tokens, heads * dim, device=dev()).bfloat16()
    v, before = k.clone(), k.clone()
    slots = torch.tensor([-1, 0, 40], dtype=torch.int64, device=dev())
    counters = torch.zeros(2, dtype=torch.int64, device=dev())
    stream = torch.cuda.current_stream().cuda_stream
    write = lambda cache, pages: _lib.lib().kv_cache_write(k.data_ptr(), v.data_ptr(), tokens, heads * dim, heads * dim,
                                                           slots.data_ptr(), fmt, cache, pages, 16, heads, dim,
                                                           counters.data_ptr(), stream)
    inside = k.data_ptr() + 128
    assert write(inside, 1) == w4.W4_ERR_ARG
    assert write(inside, 0) == w4.W4_OK
    torch.cuda.synchronize()
    assert counters.tolist() == [2, 0] and torch.equal(k, before) and torch.equal(v, before)


def test_a_block_table_without_columns():
    seqs, heads, dim = 3, 2, 64
    q = torch.randn(seqs, heads, dim, device=dev()).bfloat16()
    cache = torch.zeros(w4.kv_cache_page_bytes(w4.W4_KV_BF16, 16, heads, dim), dtype=torch.uint8, device=dev())
    lens = torch.zeros(seqs, dtype=torch.int32, device=dev())
    out = torch.full_like(q, 7.0)
    lse = torch.zeros(seqs, heads, device=dev())
    ws = torch.zeros(max(16, w4.kv_cache_attention_workspace(seqs, heads, heads, dim, 0, 16)), dtype=torch.uint8,
                     device=dev())
    stream = torch.cuda.current_stream().cuda_stream
    attend = lambda table, width: _lib.lib().kv_cache_attention(
        q.data_ptr(), seqs, heads * dim, heads, cache.data_ptr(), w4.W4_KV_BF16, 1, 16, heads, dim, table, width,
        lens.data_ptr(), 0.125, 0, out.data_ptr(), lse.data_ptr(), None, ws.data_ptr(), ws.numel(), stream)
    assert attend(out.data_ptr() + 64, 1) == w4.W4_ERR_ARG
    assert attend(out.data_ptr() + 64, 0) == w4.W4_OK
    torch.cuda.synchronize()
    assert not out.any() and (lse == -float("inf")).all()
