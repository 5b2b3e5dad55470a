"""Host-side refusals of the step plan, rotary, adapter and sampling calls, and of
their Python wrappers (no GPU: every call here returns before any HIP call)."""

import pytest
import torch

import int4_group_quantized_q4_amd as w4
from int4_group_quantized_q4_amd import _lib

FAKE = 0x100000   # 16-byte aligned, never dereferenced
BIG = 1 << 36     # far from FAKE, for buffers that must not overlap it


def at(i):
    return FAKE + i * BIG


def changed(args, **kw):
    out = dict(args)
    out.update(kw)
    return list(out.values())


def test_plan_refusals():
    f = _lib.lib().kv_cache_plan
    a = dict(lens=at(0), new=at(1), seqs=4, table=at(2), width=8, page=16, free=at(3), cap=32, count=at(4),
             lens_out=at(5), count_out=at(6), offsets=at(7), slots=at(8), positions=at(9), row_seqs=at(10), rows=64, counters=at(11),
             st=None)
    arrays = ("lens", "new", "table", "free", "count", "lens_out", "count_out", "offsets", "slots", "positions")
    for name in arrays:
        assert f(*changed(a, **{name: None})) == w4.W4_ERR_ARG, name
    for name in arrays + ("row_seqs", "counters"):
        assert f(*changed(a, **{name: a[name] + 2})) == w4.W4_ERR_ARG, name
    for name in ("slots", "counters"):
        assert f(*changed(a, **{name: a[name] + 4})) == w4.W4_ERR_ARG, name
    for b in (dict(seqs=-1), dict(width=-1), dict(cap=-1), dict(rows=-1), dict(page=0),
              # outputs in other arguments
              dict(lens_out=at(0) + 4), dict(lens_out=at(1)), dict(count_out=at(4) + 4, count=at(4) + 4, free=at(4)),
              dict(count_out=at(0)), dict(offsets=at(0) + 12), dict(slots=at(2) + 64), dict(positions=at(8) + 504),
              dict(row_seqs=at(9)), dict(counters=at(3) + 120), dict(table=at(3)), dict(free=at(1)),
              dict(counters=at(6)), dict(lens_out=at(7) + 16), dict(table=at(0) + 8)):
        assert f(*changed(a, **b)) == w4.W4_ERR_ARG, b
    for b in (dict(seqs=65536), dict(page=24), dict(page=8), dict(page=1 << 17), dict(width=1 << 27),
              dict(cap=1 << 31), dict(rows=(1 << 26) + 1)):
        assert f(*changed(a, **b)) == w4.W4_ERR_SHAPE, b


def test_rope_refusals():
    f = _lib.lib().w4a16_rope
    a = dict(q=at(0), qs=1024, qh=8, k=at(1), ks=256, kh=2, rows=4, dim=128, rot=64, layout=0, pos=at(2), freq=at(3),
             scale=1.0, qo=at(4), qos=1024, ko=at(5), kos=256, st=None)
    for name in ("q", "k", "pos", "freq", "qo", "ko"):
        assert f(*changed(a, **{name: None})) == w4.W4_ERR_ARG, name
        assert f(*changed(a, **{name: a[name] + 2})) == w4.W4_ERR_ARG, name
    for b in (dict(rows=-1), dict(qh=0), dict(kh=-1), dict(dim=0), dict(rot=0), dict(layout=2), dict(layout=-1),
              dict(scale=float("inf")), dict(scale=float("nan")), dict(qs=1016), dict(qs=1028), dict(kos=248),
              dict(q=at(0) + 8),
              # outputs in other arguments, or in place with another stride
              dict(qo=at(0), qos=2048), dict(qo=at(0) + 16), dict(qo=at(1)), dict(ko=at(0)), dict(ko=at(1), kos=264),
              dict(ko=at(4) + 64), dict(qo=at(2)), dict(ko=at(3) - 16), dict(qo=at(3)), dict(ko=at(2)),
              # slices of one buffer that reach into one another
              dict(qs=1280, ks=1280, k=at(0) + 2 * 1024, qos=1280, kos=1280, ko=at(4) + 2 * 1024 - 16),
              dict(qs=1280, ks=1280, k=at(0) + 2 * 1024, qos=1280, qo=at(0) + 2 * 64)):
        assert f(*changed(a, **b)) == w4.W4_ERR_ARG, b
    for b in (dict(dim=136), dict(dim=528), dict(rot=24), dict(rot=144), dict(qh=4096, qs=1 << 20), dict(rows=1 << 27),
              dict(qs=1 << 47)):
        assert f(*changed(a, **b)) == w4.W4_ERR_SHAPE, b
    assert f(*changed(a, rows=0, q=None, k=None, qo=None, ko=None, pos=None)) == w4.W4_OK


def test_lora_refusals():
    lib = _lib.lib()
    f = lib.w4a16_lora_add
    a = dict(x=at(0), xs=256, rows=4, K=256, ids=at(1), a=at(2), b=at(3), scaling=at(4), adapters=3, rank=16, N=512,
             y=at(5), ys=512, out=at(6), os=512, ws=at(7), ws_bytes=1 << 30, st=None)
    for name in ("x", "ids", "a", "b", "y", "out"):
        assert f(*changed(a, **{name: None})) == w4.W4_ERR_ARG, name
    for name in ("x", "ids", "a", "b", "scaling", "y", "out"):
        assert f(*changed(a, **{name: a[name] + 2})) == w4.W4_ERR_ARG, name
    for b in (dict(rows=-1), dict(K=-32), dict(N=-16), dict(adapters=-1), dict(rank=-8), dict(xs=248), dict(xs=260),
              dict(ys=504), dict(os=516),
              dict(out=at(0)), dict(out=at(1)), dict(out=at(2) + 64), dict(out=at(3)), dict(out=at(4)),
              dict(out=at(5) + 16), dict(out=at(5), os=520), dict(ws=at(0)), dict(ws=at(1)), dict(ws=at(2)),
              dict(ws=at(3)), dict(ws=at(4)), dict(ws=at(5)), dict(ws=at(6))):
        assert f(*changed(a, **b)) == w4.W4_ERR_ARG, b
    for b in (dict(K=0), dict(K=48), dict(N=24), dict(rank=0), dict(rank=12), dict(rank=264), dict(adapters=4097),
              dict(K=(1 << 20) + 32, xs=1 << 21), dict(N=(1 << 20) + 16), dict(rows=(1 << 20) + 1), dict(xs=1 << 47)):
        assert f(*changed(a, **b)) == w4.W4_ERR_SHAPE, b
    need = lib.w4a16_lora_workspace(4, 256, 512, 3, 16)
    assert need > 0
    for b in (dict(ws=None), dict(ws=at(7) + 8), dict(ws_bytes=need - 1)):
        assert f(*changed(a, **b)) == w4.W4_ERR_WORKSPACE, b
    assert f(*changed(a, rows=0, x=None, y=None, out=None, ids=None)) == w4.W4_OK
    assert f(*changed(a, N=0, y=None, out=None)) == w4.W4_OK
    assert lib.w4a16_lora_workspace(4, 256, 512, 3, 12) == 0 and lib.w4a16_lora_workspace(0, 256, 512, 3, 16) == 0


def test_sample_refusals():
    lib = _lib.lib()
    f = lib.w4a16_sample
    a = dict(z=at(0), dtype=1, rows=4, vocab=1000, stride=1000, t=at(1), k=at(2), p=at(3), m=at(4), u=at(5), tok=at(6),
             lp=at(7), ws=at(8), ws_bytes=1 << 30, st=None)
    for name in ("z", "u", "tok"):
        assert f(*changed(a, **{name: None})) == w4.W4_ERR_ARG, name
    for name in ("z", "t", "k", "p", "m", "u", "tok", "lp"):
        assert f(*changed(a, **{name: a[name] + 2})) == w4.W4_ERR_ARG, name
    for b in (dict(dtype=2), dict(dtype=-1), dict(rows=-1), dict(vocab=-1), dict(stride=999),
              dict(dtype=0, z=at(0) + 1),
              dict(tok=at(0) + 400), dict(tok=at(1)), dict(lp=at(6) + 8), dict(lp=at(5)), dict(lp=at(0)),
              dict(tok=at(2) + 12), dict(lp=at(3)), dict(tok=at(4))):
        assert f(*changed(a, **b)) == w4.W4_ERR_ARG, b
    for b in (dict(vocab=0), dict(vocab=(1 << 20) + 1, stride=1 << 21), dict(rows=65536), dict(stride=1 << 47)):
        assert f(*changed(a, **b)) == w4.W4_ERR_SHAPE, b
    need = lib.w4a16_sample_workspace(4, 1000)
    if need:
        for b in (dict(ws=None), dict(ws=at(8) + 8), dict(ws_bytes=need - 1)):
            assert f(*changed(a, **b)) == w4.W4_ERR_WORKSPACE, b
        for b in (dict(ws=at(0)), dict(ws=at(1)), dict(ws=at(5)), dict(ws=at(6))):
            assert f(*changed(a, **b)) == w4.W4_ERR_ARG, b
    assert f(*changed(a, rows=0, z=None, u=None, tok=None)) == w4.W4_OK
    assert lib.w4a16_sample_workspace(0, 1000) == 0 and lib.w4a16_sample_workspace(4, 0) == 0


def test_wrapper_refusals():
    """Shapes, types and sizes are checked before any launch; right arguments on the CPU are then refused as not on the
    device."""
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16)
    f32 = lambda *s: torch.empty(*s, dtype=torch.float32)
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8)
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32)
    i64 = lambda *s: torch.empty(*s, dtype=torch.int64)
    size = pytest.raises(ValueError, match="holds .* bytes")
    device = pytest.raises(ValueError, match="device tensor")
    plan = lambda **kw: w4.kv_cache_plan(**dict(dict(
        seq_lens=i32(4), new_tokens=i32(4), block_table=i32(4, 8), page_size=16, free_pages=i32(9), free_count=i32(1),
        seq_lens_out=i32(4), free_count_out=i32(1), row_offsets=i32(5), slots=i64(7), positions=i32(7),
        row_seqs=i32(7)), **kw))
    for kw in (dict(seq_lens=i32(3)), dict(new_tokens=i32(3)), dict(row_offsets=i32(4)), dict(positions=i32(6)),
               dict(row_seqs=i32(6)), dict(free_count=i32(0)), dict(counters=i64(1))):
        with pytest.raises(ValueError):
            plan(**kw)
    with pytest.raises(ValueError, match="seqs, width"):
        plan(block_table=i32(32))
    with device:
        plan()
    rope = lambda **kw: w4.w4a16_rope(**dict(dict(
        q=bf(3, 4, 64), k=bf(3, 2, 64), positions=i32(3), inv_freq=f32(32), q_out=bf(3, 4, 64), k_out=bf(3, 2, 64)),
        **kw))
    for kw in (dict(q_out=bf(3, 4, 48)), dict(k_out=bf(3, 3, 64)), dict(k=bf(2, 2, 64), k_out=bf(2, 2, 64)),
               dict(q=bf(3, 64, 4).transpose(1, 2)), dict(q=bf(1, 4, 64).expand(3, 4, 64)), dict(q=bf(3, 256))):
        with pytest.raises(ValueError):
            rope(**kw)
    with pytest.raises(TypeError):
        rope(q=f32(3, 4, 64), q_out=f32(3, 4, 64))
    with device:
        rope()
    lora = lambda **kw: w4.w4a16_lora_add(**dict(dict(
        x=bf(3, 64), adapter_ids=i32(3), a=bf(2, 8, 64), b=bf(2, 32, 8), scaling=f32(2), y=bf(3, 32), out=bf(3, 32),
        ws=u8(4096)), **kw))
    for kw in (dict(x=bf(3, 32)), dict(a=bf(3, 8, 64)), dict(b=bf(2, 32, 16)), dict(b=bf(2, 16, 8)), dict(y=bf(2, 32)),
               dict(out=bf(3, 16)), dict(a=bf(2, 512)), dict(x=bf(3, 1, 64)), dict(x=bf(64, 3).t())):
        with pytest.raises(ValueError):
            lora(**kw)
    with pytest.raises(TypeError):
        lora(y=f32(3, 32))
    with device:
        lora()
    sample = lambda **kw: w4.w4a16_sample(**dict(dict(logits=f32(3, 100), uniforms=f32(3), tokens=i32(3)), **kw))
    for kw in (dict(logits=f32(300)), dict(logits=f32(100, 3).t()), dict(logits=f32(1, 100).expand(3, 100))):
        with pytest.raises(ValueError):
            sample(**kw)
    with pytest.raises(TypeError):
        sample(logits=i32(3, 100))
    with device:
        sample()
