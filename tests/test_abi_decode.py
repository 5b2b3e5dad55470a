"""Host-side refusals of the norm, key-value cache and attention calls, and of
their Python wrappers (no GPU: every call here returns before any HIP call)."""

import pytest
import torch

import int4_group_quantized_q4_amd as w4
import kv_layout
from int4_group_quantized_q4_amd import _lib

FAKE = 0x100000   # 16-byte aligned, never dereferenced
BIG = 1 << 32     # far from FAKE, for buffers that must not overlap it


def changed(args, **kw):
    out = dict(args)
    out.update(kw)
    return list(out.values())


def test_norm_refusals():
    lib = _lib.lib()
    f = lib.w4a16_add_rmsnorm
    a = dict(x=FAKE, res=FAKE + BIG, w=FAKE + 2 * BIG, rows=4, d=64, eps=1e-6, off=0.0, sum=FAKE + 3 * BIG,
             y=FAKE + 4 * BIG, st=None)
    assert f(*changed(a, d=48)) == w4.W4_ERR_SHAPE
    assert f(*changed(a, d=(1 << 20) + 32)) == w4.W4_ERR_SHAPE
    assert f(*changed(a, rows=1 << 36)) == w4.W4_ERR_SHAPE
    assert f(*changed(a, rows=-1)) == w4.W4_ERR_ARG
    assert f(*changed(a, eps=-1e-6)) == w4.W4_ERR_ARG
    assert f(*changed(a, eps=float("nan"))) == w4.W4_ERR_ARG
    assert f(*changed(a, eps=float("inf"))) == w4.W4_ERR_ARG
    for name in ("x", "w", "y"):
        assert f(*changed(a, **{name: None})) == w4.W4_ERR_ARG
        assert f(*changed(a, **{name: a[name] + 8})) == w4.W4_ERR_ARG
    assert f(*changed(a, res=None)) == w4.W4_ERR_ARG                       # sum_out without a residual
    assert f(*changed(a, y=FAKE + 64)) == w4.W4_ERR_ARG                    # overlaps x without being it
    assert f(*changed(a, sum=FAKE + BIG + 16)) == w4.W4_ERR_ARG
    assert f(*changed(a, y=a["sum"])) == w4.W4_ERR_ARG
    assert f(*changed(a, y=a["w"])) == w4.W4_ERR_ARG
    assert f(*changed(a, rows=0, x=None, y=None)) == w4.W4_OK
    g = lib.w8a8_add_rmsnorm_quantize
    b = dict(x=FAKE, res=FAKE + BIG, w=FAKE + 2 * BIG, rows=4, d=64, eps=1e-6, off=0.0, sum=FAKE + 3 * BIG,
             q=FAKE + 4 * BIG, scale=FAKE + 5 * BIG, st=None)
    assert g(*changed(b, q=FAKE)) == w4.W4_ERR_ARG                         # another row pitch: not in place
    assert g(*changed(b, scale=None)) == w4.W4_ERR_ARG
    assert g(*changed(b, scale=FAKE + 5 * BIG + 2)) == w4.W4_ERR_ARG
    assert g(*changed(b, scale=FAKE + 4 * BIG + 4)) == w4.W4_ERR_ARG
    assert g(*changed(b, d=40)) == w4.W4_ERR_SHAPE


@pytest.mark.parametrize("form,code", [("bf16", 0), ("e4m3", 1), ("q4", 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_page_bytes(form, code, D):
    lib = _lib.lib()
    for page, heads in ((16, 1), (64, 3), (4096, 8)):
        assert lib.kv_cache_page_bytes(code, page, heads, D) == kv_layout.page_bytes(form, page, heads, D)


def test_page_bytes_refusals():
    lib = _lib.lib()
    for args in ((3, 16, 1, 64), (-1, 16, 1, 64), (0, 8, 1, 64), (0, 24, 1, 64), (0, 1 << 17, 1, 64), (0, 16, 0, 64),
                 (0, 16, 1025, 64), (0, 16, 1, 96), (0, 16, 1, 512), (0, 0, 1, 64)):
        assert lib.kv_cache_page_bytes(*args) == 0, args
    with pytest.raises(ValueError):
        w4.kv_cache_page_bytes(0, 24, 1, 64)


def test_write_and_read_refusals():
    lib = _lib.lib()
    a = dict(k=FAKE, v=FAKE + BIG, tokens=4, ks=256, vs=256, slots=FAKE + 2 * BIG, fmt=2, cache=FAKE + 3 * BIG,
             pages=4, page=16, heads=2, D=128, counters=None, st=None)
    w = lib.kv_cache_write
    bad = [dict(tokens=-1), dict(ks=248), dict(ks=260), dict(vs=128), dict(slots=None), dict(slots=FAKE + 2 * BIG + 4),
           dict(cache=None), dict(cache=FAKE + 3 * BIG + 8), dict(cache=FAKE), dict(cache=FAKE + BIG),
           dict(cache=FAKE + 2 * BIG), dict(slots=FAKE + 3 * BIG + 1024), dict(k=None), dict(v=FAKE + 8),
           dict(fmt=5), dict(pages=-1),
           dict(counters=FAKE + 4)]
    for b in bad:
        assert w(*changed(a, **b)) == w4.W4_ERR_ARG, b
    for b in (dict(tokens=1 << 28), dict(tokens=1 << 27), dict(page=20), dict(D=96), dict(heads=2000),
              dict(pages=1 << 31), dict(pages=1 << 30, page=65536), dict(ks=1 << 47)):
        assert w(*changed(a, **b)) == w4.W4_ERR_SHAPE, b
    assert w(*changed(a, tokens=0, k=None, v=None, slots=None, cache=None)) == w4.W4_OK
    r = dict(cache=FAKE + 3 * BIG, fmt=2, pages=4, page=16, heads=2, D=128, slots=FAKE + 2 * BIG, tokens=4, k=FAKE,
             v=FAKE + BIG, ks=256, vs=256, out=0, counters=None, st=None)
    f = lib.kv_cache_read
    # rows of k in rows of v: the same, shifted, between v's rows but too near, with another stride; k in the cache, in
    # the slots
    over = [dict(v=FAKE), dict(v=FAKE + 496), dict(v=FAKE - 16), dict(ks=512, vs=512, v=FAKE + 496),
            dict(ks=512, vs=512, v=FAKE - 528 + 1024), dict(ks=512, vs=512, v=FAKE + 1024 + 512 + 16),
            dict(ks=512, vs=1024, v=FAKE + 512), dict(k=FAKE + 3 * BIG + 64), dict(v=FAKE + 3 * BIG - 2048 + 16),
            dict(k=FAKE + 2 * BIG), dict(out=1, v=FAKE + 512)]
    for b in [dict(out=2), dict(cache=None), dict(slots=None), dict(k=FAKE + 8), dict(vs=0), dict(fmt=-1)] + over:
        assert f(*changed(r, **b)) == w4.W4_ERR_ARG, b
    assert f(*changed(r, tokens=0)) == w4.W4_OK


def test_attention_refusals():
    lib = _lib.lib()
    at = lambda i: FAKE + i * BIG
    a = dict(q=FAKE, seqs=4, qs=1024, heads=8, cache=at(1), fmt=1, pages=4, page=16, kv=2, D=128, table=at(2), width=8,
             lens=at(3), scale=0.1, window=0, out=at(4), lse=None, counters=None, ws=at(5), ws_bytes=1 << 30, st=None)
    f = lib.kv_cache_attention
    need = lib.kv_cache_attention_workspace(4, 8, 2, 128, 8, 16)
    long = lib.kv_cache_attention_workspace(4, 8, 2, 128, 1024, 16)
    assert long > need >= 0
    for b in (dict(q=None), dict(q=FAKE + 8), dict(qs=1016), dict(qs=1028), dict(cache=None), dict(fmt=3),
              dict(pages=0), dict(table=None), dict(lens=None), dict(lens=at(3) + 2), dict(out=None),
              dict(out=at(4) + 8), dict(window=-1), dict(scale=float("inf")), dict(scale=float("nan")),
              dict(scale=2.0 ** 65), dict(scale=-2.0 ** 65), dict(heads=0), dict(lse=at(6) + 2),
              dict(counters=FAKE + 4), dict(seqs=-1),
              # outputs in other arguments
              dict(out=FAKE), dict(out=FAKE + 4 * 2048 - 16), dict(out=at(1) + 128), dict(out=at(2)), dict(out=at(3)),
              dict(lse=at(4) + 64), dict(lse=at(1)), dict(width=1024, ws=FAKE), dict(width=1024, ws=at(4)),
              dict(width=1024, ws=at(2) + 4096), dict(width=1024, ws=at(1) - 4096)):
        assert f(*changed(a, **b)) == w4.W4_ERR_ARG, b
    for b in (dict(heads=7), dict(seqs=65535, heads=512, kv=32, qs=65536), dict(D=80), dict(page=48), dict(seqs=65536),
              dict(width=1 << 27), dict(heads=32768), dict(pages=1 << 30, page=65536),
              dict(qs=1 << 47)):
        assert f(*changed(a, **b)) == w4.W4_ERR_SHAPE, b
    for b in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=long - 1)):
        assert f(*changed(a, width=1024, **b)) == w4.W4_ERR_WORKSPACE, b
    assert f(*changed(a, seqs=0, q=None, cache=None, lens=None, out=None)) == w4.W4_OK
    assert lib.kv_cache_attention_workspace(0, 8, 2, 128, 8, 16) == 0
    assert lib.kv_cache_attention_workspace(4, 7, 2, 128, 8, 16) == 0


def test_wrapper_refusals():
    """Sizes, types and row layouts are checked before any launch (CPU tensors
    reach those checks; the right ones are then refused as not on the device)."""
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16)
    f32 = lambda *s: torch.empty(*s, dtype=torch.float32)
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8)
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32)
    i64 = lambda *s: torch.empty(*s, dtype=torch.int64)
    size = pytest.raises(ValueError, match="holds .* bytes")
    with size:
        w4.w4a16_add_rmsnorm(bf(4, 64), bf(3, 64), bf(64), 1e-6, None, bf(4, 64))
    with size:
        w4.w4a16_add_rmsnorm(bf(4, 64), None, bf(32), 1e-6, None, bf(4, 64))
    with size:
        w4.w4a16_add_rmsnorm(bf(4, 64), bf(4, 64), bf(64), 1e-6, bf(4, 63), bf(4, 64))
    with pytest.raises(ValueError, match="device tensor"):
        w4.w4a16_add_rmsnorm(bf(4, 64), None, bf(64), 1e-6, None, bf(4, 64))
    with pytest.raises(ValueError, match="rows, d"):
        w4.w4a16_add_rmsnorm(bf(2, 2, 64), None, bf(64), 1e-6, None, bf(4, 64))
    page = w4.kv_cache_page_bytes(w4.W4_KV_Q4, 16, 2, 64)
    rows = lambda t, **kw: dict(dict(k=bf(t, 2, 64), v=bf(t, 2, 64), slots=i64(t), format=w4.W4_KV_Q4, page_size=16,
                                     cache=u8(3 * page)), **kw)
    with pytest.raises(ValueError, match="expected"):
        w4.kv_cache_write(**rows(4, v=bf(4, 2, 128)))
    with pytest.raises(TypeError):
        w4.kv_cache_write(**rows(4, k=f32(4, 2, 64), v=f32(4, 2, 64)))
    with pytest.raises(ValueError, match="contiguous"):
        w4.kv_cache_write(**rows(4, k=bf(4, 64, 2).transpose(1, 2)))
    with pytest.raises(ValueError, match="overlap"):
        w4.kv_cache_write(**rows(4, k=bf(1, 2, 64).expand(4, 2, 64)))
    with pytest.raises(ValueError, match="device tensor"):
        w4.kv_cache_write(**rows(4))
