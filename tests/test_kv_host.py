"""Refusals of the paged K/V cache's calls, without a GPU: the C ABI's status codes in their
documented order, and the binding's argument checks."""
import ctypes
import math

import pytest
import torch

import mla_paged_latent_page_amd as mp
from test_step_host import DEV, DTYPE, FAKE, MISAL, NULLP, OK, RANGE, SHAPE, WS, lib  # noqa: F401


def cache(dtype=1, heads=8, head_dim=128, num_kv=2, page_size=16, layers=2, pages=16, batch=2, maxp=4, **over):
    d = mp.CacheDesc()
    d.blocks = d.page_table = d.cache_lengths = FAKE
    d.dtype, d.num_layers, d.num_pages, d.page_size, d.num_kv = dtype, layers, pages, page_size, num_kv
    d.num_heads, d.head_dim, d.batch_size, d.max_pages_per_seq = heads, head_dim, batch, maxp
    assert mp.lib().mla_paged_cache_default_strides(ctypes.byref(d)) == OK
    for k, v in over.items():
        setattr(d, k, v)
    return d


def scales(width=1024, page_size=16, layers=2, **over):
    s = mp.ScalesDesc()
    n = -(-width // 128)
    s.scales, s.granularity, s.stride_token = FAKE, 128, n
    s.stride_kv = n * page_size
    s.stride_layer = 2 * s.stride_kv
    s.stride_page = s.stride_layer * layers
    for k, v in over.items():
        setattr(s, k, v)
    return s


def ref(x):
    return None if x is None else ctypes.byref(x)


def write(c, s=None, k=FAKE, v=FAKE, ks=1024, vs=1024, iro=FAKE, T=5, pos=FAKE, fr=FAKE, rows=9, rope=128, layout=1, layer=1,
          fp8=False):
    a = (k, v, ks, vs, iro, T, pos, fr, rows, rope, layout, ref(c))
    return mp.lib().kv_write_paged_fp8(*a, ref(s), layer, None) if fp8 else mp.lib().kv_write_paged(*a, layer, None)


def gather(c, s=None, bro=FAKE, co=FAKE, M=5, layer=1, k=FAKE, v=FAKE, fp8=False):
    if fp8:
        return mp.lib().kv_gather_paged_fp8_cache(bro, co, M, ref(c), ref(s), layer, k, v, None)
    return mp.lib().kv_gather_paged(bro, co, M, ref(c), layer, k, v, None)


def attend(c, s=None, q=FAKE, qs=4096, iro=FAKE, T=5, H=32, scale=0.1, window=0, sinks=0, layer=1, out=FAKE, lse=FAKE,
           ws=FAKE, size=1 << 40, fp8=False):
    a = (q, qs, iro, T, H, scale, window, sinks, ref(c))
    b = (layer, out, lse, ws, size, None)
    return mp.lib().kv_attention_paged_fp8_cache(*a, ref(s), *b) if fp8 else mp.lib().kv_attention_paged(*a, *b)


def test_write_refuses(lib):  # noqa: F811
    c = cache()
    assert write(c) == DEV and write(c, T=0, k=None, v=None, iro=None, pos=None, fr=None) == OK
    assert write(c, pos=None) == DEV and write(c, rope=0, fr=None, rows=0) == DEV
    assert write(None) == NULLP and write(c, fr=None) == NULLP
    for name in ("k", "v", "iro"):
        assert write(c, **{name: None}) == NULLP
    for over in (dict(blocks=None), dict(page_table=None), dict(cache_lengths=None)):
        assert write(cache(**over)) == NULLP
    for kw in (dict(T=-1), dict(rope=-8), dict(rope=136), dict(rope=4), dict(rope=24), dict(rows=0), dict(layout=2),
               dict(ks=1016), dict(vs=1016), dict(ks=-8)):
        assert write(c, **kw) == SHAPE, kw
    assert write(c, rope=24, layout=0) == DEV and write(c, T=1, ks=0, vs=0) == DEV
    assert write(cache(num_kv=1)) == SHAPE and write(cache(head_dim=124)) == SHAPE
    assert write(cache(heads=8192), ks=1 << 20, vs=1 << 20) == DEV
    assert write(cache(heads=8193), ks=1 << 21, vs=1 << 21) == SHAPE
    assert write(cache(dtype=0)) == DTYPE and write(cache(dtype=2)) == DTYPE
    for kw in (dict(k=FAKE + 2), dict(v=FAKE + 8), dict(ks=1028), dict(vs=1028), dict(fr=FAKE + 4), dict(pos=FAKE + 2)):
        assert write(c, **kw) == MISAL, kw
    assert write(cache(blocks=FAKE + 8)) == MISAL and write(c, layer=2) == RANGE
    c8, s8 = cache(dtype=2), scales()
    assert write(c8, s8, fp8=True) == DEV and write(c8, None, fp8=True) == NULLP and write(c, s8, fp8=True) == DTYPE
    assert write(c8, scales(scales=None), fp8=True) == NULLP and write(c8, scales(scales=FAKE + 2), fp8=True) == MISAL
    for over in (dict(granularity=64), dict(stride_token=7), dict(stride_kv=7), dict(stride_page=0)):
        assert write(c8, scales(**over), fp8=True) == SHAPE, over
    assert write(cache(dtype=2, heads=1, head_dim=8), scales(8), ks=8, vs=8, rope=8, layout=0, fp8=True) == MISAL


def test_gather_refuses(lib):  # noqa: F811
    c = cache()
    assert gather(c) == DEV and gather(cache(dtype=0)) == DEV and gather(cache(cache_lengths=None)) == DEV
    assert gather(c, M=0, bro=None, co=None, k=None, v=None) == OK and gather(c, M=-1) == SHAPE
    for name in ("bro", "co", "k", "v"):
        assert gather(c, **{name: None}) == NULLP
    assert gather(None) == NULLP and gather(cache(num_kv=1)) == SHAPE and gather(cache(dtype=2)) == DTYPE
    assert gather(c, k=FAKE + 8) == MISAL and gather(c, v=FAKE + 4) == MISAL and gather(c, layer=2) == RANGE
    assert gather(cache(heads=8193)) == SHAPE
    c8 = cache(dtype=2)
    assert gather(c8, scales(), fp8=True) == DEV and gather(c8, fp8=True) == NULLP
    assert gather(c, scales(), fp8=True) == DTYPE and gather(c8, scales(granularity=32), fp8=True) == SHAPE


def test_attention_refuses(lib):  # noqa: F811
    c = cache()
    assert attend(c) == DEV and attend(c, T=0, q=None, iro=None, out=None, ws=None, size=0) == OK
    assert attend(cache(dtype=0)) == DEV and attend(c, lse=None) == DEV and attend(c, window=7, sinks=3) == DEV
    assert attend(c, scale=-1.0) == DEV and attend(c, scale=0.0) == DEV and attend(None) == NULLP
    for name in ("q", "iro", "out", "ws"):
        assert attend(c, **{name: None}) == NULLP
    for over in (dict(blocks=None), dict(page_table=None), dict(cache_lengths=None)):
        assert attend(cache(**over)) == NULLP
    for kw in (dict(T=-1), dict(H=0), dict(H=-8), dict(H=12), dict(scale=math.nan), dict(scale=math.inf), dict(window=-1),
               dict(sinks=-1), dict(qs=4088), dict(scale=2.0 ** 127), dict(T=1 << 26)):
        assert attend(c, **kw) == SHAPE, kw
    assert attend(cache(num_kv=1)) == SHAPE and attend(cache(head_dim=264), qs=1 << 20) == SHAPE
    assert attend(cache(head_dim=4), qs=1 << 20) == SHAPE and attend(cache(head_dim=256), qs=1 << 20) == DEV
    assert attend(cache(page_size=1 << 16, maxp=1 << 15)) == SHAPE
    assert attend(cache(dtype=2)) == DTYPE
    for kw in (dict(q=FAKE + 8), dict(qs=4100), dict(out=FAKE + 4), dict(lse=FAKE + 1), dict(ws=FAKE + 128)):
        assert attend(c, **kw) == MISAL, kw
    assert attend(c, layer=2) == RANGE
    need = mp.kv_attention_workspace_size(5, 32, 8, 128)
    assert need > 0 and attend(c, size=need) == DEV and attend(c, size=need - 1) == WS
    for a in ((-1, 32, 8, 128), (5, 0, 8, 128), (5, 32, 0, 128), (5, 12, 8, 128), (5, 32, 8, 0), (5, 32, 8, 257)):
        assert mp.kv_attention_workspace_size(*a) == 0
    c8 = cache(dtype=2)
    assert attend(c8, scales(), fp8=True) == DEV and attend(c8, fp8=True) == NULLP
    assert attend(c, scales(), fp8=True) == DTYPE and attend(c8, scales(stride_token=7), fp8=True) == SHAPE
    assert attend(c8, scales(scales=FAKE + 1), fp8=True) == MISAL


# ---------------------------------------------------------------------------
# the binding (host tensors: a call whose arguments are right stops at the residency check)
# ---------------------------------------------------------------------------
BF16 = torch.bfloat16
IRO = torch.tensor([0, 2, 5], dtype=torch.int32)


def host_cache(dtype=BF16, heads=2, D=64, with_scales=False):
    pool = torch.zeros((4, 2, 2, 16, heads, D), dtype=dtype)
    sc = torch.zeros((4, 2, 2, 16, -(-heads * D // 128))) if with_scales else None
    return mp.PagedKVCache(pool, torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), scales=sc)


def test_binding_write():
    k, v = torch.zeros((5, 2, 64), dtype=BF16), torch.zeros((5, 6, 64), dtype=BF16)[:, 4:]
    fr, pos = torch.zeros((9, 64)), torch.zeros(5, dtype=torch.int32)

    def call(k=k, v=v, iro=IRO, c=None, fp8=False, **kw):
        if fp8:
            mp.kv_write_paged_fp8(k, v, iro, c or host_cache(torch.uint8, with_scales=True), 1, **kw)
        else:
            mp.kv_write_paged(k, v, iro, c or host_cache(), 1, **kw)
    for kw in ({}, dict(freqs_cis=fr), dict(freqs_cis=fr, positions=pos, layout="half"), dict(fp8=True)):
        with pytest.raises(ValueError, match="current GPU"):
            call(**kw)
    for kw, msg in ((dict(k=None), "k must be"), (dict(k=k[0]), "k must be"), (dict(v=None), "v must be"),
                    (dict(v=v[:4]), "v must be"), (dict(k=k[..., :32]), "k must be"), (dict(k=k.float()), "k must be of dtype"),
                    (dict(v=torch.zeros((5, 64, 2), dtype=BF16).transpose(1, 2)), "contiguous"),
                    (dict(iro=IRO[:2]), "input_row_offsets"), (dict(positions=pos[:4]), "positions"),
                    (dict(freqs_cis=fr[0]), "freqs_cis"), (dict(freqs_cis=fr.double()), "freqs_cis must be of dtype"),
                    (dict(layout="both"), "layout"), (dict(fp8=True, c=host_cache(torch.uint8)), "no scale pool")):
        with pytest.raises(ValueError, match=msg):
            call(**kw)


def test_binding_gather():
    k, v = torch.zeros((5, 2, 64), dtype=BF16), torch.zeros((5, 2, 64), dtype=BF16)
    co = torch.zeros(2, dtype=torch.int32)
    for c, call in ((host_cache(), mp.kv_gather_paged),
                    (host_cache(torch.uint8, with_scales=True), mp.kv_gather_paged_fp8_cache)):
        with pytest.raises(ValueError, match="current GPU"):
            call(IRO, co, 5, c, 1, k, v)
        for args, msg in (((IRO[:2], co, 5, c, 1, k, v), "buffer_row_offsets"), ((IRO, co[:1], 5, c, 1, k, v), "cache_offsets"),
                          ((IRO, co, 6, c, 1, k, v), "k_buffer"), ((IRO, co, 5, c, 1, k, v[:4]), "v_buffer"),
                          ((IRO, co, 5, c, 1, k.float(), v), "k_buffer must be of dtype"),
                          ((IRO, co, 5, c, 1, k, None), "v_buffer")):
            with pytest.raises(ValueError, match=msg):
                call(*args)


def test_binding_attention():
    q = torch.zeros((5, 10, 64), dtype=BF16)[:, :4]
    out, ws, lse = torch.zeros((5, 4, 64), dtype=BF16), torch.zeros(1 << 12, dtype=torch.uint8), torch.zeros((5, 4))

    def call(q=q, iro=IRO, c=None, out=out, ws=ws, lse=lse, scale=0.1, **kw):
        mp.kv_attention_paged(q, iro, scale, c or host_cache(), 1, out, ws, lse=lse, **kw)
    for kw, msg in (({}, "current GPU"), (dict(lse=None, window=5, sinks=2), "current GPU"), (dict(q=q[0]), "q must be"),
                    (dict(q=q[..., :32]), "q must be"), (dict(q=q.float()), "q must be of dtype"),
                    (dict(out=out[:, :3]), "out must be"), (dict(out=out.float()), "out must be of dtype"),
                    (dict(iro=IRO[:2]), "input_row_offsets"), (dict(lse=lse[:, :2]), "lse"), (dict(ws=None), "workspace"),
                    (dict(window=-1), "window"), (dict(window=1 << 32), "window"), (dict(sinks=1 << 31), "sinks"),
                    (dict(c=host_cache(torch.float32)), "q must be of dtype")):
        with pytest.raises(ValueError, match=msg):
            call(**kw)
    with pytest.raises(ValueError, match="no scale pool"):
        mp.kv_attention_paged_fp8_cache(q, IRO, 0.1, host_cache(torch.uint8), 1, out, ws)
