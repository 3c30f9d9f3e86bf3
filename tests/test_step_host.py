"""Refusals of the speculative-decoding step's calls, without a GPU: the C ABI's status
codes in their documented order, and the binding's argument checks."""
import ctypes
import math
import os

import pytest
import torch

import mla_paged_latent_page_amd as mp

OK, NULLP, SHAPE, DTYPE, MISAL, RANGE, WS, DEV, HIP = range(9)
FAKE = 0x100000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mp.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return mp.lib()


def cache_desc(dtype=1, num_kv=1, head_dim=576, page_size=16, layers=2, pages=16, batch=2, maxp=4, **over):
    d = mp.CacheDesc()
    d.blocks = d.page_table = d.cache_lengths = FAKE
    d.dtype, d.num_layers, d.num_pages, d.page_size, d.num_kv = dtype, layers, pages, page_size, num_kv
    d.num_heads, d.head_dim, d.batch_size, d.max_pages_per_seq = 1, head_dim, batch, maxp
    assert mp.lib().mla_paged_cache_default_strides(ctypes.byref(d)) == OK
    for k, v in over.items():
        setattr(d, k, v)
    return d


def scales_desc(head_dim=576, page_size=16, layers=2, **over):
    s = mp.ScalesDesc()
    n = -(-head_dim // 128)
    s.scales, s.granularity, s.stride_token = FAKE, 128, n
    s.stride_kv = s.stride_layer = n * page_size
    s.stride_page = s.stride_layer * layers
    for k, v in over.items():
        setattr(s, k, v)
    return s


def freqs(lib, theta=1e4, factor=1.0, fast=32.0, slow=1.0, amp=1.0, scaling=0, orig=0, first=0, rows=8, R=64, out=FAKE,
          null=False):
    p = mp.RopeParams(theta, factor, fast, slow, amp, scaling, orig)
    return lib.mla_rope_freqs(None if null else ctypes.byref(p), first, rows, R, out, None)


def test_rope_freqs_refusals(lib):
    assert freqs(lib, null=True) == NULLP and freqs(lib, out=None) == NULLP
    for bad in (dict(theta=0.0), dict(theta=-1.0), dict(theta=math.nan), dict(amp=math.inf), dict(scaling=3),
                dict(scaling=1, factor=0.0), dict(scaling=2, orig=0), dict(scaling=2, orig=9, theta=1.0),
                dict(scaling=2, orig=9, fast=0.0), dict(scaling=2, orig=9, slow=math.nan), dict(R=63), dict(R=0),
                dict(R=514), dict(rows=-1), dict(first=-1), dict(first=2 ** 31 - 1, rows=2)):
        assert freqs(lib, **bad) == SHAPE, bad
    assert freqs(lib, out=FAKE + 4) == MISAL
    assert freqs(lib, rows=0, out=None) == OK
    assert freqs(lib) == DEV and freqs(lib, scaling=2, orig=4096, factor=4.0) == DEV


def test_rope_freqs_refuses_angles_beyond_binary64(lib):
    # 2^50 quarter turns are 1.77e15 rad.
    assert freqs(lib, theta=1e-300) == SHAPE and freqs(lib, scaling=1, factor=1e-320) == SHAPE
    assert freqs(lib, scaling=1, factor=1e-9, first=10 ** 7) == SHAPE
    assert freqs(lib, scaling=1, factor=1e-9, first=10 ** 6) == DEV


def rope_q(lib, q=FAKE, st=16 * 192, sh=192, T=5, H=16, nope=128, R=64, dt=1, pos=FAKE, fr=FAKE, ms=100, lay=0, out=FAKE,
           ost=None, osh=None):
    return lib.mla_rope_q(q, st, sh, T, H, nope, R, dt, pos, fr, ms, lay, out, st if ost is None else ost,
                          sh if osh is None else osh, None)


def test_rope_q_refusals(lib):
    for k in ("q", "pos", "fr", "out"):
        assert rope_q(lib, **{k: None}) == NULLP
    for bad in (dict(T=-1), dict(H=0), dict(nope=-8), dict(nope=4104, sh=8192), dict(R=0), dict(R=12), dict(R=520, sh=1024),
                dict(R=24, lay=1), dict(lay=2), dict(ms=0), dict(sh=184), dict(osh=184), dict(st=-16), dict(ost=64)):
        assert rope_q(lib, **bad) == SHAPE, bad
    assert rope_q(lib, dt=2) == DTYPE
    for bad in (dict(q=FAKE + 8), dict(out=FAKE + 2), dict(fr=FAKE + 4), dict(pos=FAKE + 2), dict(st=16 * 192 + 4),
                dict(sh=196), dict(nope=124)):
        assert rope_q(lib, **bad) == MISAL, bad
    assert rope_q(lib, T=0, q=None, pos=None, fr=None, out=None) == OK
    assert rope_q(lib) == DEV


def write_at(lib, d, s=None, x=FAKE, iro=FAKE, T=5, pos=FAKE, gamma=FAKE, eps=1e-6, fr=FAKE, ms=100, K=512, lay=0, layer=1):
    if s is None:
        return lib.mla_write_latent_paged_at(x, iro, T, pos, gamma, eps, fr, ms, K, lay, ctypes.byref(d), layer, None)
    return lib.mla_write_latent_paged_fp8_at(x, iro, T, pos, gamma, eps, fr, ms, K, lay, ctypes.byref(d),
                                             ctypes.byref(s), layer, None)


def test_write_at_refusals(lib):
    for d, s in ((cache_desc(), None), (cache_desc(dtype=2), scales_desc())):
        for k in ("x", "iro", "pos", "gamma", "fr"):
            assert write_at(lib, d, s, **{k: None}) == NULLP
        for bad in (dict(T=-1), dict(K=0), dict(K=516), dict(K=640), dict(eps=-1.0), dict(lay=2), dict(ms=0)):
            assert write_at(lib, d, s, **bad) == SHAPE, bad
        assert write_at(lib, d, s, x=FAKE + 2) == MISAL and write_at(lib, d, s, pos=FAKE + 1) == MISAL
        assert write_at(lib, d, s, layer=2) == RANGE
        assert write_at(lib, d, s, T=0) == OK and write_at(lib, d, s) == DEV
    assert write_at(lib, cache_desc(head_dim=536), lay=1) == SHAPE       # a rope part of 24 has no aligned halves
    assert write_at(lib, cache_desc(dtype=0)) == DTYPE
    assert write_at(lib, cache_desc(), scales_desc()) == DTYPE
    assert write_at(lib, cache_desc(dtype=2), scales_desc(granularity=64)) == SHAPE


def attend(lib, d, s=None, q=FAKE, iro=FAKE, T=5, H=16, mask=FAKE, words=1, scale=0.1, K=512, layer=1, out=FAKE, lse=FAKE,
           ws=FAKE, nbytes=None):
    if nbytes is None:
        nbytes = lib.mla_tree_attention_workspace_size(max(T, 0), max(H, 1), min(max(K, 8), 512))
    if s is None:
        return lib.mla_tree_attention_paged(q, iro, T, H, mask, words, scale, K, ctypes.byref(d), layer, out, lse, ws,
                                            nbytes, None)
    return lib.mla_tree_attention_paged_fp8_cache(q, iro, T, H, mask, words, scale, K, ctypes.byref(d),
                                                  ctypes.byref(s), layer, out, lse, ws, nbytes, None)


def test_tree_attention_refusals(lib):
    for d, s in ((cache_desc(), None), (cache_desc(dtype=2), scales_desc())):
        for k in ("q", "iro", "out", "ws"):
            assert attend(lib, d, s, **{k: None}) == NULLP
        for bad in (dict(T=-1), dict(H=0), dict(K=0), dict(K=12), dict(K=520), dict(scale=math.nan), dict(scale=math.inf),
                    dict(words=0), dict(words=-1), dict(mask=None), dict(T=2 ** 20, H=128)):
            assert attend(lib, d, s, **bad) == SHAPE, bad
        for bad in (dict(q=FAKE + 8), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(mask=FAKE + 4), dict(ws=FAKE + 128)):
            assert attend(lib, d, s, **bad) == MISAL, bad
        assert attend(lib, d, s, layer=2) == RANGE
        need = lib.mla_tree_attention_workspace_size(5, 16, 512)
        assert attend(lib, d, s, nbytes=need - 1) == WS
        assert attend(lib, d, s, T=0, q=None, out=None, ws=None, nbytes=0) == OK
        assert attend(lib, d, s) == DEV and attend(lib, d, s, mask=None, words=0, lse=None) == DEV
    assert attend(lib, cache_desc(num_kv=2)) == SHAPE
    assert attend(lib, cache_desc(head_dim=580)) == SHAPE
    assert attend(lib, cache_desc(page_size=2 ** 16, maxp=2 ** 15)) == SHAPE
    assert attend(lib, cache_desc(dtype=2)) == DTYPE
    assert attend(lib, cache_desc(dtype=1), scales_desc()) == DTYPE
    assert attend(lib, cache_desc(cache_lengths=None)) == NULLP


def test_tree_attention_workspace_size(lib):
    size = lib.mla_tree_attention_workspace_size
    assert size(-1, 16, 512) == 0 and size(4, 0, 512) == 0 and size(4, 16, 0) == 0 and size(4, 16, 520) == 0
    assert 0 < size(1, 16, 512) < size(1, 128, 512) == size(1000, 128, 512)


def test_page_calls_refuse(lib):
    def copy(d, s=None, src=FAKE, dst=FAKE, n=3):
        return lib.mla_copy_pages(src, dst, n, ctypes.byref(d) if d else None, ctypes.byref(s) if s else None, None)

    def fork(d, s=None, a=FAKE, b=FAKE, c=FAKE, refs=FAKE, n=3):
        return lib.mla_fork_paged(a, b, c, n, refs, ctypes.byref(d) if d else None, ctypes.byref(s) if s else None, None)

    def free(d, a=FAKE, refs=FAKE, lst=FAKE, cnt=FAKE, n=3):
        return lib.mla_free_paged(a, n, refs, lst, cnt, ctypes.byref(d) if d else None, None)

    def compact(d, s=None, a=FAKE, o=FAKE, n=3):
        return lib.mla_compact_paged(a, o, n, ctypes.byref(d) if d else None, ctypes.byref(s) if s else None, None)
    for call in (copy, fork, free, compact):
        d = cache_desc()
        assert call(None) == NULLP and call(d, n=-1) == SHAPE and call(d, n=0) == OK and call(d) == DEV
        assert call(cache_desc(num_kv=2, head_dim=128)) == DEV and call(cache_desc(dtype=0)) == DEV
        assert call(cache_desc(num_kv=3)) == SHAPE and call(cache_desc(page_size=0)) == SHAPE
        assert call(cache_desc(dtype=9)) == DTYPE
    for call in (copy, fork, compact):
        assert call(cache_desc(dtype=2)) == NULLP and call(cache_desc(), scales_desc()) == SHAPE
        assert call(cache_desc(dtype=2), scales_desc()) == DEV
        assert call(cache_desc(dtype=2), scales_desc(granularity=64)) == SHAPE
        assert call(cache_desc(blocks=None)) == NULLP and call(cache_desc(blocks=FAKE + 8)) == MISAL
    assert copy(cache_desc(), src=None) == NULLP and copy(cache_desc(), dst=None) == NULLP
    for k in ("a", "b", "c", "refs"):
        assert fork(cache_desc(), **{k: None}) == NULLP
    for k in ("a", "refs", "lst", "cnt"):
        assert free(cache_desc(), **{k: None}) == NULLP
    for k in ("a", "o"):
        assert compact(cache_desc(), **{k: None}) == NULLP
    assert free(cache_desc(blocks=None)) == DEV and free(cache_desc(dtype=2)) == DEV
    assert free(cache_desc(), n=65537) == SHAPE
    for call in (fork, free, compact):
        assert call(cache_desc(cache_lengths=None)) == NULLP and call(cache_desc(page_table=None)) == NULLP


# ---------------------------------------------------------------------------
# the binding (host tensors: a call whose arguments are right stops at the residency check)
# ---------------------------------------------------------------------------
bf16 = torch.bfloat16


def host_cache(dtype=bf16, D=576, batch=2, scales=False):
    pool = torch.zeros((4, 2, 1, 16, 1, D), dtype=dtype)
    sc = torch.zeros((4, 2, 1, 16, -(-D // 128))) if scales else None
    return mp.PagedKVCache(pool, torch.zeros((batch, 2), dtype=torch.int32), torch.zeros(batch, dtype=torch.int32),
                           scales=sc)


IRO = torch.tensor([0, 2, 5], dtype=torch.int32)


def test_binding_rope():
    q, pos, fr = torch.zeros((5, 4, 192), dtype=bf16), torch.zeros(5, dtype=torch.int32), torch.zeros((9, 64))
    with pytest.raises(ValueError, match="current GPU"):
        mp.mla_rope_q(q, pos, fr, q)
    for args, kw, msg in (((q[0], pos, fr, q), {}, "q must be"), ((q, pos, fr, q[:, :2]), {}, "shape"),
                          ((q, pos, fr, q.float()), {}, "dtype"), ((q.half(), pos, fr, q.half()), {}, "dtype"),
                          ((q, pos[:3], fr, q), {}, "positions"), ((q, pos, torch.zeros((9, 32)), q), {}, "wide"),
                          ((q, pos, fr, q), dict(layout="both"), "layout"), ((q, pos, fr.double(), q), {}, "dtype")):
        with pytest.raises(ValueError, match=msg):
            mp.mla_rope_q(*args, **kw)
    with pytest.raises(ValueError, match="scaling"):
        mp.mla_rope_freqs(fr, scaling="cubic")
    with pytest.raises(ValueError, match="rows, d_rope"):
        mp.mla_rope_freqs(fr[0])
    with pytest.raises(ValueError, match="current GPU"):
        mp.mla_rope_freqs(fr)


def test_binding_write_at():
    x, g, fr = torch.zeros((5, 576), dtype=bf16), torch.zeros(512), torch.zeros((9, 64))
    pos = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="current GPU"):
        mp.mla_write_latent_paged_at(x, IRO, pos, g, 1e-6, fr, 512, host_cache(), 1)
    with pytest.raises(ValueError, match="positions must have"):
        mp.mla_write_latent_paged_at(x, IRO, pos[:4], g, 1e-6, fr, 512, host_cache(), 1)
    with pytest.raises(ValueError, match="layout"):
        mp.mla_write_latent_paged_fp8_at(x, IRO, pos, g, 1e-6, fr, 512, host_cache(torch.uint8, scales=True), 1, layout="")
    with pytest.raises(ValueError, match="no scale pool"):
        mp.mla_write_latent_paged_fp8_at(x, IRO, pos, g, 1e-6, fr, 512, host_cache(torch.uint8), 1)


def test_binding_tree_attention():
    q, out = torch.zeros((5, 4, 576), dtype=bf16), torch.zeros((5, 4, 512), dtype=bf16)
    mask, ws, lse = torch.zeros((5, 1), dtype=torch.int64), torch.zeros(1 << 24, dtype=torch.uint8), torch.zeros((5, 4))

    def call(q=q, iro=IRO, mask=mask, c=None, out=out, ws=ws, lse=lse):
        mp.mla_tree_attention_paged(q, iro, mask, 0.1, 512, c or host_cache(), 1, out, ws, lse=lse)
    for kw, msg in ((dict(), "current GPU"), (dict(q=q[0]), "q_latent must be"), (dict(q=q[:, :, :512]), "wide"),
                    (dict(q=q.float()), "q_latent must be of dtype"), (dict(q=q.transpose(0, 1)), "out_latent|contiguous"),
                    (dict(out=out[:, :, :500]), "out_latent"), (dict(out=out.float()), "out_latent must be of dtype"),
                    (dict(iro=IRO[:2]), "input_row_offsets"), (dict(mask=mask[:4]), "tree_mask"),
                    (dict(mask=mask.int()), "tree_mask"), (dict(lse=lse[:, :2]), "lse"), (dict(lse=lse.double()), "lse"),
                    (dict(ws=None), "workspace"), (dict(c=host_cache(torch.float32)), "of dtype")):
        with pytest.raises(ValueError, match=msg):
            call(**kw)
    with pytest.raises(ValueError, match="no scale pool"):
        mp.mla_tree_attention_paged_fp8_cache(q, IRO, mask, 0.1, 512, host_cache(torch.uint8), 1, out, ws)


def test_binding_pages():
    three, two = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    refs = torch.zeros(4, dtype=torch.int32)
    c = host_cache()
    for call, msg in ((lambda: mp.mla_copy_pages(three, two, c), "same number"),
                      (lambda: mp.mla_copy_pages(three, three, c), "current GPU"),
                      (lambda: mp.mla_copy_pages(three.float(), three, c), "32-bit"),
                      (lambda: mp.mla_fork_paged(three, three, two, refs, c), "same number"),
                      (lambda: mp.mla_fork_paged(three, three, three, refs[:3], c), "ref_counts"),
                      (lambda: mp.mla_fork_paged(three, three, three, refs, c), "current GPU"),
                      (lambda: mp.mla_free_paged(three, refs, refs[:2], two, c), "free_list"),
                      (lambda: mp.mla_free_paged(three, refs, refs, two[:0], c), "free_count"),
                      (lambda: mp.mla_compact_paged(three, two, c), "accepted_offsets"),
                      (lambda: mp.mla_compact_paged(three, three, c), "current GPU")):
        with pytest.raises(ValueError, match=msg):
            call()
