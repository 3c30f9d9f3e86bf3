"""The paged K/V cache's operators at the edges of what they accept: rows behind the last request, values near the
largest that the sums hold, calls of several launches, positions below 2^31, large pages, thousands of requests."""
import math

import numpy as np
import pytest
import torch

import mla_paged_latent_page_amd as mp
import workloads as W
from plain_kv import KvCase, cast_pool, check_kv_attention, rotated
from plain_step import HALF_BF16, U32, i32
from test_gpu_kv_cache import attend, cache_of, same, written

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def write(case, k, v, iro=None, **kw):
    (mp.kv_write_paged_fp8 if case.dtype == "e4m3" else mp.kv_write_paged)(k, v, case.iro if iro is None else iro,
                                                                          cache_of(case), case.layer, **kw)


def raw(pool):
    return pool.view(torch.uint8 if pool.element_size() == 1 else torch.int16)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens, new, pad", [([5], [3], 1), ([0, 30, 7], [2, 0, 9], 40), ([17], [0], 6),
                                            ([3] * 70, [1] * 69 + [0], 200)])
def test_writes_behind_the_last_request_are_skipped(lens, new, pad, dtype, given):
    # a call with more tokens than the requests have, as a step captured with a fixed count makes it: the last
    # request has room for them, and nothing of it may change
    KH, D = 2, 64
    case = KvCase(70, [n + 300 for n in lens], new, KH, KH, D, dtype=dtype)
    case.lens = np.asarray(lens)
    case.dev.cache_lengths.copy_(i32(lens, "cuda"))
    T = case.T + pad
    g = torch.Generator(device="cuda").manual_seed(70)
    k, v = (torch.randn((T, KH, D), generator=g, device="cuda").to(BF16) for _ in range(2))
    table = torch.from_numpy(W.rope_table(400, D)).cuda()
    pos = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, new)] + [np.zeros(pad, np.int64)])
    more = dict(freqs_cis=table, layout="half", positions=i32(pos, "cuda") if given else None)
    before = case.dev.pool.clone()
    scales = None if case.dev.scales is None else case.dev.scales.clone()
    write(case, k[:case.T], v[:case.T], **dict(more, positions=i32(pos[:case.T], "cuda") if given else None))
    want, swant = case.dev.pool.clone(), None if scales is None else case.dev.scales.clone()
    case.dev.pool.copy_(before)
    if scales is not None:
        case.dev.scales.copy_(scales)
    k[case.T:], v[case.T:] = math.nan, math.inf
    write(case, k, v, **more)
    unchanged = same(raw(case.dev.pool), raw(want))
    assert unchanged
    if scales is not None:
        unchanged = same(case.dev.scales.view(torch.int32), swant.view(torch.int32))
        assert unchanged
    if case.T:
        page, slot = written(case, new)
        changed = not same(raw(want)[page, 1, :, slot], raw(before)[page, 1, :, slot])
        assert changed


# ---------------------------------------------------------------------------
# values near the largest that the sums hold
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("lens, new, H, KH", [([255], [1], 8, 2), ([100, 3], [156, 1], 4, 2)])
@pytest.mark.parametrize("D, dtype", [(64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "e4m3"), (80, "bf16"), (80, "e4m3"),
                                      (64, "f32")])
def test_values_just_inside_the_limit(lens, new, H, KH, D, dtype):
    # |V| x rows seen just below 2^119, and scores that grow by just less than the 2^8 that weights may reach while
    # their reference lags
    case = KvCase(71, lens, new, H, KH, D, dtype=dtype)
    rows = int((case.lens + case.new).max())
    top = 2.0 ** 119 / rows * 0.99
    case.q.zero_()
    case.q[:, :, 0] = 1.0
    case.scale = math.log(2.0)
    for b, (n, m) in enumerate(zip(lens, new)):
        page, slot = case.where(b, range(n + m))
        k = torch.zeros((n + m, KH, D), device="cuda")
        k[64:, :, 0] = 7.5
        sign = torch.randint(0, 2, (n + m, KH, D), device="cuda", generator=torch.Generator("cuda").manual_seed(b)) * 2 - 1
        sign[:, :, :8] = 1
        if dtype == "e4m3":
            case.dev.pool[page, 1, 0, slot] = k.to(torch.float8_e4m3fn).view(torch.uint8)
            case.dev.pool[page, 1, 1, slot] = (448.0 * sign).to(torch.float8_e4m3fn).view(torch.uint8)
            case.dev.scales[page, 1, 0, slot] = 1.0
            case.dev.scales[page, 1, 1, slot] = top / 448
        else:
            case.dev.pool[page, 1, 0, slot] = k.to(case.dev.pool.dtype)
            case.dev.pool[page, 1, 1, slot] = (top * sign).to(case.dev.pool.dtype)
    out, z = attend(case)
    check_kv_attention(case, out, z)
    assert bool((out[:, :, :8].double() > top * 0.98).all())


# ---------------------------------------------------------------------------
# calls in several launches
# ---------------------------------------------------------------------------
def paged(shape, layer_dtype, lengths, page_size, scales=None, seed=72):
    """A pool of one layer for requests of the given capacities, its pages in random order, and (page, slot) of a
    request's positions."""
    need = [-(-n // page_size) for n in lengths]
    order = np.random.default_rng(seed).permutation(sum(need))
    table = np.zeros((len(need), max(need)), np.int64)
    for b, at in enumerate(np.cumsum([0] + need[:-1])):
        table[b, :need[b]] = order[at:at + need[b]]
    pool = torch.empty((sum(need), 1, 2, page_size, *shape), dtype=layer_dtype, device="cuda")
    sc = None if scales is None else torch.empty((sum(need), 1, 2, page_size, scales), device="cuda")
    cache = mp.PagedKVCache(pool, i32(table, "cuda"), torch.zeros(len(need), dtype=torch.int32, device="cuda"), scales=sc)
    dev = torch.from_numpy(table).cuda()

    def where(b, positions):
        p = torch.as_tensor(positions, device="cuda")
        return dev[b, p // page_size], p % page_size
    return cache, where


def test_writes_and_reads_in_several_launches():
    # rows of 2^20 columns: 4,096 tokens to a launch; the first token of the second one is inside the second request
    KH, D = 4096, 256
    seq = [3000, 1099]
    T = sum(seq)
    g = torch.Generator(device="cuda").manual_seed(73)
    k, v = (torch.randn((T, KH, D), generator=g, device="cuda", dtype=BF16) for _ in range(2))
    cache, where = paged((KH, D), BF16, seq, 64)
    iro = i32([0, 3000, T], "cuda")
    mp.kv_write_paged(k, v, iro, cache, 0)
    for b, first in ((0, 0), (1, 3000)):
        for lo in range(0, seq[b], 256):
            hi = min(lo + 256, seq[b])
            page, slot = where(b, range(lo, hi))
            for side, x in ((0, k), (1, v)):
                right = same(cache.pool[page, 0, side, slot], x[first + lo:first + hi])
                assert right, (b, lo, side)
    kb, vb = torch.zeros_like(k), torch.zeros_like(v)
    mp.kv_gather_paged(iro, i32([0, 0], "cuda"), T, cache, 0, kb, vb)
    for lo in range(0, T, 256):
        right = same(kb[lo:lo + 256], k[lo:lo + 256]) and same(vb[lo:lo + 256], v[lo:lo + 256])
        assert right, lo


def test_quantising_writes_and_reads_in_several_launches():
    # ... into an e4m3 cache, rotated at given positions; and reads of more than 8,192 of its rows
    KH, D = 4096, 256
    seq = [3000, 1099]
    T = sum(seq)
    g = torch.Generator(device="cuda").manual_seed(74)
    k, v = (torch.randn((T, KH, D), generator=g, device="cuda", dtype=BF16) for _ in range(2))
    cache, where = paged((KH, D), torch.uint8, seq, 64, scales=KH * D // 128)
    table = torch.from_numpy(W.rope_table(500, 128)).cuda()
    pos = np.arange(T) * 7 % 500
    mp.kv_write_paged_fp8(k, v, i32([0, 3000, T], "cuda"), cache, 0, positions=i32(pos, "cuda"), freqs_cis=table, layout="half")
    edges = [0, 1, 2999, 3000, 4094, 4095, 4096, 4097, 4098]
    for t in edges:
        b = int(t >= 3000)
        page, slot = where(b, [t - 3000 * b])
        kr, mag = rotated(k[t:t + 1].double(), table.double()[pos[t]][None], 128, True)
        for side, ref, mag in ((0, kr, mag), (1, v[t:t + 1].double(), v[t:t + 1].double().abs())):
            sc = cache.scales[page, 0, side, slot].double()
            want = ref.view(1, -1, 128).abs().amax(2) / 448
            assert bool(((sc - want).abs() <= want * 4 * U32).all()), t
            sc = sc.repeat_interleave(128, 1).view(1, KH, D)
            got = cast_pool(cache.pool[page, 0, side, slot], "e4m3") * sc
            # as in test_write: two products and a sum, half a step of the code, half its smallest step
            tol = mag * 2 * U32 + ref.abs() * 2.0 ** -4 * 1.001 + sc * 2.0 ** -10
            assert bool(((got - ref).abs() <= tol).all()), (t, side)
    del k, v
    M = 2 * T - 4       # 8,194 rows: of the first request, the second, and all but four of both again
    again = [3000, 1099, 2998, 1097]
    four = mp.PagedKVCache(cache.pool, cache.page_table[[0, 1, 0, 1]].contiguous(), cache.cache_lengths[[0, 1, 0, 1]].contiguous(),
                           scales=cache.scales)
    kb, vb = (torch.zeros((M, KH, D), dtype=BF16, device="cuda") for _ in range(2))
    mp.kv_gather_paged_fp8_cache(i32(np.concatenate([[0], np.cumsum(again)]), "cuda"), i32([0, 0, 2, 2], "cuda"), M, four, 0,
                                 kb, vb)
    for r, b, p in ((0, 0, 0), (2999, 0, 2999), (3000, 1, 0), (4098, 1, 1098), (4099, 0, 2), (7097, 1, 2), (8190, 1, 1095),
                    (8191, 1, 1096), (8192, 1, 1097), (8193, 1, 1098)):
        page, slot = where(b, [p])
        for side, got in ((0, kb), (1, vb)):
            sc = cache.scales[page, 0, side, slot].repeat_interleave(128, 1).view(1, KH, D)
            ref = cache.pool[page, 0, side, slot].view(torch.float8_e4m3fn).float() * sc
            assert same(got[r:r + 1], ref.to(BF16)), (r, side)


def test_attention_in_several_launches():
    # the general form takes 2^23 tokens x key heads in a launch: 2^20 + 5 tokens of 16 heads
    T, H, D, window = (1 << 20) + 5, 16, 8, 3
    cache, where = paged((H, D), torch.float32, [T], 1024)
    g = torch.Generator(device="cuda").manual_seed(75)
    cache.pool.normal_(generator=g)
    q = torch.randn((T, H, D), generator=g, device="cuda")
    out, z = torch.zeros_like(q), torch.zeros((T, H), device="cuda")
    ws = torch.empty(mp.kv_attention_workspace_size(T, H, H, D), dtype=torch.uint8, device="cuda")
    mp.kv_attention_paged(q, i32([0, T], "cuda"), 0.5, cache, 0, out, ws, window=window, sinks=1, lse=z)
    page, slot = where(0, range(T))
    K, V = (cache.pool[page, 0, side, slot] for side in (0, 1))
    step = 1 << 17
    for lo in range(0, T, step):
        t = torch.arange(lo, min(lo + step, T), device="cuda")
        at = torch.stack([t - 2, t - 1, t, torch.zeros_like(t)])          # the window, and the sink where it is not in it
        seen = (at >= 0) & torch.cat([torch.ones_like(at[:3], dtype=torch.bool), (t > 2)[None]])
        at = at.clamp_min(0)
        k, v, x = K[at].double(), V[at].double(), q[t].double()
        s = ((k * x).sum(3) * 0.5).masked_fill(~seen[:, :, None], -math.inf)
        mags = ((k * x).abs().sum(3) * 0.5).amax(0)
        ref = torch.logsumexp(s, 0)
        w = torch.exp(s - ref)
        o, mag = (w[..., None] * v).sum(0), (w[..., None] * v.abs()).sum(0)
        # the bounds of tests/plain_kv.py, of four rows
        ds = mags * (D + 8) * U32
        tol = mag * (2 * ds + 2.0 ** -20 + 12 * U32)[..., None] + o.abs() * 2 * U32 + 1e-30
        assert bool(((out[t].double() - o).abs() <= tol).all()), lo
        assert bool(((z[t].double() - ref).abs() <= ds + 2.0 ** -20 + 12 * U32 + ref.abs() * 2 * U32).all()), lo


# ---------------------------------------------------------------------------
# far positions and large pages
# ---------------------------------------------------------------------------
def plain_window(q, K, V, scale, seen):
    """out, lse and their bounds (tests/plain_kv.py) of q [T, H, D] over rows K, V [n, KH, D], float64."""
    T, H, D = q.shape
    G = H // K.shape[1]
    out, lse, tol, ltol = [], [], [], []
    for h in range(H):
        k, v, x = K[:, h // G].contiguous(), V[:, h // G].contiguous(), q[:, h].double()
        s = ((x @ k.t().contiguous()) * scale).masked_fill(~seen, -math.inf)
        ds = ((x.abs() @ k.abs().t().contiguous()) * scale).masked_fill(~seen, 0.0).amax(1) * (D + 8) * U32
        z = torch.logsumexp(s, 1)
        w = torch.exp(s - z[:, None])
        o, mag = w @ v, w @ v.abs()
        many = 3 * seen.sum(1) * U32
        half = 0.0 if q.dtype == torch.float32 else HALF_BF16
        out.append(o)
        lse.append(z)
        tol.append(mag * (2 * ds + 2.0 ** -20 + many + half)[:, None] + o.abs() * max(half, 2 * U32) * 1.02 + 1e-30)
        ltol.append(ds + 2.0 ** -20 + many + z.abs() * 2 * U32)
    return [torch.stack(x, 1) for x in (out, lse, tol, ltol)]


@pytest.mark.parametrize("page_size, pages", [(1 << 20, 2047), ((1 << 20) - 24, 2047), (999999, 2147)])
@pytest.mark.parametrize("D, dtype", [(64, "bf16"), (64, "e4m3"), (80, "bf16")])
def test_positions_near_the_largest(D, dtype, page_size, pages):
    # all logical pages of a request are three pages of the pool, its own; new tokens cross into the last page and end
    # at the last position, below 2^31; a window and two sinks
    H, KH, window, sinks = 4, 1, 100, 2
    capacity = page_size * pages
    assert 2 ** 31 - 2 ** 21 < capacity < 2 ** 31
    lens, new = [capacity - page_size - 10, capacity - 20], [30, 20]
    fp8 = dtype == "e4m3"
    T = sum(new)
    pool = torch.zeros((6, 1, 2, page_size, KH, D), dtype=torch.uint8 if fp8 else BF16, device="cuda")
    scales = torch.ones((6, 1, 2, page_size, 1), device="cuda") if fp8 else None
    table = torch.stack([torch.arange(pages) % 3, 3 + (torch.arange(pages) * 2 + 1) % 3]).int().cuda()
    cache = mp.PagedKVCache(pool, table, i32(lens, "cuda"), scales=scales)
    g = torch.Generator(device="cuda").manual_seed(76)
    iro = i32([0, 30, 50], "cuda")
    # rows behind the window and at the start, then the new ones by the call
    rows, at = [], []
    for b, n in enumerate(lens):
        p = torch.cat([torch.arange(0, sinks), torch.arange(n - window, n)]).cuda()
        x = torch.randn((2, len(p), KH, D), generator=g, device="cuda")
        page, slot = table[b, p // page_size].long(), p % page_size
        for side in (0, 1):
            pool[page, 0, side, slot] = x[side].to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x[side].to(BF16)
        at.append(torch.cat([p, torch.arange(n, n + new[b], device="cuda")]))
    k, v = (torch.randn((T, KH, D), generator=g, device="cuda").to(BF16) for _ in range(2))
    (mp.kv_write_paged_fp8 if fp8 else mp.kv_write_paged)(k, v, iro, cache, 0)
    M = [100 + n for n in new]
    kb, vb = (torch.empty((sum(M), KH, D), dtype=BF16, device="cuda") for _ in range(2))
    (mp.kv_gather_paged_fp8_cache if fp8 else mp.kv_gather_paged)(i32([0, M[0], sum(M)], "cuda"),
                                                                 i32([n - 100 for n in lens], "cuda"), sum(M), cache, 0, kb, vb)
    q = torch.randn((T, H, D), generator=g, device="cuda").to(BF16)
    out, z = torch.empty_like(q), torch.empty((T, H), device="cuda")
    ws = torch.empty(mp.kv_attention_workspace_size(T, H, KH, D), dtype=torch.uint8, device="cuda")
    (mp.kv_attention_paged_fp8_cache if fp8 else mp.kv_attention_paged)(q, iro, 0.125, cache, 0, out, ws, window=window,
                                                                       sinks=sinks, lse=z)
    for b, (n, m) in enumerate(zip(lens, new)):
        t0 = [0, 30][b]
        p, own = at[b], slice(t0, t0 + m)
        page, slot = table[b, p // page_size].long(), p % page_size
        rows = []
        for side in (0, 1):
            r = cast_pool(pool[page, 0, side, slot], dtype)
            rows.append(r * scales[page, 0, side, slot].double()[:, :, None] if fp8 else r)
        read = torch.stack([kb, vb])[:, sum(M[:b]):sum(M[:b]) + M[b]].double()
        assert same(read, torch.stack(rows)[:, sinks:].float().to(BF16).double())
        if not fp8:
            assert same(rows[0][-m:], k[own].double()) and same(rows[1][-m:], v[own].double())
        me = torch.arange(n, n + m, device="cuda")[:, None]
        seen = (p <= me) & ((me - p < window) | (p < sinks))
        ref, zref, tol, ltol = plain_window(q[own], rows[0], rows[1], 0.125, seen)
        assert bool(((out[own].double() - ref).abs() <= tol).all()) and bool(((z[own].double() - zref).abs() <= ltol).all())


@pytest.mark.parametrize("page_size", [264, 1000, 4104, 1 << 16, 3001])
@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (64, "e4m3"), (80, "f32")])
def test_large_pages(D, dtype, page_size):
    case = KvCase(77, [page_size - 3, 2 * page_size + 5 if page_size < 10000 else 7, 0], [9, 70, 1], 4, 2, D, page_size=page_size,
                  dtype=dtype)
    check_kv_attention(case, *attend(case))


def test_thousands_of_requests():
    rng = np.random.default_rng(78)
    lens, new = rng.integers(0, 40, 3000), rng.choice([0, 1, 1, 2], 3000)
    case = KvCase(78, lens, new, 2, 1, 64)
    check_kv_attention(case, *attend(case))


# ---------------------------------------------------------------------------
# a step captured with a fixed number of tokens
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (64, "e4m3"), (80, "bf16")])
def test_captured_steps_with_fewer_tokens(D, dtype):
    H, KH, T, fp8 = 8, 2, 24, dtype == "e4m3"
    case = KvCase(79, [400, 30, 250], [16, 16, 16], H, KH, D, dtype=dtype)
    base = [400, 30, 250]
    cache = cache_of(case)
    table = torch.from_numpy(W.rope_table(600, D)).cuda()
    g = torch.Generator(device="cuda").manual_seed(79)
    x = torch.randn((T, H + 2 * KH, D), generator=g, device="cuda").to(BF16)
    pos, iro = i32(np.zeros(T), "cuda"), i32([0, 8, 16, 24], "cuda")
    q, out, z = torch.empty((T, H, D), dtype=BF16, device="cuda"), torch.empty((T, H, D), dtype=BF16, device="cuda"), \
        torch.empty((T, H), device="cuda")
    ws = torch.empty(mp.kv_attention_workspace_size(T, H, KH, D), dtype=torch.uint8, device="cuda")

    def step(n):
        mp.mla_rope_q(x[:n, :H], pos[:n], table, q[:n], d_nope=0, layout="half")
        (mp.kv_write_paged_fp8 if fp8 else mp.kv_write_paged)(x[:n, H:H + KH], x[:n, H + KH:], iro, cache, 1, positions=pos[:n],
                                                              freqs_cis=table, layout="half")
        (mp.kv_attention_paged_fp8_cache if fp8 else mp.kv_attention_paged)(q[:n], iro, case.scale, cache, 1, out[:n], ws,
                                                                           lse=z[:n])
    case.dev.cache_lengths.copy_(i32(base, "cuda"))
    before = case.dev.pool.clone()
    step(T)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(T)
    for seq in ([1, 1, 1], [8, 8, 8], [0, 3, 2], [10, 0, 0], [0, 0, 0], [1, 14, 1]):
        n = sum(seq)
        iro.copy_(i32(np.concatenate([[0], np.cumsum(seq)]), "cuda"))
        p = np.concatenate([np.arange(m) + b for b, m in zip(base, seq)] + [np.zeros(T - n)])
        pos.copy_(i32(p, "cuda"))
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        x[n:] = math.nan
        case.dev.pool.copy_(before)
        out.fill_(7.0)
        z.fill_(7.0)
        if n:
            step(n)
        want = [t.clone() for t in (case.dev.pool, out, z)]
        case.dev.pool.copy_(before)
        out.fill_(7.0)
        z.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        unchanged = same(raw(case.dev.pool), raw(want[0]))
        assert unchanged and same(out, want[1]) and same(z, want[2]), seq
