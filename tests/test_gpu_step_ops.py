"""The speculative-decoding step on the GPU against plain 64-bit forms: rotary
positions, latent writes at given positions, tree attention, page upkeep."""
import math

import numpy as np
import pytest
import torch

import mla_paged_latent_page_amd as mp
import workloads as W
from plain_step import (HALF_BF16, U32, AttentionCase, check_attention, frequencies, i32, mask_tensor, rotate)
from gpu_util import check_guards, guarded_empty

pytestmark = pytest.mark.gpu


def same(a, b):
    return bool(torch.equal(a, b))


def cache_of(case_or_dc):
    dc = getattr(case_or_dc, "dev", case_or_dc)
    return mp.PagedKVCache(dc.pool, dc.page_table, dc.cache_lengths, scales=dc.scales)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("first, rows, dim, scaling, factor, amplitude", [
    (0, 1, 2, "none", 1.0, 1.0), (0, 1000, 64, "none", 1.0, 1.0), (5, 333, 6, "linear", 4.0, 1.0),
    (1 << 20, 777, 64, "by_parts", 40.0, 1.37), (0, 4097, 128, "by_parts", 8.0, 0.9), (0, 9, 512, "by_parts", 2.5, 1.0),
    ((1 << 31) - 50, 50, 64, "none", 1.0, 1.0)])
def test_rope_freqs(first, rows, dim, scaling, factor, amplitude):
    out = guarded_empty((rows, dim), torch.float32)
    mp.mla_rope_freqs(out, theta=10000.0, first_position=first, scaling=scaling, factor=factor,
                      original_max_position=4096, amplitude=amplitude)
    check_guards("rope_freqs")
    f = frequencies(dim, 10000.0, scaling, factor, 4096)
    ang = (first + np.arange(rows, dtype=np.float64))[:, None] * f
    ref = np.stack([np.cos(ang), np.sin(ang)], 2).reshape(rows, dim) * amplitude
    # One rounding (at most 2^-24 of the amplitude), and a binary64 angle of a turns is off by
    # a 2^-52 turns, twice (the table's and the reference's).
    tol = amplitude * (U32 + 4 * np.repeat(np.abs(ang), 2, axis=1) * 2.0 ** -52)
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("T, H, nope, R, half, dtype, inplace, strided", [
    (1, 1, 128, 64, False, "bf16", False, False), (3, 16, 128, 64, True, "bf16", True, False),
    (7, 5, 64, 8, False, "bf16", False, True), (2, 130, 128, 64, True, "bf16", False, True),
    (65, 20, 0, 16, True, "f32", False, False), (9, 3, 4, 512, False, "f32", True, False),
    (5, 128, 128, 64, False, "bf16", True, True), (4, 2, 200, 512, True, "bf16", False, False),
    (6, 70, 12, 48, True, "f32", True, True)])
def test_rope_q(T, H, nope, R, half, dtype, inplace, strided):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + H)
    D = nope + R
    pad = 16 if strided else 0
    wide = torch.randn((T, H + (1 if strided else 0), D + pad), generator=g, device="cuda").to(dt)
    q = wide[:, :H, :D]
    before = wide.clone()
    table = torch.from_numpy(W.rope_table(500, R)).cuda()
    pos = i32(np.random.default_rng(T).integers(0, 520, T), "cuda")     # some past the table: its last row
    out = q if inplace else guarded_empty((T, H, D), dt)
    mp.mla_rope_q(q, pos, table, out, d_nope=nope, layout="half" if half else "interleaved")
    check_guards("rope_q")
    x = before[:, :H, :D].double()
    tab = table.double()[pos.long().clamp(max=499)][:, None]
    ref, mag = rotate(x[..., nope:], tab, half)
    assert same(out[..., :nope], before[:, :H, :nope])
    # two products and a sum in binary32, then one rounding to the type
    tol = mag * 2 * U32 + ref.abs() * (HALF_BF16 * 1.01 if dt == torch.bfloat16 else U32)
    assert bool(((out[..., nope:].double() - ref).abs() <= tol).all())
    if strided:
        assert same(wide[:, :, D:], before[:, :, D:]) and same(wide[:, H:], before[:, H:])
    if not inplace:
        assert same(wide, before)


@pytest.mark.parametrize("K, R, half, dtype, page_size", [
    (512, 64, False, "bf16", 16), (512, 64, True, "bf16", 7), (64, 16, True, "bf16", 1), (256, 512, True, "bf16", 16),
    (512, 64, True, "e4m3", 16), (128, 32, False, "e4m3", 5), (512, 0, False, "bf16", 16)])
def test_latent_write_at(K, R, half, dtype, page_size):
    case = W.latent_write_case("at", seed=K + R, seq_lens=[3, 0, 17, 1, 9], start_lengths=[0, 5, 30, 100, 16],
                               page_size=page_size, K=K, R=R, dtype=dtype, max_seq_len=200)
    dc, t = W.device_latent_write(case)
    before = dc.pool.clone()
    rng = np.random.default_rng(3)
    pos = rng.integers(0, 200, case.T)
    call = mp.mla_write_latent_paged_fp8_at if dtype == "e4m3" else mp.mla_write_latent_paged_at
    call(t["x"], t["input_row_offsets"], i32(pos, "cuda"), t["gamma"], case.eps, t["freqs"] if R else None, K,
         cache_of(dc), 1, layout="half" if half else "interleaved")
    x = t["x"].double()
    lat = x[:, :K]
    lat = t["gamma"].double() * lat / torch.sqrt((lat * lat).mean(1, keepdim=True) + case.eps)
    ref, mag = lat, lat.abs()
    if R:
        rot, m = rotate(x[:, K:], t["freqs"].double()[torch.from_numpy(pos).cuda()], half)
        ref, mag = torch.cat([lat, rot], 1), torch.cat([mag, m], 1)
    offs = np.concatenate([[0], np.cumsum([3, 0, 17, 1, 9])])
    where = [(int(case.cache.page_table[b, (l + i) // page_size]), (l + i) % page_size)
             for b, l in enumerate([0, 5, 30, 100, 16]) for i in range(offs[b + 1] - offs[b])]
    page, slot = (torch.tensor(v, device="cuda") for v in zip(*where))
    got = dc.pool[page, 1, 0, slot, 0]
    # binary32: the sum of K squares, a root and a division, three products; then one rounding
    err32 = mag * (K + 8) * U32
    if dtype == "e4m3":
        sc = dc.scales[page, 1, 0, slot].double().repeat_interleave(128, 1)[:, :K + R]
        got = got.view(torch.float8_e4m3fn).float().double() * sc
        # a code is off by half a step, 2^-4 of its value, or half the smallest step, 2^-10
        tol = err32 + ref.abs() * 2.0 ** -4 * 1.001 + sc * 2.0 ** -10
    else:
        got, tol = got.double(), err32 + ref.abs() * HALF_BF16 * 1.001
    assert bool(((got - ref).abs() <= tol).all())
    keep = torch.ones(dc.pool.shape[:4], dtype=torch.bool, device="cuda")
    keep[page, 1, 0, slot] = False
    raw = torch.uint8 if dtype == "e4m3" else torch.int16
    assert same(dc.pool.view(raw)[keep], before.view(raw)[keep])


def test_latent_write_at_its_own_positions_is_the_plain_write():
    for dtype in ("bf16", "e4m3"):
        case = W.latent_write_case("same", seed=5, seq_lens=[40, 3], start_lengths=[7, 90], page_size=16, dtype=dtype)
        dc, t = W.device_latent_write(case)
        other, _ = W.device_latent_write(case)
        pos = i32(list(range(7, 47)) + [90, 91, 92], "cuda")
        args = (t["gamma"], case.eps, t["freqs"], 512)
        if dtype == "e4m3":
            mp.mla_write_latent_paged_fp8(t["x"], t["input_row_offsets"], *args, cache_of(dc), 1)
            mp.mla_write_latent_paged_fp8_at(t["x"], t["input_row_offsets"], pos, *args, cache_of(other), 1)
            assert same(dc.scales.view(torch.int32), other.scales.view(torch.int32))
        else:
            mp.mla_write_latent_paged(t["x"], t["input_row_offsets"], *args, cache_of(dc), 1)
            mp.mla_write_latent_paged_at(t["x"], t["input_row_offsets"], pos, *args, cache_of(other), 1)
        assert same(dc.pool.view(torch.uint8), other.pool.view(torch.uint8))


# ---------------------------------------------------------------------------
# tree attention
# ---------------------------------------------------------------------------
def attend(case, lse=True, workspace=None, stream=None):
    dt = case.q.dtype
    out = guarded_empty((case.T, case.H, case.K), dt)
    out.fill_(7.25)
    z = guarded_empty((case.T, case.H), torch.float32)
    z.fill_(7.25)
    size = mp.mla_tree_attention_workspace_size(case.T, case.H, case.K)
    if workspace is None:
        workspace = guarded_empty((size,), torch.uint8)
        workspace.fill_(0xFF)     # NaN as floats: nothing in it has to start at zero
    call = mp.mla_tree_attention_paged_fp8_cache if case.host.dtype == "e4m3" else mp.mla_tree_attention_paged
    call(case.q, case.iro, case.mask, case.scale, case.K, cache_of(case), case.layer, out, workspace,
         lse=z if lse else None, stream=stream)
    check_guards("tree attention")
    return out, z


SHAPES = [
    # lens, new, heads, page_size, mask
    ([0], [1], 1, 16, "chain"),
    ([5], [1], 16, 16, "chain"),
    ([31, 32, 33, 63, 64, 65], [1] * 6, 16, 16, "chain"),
    ([127, 128, 129, 1000], [1] * 4, 128, 128, "chain"),
    ([0, 700, 3, 0], [3, 0, 1, 33], 20, 7, "chain"),
    ([100, 257, 0], [8, 64, 5], 16, 16, "tree"),
    ([40, 0, 9], [100, 65, 1], 3, 1, "tree"),
    ([0, 0, 40, 17], [4, 1, 30, 64], 128, 64, "holes"),
    ([2000, 1], [2, 130], 33, 100, "holes"),
    ([4000, 333, 1500], [7, 1, 12], 128, 128, "tree"),
    ([9000], [1], 5, 16, "chain"),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("lens, new, heads, page_size, mask", SHAPES)
def test_tree_attention(lens, new, heads, page_size, mask, dtype):
    case = AttentionCase(len(lens) * 100 + heads, lens, new, heads, page_size=page_size, mask=mask, dtype=dtype)
    check_attention(case, *attend(case))


@pytest.mark.parametrize("K, R, dtype", [(64, 16, "f32"), (64, 16, "bf16"), (512, 0, "bf16"), (256, 64, "bf16"),
                                         (8, 8, "f32"), (128, 64, "e4m3"), (512, 512, "bf16"), (256, 128, "e4m3")])
def test_tree_attention_other_row_widths(K, R, dtype):
    case = AttentionCase(K + R, [50, 0, 300], [3, 9, 1], 6, K=K, R=R, dtype=dtype, mask="tree")
    check_attention(case, *attend(case))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_tree_attention_large_scores(dtype):
    # scores of several hundred: the running maximum moves a lot, most weights vanish
    case = AttentionCase(77, [700, 64], [5, 20], 24, mask="tree", q_std=60.0, dtype=dtype)
    out, z = attend(case)
    ref, zref, _, ltol = case.reference()
    # the weights' error bound is vacuous at such scores; the sums' bound is not
    assert bool(torch.isfinite(out.double()).all())
    assert bool(((z.double() - zref).abs() <= ltol).all())
    # where one row holds nearly all the weight the output is that row
    assert float((out.double() - ref).abs().max()) < 0.5


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_tree_attention_rows_a_token_does_not_see_may_hold_anything(dtype):
    new = [6, 40]
    case = AttentionCase(5, [70, 10], new, 32, mask="tree", dtype=dtype)
    # token 4 of request 0 and token 20 of request 1 hold NaN and infinities; only they see themselves
    bad = {0: 4, 1: 20}
    rows = []
    for b in (0, 1):
        case.seen[b] = [m & ~(1 << bad[b]) | ((1 << bad[b]) if i == bad[b] else 0) for i, m in enumerate(case.seen[b])]
        rows += case.seen[b]
    case.mask = mask_tensor(rows, 1, "cuda")
    for b in (0, 1):
        p = int(case.lens[b]) + bad[b]
        page, slot = int(case.host.page_table[b, p // 16]), p % 16
        row = case.dev.pool[page, 1, 0, slot, 0]
        if dtype == "e4m3":
            row[::3] = 0x7F
            case.dev.scales[page, 1, 0, slot, 1] = math.inf
        else:
            row[::3] = math.nan
            row[1::3] = math.inf
            row[2::3] = -math.inf
    out, z = attend(case)
    seers = torch.tensor([bad[0], new[0] + bad[1]], device="cuda")
    assert bool(torch.isnan(out[seers]).all()) and bool(torch.isnan(z[seers]).all())
    # the others: as if those rows were never there
    keep = torch.ones(sum(new), dtype=torch.bool, device="cuda")
    keep[seers] = False
    for b in (0, 1):
        p = int(case.lens[b]) + bad[b]
        page, slot = int(case.host.page_table[b, p // 16]), p % 16
        case.dev.pool[page, 1, 0, slot, 0] = 0
        if dtype == "e4m3":
            case.dev.scales[page, 1, 0, slot] = 1.0
    ref, zref, tol, ltol = case.reference()
    assert bool(((out.double() - ref).abs()[keep] <= tol[keep]).all())
    assert bool(((z.double() - zref).abs()[keep] <= ltol[keep]).all())


def test_tree_attention_padded_batch_and_no_lse():
    case = AttentionCase(6, [50, 2000], [3, 4], 16, mask="tree", extra_tokens=5)
    out, z = attend(case)
    check_attention(case, out, z)
    assert bool((out[7:] == 7.25).all()) and bool((z[7:] == 7.25).all())
    again, z2 = attend(case, lse=False)
    assert same(out, again) and bool((z2 == 7.25).all())


def test_tree_attention_mask_narrower_than_the_draft():
    case = AttentionCase(8, [20], [90], 8, mask="tree", words=1)   # drafted rows 64.. are seen by nobody
    check_attention(case, *attend(case))


def test_tree_attention_positions_past_the_page_table_are_not_seen():
    case = AttentionCase(9, [100, 30], [4, 2], 16, mask="chain", page_size=16)
    full = case.dev.page_table.shape[1] * 16
    out, z = attend(case)
    case.dev.cache_lengths.copy_(i32([0xFFFFFFFF, 30], "cuda"))    # a length no page table holds
    got, z2 = attend(case)
    assert same(got[4:], out[4:]) and full >= 104
    case.dev.cache_lengths.copy_(i32([full, 30], "cuda"))
    capped, z3 = attend(case)
    assert same(capped[4:], out[4:])


def test_tree_attention_twice_is_the_same_bits():
    case = AttentionCase(10, [5000, 1200, 60], [3, 17, 1], 128, mask="tree", page_size=64)
    a, za = attend(case)
    b, zb = attend(case)
    assert same(a, b) and same(za, zb)


def test_tree_attention_far_pages():
    # page offsets past 2^32 bytes
    page, pages = 64, 66000
    pool = torch.zeros((pages, 1, 1, page, 1, 576), dtype=torch.bfloat16, device="cuda")
    case = AttentionCase(11, [150], [2], 16, page_size=64)
    far = [65999, 3, 60001]
    for i, f in enumerate(far):
        pool[f, 0] = case.dev.pool[int(case.host.page_table[0, i]), 1]
    table = i32([far], "cuda")
    out, z = attend(case)
    got, gz = torch.empty_like(out), torch.empty_like(z)
    ws = torch.empty(mp.mla_tree_attention_workspace_size(2, 16, 512), dtype=torch.uint8, device="cuda")
    mp.mla_tree_attention_paged(case.q, case.iro, None, case.scale, 512,
                                mp.PagedKVCache(pool, table, case.dev.cache_lengths), 0, got, ws, lse=gz)
    assert same(out, got) and same(z, gz)


def test_tree_attention_captured_and_replayed():
    case = AttentionCase(12, [3000, 500], [4, 1], 64, mask="tree", page_size=32)
    cache = cache_of(case)
    out = torch.zeros((case.T, case.H, 512), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros((case.T, case.H), device="cuda")
    ws = torch.empty(mp.mla_tree_attention_workspace_size(case.T, case.H, 512), dtype=torch.uint8, device="cuda")

    def call():
        mp.mla_tree_attention_paged(case.q, case.iro, case.mask, case.scale, 512, cache, 1, out, ws, lse=z)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([3000, 500], [40, 499], [1, 0], [3000, 500]):
        case.dev.cache_lengths.copy_(i32(lens, "cuda"))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got, gz = out.clone(), z.clone()
        call()
        torch.cuda.synchronize()
        assert same(got, out) and same(gz, z)


def test_tree_attention_on_another_stream():
    case = AttentionCase(13, [1500], [5], 32, mask="tree")
    ref, zr = attend(case)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, z = attend(case, stream=s)
    s.synchronize()
    assert same(out, ref) and same(z, zr)


# ---------------------------------------------------------------------------
# page upkeep
# ---------------------------------------------------------------------------
def pages_case(seed, lens, page_size, dtype, layers=3, num_kv=1, spare=10, batch=None, extra=0, D=576, max_pages=None):
    """A pool whose every byte is distinct noise, and its page table."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    need = [-(-(l + extra) // page_size) for l in lens]
    pages = sum(need) + spare
    perm = rng.permutation(pages)
    batch = batch or len(lens)
    table = np.full((batch, max_pages or max(1, max(need)) + 1), 0xFFFFFFFF, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    eb = {"bf16": 2, "f32": 4, "e4m3": 1}[dtype]
    raw = torch.randint(0, 256, (pages, layers, num_kv, page_size, 1, D * eb), generator=g, device="cuda",
                        dtype=torch.uint8)
    pool = {"bf16": lambda: raw.view(torch.bfloat16), "f32": lambda: raw.view(torch.float32), "e4m3": lambda: raw}[dtype]()
    scales = torch.rand((pages, layers, num_kv, page_size, -(-D // 128)), generator=g, device="cuda") if eb == 1 else None
    lengths = np.zeros(batch, np.int64)
    lengths[:len(lens)] = lens
    cache = mp.PagedKVCache(pool, i32(table, "cuda"), i32(lengths, "cuda"), scales=scales)
    return cache, table, perm[at:], need


def raw_of(pool):
    return pool.view(torch.uint8)


@pytest.mark.parametrize("dtype, num_kv, page_size", [("bf16", 1, 16), ("f32", 2, 3), ("e4m3", 1, 128), ("bf16", 2, 1)])
def test_copy_pages(dtype, num_kv, page_size):
    cache, _, spare, _ = pages_case(1, [100, 40], page_size, dtype, num_kv=num_kv)
    n = cache.pool.shape[0]
    src = [int(cache.page_table[0, 0]), int(cache.page_table[1, 0]), int(cache.page_table[0, 1]), n, 2 ** 32 - 1, 0]
    dst = [int(spare[0]), int(spare[1]), int(spare[2]), int(spare[3]), int(spare[4]), n]
    want, sw = raw_of(cache.pool).clone(), None if cache.scales is None else cache.scales.clone()
    for a, b in [(a, b) for a, b in zip(src, dst) if 0 <= a < n and b < n]:
        want[b] = raw_of(cache.pool)[a]
        if sw is not None:
            sw[b] = cache.scales[a]
    mp.mla_copy_pages(i32(src, "cuda"), i32(dst, "cuda"), cache)
    assert same(raw_of(cache.pool), want)
    assert sw is None or same(cache.scales, sw)


def fork_reference(cache, table, refs, lens, parents, children, fresh):
    ps = cache.pool.shape[3]
    pool, sc = raw_of(cache.pool).clone(), None if cache.scales is None else cache.scales.clone()
    table, refs, lens = table.copy(), refs.copy(), lens.copy()
    for p, c, f in zip(parents, children, fresh):
        if p >= len(lens) or c >= len(lens) or p == c:
            continue
        L = min(int(lens[p]), table.shape[1] * ps)
        full, part = L // ps, L % ps
        if part and f >= cache.pool.shape[0]:
            continue
        table[c, :full] = table[p, :full]
        for pg in table[p, :full]:
            refs[pg] += 1
        if part:
            src = int(table[p, full])
            table[c, full] = f
            refs[f] = 1
            pool[f, :, :, :part] = pool[src, :, :, :part]
            if sc is not None:
                sc[f, :, :, :part] = sc[src, :, :, :part]
        lens[c] = L
    return pool, sc, table, refs, lens


@pytest.mark.parametrize("dtype, page_size", [("bf16", 16), ("e4m3", 7), ("f32", 1), ("bf16", 128)])
def test_fork_and_free(dtype, page_size):
    lens = [100, 0, 33, 128]
    cache, table, spare, need = pages_case(2, lens, page_size, dtype, batch=12)
    pages = cache.pool.shape[0]
    refs = np.zeros(pages, np.int64)
    for b, n in enumerate(need):
        refs[table[b, :n]] += 1
    parents, children = [0, 0, 2, 1, 3, 3, 99, 2], [4, 5, 6, 7, 8, 9, 10, 2]
    fresh = list(spare[:8])
    parents.append(0), children.append(11), fresh.append(pages)     # no page: skipped where one is needed
    lens64 = cache.cache_lengths.cpu().numpy().astype(np.int64)
    pool, sc, t2, r2, l2 = fork_reference(cache, table, refs, lens64, parents, children, fresh)
    rt = i32(refs, "cuda")
    mp.mla_fork_paged(i32(parents, "cuda"), i32(children, "cuda"), i32(fresh, "cuda"), rt, cache)
    assert same(raw_of(cache.pool), pool) and (sc is None or same(cache.scales, sc))
    assert same(cache.page_table, i32(t2, "cuda")) and same(rt, i32(r2, "cuda"))
    assert same(cache.cache_lengths, i32(l2, "cuda"))

    # free: two children (one of them listed twice), a parent, an empty request, one past the batch
    gone = [5, 0, 5, 1, 500, 8]
    r3, t3, l3, freed = r2.copy(), t2.copy(), l2.copy(), set()
    for b in gone:
        if b >= 12:
            continue
        for i in range(-(-int(l3[b]) // page_size)):
            pg = int(t3[b, i])
            t3[b, i] = 0xFFFFFFFF
            if r3[pg] > 0:
                r3[pg] -= 1
                if r3[pg] == 0:
                    freed.add(pg)
        l3[b] = 0
    lst = torch.full((pages,), -7, dtype=torch.int32, device="cuda")
    cnt = i32([2], "cuda")
    before = raw_of(cache.pool).clone()
    mp.mla_free_paged(i32(gone, "cuda"), rt, lst, cnt, cache)
    assert same(rt, i32(r3, "cuda")) and same(cache.page_table, i32(t3, "cuda"))
    assert same(cache.cache_lengths, i32(l3, "cuda")) and same(raw_of(cache.pool), before)
    assert int(cnt[0]) == 2 + len(freed)
    assert lst[:2 + len(freed)].tolist() == [-7, -7] + sorted(freed)
    assert bool((lst[2 + len(freed):] == -7).all())


def test_free_many_pages_and_a_full_list():
    # more pages than one step of the ordered walk, several holders of each, counts at 0 left alone
    pages, ps = 40000, 4
    pool = torch.zeros((pages, 1, 1, ps, 1, 8), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(0)
    table = np.stack([rng.permutation(pages)[:20000] for _ in range(3)])
    refs = np.zeros(pages, np.int64)
    for b in range(3):
        refs[table[b]] += 1
    zero = table[0, :50]
    held = refs.copy()
    held[zero] = 0
    cache = mp.PagedKVCache(pool, i32(table, "cuda"), i32([80000, 79999, 5], "cuda"))
    rt, lst, cnt = i32(held, "cuda"), i32(np.zeros(pages), "cuda"), i32([pages - 100], "cuda")
    want = held.copy()
    for b in (0, 1):
        want[table[b]] = np.maximum(want[table[b]] - 1, 0)
    freed = np.nonzero((want == 0) & (held > 0))[0]
    mp.mla_free_paged(i32([1, 0], "cuda"), rt, lst, cnt, cache)
    assert same(rt, i32(want, "cuda"))
    assert int(cnt[0]) == pages and len(freed) > 100
    assert lst[pages - 100:].tolist() == freed[:100].tolist() and bool((lst[:pages - 100] == 0).all())


@pytest.mark.parametrize("dtype, page_size, num_kv", [("bf16", 16, 1), ("e4m3", 5, 1), ("f32", 1, 2), ("bf16", 64, 2)])
def test_compact(dtype, page_size, num_kv):
    lens = [0, 100, 15, 33, 64]
    cache, table, _, _ = pages_case(3, lens, page_size, dtype, num_kv=num_kv, extra=40)
    picks = [[0, 1, 2], [0, 2, 3, 4, 9, 10, 11, 12, 13, 30, 39], [], [5], [1, 2, 3, 4, 5, 6, 7, 8, 9, 10]]
    pool, sc = raw_of(cache.pool).clone(), None if cache.scales is None else cache.scales.clone()
    for b, p in enumerate(picks):
        for i, a in enumerate(p):       # one after another, in ascending order
            s, d = lens[b] + a, lens[b] + i
            sp, dp = int(table[b, s // page_size]), int(table[b, d // page_size])
            pool[dp, :, :, d % page_size] = pool[sp, :, :, s % page_size].clone()
            if sc is not None:
                sc[dp, :, :, d % page_size] = sc[sp, :, :, s % page_size].clone()
    acc = i32(sum(picks, []), "cuda")
    off = i32(np.concatenate([[0], np.cumsum([len(p) for p in picks])]), "cuda")
    mp.mla_compact_paged(acc, off, cache)
    assert same(raw_of(cache.pool), pool)
    assert sc is None or same(cache.scales, sc)


@pytest.mark.parametrize("dtype, layers", [("bf16", 2), ("e4m3", 5)])
def test_compact_long_drafts(dtype, layers):
    # more accepted rows than a wave has lanes, in one request between two others
    lens, rng = [3, 77, 40], np.random.default_rng(5)
    cache, table, _, _ = pages_case(5, lens, 16, dtype, layers=layers, extra=300)
    picks = [[7], sorted(rng.choice(300, 171, replace=False).tolist()), list(range(64)) + [65, 200]]
    pool, sc = raw_of(cache.pool).clone(), None if cache.scales is None else cache.scales.clone()
    for b, p in enumerate(picks):
        for i, a in enumerate(p):
            s, d = lens[b] + a, lens[b] + i
            sp, dp = int(table[b, s // 16]), int(table[b, d // 16])
            pool[dp, :, :, d % 16] = pool[sp, :, :, s % 16].clone()
            if sc is not None:
                sc[dp, :, :, d % 16] = sc[sp, :, :, s % 16].clone()
    acc = i32(sum(picks, []), "cuda")
    mp.mla_compact_paged(acc, i32([0, 1, 172, 238], "cuda"), cache)
    assert same(raw_of(cache.pool), pool)
    assert sc is None or same(cache.scales, sc)


def test_compact_positions_without_a_slot_are_skipped():
    cache, table, _, _ = pages_case(4, [10, 10], 16, "bf16", extra=20)
    before = raw_of(cache.pool).clone()
    # past the page table, past 2^32 with the length added, and a page id past the pool
    cache.page_table[1, 1] = 10 ** 6
    mp.mla_compact_paged(i32([1000, 0xFFFFFFFF, 7], "cuda"), i32([0, 2, 3], "cuda"), cache)
    assert same(raw_of(cache.pool), before)


# ---------------------------------------------------------------------------
# the whole step
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_drafted_step(dtype):
    """Rotate, absorb, write, attend, then accept a path, move its rows, fork a request and
    attend again: the outputs of the accepted tokens do not change by more than the bound of
    either call, and the fork answers as its parent, bit for bit."""
    H, ps, rng = 16, 16, np.random.default_rng(1)
    lens, new = np.array([45, 130]), np.array([7, 5])
    base = AttentionCase(20, lens, new, H, page_size=ps, mask="tree", dtype=dtype)
    T = int(new.sum())
    # a third, free row of the page table and two spare pages for the fork
    table = np.full((3, base.host.page_table.shape[1] + 1), 0xFFFFFFFF, np.int64)
    table[:2, :-1] = base.host.page_table
    spare = [p for p in range(base.host.num_pages) if p not in set(base.host.page_table.flatten().tolist())]
    lengths = i32([45, 130, 0], "cuda")
    cache = mp.PagedKVCache(base.dev.pool, i32(table, "cuda"), lengths, scales=base.dev.scales)
    freqs = torch.empty((300, 64), device="cuda")
    mp.mla_rope_freqs(freqs, scaling="by_parts", factor=4.0, original_max_position=64)
    depth = np.concatenate([[bin(m).count("1") - 1 for m in r] for r in base.seen])
    pos = i32(np.repeat(lens, new) + depth, "cuda")
    iro = i32([0, 7, 12, 12], "cuda")
    absorb = W.absorb_case("step", seed=3, T=T, H=H)
    at = W.device_absorb(absorb)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((T, 576), generator=g, device="cuda").to(torch.bfloat16)
    gamma = torch.rand(512, generator=g, device="cuda") + 0.5

    q = torch.empty_like(at["q"])
    mp.mla_rope_q(at["q"], pos, freqs, q)
    ql = torch.empty((T, H, 576), dtype=torch.bfloat16, device="cuda")
    mp.mla_absorb_q(q, at["w_uk"], ql)
    if dtype == "e4m3":
        mp.mla_write_latent_paged_fp8_at(x, iro, pos, gamma, 1e-6, freqs, 512, cache, 1)
    else:
        mp.mla_write_latent_paged_at(x, iro, pos, gamma, 1e-6, freqs, 512, cache, 1)
    call = mp.mla_tree_attention_paged_fp8_cache if dtype == "e4m3" else mp.mla_tree_attention_paged
    out = torch.empty((T, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((T, H), device="cuda")
    ws = torch.empty(mp.mla_tree_attention_workspace_size(T, H, 512), dtype=torch.uint8, device="cuda")
    call(ql, iro, base.mask, base.scale, 512, cache, 1, out, ws, lse=lse)
    base.q = ql
    check_attention(base, out, lse)      # the reference reads the rows that the write stored
    tol = base.reference()[2]

    # accept the path of the deepest token of each request
    paths = []
    for b in range(2):
        best = max(base.seen[b], key=lambda m: (bin(m).count("1"), m))
        paths.append([j for j in range(int(new[b])) if (best >> j) & 1])
    mp.mla_compact_paged(i32(sum(paths, []), "cuda"), i32([0, len(paths[0]), len(paths[0]) + len(paths[1]),
                                                          len(paths[0]) + len(paths[1])], "cuda"), cache)
    # fork request 0, all its accepted rows cached, into row 2
    took = i32([lens[0] + len(paths[0]), lens[1] + len(paths[1]), 0], "cuda")
    lengths.copy_(took)
    refs = np.zeros(base.host.num_pages, np.int64)
    for b in range(2):
        refs[table[b, :-(-int(lens[b] + new[b]) // ps)]] = 1
    rt = i32(refs, "cuda")
    mp.mla_fork_paged(i32([0], "cuda"), i32([2], "cuda"), i32([spare[0]], "cuda"), rt, cache)
    # the accepted tokens again, now as a chain behind the old lengths, for requests 0, 1 and the fork
    lengths.copy_(i32([lens[0], lens[1], lens[0]], "cuda"))
    n0, n1 = len(paths[0]), len(paths[1])
    pick = torch.tensor(paths[0] + [7 + j for j in paths[1]] + paths[0], device="cuda")
    T2 = len(pick)
    out2 = torch.empty((T2, H, 512), dtype=torch.bfloat16, device="cuda")
    ws2 = torch.empty(mp.mla_tree_attention_workspace_size(T2, H, 512), dtype=torch.uint8, device="cuda")
    call(ql[pick].contiguous(), i32([0, n0, n0 + n1, T2], "cuda"), None, base.scale, 512, cache, 1, out2, ws2)
    assert same(out2[:n0], out2[n0 + n1:])
    assert bool(((out2[:n0 + n1].double() - out[pick[:n0 + n1]].double()).abs() <= 2 * tol[pick[:n0 + n1]]).all())
