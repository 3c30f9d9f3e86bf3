"""The paged K/V cache's operators on the GPU against plain 64-bit forms: rotating and quantising
writes, reading back, attention with and without a window."""
import math

import numpy as np
import pytest
import torch

import mla_paged_latent_page_amd as mp
import workloads as W
from gpu_util import check_guards, guarded_empty
from plain_kv import KvCase, cast_pool, check_kv_attention, quantised, rotated
from plain_step import HALF_BF16, U32, i32

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def same(a, b):
    return bool(torch.equal(a, b))


def cache_of(case):
    return mp.PagedKVCache(case.dev.pool, case.dev.page_table, case.dev.cache_lengths, scales=case.dev.scales)


def attend(case, lse=True, workspace=None, stream=None, q=None, guard=True):
    q = case.q if q is None else q
    out = guarded_empty((case.T, case.H, case.D), case.q.dtype) if guard else torch.empty_like(case.q)
    z = guarded_empty((case.T, case.H), torch.float32) if lse and guard else \
        torch.empty((case.T, case.H), device="cuda") if lse else None
    out.fill_(7.0)
    if lse:
        z.fill_(7.0)
    if workspace is None:
        size = mp.kv_attention_workspace_size(case.T, case.H, case.KH, case.D)
        workspace = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    call = mp.kv_attention_paged_fp8_cache if case.dtype == "e4m3" else mp.kv_attention_paged
    call(q, case.iro, case.scale, cache_of(case), case.layer, out, workspace, window=case.window, sinks=case.sinks,
         lse=z, stream=stream)
    if guard:
        check_guards("kv_attention")
    return out, z


# ---------------------------------------------------------------------------
# writes
# ---------------------------------------------------------------------------
def written(case, seq):
    """(page, slot) of every new token, in order."""
    pages, slots = zip(*(case.where(b, range(int(n), int(n) + m)) for b, (n, m) in enumerate(zip(case.lens, seq)) if m))
    return torch.cat(pages), torch.cat(slots)


@pytest.mark.parametrize("KH, D, rope, half, dtype, page_size, fused, given", [
    (8, 128, 128, True, "bf16", 16, True, False), (8, 128, 128, False, "e4m3", 16, True, False),
    (2, 64, 64, True, "e4m3", 7, False, True), (3, 64, 32, False, "e4m3", 1, True, True),
    (1, 8, 8, False, "bf16", 5, False, False), (1, 16, 16, True, "e4m3", 64, True, False),
    (5, 112, 0, False, "e4m3", 16, False, False), (5, 112, 48, True, "bf16", 100, True, True),
    (2, 256, 256, True, "e4m3", 16, False, False), (16, 256, 64, False, "bf16", 32, True, False),
    (40, 80, 80, True, "e4m3", 16, True, True)])
def test_write(KH, D, rope, half, dtype, page_size, fused, given):
    lens, seq = [0, 5, 30, 100, 16, 3], [3, 0, 17, 1, 9, 40]
    case = KvCase(KH + D, lens, seq, KH, KH, D, page_size=page_size, dtype=dtype)
    T = case.T
    g = torch.Generator(device="cuda").manual_seed(D)
    wide = torch.randn((T, 3 * KH, D), generator=g, device="cuda").to(BF16)
    k, v = (wide[:, KH:2 * KH], wide[:, 2 * KH:]) if fused else (wide[:, :KH].contiguous(), wide[:, KH:2 * KH].contiguous())
    k[1] = 0
    v[2, 0] = 0
    table = torch.from_numpy(W.rope_table(120, rope)).cuda() if rope else None
    own = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, seq)])
    pos = np.random.default_rng(1).integers(0, 130, T) if given else own      # some past the table: its last row
    before, sbefore = case.dev.pool.clone(), None if case.dev.scales is None else case.dev.scales.clone()
    call = mp.kv_write_paged_fp8 if dtype == "e4m3" else mp.kv_write_paged
    call(k, v, case.iro, cache_of(case), 1, positions=i32(pos, "cuda") if given else None, freqs_cis=table,
         layout="half" if half else "interleaved")
    tab = table.double()[torch.from_numpy(pos).cuda().clamp(max=119)] if rope else None
    page, slot = written(case, seq)
    kr, kmag = rotated(k.double(), tab, rope, half)
    for side, ref, mag in ((0, kr, kmag), (1, v.double(), v.double().abs())):
        got = case.dev.pool[page, 1, side, slot]
        err32 = mag * 2 * U32        # two products and a sum in binary32
        if dtype == "e4m3":
            # a code is off by half a step, 2^-4 of its value, or half the smallest step, 2^-10
            sc = case.dev.scales[page, 1, side, slot].double()
            amax = torch.nn.functional.pad(ref.reshape(T, -1).abs(), (0, -KH * D % 128)).view(T, -1, 128).amax(2)
            want = torch.where(amax == 0, 448.0, amax) / 448
            assert bool(((sc - want).abs() <= want * 4 * U32).all())
            sc = sc.repeat_interleave(128, 1)[:, :KH * D].view(T, KH, D)
            got = cast_pool(got, dtype) * sc
            tol = err32 + ref.abs() * 2.0 ** -4 * 1.001 + sc * 2.0 ** -10
        else:
            got, tol = got.double(), err32 + ref.abs() * HALF_BF16 * 1.001
        assert bool(((got - ref).abs() <= tol).all())
    keep = torch.ones(case.dev.pool.shape[:4], dtype=torch.bool, device="cuda")
    keep[page, 1, :, slot] = False
    raw = torch.uint8 if dtype == "e4m3" else torch.int16
    assert same(case.dev.pool.view(raw)[keep], before.view(raw)[keep])
    if sbefore is not None:
        assert same(case.dev.scales.view(torch.int32)[keep], sbefore.view(torch.int32)[keep])


def test_write_codes_are_the_documented_quotients():
    # no rotation: amax, quotient and rounding in binary32, bit for bit; blocks of very small and large values
    case = KvCase(3, [4], [6], 4, 4, 64, dtype="e4m3")
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((6, 4, 64), generator=g, device="cuda") for _ in range(2))
    for i, f in enumerate((1.0, 1e-30, 2.0 ** -127, 1e30, 0.0, 1e38)):
        k[i] *= f
    k, v = k.clamp(-3e38, 3e38).to(BF16), v.to(BF16)
    mp.kv_write_paged_fp8(k, v, case.iro, cache_of(case), 1)
    page, slot = written(case, [6])
    for side, x in ((0, k), (1, v)):
        codes, scales = quantised(x.double().view(6, 256))
        assert same(case.dev.pool[page, 1, side, slot].view(6, 256), codes.view(torch.uint8))
        assert same(case.dev.scales[page, 1, side, slot], scales)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_writes_without_a_slot_are_skipped(dtype):
    case = KvCase(5, [10, 30, 3], [8, 4, 2], 2, 2, 128, page_size=8, dtype=dtype)
    case.dev.page_table[0, 2] = case.dev.pool.shape[0]       # positions 16 and 17: a page past the pool
    case.dev.cache_lengths[1] = 1 << 20                      # past the page table
    case.dev.cache_lengths[2] = -1                           # 2^32 - 1, then past 2^32
    before = case.dev.pool.clone()
    k = torch.full((14, 2, 128), 3.0, dtype=BF16, device="cuda")
    (mp.kv_write_paged_fp8 if dtype == "e4m3" else mp.kv_write_paged)(k, -k, case.iro, cache_of(case), 1)
    page, slot = case.where(0, range(10, 16))
    keep = torch.ones(case.dev.pool.shape[:4], dtype=torch.bool, device="cuda")
    keep[page, 1, :, slot] = False
    raw = torch.uint8 if dtype == "e4m3" else torch.int16
    assert same(case.dev.pool.view(raw)[keep], before.view(raw)[keep])
    got = cast_pool(case.dev.pool[page, 1, :, slot], dtype)
    want = 448.0 if dtype == "e4m3" else 3.0
    assert bool((got[:, 0] == want).all()) and bool((got[:, 1] == -want).all())


@pytest.mark.parametrize("requests", [1, 64, 65, 300])
def test_write_finds_each_tokens_request(requests):
    rng = np.random.default_rng(requests)
    seq = rng.choice([0, 1, 2, 5], requests)
    seq[-1] = 3
    case = KvCase(6, rng.integers(0, 9, requests), seq, 1, 1, 16, page_size=4)
    x = torch.arange(case.T, device="cuda").to(BF16)[:, None, None].expand(-1, 1, 16).contiguous()
    mp.kv_write_paged(x, -x, case.iro, cache_of(case), 1)
    page, slot = written(case, seq)
    assert same(case.dev.pool[page, 1, 0, slot], x) and same(case.dev.pool[page, 1, 1, slot], -x)


# ---------------------------------------------------------------------------
# reading back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("KH, D, page_size, dtype", [
    (8, 128, 16, "bf16"), (8, 128, 16, "e4m3"), (1, 8, 3, "bf16"), (1, 16, 3, "e4m3"), (2, 64, 1, "f32"), (1, 4, 5, "f32"),
    (5, 112, 100, "e4m3"), (3, 80, 7, "bf16"), (40, 256, 16, "f32")])
def test_gather(KH, D, page_size, dtype):
    lens = [70, 0, 5, 33, 128]
    first = [3, 0, 5, 32, 0]
    case = KvCase(KH + D, lens, [0] * 5, KH, KH, D, page_size=page_size, dtype=dtype)
    rows = [n - f for n, f in zip(lens, first)]
    M = sum(rows)
    dt = {"bf16": BF16, "e4m3": BF16, "f32": torch.float32}[dtype]
    k, v = guarded_empty((M, KH, D), dt), guarded_empty((M, KH, D), dt)
    call = mp.kv_gather_paged_fp8_cache if dtype == "e4m3" else mp.kv_gather_paged
    call(i32(np.concatenate([[0], np.cumsum(rows)]), "cuda"), i32(first, "cuda"), M, cache_of(case), 1, k, v)
    check_guards("kv_gather")
    for side, got in ((0, k), (1, v)):
        if dtype == "e4m3":    # the product in binary32, then one rounding
            ref = torch.cat([case.rows64(b, side, range(f, n)) for b, (f, n) in enumerate(zip(first, lens)) if f < n])
            assert same(got, ref.float().to(BF16))
        else:
            where = [case.where(b, range(f, n)) for b, (f, n) in enumerate(zip(first, lens)) if f < n]
            ref = torch.cat([case.dev.pool[p, 1, side, s] for p, s in where])
            raw = torch.int16 if dtype == "bf16" else torch.int32
            assert same(got.view(raw), ref.view(raw))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
CASES = [
    # lens, new, heads, kv_heads, head_dim, page_size, window, sinks
    ([5], [1], 1, 1, 8, 16, 0, 0),
    ([0], [1], 8, 8, 128, 16, 0, 0),
    ([0, 1, 2, 63, 64, 65], [1] * 6, 8, 2, 128, 16, 0, 0),
    ([300, 0, 65], [4, 0, 9], 14, 2, 64, 3, 0, 0),
    ([700, 20], [3, 1], 32, 8, 128, 100, 0, 0),
    ([0, 90], [70, 200], 10, 2, 128, 64, 0, 0),
    ([33], [129], 7, 1, 64, 16, 0, 0),
    ([100, 7, 0], [3, 20, 40], 12, 12, 80, 16, 0, 0),
    ([50, 4], [2, 130], 9, 3, 112, 7, 0, 0),
    ([64, 3], [5, 1], 4, 2, 256, 16, 0, 0),
    ([500, 20], [3, 1], 8, 2, 128, 16, 100, 4),
    ([500, 0, 30], [80, 300, 1], 16, 4, 64, 32, 64, 3),
    ([200, 10], [150, 40], 6, 3, 128, 100, 1, 0),
    ([200, 10], [150, 40], 6, 3, 128, 16, 1, 1),
    ([900], [260], 8, 1, 128, 64, 130, 70),
    ([60, 900], [8, 1], 5, 1, 80, 16, 33, 200),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("lens, new, H, KH, D, page_size, window, sinks", CASES)
def test_attention(lens, new, H, KH, D, page_size, window, sinks, dtype):
    if dtype == "e4m3" and KH * D % 16:
        pytest.skip("rows of codes are multiples of 16 bytes")
    case = KvCase(H + D, lens, new, H, KH, D, page_size=page_size, dtype=dtype, window=window, sinks=sinks)
    check_kv_attention(case, *attend(case))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D", [64, 128, 80])
def test_rows_behind_the_last_sequence_are_left(D, dtype):
    case = KvCase(2, [30, 2], [5, 70], 8, 2, D, dtype=dtype, extra_tokens=4)
    case.q[-4:] = math.nan
    out, z = attend(case)
    assert bool((out[-4:] == 7.0).all()) and bool((z[-4:] == 7.0).all())
    check_kv_attention(case, out, z)


def test_views_and_no_lse():
    for D, dtype in ((128, "bf16"), (64, "e4m3"), (80, "f32")):
        case = KvCase(4, [30, 2], [5, 70], 8, 2, D, dtype=dtype)
        ref, _ = attend(case)
        wide = torch.full((case.T, 12, D), math.nan, dtype=case.q.dtype, device="cuda")
        wide[:, 2:10] = case.q
        got, z = attend(case, lse=False, q=wide[:, 2:10])
        assert z is None and same(got, ref)


@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (64, "bf16"), (128, "e4m3"), (80, "f32")])
def test_positions_past_the_page_table_are_not_seen(D, dtype):
    # a table of 64 positions: tokens at 60 .. 67, then with a window that lies behind it
    case = KvCase(5, [56], [8], 4, 2, D, page_size=16, dtype=dtype)
    case.dev.cache_lengths[0] = 60
    out, z = attend(case)
    full = KvCase(5, [56], [8], 4, 2, D, page_size=16, dtype=dtype)     # its last row is position 63
    ref, zref, tol, ltol = full.reference()
    case.window = 4
    far, zfar = attend(case)     # tokens 7 .. see 64 .. only
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(far[:7]).all())
    assert bool((far[7] == 0).all()) and bool((zfar[7] == -math.inf).all())
    case.sinks = 1
    one, zone = attend(case)
    v = case.rows64(0, 1, [0])[0].repeat_interleave(2, dim=0)
    assert bool(((one[7].double() - v).abs() <= v.abs() * HALF_BF16 * 2.01).all()) and bool(torch.isfinite(zone).all())
    case.sinks, case.window = 0, 0
    case.q[3] = full.q[7]        # token 3 is at position 63 and sees what the full case's last one sees
    out, z = attend(case)
    assert bool(((out[3].double() - ref[7]).abs() <= tol[7]).all()) and bool(((z[3] - zref[7]).abs() <= ltol[7]).all())
