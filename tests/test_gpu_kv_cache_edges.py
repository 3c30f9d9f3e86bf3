"""The paged K/V cache's operators where they can go wrong: values that are not finite, shares and their
joins, scales of either sign, strided and far pools, other streams, captured graphs, and all of them together."""
import math

import numpy as np
import pytest
import torch

import mla_paged_latent_page_amd as mp
import workloads as W
from plain_kv import KvCase, check_kv_attention, quantised, rotated
from plain_step import HALF_BF16, U32, i32
from test_gpu_kv_cache import attend, cache_of, same

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------
# lens, new, heads per key head, window, sinks, position
PLANTS = [
    (200, 8, 4, 0, 0, 203),          # few rows, inside the tokens' own rows
    (100, 300, 4, 0, 0, 150),        # many rows
    (100, 300, 1, 0, 0, 399),        # only the last token sees it
    (500, 300, 2, 64, 0, 520),       # leaves the window again
    (500, 9, 2, 64, 4, 3),           # a sink
    (500, 300, 2, 64, 4, 4),         # just behind the sinks, seen by nobody
    (500, 300, 2, 600, 4, 4),        # ... and by some
    (1000, 2, 8, 0, 0, 70),          # far from every edge: seen by all
]


@pytest.mark.parametrize("what", ["v nan", "v inf", "k nan", "k scale", "v scale"])
@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (64, "bf16"), (128, "e4m3"), (64, "e4m3"), (80, "e4m3"), (80, "bf16"),
                                      (64, "f32")])
@pytest.mark.parametrize("lens, new, G, window, sinks, at", PLANTS)
def test_what_a_token_does_not_see_may_hold_anything(lens, new, G, window, sinks, at, D, dtype, what):
    fp8 = dtype == "e4m3"
    if "scale" in what and not fp8 or what == "v inf" and fp8:
        pytest.skip("no such value in this cache")
    KH = 2
    case = KvCase(at + D, [lens], [new], KH * G, KH, D, page_size=16, dtype=dtype, window=window, sinks=sinks)
    ref, zref, tol, ltol = case.reference()
    page, slot = case.where(0, [at])
    page, slot, side = int(page[0]), int(slot[0]), 0 if what[0] == "k" else 1
    col = torch.arange(KH * D, device="cuda").view(KH, D)
    if "scale" in what:
        case.dev.scales[page, 1, side, slot, 0] = math.nan if side == 0 else math.inf
        bad = col < 128
    else:
        value = 0x7F if fp8 else math.inf if what == "v inf" else math.nan
        case.dev.pool[page, 1, side, slot, 1, 5] = value
        bad = col == D + 5
    bad = bad.any(1, keepdim=True).expand(KH, D) if side == 0 else bad
    bad = bad.repeat_interleave(G, 0)
    out, z = attend(case)
    sees = case.seen(0)[:, at]
    hit = sees[:, None, None] & bad
    free = ~hit
    if "scale" in what and D != 80 and side == 1:      # every column of a head with such a scale may be lost
        free &= ~(sees[:, None, None] & bad.any(1, keepdim=True))
    assert not bool(torch.isfinite(out[hit]).any())
    if what == "v inf":
        assert bool((out[hit] == math.inf).all())
    assert bool(torch.isfinite(out[free]).all())
    assert bool(((out.double() - ref).abs() <= tol)[free].all())
    zhit = sees[:, None] & bad.any(1) if side == 0 else torch.zeros_like(z, dtype=torch.bool)
    assert not bool(torch.isfinite(z[zhit]).any())
    assert bool(((z.double() - zref).abs() <= ltol)[~zhit].all())


@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (64, "bf16"), (80, "bf16"), (64, "f32")])
def test_infinite_scores(D, dtype):
    # a key of +infinity in one column: heads whose query is positive there have a score of +infinity, the others
    # one of -infinity, a weight of 0
    at = 150
    case = KvCase(60, [140], [70], 8, 2, D, dtype=dtype)
    flip = torch.arange(8, device="cuda") % 2 * 2 - 1
    case.q[:, :, 3] = (case.q[:, :, 3].abs() + 0.1) * flip
    page, slot = case.where(0, [at])
    sees = case.seen(0)[:, at]
    hidden = case.seen(0)
    clean = case.reference()
    hidden[:, at] = False
    case.seen = lambda b: hidden
    without = case.reference()
    case.dev.pool[int(page[0]), 1, 0, int(slot[0]), :, 3] = math.inf
    out, z = attend(case)
    lost = sees[:, None] & (flip > 0)
    assert not bool(torch.isfinite(out[lost]).any()) and not bool(torch.isfinite(z[lost]).any())
    for (ref, zref, tol, ltol), rows in ((clean, ~sees[:, None] & (flip != 0)), (without, sees[:, None] & (flip < 0))):
        assert bool(((out.double() - ref).abs() <= tol)[rows].all())
        assert bool(((z.double() - zref).abs() <= ltol)[rows].all())


def test_written_values_that_are_not_finite():
    case = KvCase(61, [4], [3], 2, 2, 128, dtype="e4m3")
    g = torch.Generator(device="cuda").manual_seed(61)
    k, v = (torch.randn((3, 2, 128), generator=g, device="cuda").to(BF16) for _ in range(2))
    want = k.clone()
    k[0, 0, 3], k[1, 0, 3], k[1, 1, 5], v[2] = math.nan, math.inf, -math.inf, math.nan
    want[0, 0, 3] = 0
    mp.kv_write_paged_fp8(k, v, case.iro, cache_of(case), 1)
    page, slot = case.where(0, range(4, 7))
    codes, scales = quantised(want.double().view(3, 256))
    got, sc = case.dev.pool[page, 1, 0, slot].view(3, 256), case.dev.scales[page, 1, 0, slot]
    keep = torch.ones(256, dtype=torch.bool, device="cuda")
    keep[3] = False
    assert same(got[0, keep], codes.view(torch.uint8)[0, keep]) and same(sc[0], scales[0])
    assert int(got[0, 3]) & 0x7F == 0x7F and bool(torch.isinf(sc[1]).all())
    assert same(got[2], codes.view(torch.uint8)[2]) and same(sc[2], scales[2])
    assert bool((case.dev.pool[page, 1, 1, slot][2] & 0x7F == 0x7F).all())


# ---------------------------------------------------------------------------
# shares, joins, shapes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("lens, new, H, KH, D, page_size, window, sinks", [
    ([20000], [1], 8, 2, 128, 16, 0, 0),                   # one request over all shares
    ([33000], [1], 1, 1, 64, 8, 0, 0),
    ([9000], [200], 8, 1, 64, 3, 0, 0),                    # more tiles than page ids are held for
    ([7000], [130], 4, 2, 128, 1, 0, 0),
    ([6000], [100], 6, 1, 128, 24, 5000, 100),
    ([5000, 0, 40, 4000, 9], [1, 0, 0, 3, 0], 8, 4, 128, 16, 0, 0),
    (list(range(0, 1400, 20)), [1] * 70, 8, 2, 64, 16, 0, 0),      # more requests than 64 lanes
    ([3000] * 33 + [0] * 33, [1] * 33 + [0, 2] * 16 + [1], 4, 1, 128, 16, 0, 0),
    ([10, 700, 64, 0], [128, 129, 256, 257], 1, 1, 64, 16, 0, 0),  # rows of an item, and one more
    ([700, 10], [43, 86], 3, 1, 128, 48, 0, 0),
    ([700, 10], [1, 3], 160, 1, 64, 16, 0, 0),             # a token's heads in two items
    ([300], [2], 64, 64, 64, 128, 0, 0),
    ([63, 64, 127, 128, 129], [2] * 5, 4, 2, 128, 16, 64, 64),
    ([63, 64, 127, 128, 129], [70, 1, 64, 65, 130], 4, 1, 64, 16, 63, 65),
    ([400, 1000], [65, 300], 2, 1, 128, 8, 128, 1),
])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_shares_and_joins(lens, new, H, KH, D, page_size, window, sinks, dtype):
    case = KvCase(H + D, lens, new, H, KH, D, page_size=page_size, dtype=dtype, window=window, sinks=sinks)
    out, z = attend(case)
    check_kv_attention(case, out, z)
    again, z2 = attend(case)
    assert same(out, again) and same(z, z2)


@pytest.mark.parametrize("D, dtype", [(64, "bf16"), (64, "e4m3"), (80, "f32")])
def test_many_requests(D, dtype):
    rng = np.random.default_rng(14)
    lens, new = rng.integers(0, 200, 300), rng.choice([0, 0, 1, 2, 40], 300)
    new[5], new[299] = 70, 1
    case = KvCase(14, lens, new, 4, 2, D, dtype=dtype)
    check_kv_attention(case, *attend(case))
    rows = np.minimum(lens, rng.integers(0, 60, 300))
    M = int(rows.sum())
    dt = torch.float32 if dtype == "f32" else BF16
    kb, vb = torch.empty((M, 2, D), dtype=dt, device="cuda"), torch.empty((M, 2, D), dtype=dt, device="cuda")
    call = mp.kv_gather_paged_fp8_cache if dtype == "e4m3" else mp.kv_gather_paged
    call(i32(np.concatenate([[0], np.cumsum(rows)]), "cuda"), i32(lens - rows, "cuda"), M, cache_of(case), 1, kb, vb)
    for side, got in ((0, kb), (1, vb)):
        want = torch.cat([case.rows64(b, side, range(n - m, n)) for b, (n, m) in enumerate(zip(lens, rows)) if m])
        assert same(got, want.float().to(dt))


@pytest.mark.parametrize("page_size", [16, 3])
@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (128, "e4m3"), (64, "e4m3"), (80, "f32")])
def test_page_ids_past_the_pool_stay_with_their_request(D, dtype, page_size):
    # reads clamp them: the request's own outputs are unspecified, the others' are not touched
    case = KvCase(15, [300, 40, 200], [2, 5, 140], 8, 2, D, page_size=page_size, dtype=dtype)
    ref, zref = attend(case)
    case.dev.page_table[0, :3] = -1
    case.dev.page_table[0, 3] = case.dev.pool.shape[0]
    out, z = attend(case)
    assert same(out[2:], ref[2:]) and same(z[2:], zref[2:])


@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (64, "e4m3"), (80, "f32")])
def test_windows_without_effect(D, dtype):
    # sinks without a window, and a window longer than every context, change nothing
    case = KvCase(16, [300, 0], [3, 200], 4, 2, D, dtype=dtype)
    ref, zref = attend(case)
    case.sinks = 7
    out, z = attend(case)
    assert same(out, ref) and same(z, zref)
    for case.window, case.sinks in ((304, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
        check_kv_attention(case, *attend(case))


@pytest.mark.parametrize("scale", [-0.125, 0.0, 2.0 ** -40, -2.0 ** -135, 1.0])
@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (64, "e4m3"), (80, "f32")])
def test_scales_of_either_sign(scale, D, dtype):
    case = KvCase(9, [300, 20], [5, 90], 8, 2, D, dtype=dtype, q_std=0.25 if abs(scale) == 1 else 1.0)
    case.scale = scale
    check_kv_attention(case, *attend(case))


@pytest.mark.parametrize("D, dtype, q, k, scale", [(128, "bf16", 2.0 ** 50, 2.0 ** 50, 2.0 ** -104),
                                                  (64, "bf16", 2.0 ** 40, 2.0 ** 23, 2.0 ** -66),
                                                  (64, "bf16", 2.0 ** 40, 2.0 ** 21, -2.0 ** -64),
                                                  (128, "bf16", 2.0 ** -14, 2.0 ** -13, 2.0 ** 25),
                                                  (64, "bf16", 2.0 ** -14, 2.0 ** -13, -2.0 ** 27),
                                                  (128, "bf16", 2.0 ** -45, 2.0 ** -45, 2.0 ** 86)])
def test_small_and_large_scales(D, dtype, q, k, scale):
    # scores of ordinary size from queries, keys and scales that are not
    case = KvCase(12, [0, 0, 300, 1], [1, 3, 5, 140], 8, 2, D, dtype=dtype)
    case.q *= q
    case.dev.pool[:, :, 0] *= k
    case.scale = scale
    check_kv_attention(case, *attend(case))


def test_rows_far_apart():
    # 16 MiB between token rows
    case = KvCase(13, [40, 3], [3, 90], 8, 2, 128)
    ref, zref = attend(case)
    case.dev.pool = apart(case.dev.pool, 4 * 16 * (1 << 23) + 128, (1 << 23) - 256)
    out, z = attend(case)
    assert same(out, ref) and same(z, zref)


@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (64, "bf16"), (128, "e4m3"), (80, "f32")])
def test_scores_far_from_nought(D, dtype):
    # keys along the queries: scores grow along the sequence by far more than a weight's range, then fall again
    case = KvCase(10, [700], [3], 4, 1, D, dtype=dtype)
    case.q[:] = case.q[:1, :1]
    u = case.q[0, 0].double()
    ramp = torch.cat([torch.linspace(0, 60, 400), torch.linspace(60, -60, 303)]).double().cuda()
    rows = (ramp[:, None] * u / (u @ u) / case.scale)
    page, slot = case.where(0, range(703))
    if dtype == "e4m3":
        codes, sc = quantised(rows)
        case.dev.pool[page, 1, 0, slot] = codes.view(torch.uint8).view(703, 1, D)
        case.dev.scales[page, 1, 0, slot] = sc
    else:
        case.dev.pool[page, 1, 0, slot] = rows.to(case.dev.pool.dtype).view(703, 1, D)
    check_kv_attention(case, *attend(case))


# ---------------------------------------------------------------------------
# pools
# ---------------------------------------------------------------------------
def apart(t, page_stride, extra=0):
    """A copy of t [pages, layers, kv, slots, ...] whose pages lie page_stride elements apart and whose rows have
    `extra` elements between them."""
    width = t[0, 0, 0, 0].numel()
    st, n = width + extra, t.shape
    strides = [page_stride, n[2] * n[3] * st + 64, n[3] * st + 32, st]
    assert strides[1] * n[1] <= page_stride
    raw = torch.empty((n[0] - 1) * page_stride + n[1] * strides[1], dtype=t.dtype, device=t.device)
    inner = [t.shape[5], 1] if t.dim() == 6 else [1]
    view = raw.as_strided(n, strides + inner)
    view.copy_(t)
    return view


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (64, "bf16"), (128, "e4m3"), (64, "e4m3"), (112, "e4m3"), (80, "f32")])
def test_pools_with_rows_apart(D, dtype, far):
    lens, new, KH = [300, 0, 20], [4, 130, 1], 2
    case = KvCase(11, lens, new, 8, KH, D, page_size=16, dtype=dtype)
    # far: the last page in use begins past 2^32 elements
    top = max(int(case.where(b, range(n + m))[0].max()) for b, (n, m) in enumerate(zip(lens, new)))
    step = ((1 << 32) // top // 512 + 1) * 512 if far else 1 << 17
    ref, zref = attend(case)
    case.dev.pool = apart(case.dev.pool, step, 16 if dtype != "f32" else 4)
    if dtype == "e4m3":
        case.dev.scales = apart(case.dev.scales, step // 8 if far else 1 << 14, 3)
    out, z = attend(case)
    assert same(out, ref) and same(z, zref)
    # what was written to such a pool is read back from it
    rows = [n + m for n, m in zip(lens, new)]
    M = sum(rows)
    if dtype != "f32":
        g = torch.Generator(device="cuda").manual_seed(D)
        k, v = (torch.randn((case.T, KH, D), generator=g, device="cuda").to(BF16) for _ in range(2))
        (mp.kv_write_paged_fp8 if dtype == "e4m3" else mp.kv_write_paged)(k, v, case.iro, cache_of(case), 1)
    dt = torch.float32 if dtype == "f32" else BF16
    kb, vb = torch.empty((M, KH, D), dtype=dt, device="cuda"), torch.empty((M, KH, D), dtype=dt, device="cuda")
    call = mp.kv_gather_paged_fp8_cache if dtype == "e4m3" else mp.kv_gather_paged
    call(i32(np.concatenate([[0], np.cumsum(rows)]), "cuda"), i32([0] * 3, "cuda"), M, cache_of(case), 1, kb, vb)
    for side, got in ((0, kb), (1, vb)):
        want = torch.cat([case.rows64(b, side, range(n)) for b, n in enumerate(rows)])
        assert same(got, want.float().to(dt))
    if dtype == "bf16":
        new_rows = torch.cat([torch.arange(n, n + m) + o for n, m, o in
                              zip(lens, new, np.concatenate([[0], np.cumsum(rows)[:-1]]))]).cuda()
        assert same(kb[new_rows], k) and same(vb[new_rows], v)


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D, dtype", [(128, "bf16"), (64, "e4m3"), (80, "f32")])
def test_other_streams(D, dtype):
    cases = [KvCase(20 + i, [900 * i, 30], [1, 40], 8, 2, D, dtype=dtype) for i in range(3)]
    ref = [attend(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    call = mp.kv_attention_paged_fp8_cache if dtype == "e4m3" else mp.kv_attention_paged
    bufs = [(torch.empty_like(c.q), torch.empty((c.T, c.H), device="cuda"),
             torch.empty(mp.kv_attention_workspace_size(c.T, c.H, c.KH, c.D), dtype=torch.uint8, device="cuda"))
            for c in cases]
    for turn in range(4):
        for out, z, ws in bufs:
            out.fill_(7.0)
            z.fill_(7.0)
            ws.fill_(0xFF)
        for c, s, (out, z, ws) in zip(cases, streams, bufs):
            s.wait_stream(torch.cuda.current_stream())
            if turn % 2:
                call(c.q, c.iro, c.scale, cache_of(c), 1, out, ws, lse=z, stream=s)
            else:
                with torch.cuda.stream(s):
                    call(c.q, c.iro, c.scale, cache_of(c), 1, out, ws, lse=z)
        torch.cuda.synchronize()
        for (out, z, _), (o, zo) in zip(bufs, ref):
            assert same(out, o) and same(z, zo)


def step_buffers(case):
    g = torch.Generator(device="cuda").manual_seed(case.T)
    kv = torch.randn((case.T, 2, case.KH, case.D), generator=g, device="cuda").to(BF16)
    size = mp.kv_attention_workspace_size(case.T, case.H, case.KH, case.D)
    return dict(kv=kv, pos=i32(np.zeros(case.T), "cuda"), q2=torch.empty_like(case.q), out=torch.empty_like(case.q),
                table=torch.from_numpy(W.rope_table(4096, case.D)).cuda(),
                z=torch.empty((case.T, case.H), device="cuda"),
                ws=torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"))


def step(case, b):
    """One layer of one step as a model runs it: rotate the queries, write the new rows, attend."""
    fp8 = case.dtype == "e4m3"
    cache = cache_of(case)
    mp.mla_rope_q(case.q, b["pos"], b["table"], b["q2"], d_nope=0, layout="half")
    (mp.kv_write_paged_fp8 if fp8 else mp.kv_write_paged)(b["kv"][:, 0], b["kv"][:, 1], case.iro, cache, 1,
                                                          positions=b["pos"], freqs_cis=b["table"], layout="half")
    (mp.kv_attention_paged_fp8_cache if fp8 else mp.kv_attention_paged)(
        b["q2"], case.iro, case.scale, cache, 1, b["out"], b["ws"], window=case.window, sinks=case.sinks, lse=b["z"])


@pytest.mark.parametrize("D, dtype, window", [(128, "bf16", 0), (64, "e4m3", 100), (80, "bf16", 0)])
def test_captured_steps_replay(D, dtype, window):
    # two graphs, each with its own workspace, replayed in turn and at once, lengths moving between replays
    cases = [KvCase(30, [1000, 5, 600], [1, 1, 1], 8, 2, D, dtype=dtype, window=window),
             KvCase(31, [300], [140], 4, 1, D, dtype=dtype, window=window)]
    bufs, graphs = [step_buffers(c) for c in cases], []
    streams = [torch.cuda.Stream() for _ in cases]
    for c, b in zip(cases, bufs):
        step(c, b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(c, b)
        graphs.append(graph)
    for turn in range(4):
        want = []
        for c, b in zip(cases, bufs):
            c.dev.cache_lengths.copy_(i32(c.lens - (3 - turn) * 7 % (c.lens.min() + 1), "cuda"))
            p = np.concatenate([np.arange(m) + n for n, m in zip(c.dev.cache_lengths.tolist(), c.new.tolist())])
            b["pos"].copy_(i32(p, "cuda"))
            c.q.mul_(-1.0 if turn == 2 else 0.75)
            b["kv"].mul_(0.5 if turn == 1 else -1.25)
            step(c, b)                       # eager
            want.append((b["out"].clone(), b["z"].clone(), c.dev.pool.clone()))
            b["out"].zero_()
            b["z"].zero_()
            for i, (n, m) in enumerate(zip(c.dev.cache_lengths.tolist(), c.new.tolist())):
                page, slot = c.where(i, range(n, n + m))
                c.dev.pool[page, 1, :, slot] = 0
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            if turn % 2:
                with torch.cuda.stream(s):
                    g.replay()
            else:
                g.replay()
        torch.cuda.synchronize()
        raw = torch.uint8 if dtype == "e4m3" else torch.int16
        for c, b, (out, z, pool) in zip(cases, bufs, want):
            assert same(b["out"], out) and same(b["z"], z) and same(c.dev.pool.view(raw), pool.view(raw))


# ---------------------------------------------------------------------------
# a request's life
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("KH, G, D, dtype, half", [(2, 4, 128, "bf16", True), (4, 2, 64, "e4m3", False),
                                                  (3, 5, 80, "bf16", True)])
def test_prompt_steps_fork_and_read_back(KH, G, D, dtype, half):
    """A prompt in chunks, steps of one token, a fork, steps of both, the rows read back, all on one cache: every
    output against the 64-bit attention of the rows that the cache then holds."""
    fp8, H = dtype == "e4m3", KH * G
    case = KvCase(40, [150, 150], [1, 1], H, KH, D, page_size=16, dtype=dtype)
    cache, total = cache_of(case), 130
    g = torch.Generator(device="cuda").manual_seed(40)
    table = torch.from_numpy(W.rope_table(200, D)).cuda()
    tab64 = table.double()
    case.dev.cache_lengths.zero_()
    lens = [0, 0]
    spare = sorted(set(range(case.dev.pool.shape[0])) - set(case.host.page_table.reshape(-1).tolist()))
    refs = torch.zeros(case.dev.pool.shape[0], dtype=torch.int32, device="cuda")
    for p in case.host.page_table.reshape(-1).tolist():
        if 0 <= p < refs.numel():
            refs[p] = 1
    plan = [(70, 0), (47, 0), (1, 0), (1, 0), "fork", (1, 1), (1, 1), (5, 3)]
    for move in plan:
        if move == "fork":
            dst = spare[0] if spare else int(case.dev.page_table[1, 0])
            refs[dst] = 0
            mp.mla_fork_paged(i32([0], "cuda"), i32([1], "cuda"), i32([dst], "cuda"), refs, cache)
            lens[1] = lens[0]
            assert case.dev.cache_lengths.tolist() == lens
            case.host.page_table = case.dev.page_table.cpu().numpy().astype(np.int64)
            continue
        T = sum(move)
        x = torch.randn((T, H + 2 * KH, D), generator=g, device="cuda").to(BF16)
        pos = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, move)])
        iro, p = i32(np.concatenate([[0], np.cumsum(move)]), "cuda"), i32(pos, "cuda")
        q = torch.empty((T, H, D), dtype=BF16, device="cuda")
        mp.mla_rope_q(x[:, :H], p, table, q, d_nope=0, layout="half" if half else "interleaved")
        (mp.kv_write_paged_fp8 if fp8 else mp.kv_write_paged)(
            x[:, H:H + KH], x[:, H + KH:], iro, cache, 1, freqs_cis=table, layout="half" if half else "interleaved")
        out, z = torch.empty_like(q), torch.empty((T, H), device="cuda")
        ws = torch.empty(mp.kv_attention_workspace_size(T, H, KH, D), dtype=torch.uint8, device="cuda")
        (mp.kv_attention_paged_fp8_cache if fp8 else mp.kv_attention_paged)(q, iro, case.scale, cache, 1, out, ws, lse=z)
        case.lens, case.new, case.T, case.q = np.asarray(lens), np.asarray(move), T, q
        check_kv_attention(case, out, z)
        # the written rows: rotated keys, in the cache's type
        ref, mag = rotated(x[:, H:H + KH].double(), tab64[torch.from_numpy(pos).cuda()], D, half)
        got = torch.cat([case.rows64(b, 0, range(n, n + m)) for b, (n, m) in enumerate(zip(lens, move)) if m])
        step = ref.abs().amax() / 448 * 2.0 ** -10 if fp8 else 0.0
        assert bool(((got - ref).abs() <= mag * 3 * U32 + ref.abs() * (2.0 ** -4 if fp8 else HALF_BF16) * 1.001 + step).all())
        lens = [n + m for n, m in zip(lens, move)]
        case.dev.cache_lengths.copy_(i32(lens, "cuda"))
    M = sum(lens)
    kb, vb = (torch.empty((M, KH, D), dtype=BF16, device="cuda") for _ in range(2))
    (mp.kv_gather_paged_fp8_cache if fp8 else mp.kv_gather_paged)(i32([0, lens[0], M], "cuda"), i32([0, 0], "cuda"), M,
                                                                 cache, 1, kb, vb)
    for side, got in ((0, kb), (1, vb)):
        want = torch.cat([case.rows64(b, side, range(n)) for b, n in enumerate(lens)])
        assert same(got, want.float().to(BF16))


def test_projected_rows_are_attended():
    # kv_matmul_paged writes the rows that the attention reads
    case = KvCase(41, [40, 0], [3, 150], 8, 2, 128)
    g = torch.Generator(device="cuda").manual_seed(41)
    h = torch.randn((case.T, 256), generator=g, device="cuda").to(BF16)
    w = (torch.randn((256, 512), generator=g, device="cuda") / 16).to(BF16)
    mp.kv_matmul_paged(h, case.iro, w, cache_of(case), 1)
    check_kv_attention(case, *attend(case))
    y = (h.double() @ w.double()).view(case.T, 2, 2, 128)
    mag = (h.double().abs() @ w.double().abs()).view(y.shape)[:, 1]
    got = torch.cat([case.rows64(b, 1, range(n, n + m)) for b, (n, m) in enumerate(zip([40, 0], [3, 150]))])
    assert bool(((got - y[:, 1]).abs() <= y[:, 1].abs() * HALF_BF16 * 1.01 + mag * 256 * U32).all())
