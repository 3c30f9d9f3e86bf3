"""The drafted step's calls at the ends of their documented ranges."""
import math

import numpy as np
import pytest
import torch

import mla_paged_latent_page_amd as mp
import workloads as W
from gpu_util import check_guards, guarded_empty
from plain_step import HALF_BF16, U32, AttentionCase, check_attention, i32
from test_gpu_step_ops import attend, cache_of, raw_of, same

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# values that are not finite in a row that is seen
# ---------------------------------------------------------------------------
def row_at(case, b, p):
    """Cache row at position p of request b, and its scales."""
    ps = case.host.page_size
    page, slot = int(case.host.page_table[b, p // ps]), p % ps
    return case.dev.pool[page, case.layer, 0, slot, 0], (case.dev.scales[page, case.layer, 0, slot]
                                                         if case.host.dtype == "e4m3" else None)


def without(case, drop):
    """float64 outputs, log-sum-exps and their bounds (those of AttentionCase.reference) where no
    token sees position drop[b] of request b; and which tokens saw it."""
    out = torch.zeros((case.T, case.H, case.K), dtype=torch.float64, device="cuda")
    lse, tol, ltol = torch.zeros_like(out[..., 0]), torch.zeros_like(out), torch.zeros_like(out[..., 0])
    saw, at = torch.zeros(case.T, dtype=torch.bool, device="cuda"), 0
    for b, n in enumerate(case.new.tolist()):
        rows, cached = case.rows64(b), int(case.lens[b])
        for i in range(n):
            p = list(range(cached)) + [cached + j for j in range(n) if (case.seen[b][i] >> j) & 1]
            saw[at + i] = drop[b] in p
            r = rows[[x for x in p if x != drop[b]]]
            q = case.q[at + i].double()
            s = (q @ r.t().contiguous()) * case.scale
            ds = ((q.abs() @ r.abs().t().contiguous()) * case.scale).amax(dim=1) * (case.D + 8) * U32
            z = torch.logsumexp(s, dim=1)
            w = torch.exp(s - z[:, None])
            o, mag = w @ r[:, :case.K], w @ r[:, :case.K].abs()
            rel = 2 * ds + 2.0 ** -20 + 3 * r.shape[0] * U32 + (0.0 if case.host.dtype == "f32" else HALF_BF16)
            out[at + i], lse[at + i] = o, z
            tol[at + i] = mag * rel[:, None] + o.abs() * (2 * U32 if case.host.dtype == "f32" else HALF_BF16) * 1.02 + 1e-30
            ltol[at + i] = ds + 2.0 ** -20 + 3 * r.shape[0] * U32 + z.abs() * 2 * U32
        at += n
    return out, lse, tol, ltol, saw


INFINITE = [
    # lens, new, heads, page_size, mask
    ([70, 33], [3, 4], 16, 16, "chain"),       # narrow items
    ([70, 33], [3, 4], 16, 5, "tree"),
    ([150, 40], [2, 1], 100, 16, "tree"),      # two workgroups side by side
    ([70, 9], [9, 40], 16, 16, "tree"),        # wide
    ([33, 300], [20, 5], 64, 12, "chain"),
    ([9000, 5000], [2, 3], 16, 64, "tree"),    # split items
    ([4000, 64], [9, 40], 16, 128, "tree"),
]


@pytest.mark.parametrize("where", ["drafted", "cached"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("lens, new, heads, page_size, mask", INFINITE)
def test_an_infinity_in_a_row_that_is_seen(lens, new, heads, page_size, mask, dtype, where):
    """Score + infinity or NaN: the output is NaN.  Score - infinity: the weight is 0, and 0 times
    infinity is NaN in the columns the infinity is in (e4m3: those of the block whose scale it is)
    and there alone.  Other tokens do not notice."""
    case = AttentionCase(sum(lens) + heads, lens, new, heads, page_size=page_size, mask=mask, dtype=dtype)
    # the row of the first drafted token (seen by it and its descendants), or of a cached one
    drop = [l if where == "drafted" else l // 2 for l in lens]
    out, lse, tol, ltol, saw = without(case, drop)
    bad = torch.zeros(case.K, dtype=torch.bool, device="cuda")
    if dtype == "e4m3":
        # All products of block 2 have one sign: positive codes there, and queries of one sign per head.
        block = slice(256, 384)
        sign = torch.where(torch.arange(heads, device="cuda") % 2 == 0, 1.0, -1.0).to(case.q.dtype)
        case.q[:, :, block] = (case.q[:, :, block].abs() + 0.01) * sign[:, None]
        out, lse, tol, ltol, saw = without(case, drop)
        bad[block] = True
        up = (sign > 0).expand(case.T, heads)
        for b in range(2):
            row, sc = row_at(case, b, drop[b])
            row[block] = 0x38          # 1.0
            sc[2] = math.inf
    else:
        column = 77
        bad[column] = True
        up = case.q[:, :, column] > 0
        assert bool((case.q[:, :, column] != 0).all())
        for b in range(2):
            row_at(case, b, drop[b])[0][column] = math.inf
    got, z = attend(case)
    live = int(case.new.sum())
    got, z, up = got[:live].double(), z[:live].double(), up[:live]
    finite = ~(saw[:, None] & up)
    assert bool((saw[:, None] & up).any()) and bool((saw[:, None] & ~up).any())
    assert bool(torch.isnan(got[~finite]).all()) and bool(torch.isnan(z[~finite]).all())
    nan = (saw[:, None] & ~up)[:, :, None] & bad
    assert bool(torch.isnan(got[nan]).all()), "a weight of 0 times infinity is NaN"
    ok = finite[:, :, None] & ~nan
    assert bool(((got - out).abs()[ok] <= tol[ok]).all())
    assert bool(((z - lse).abs()[finite] <= ltol[finite]).all())


@pytest.mark.parametrize("heads, new", [(16, [2, 3]), (128, [1, 2]), (16, [9, 20])])
def test_an_infinity_in_rope_columns_has_no_column_of_the_output(heads, new):
    case = AttentionCase(heads, [100, 31], new, heads, mask="chain")
    case.seen = [[(1 << (i + 1)) - 1 for i in range(n)] for n in new]
    drop = [100, 31]
    out, lse, tol, ltol, saw = without(case, drop)
    for b in range(2):
        row_at(case, b, drop[b])[0][520] = math.inf
    got, z = attend(case)
    finite = case.q[:, :, 520] < 0
    assert bool(saw.all()) and bool(torch.isnan(got[~finite]).all())
    assert bool(((got.double() - out).abs()[finite] <= tol[finite]).all())
    assert bool(((z.double() - lse).abs()[finite] <= ltol[finite]).all())


# ---------------------------------------------------------------------------
# offsets out of order
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("heads", [16, 128])
def test_offsets_that_decrease_stay_inside_the_outputs(heads, dtype):
    case = AttentionCase(heads, [70, 33, 5, 90], [3, 4, 1, 2], heads, mask="tree", dtype=dtype)
    good = case.iro
    for offsets in ([0, 7, 3, 8, 10], [4, 0, 10, 2, 9], [0, 10, 0, 10, 10], [0, 0xFFFFFFFF, 1, 2, 3], [9, 8, 7, 6, 5]):
        case.iro = i32(offsets, "cuda")
        attend(case)           # (the guards beside outputs and workspace)
    case.iro = good
    check_attention(case, *attend(case))


def test_offsets_that_name_every_token_in_every_second_request():
    # as many units of work as pass 2^32 when each request is believed
    T, heads, requests, ps = 2000, 128, 2000, 128
    case = AttentionCase(1, [1], [1], heads, page_size=ps)
    q = torch.zeros((T, heads, 576), dtype=torch.bfloat16, device="cuda")
    out = guarded_empty((T, heads, 512), torch.bfloat16)
    lse = guarded_empty((T, heads), torch.float32)
    ws = guarded_empty((mp.mla_tree_attention_workspace_size(T, heads, 512),), torch.uint8)
    table = torch.zeros((requests, 1024), dtype=torch.int32, device="cuda")
    lengths = torch.full((requests,), 1024 * ps - 5, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, T] * (requests // 2) + [T], dtype=torch.int32, device="cuda")
    mp.mla_tree_attention_paged(q, offsets, None, 0.1, 512, mp.PagedKVCache(case.dev.pool, table, lengths), 1, out, ws,
                                lse=lse)
    check_guards("tree attention")


# ---------------------------------------------------------------------------
# more work-items than one launch holds (2^32 in a dimension)
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype, T, H", [("bf16", (1 << 20) + 3, 16), ("bf16", 3, (1 << 24) // 3 + 9), ("e4m3", 1 << 22, 5)])
def test_attention_of_more_than_2_24_pairs(dtype, T, H):
    # rows of 16 columns; the table holds one page of 8 positions
    D, K, ps = 16, 8, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((T, H, D), generator=g, device="cuda").to(torch.bfloat16)
    if dtype == "e4m3":
        pool = torch.randn((2, 1, 1, ps, 1, D), generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        scales = torch.rand((2, 1, 1, ps, 1), generator=g, device="cuda") + 0.5
        rows = pool[1, 0, 0, :, 0].view(torch.float8_e4m3fn).float() * scales[1, 0, 0]
    else:
        pool, scales = torch.randn((2, 1, 1, ps, 1, D), generator=g, device="cuda").to(torch.bfloat16), None
        rows = pool[1, 0, 0, :, 0].float()
    cache = mp.PagedKVCache(pool, i32([[1]], "cuda"), i32([6], "cuda"), scales=scales)
    out = torch.full((T, H, K), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    ws = torch.empty(mp.mla_tree_attention_workspace_size(T, H, K), dtype=torch.uint8, device="cuda")
    call = mp.mla_tree_attention_paged if scales is None else mp.mla_tree_attention_paged_fp8_cache
    call(q, i32([0, T], "cuda"), None, 0.25, K, cache, 0, out, ws, lse=lse)
    pick = torch.unique(torch.cat([torch.randint(0, T * H, (4000,), generator=g, device="cuda"),
                                   torch.arange(T * H - 500, T * H, device="cuda"), torch.arange(500, device="cuda"),
                                   torch.arange((1 << 23) - 50, (1 << 23) + 50, device="cuda"),
                                   torch.arange((1 << 24) - 50, (1 << 24) + 50, device="cuda")]))
    pick = pick[pick < T * H]
    x = q.view(-1, D)[pick].double()
    r = rows.double()
    s = x @ r.t().contiguous() * 0.25
    last = 6 + (pick // H).clamp(max=1)             # the newest position that the token sees
    s = torch.where(torch.arange(ps, device="cuda")[None] <= last[:, None], s, -math.inf)
    ref = torch.softmax(s, 1) @ r[:, :K]
    mag = torch.softmax(s, 1) @ r[:, :K].abs()
    ds = ((x.abs() @ r.abs().t().contiguous()) * 0.25).amax(1) * (D + 8) * U32
    tol = mag * (2 * ds + 2.0 ** -20 + 3 * ps * U32)[:, None] + ref.abs() * HALF_BF16 * 1.02 + 1e-30
    assert bool(((out.view(-1, K)[pick].double() - ref).abs() <= tol).all())
    z = torch.logsumexp(s, 1)
    assert bool(((lse.view(-1)[pick].double() - z).abs() <= ds + 2.0 ** -20 + 3 * ps * U32 + z.abs() * 2 * U32).all())


@pytest.mark.parametrize("T, H, half", [((1 << 24) + 5, 1, False), (1, (1 << 22) + 70, True), (2, (1 << 22) + 70, False)])
def test_rope_q_of_more_than_one_grid(T, H, half):
    g = torch.Generator(device="cuda").manual_seed(2)
    R = 16
    q = torch.randn((T, H, 8 + R), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.from_numpy(W.rope_table(500, R)).cuda()
    pos = torch.randint(0, 500, (T,), generator=g, device="cuda").to(torch.int32)
    out = torch.full_like(q, 7.0)
    mp.mla_rope_q(q, pos, table, out, d_nope=8, layout="half" if half else "interleaved")
    assert same(out[..., :8], q[..., :8])
    for lo in range(0, T * H, 1 << 22):
        x = q.view(-1, 8 + R)[lo:lo + (1 << 22), 8:].double()
        tab = table.double()[pos[torch.arange(lo, lo + x.shape[0], device="cuda") // H].long()]
        c, s = tab[:, 0::2], tab[:, 1::2]
        x0, x1 = x.chunk(2, 1) if half else (x[:, 0::2], x[:, 1::2])
        y0, y1 = x0 * c - x1 * s, x0 * s + x1 * c
        m0, m1 = (x0 * c).abs() + (x1 * s).abs(), (x0 * s).abs() + (x1 * c).abs()
        y = out.view(-1, 8 + R)[lo:lo + (1 << 22), 8:].double()
        g0, g1 = y.chunk(2, 1) if half else (y[:, 0::2], y[:, 1::2])
        for got, ref, mag in ((g0, y0, m0), (g1, y1, m1)):
            assert bool(((got - ref).abs() <= mag * 2 * U32 + ref.abs() * HALF_BF16 * 1.01).all())


# ---------------------------------------------------------------------------
# positions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_latent_writes_past_position_2_32_store_nothing(dtype, half):
    case = W.latent_write_case("far", seed=3, seq_lens=[6, 3], start_lengths=[0, 20], page_size=16, K=512, R=64,
                               dtype=dtype, max_seq_len=100)
    dc, t = W.device_latent_write(case)
    dc.cache_lengths.copy_(i32([2 ** 32 - 2, 2 ** 32 - 1], "cuda"))
    before, scales = raw_of(dc.pool).clone(), None if dc.scales is None else dc.scales.clone()
    args = (t["gamma"], case.eps, t["freqs"], 512, cache_of(dc), 1)
    layout = "half" if half else "interleaved"
    if dtype == "e4m3":
        mp.mla_write_latent_paged_fp8_at(t["x"], t["input_row_offsets"], i32(np.arange(9), "cuda"), *args, layout=layout)
        mp.mla_write_latent_paged_fp8(t["x"], t["input_row_offsets"], *args)
    else:
        mp.mla_write_latent_paged_at(t["x"], t["input_row_offsets"], i32(np.arange(9), "cuda"), *args, layout=layout)
        mp.mla_write_latent_paged(t["x"], t["input_row_offsets"], *args)
    assert same(raw_of(dc.pool), before)
    assert scales is None or same(dc.scales.view(torch.int32), scales.view(torch.int32))


@pytest.mark.parametrize("heads", [1, 2])
def test_kv_products_past_position_2_32_store_nothing(heads):
    case = W.kv_matmul_case("far", seed=1, seq_lens=[6, 300], start_lengths=[0, 20], hidden_dim=256, num_kv_heads=heads,
                            head_dim=128, page_size=16)
    dc, t = W.device_kv(case)
    dc.cache_lengths.copy_(i32([2 ** 32 - 2, 2 ** 32 - 299], "cuda"))
    before = raw_of(dc.pool).clone()
    mp.kv_matmul_paged(t["hidden"], t["input_row_offsets"], t["weight"], cache_of(dc), case.layer_idx)
    assert same(raw_of(dc.pool), before)


@pytest.mark.parametrize("at", [False, True])
def test_latent_writes_of_more_than_2_27_tokens(at):
    # rows of 8 columns; all but the first 16 tokens of the first request lie past its page table
    T = (1 << 27) + 9
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros((T, 8), dtype=torch.bfloat16, device="cuda")
    x[:16] = torch.randn((16, 8), generator=g, device="cuda").to(torch.bfloat16)
    x[-5:] = torch.randn((5, 8), generator=g, device="cuda").to(torch.bfloat16)
    pool = torch.zeros((4, 1, 1, 16, 1, 8), dtype=torch.bfloat16, device="cuda")
    cache = mp.PagedKVCache(pool, i32([[2], [1]], "cuda"), i32([0, 3], "cuda"))
    gamma = torch.rand(8, generator=g, device="cuda") + 0.5
    offsets = i32([0, T - 5, T], "cuda")
    if at:
        pos = torch.zeros(T, dtype=torch.int32, device="cuda")
        mp.mla_write_latent_paged_at(x, offsets, pos, gamma, 1e-6, None, 8, cache, 0)
    else:
        mp.mla_write_latent_paged(x, offsets, gamma, 1e-6, None, 8, cache, 0)
    want = torch.zeros((4, 16, 8), dtype=torch.float64, device="cuda")
    for page, slots, rows in ((2, slice(0, 16), x[:16]), (1, slice(3, 8), x[-5:])):
        r = rows.double()
        want[page, slots] = gamma.double() * r / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-6)
    got = pool[:, 0, 0, :, 0].double()
    # binary32: the sum of 8 squares, a root and a division, three products; then one rounding
    assert bool(((got - want).abs() <= want.abs() * (16 * U32 + HALF_BF16 * 1.001)).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_compaction_past_position_2_32(dtype):
    # a length close to 2^32 in a table that reaches past it
    ps, pages, D = 1 << 20, 3, 16
    raw = torch.randint(0, 256, (pages, 1, 1, ps, 1, D * (1 if dtype == "e4m3" else 2)), dtype=torch.uint8, device="cuda")
    pool = raw if dtype == "e4m3" else raw.view(torch.bfloat16)
    scales = torch.rand((pages, 1, 1, ps, 1), device="cuda") if dtype == "e4m3" else None
    table = torch.full((1, 4098), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, 4095], table[0, 4096] = 0, 1, 2
    cache = mp.PagedKVCache(pool, table, i32([2 ** 32 - 5], "cuda"), scales=scales)
    accepted = [2, 9, 0xFFFFFFFF]       # positions 2^32 - 3, 2^32 + 4 and one past the table
    tensors = [raw_of(pool)] + ([] if scales is None else [scales])
    want = [t.clone() for t in tensors]
    for w, t in zip(want, tensors):
        w[1, 0, 0, ps - 5], w[1, 0, 0, ps - 4] = t[1, 0, 0, ps - 3], t[2, 0, 0, 4]
    mp.mla_compact_paged(i32(accepted, "cuda"), i32([0, 3], "cuda"), cache)
    assert all(same(w, t) for w, t in zip(want, tensors))


# ---------------------------------------------------------------------------
# scales and scores at the ends of binary32
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("scale", [3e38, -3e38])
def test_a_scale_close_to_the_largest_number(scale, heads, dtype):
    # queries of zero: every score is 0, the output the mean
    case = AttentionCase(9, [200, 33], [2, 3], heads, mask="tree", dtype=dtype)
    case.q.zero_()
    case.scale = scale
    check_attention(case, *attend(case))


@pytest.mark.parametrize("length", ["capacity", "two less", "2^32 - 1", "2^31"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("heads, mask", [(16, "chain"), (16, "tree"), (64, "tree"), (128, "chain")])
def test_attention_sees_the_positions_of_the_page_table(heads, mask, dtype, length):
    """Request 0's length at and past what its table's row holds: the answer is that of the
    positions below it alone."""
    capacity, n = 112, 4
    case = AttentionCase(heads, [capacity - n, 30], [n, 2], heads, mask=mask, dtype=dtype, page_size=16)
    assert case.dev.page_table.shape[1] * 16 == capacity
    cached = {"capacity": capacity, "two less": capacity - 2, "2^32 - 1": capacity, "2^31": capacity}[length]
    word = {"capacity": capacity, "two less": capacity - 2, "2^32 - 1": 2 ** 32 - 1, "2^31": 2 ** 31}[length]
    case.dev.cache_lengths.copy_(i32([word, 30], "cuda"))
    got, z = attend(case)
    # the reference: a request of `cached` rows whose drafted rows past the capacity nobody sees
    rows = case.rows64(0)          # all positions below the capacity
    kept = capacity - cached
    case.lens = np.array([cached, 30])
    case.seen[0] = [m & ((1 << kept) - 1) for m in case.seen[0]]
    pad = torch.cat([rows, torch.zeros((cached + n - capacity, case.D), dtype=torch.float64, device="cuda")])
    second = case.rows64(1)
    case.rows64 = lambda b: second if b else pad
    check_attention(case, got, z)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("heads", [5, 24, 128])
def test_outputs_at_large_scores(heads, dtype):
    """Scores of several hundred: the bound of AttentionCase.reference with the weights' factor
    exp(2 ds) written out (there it is taken to first order), nothing looser."""
    case = AttentionCase(78 + heads, [700, 64], [5, 6], heads, mask="tree", q_std=40.0, dtype=dtype)
    got, z = attend(case)
    ref, zref, tol, ltol = case.reference()
    at, extra = 0, torch.zeros_like(tol)
    for b, n in enumerate(case.new.tolist()):
        rows = case.rows64(b)
        for i in range(n):
            keep = [p for p in range(rows.shape[0]) if p < case.lens[b] or (case.seen[b][i] >> (p - int(case.lens[b]))) & 1]
            r, q = rows[keep], case.q[at + i].double()
            ds = ((q.abs() @ r.abs().t().contiguous()) * case.scale).amax(dim=1) * (case.D + 8) * U32
            w = torch.softmax((q @ r.t().contiguous()) * case.scale, dim=1)
            extra[at + i] = (w @ r[:, :case.K].abs()) * (torch.expm1(2 * ds) - 2 * ds)[:, None]
        at += n
    assert bool(((got.double() - ref).abs() <= tol + extra).all())
    assert bool(((z.double() - zref).abs() <= ltol).all())


# ---------------------------------------------------------------------------
# a step captured and replayed
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_step_of_all_calls_captured_and_replayed(dtype):
    """Free, fork, copy, rotate, write, attend and compact in one graph, replayed over changed inputs,
    with eager calls between; every buffer as the eager calls leave it."""
    H, ps, lens, new = 16, 16, [45, 130, 45, 0], [3, 5, 2, 0]
    base = AttentionCase(31, lens[:3], new[:3], H, page_size=ps, mask="tree", dtype=dtype)
    used = set(base.host.page_table.flatten().tolist())
    spare = [p for p in range(base.host.num_pages) if p not in used]
    assert len(spare) >= 2
    table = np.full((4, base.host.page_table.shape[1]), 0xFFFFFFFF, np.int64)
    table[:3] = base.host.page_table
    refs = np.zeros(base.host.num_pages, np.int64)
    for b in range(3):
        refs[table[b, :-(-(lens[b] + new[b]) // ps)]] += 1
    T = base.T
    g = torch.Generator(device="cuda").manual_seed(4)
    d = dict(pool=base.dev.pool.clone(), table=i32(table, "cuda"), lengths=i32(lens, "cuda"), refs=i32(refs, "cuda"),
             list=torch.full((base.host.num_pages,), -1, dtype=torch.int32, device="cuda"), count=i32([0], "cuda"),
             q=torch.zeros((T, H, 192), dtype=torch.bfloat16, device="cuda"),
             out=torch.zeros((T, H, 512), dtype=torch.bfloat16, device="cuda"), lse=torch.zeros((T, H), device="cuda"),
             freqs=torch.zeros((200, 64), device="cuda"))
    if base.dev.scales is not None:
        d["scales"] = base.dev.scales.clone()
    cache = mp.PagedKVCache(d["pool"], d["table"], d["lengths"], scales=d.get("scales"))
    iro = i32([0, 3, 8, 10, 10], "cuda")
    pos = i32([45, 46, 46, 130, 131, 132, 131, 133, 45, 46], "cuda")
    qin = torch.zeros_like(d["q"])
    x = torch.zeros((T, 576), dtype=torch.bfloat16, device="cuda")
    gamma = torch.rand(512, generator=g, device="cuda") + 0.5
    ws = torch.empty(mp.mla_tree_attention_workspace_size(T, H, 512), dtype=torch.uint8, device="cuda")
    ids = {k: i32(v, "cuda") for k, v in dict(gone=[3], parent=[0], child=[3], fresh=[spare[0]], src=[int(table[1, 0])],
                                             dst=[spare[1]], accepted=[0, 2, 1, 4], offsets=[0, 2, 4, 4, 4]).items()}

    def step():
        d["count"].zero_()
        mp.mla_free_paged(ids["gone"], d["refs"], d["list"], d["count"], cache)
        mp.mla_fork_paged(ids["parent"], ids["child"], ids["fresh"], d["refs"], cache)
        mp.mla_copy_pages(ids["src"], ids["dst"], cache)
        mp.mla_rope_freqs(d["freqs"], scaling="linear", factor=2.0)
        mp.mla_rope_q(qin, pos, d["freqs"], d["q"], layout="half")
        write = mp.mla_write_latent_paged_fp8_at if dtype == "e4m3" else mp.mla_write_latent_paged_at
        write(x, iro, pos, gamma, 1e-6, d["freqs"], 512, cache, 1, layout="half")
        call = mp.mla_tree_attention_paged_fp8_cache if dtype == "e4m3" else mp.mla_tree_attention_paged
        call(base.q, iro, base.mask, base.scale, 512, cache, 1, d["out"], ws, lse=d["lse"])
        mp.mla_compact_paged(ids["accepted"], ids["offsets"], cache)

    def fill(seed):
        g.manual_seed(seed)
        qin.copy_(torch.randn(qin.shape, generator=g, device="cuda"))
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))

    def state():
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in d.items()}

    def put(s):
        for k, v in s.items():
            d[k].copy_(v)
        torch.cuda.synchronize()
    start = state()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    put(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        fill(seed)
        before = state()
        graph.replay()
        got = state()
        put(before)
        step()
        want = state()
        for k in want:
            assert same(got[k].view(torch.uint8), want[k].view(torch.uint8)), (seed, k)
        assert bool(torch.isfinite(want["out"].float()).all()) and int(want["lengths"][3]) == 45
