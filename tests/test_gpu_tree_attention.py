"""Tree attention on the matrix cores at the edges of its work split: items of 64 and of 128
query rows, shares that begin and end inside a request, more requests than a wave has lanes."""
import math

import numpy as np
import pytest
import torch

import mla_paged_latent_page_amd as mp
from plain_step import AttentionCase, check_attention, mask_tensor
from test_gpu_step_ops import attend, cache_of, same

pytestmark = pytest.mark.gpu

# An average of at most 64 query rows per request takes the narrow items.
NARROW = [
    # lens, new, heads, page_size, mask
    ([9000, 3, 77], [1, 2, 4], 16, 100, "tree"),
    ([0, 1, 2, 31, 33, 64], [1] * 6, 5, 3, "chain"),
    ([40000], [3], 20, 128, "tree"),
    ([70, 0, 500], [4, 0, 4], 16, 7, "holes"),
    ([300, 65], [4, 4], 16, 64, "tree"),            # 64 rows
    ([1000, 20, 20, 20], [12, 1, 1, 1], 16, 16, "chain"),   # three items of one request
    ([2049, 4095], [1, 2], 33, 8, "tree"),
]
# At most 128: two workgroups side by side.
TWINS = [
    ([30000], [1], 128, 16, "chain"),
    ([0, 0], [2, 1], 64, 5, "chain"),
    ([300], [5], 13, 64, "tree"),                   # 65 rows
    ([2000, 10, 700], [12, 1, 5], 16, 16, "tree"),  # 192, 16 and 80 rows
    ([5000, 0, 63], [8, 0, 8], 16, 100, "holes"),
    ([12345, 1], [3, 1], 64, 128, "tree"),
]
WIDE = [
    ([9000, 3], [8, 20], 16, 100, "tree"),
    ([64, 64], [10, 9], 16, 40, "holes"),
    ([500], [600], 16, 128, "chain"),
    ([20000, 7], [9, 1], 64, 16, "tree"),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens, new, heads, page_size, mask", NARROW + TWINS + WIDE)
def test_shares(lens, new, heads, page_size, mask, dtype):
    case = AttentionCase(heads + lens[0], lens, new, heads, page_size=page_size, mask=mask, dtype=dtype)
    check_attention(case, *attend(case))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [16, 100, 220])
def test_more_requests_than_lanes(heads, dtype):
    rng = np.random.default_rng(heads)
    lens, new = rng.integers(0, 300, 150), rng.choice([0, 1, 1, 2], 150)
    lens[149], new[149] = 1500, 3
    case = AttentionCase(3, lens, new, heads, page_size=16, mask="tree", dtype=dtype)
    check_attention(case, *attend(case))


@pytest.mark.parametrize("heads", [16, 128])
def test_one_request_behind_many_empty_ones(heads):
    lens, new = np.zeros(300, np.int64), np.zeros(300, np.int64)
    lens[299], new[299] = 700, 2
    case = AttentionCase(4, lens, new, heads, page_size=16, mask="chain")
    check_attention(case, *attend(case))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_narrow_items_and_rows_a_token_does_not_see(dtype):
    # The last drafted row of either request holds NaN and infinities; only its own token sees it.
    lens, new = [70, 10], [3, 4]
    case = AttentionCase(5, lens, new, 16, mask="chain", dtype=dtype)
    case.seen = [[(1 << (i + 1)) - 1 for i in range(n)] for n in new]
    case.mask = mask_tensor([m for r in case.seen for m in r], 1, "cuda")
    for b in (0, 1):
        p = lens[b] + new[b] - 1
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
    seers = torch.tensor([2, 6], device="cuda")
    assert bool(torch.isnan(out[seers]).all()) and bool(torch.isnan(z[seers]).all())
    keep = torch.ones(7, dtype=torch.bool, device="cuda")
    keep[seers] = False
    for b in (0, 1):     # as if those rows were never there
        p = lens[b] + new[b] - 1
        page, slot = int(case.host.page_table[b, p // 16]), p % 16
        case.dev.pool[page, 1, 0, slot, 0] = 0
        if dtype == "e4m3":
            case.dev.scales[page, 1, 0, slot] = 1.0
    ref, zref, tol, ltol = case.reference()
    assert bool(((out.double() - ref).abs()[keep] <= tol[keep]).all())
    assert bool(((z.double() - zref).abs()[keep] <= ltol[keep]).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("heads", [16, 128])
def test_a_negative_scale_is_negated_queries(heads, dtype):
    case = AttentionCase(6, [200, 33], [2, 3], heads, mask="tree", dtype=dtype)
    case.q = -case.q
    ref, zref = attend(case)
    case.q, case.scale = -case.q, -case.scale
    out, z = attend(case)
    assert same(out, ref) and same(z, zref)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_a_scale_of_zero_is_a_mean(dtype):
    case = AttentionCase(7, [200, 33], [2, 3], 16, mask="tree", dtype=dtype)
    case.scale = 0.0
    check_attention(case, *attend(case))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads, page_size", [(16, 16), (128, 16), (16, 5), (128, 5)])
def test_rows_apart_in_the_pool(heads, page_size, dtype):
    case = AttentionCase(8, [400, 31], [2, 1], heads, page_size=page_size, mask="tree", dtype=dtype)
    ref, zref = attend(case)
    pool = case.dev.pool
    apart = torch.full((*pool.shape[:4], 3, 576), 0x7F if dtype == "e4m3" else math.nan, dtype=pool.dtype, device="cuda")
    apart[..., 1:2, :] = pool
    out, z = torch.empty_like(ref), torch.empty_like(zref)
    ws = torch.empty(mp.mla_tree_attention_workspace_size(case.T, heads, 512), dtype=torch.uint8, device="cuda")
    call = mp.mla_tree_attention_paged_fp8_cache if dtype == "e4m3" else mp.mla_tree_attention_paged
    call(case.q, case.iro, case.mask, case.scale, 512,
         mp.PagedKVCache(apart[..., 1:2, :], case.dev.page_table, case.dev.cache_lengths, scales=case.dev.scales), 1, out,
         ws, lse=z)
    assert same(out, ref) and same(z, zref)


def test_two_graphs_at_once():
    cases = [AttentionCase(20, [5000, 80], [3, 2], 16, mask="tree", page_size=64),
             AttentionCase(21, [1200, 3000, 9], [9, 1, 20], 128, mask="tree", page_size=64, dtype="e4m3")]
    runs = []
    for case in cases:
        out = torch.empty((case.T, case.H, 512), dtype=torch.bfloat16, device="cuda")
        z = torch.empty((case.T, case.H), device="cuda")
        ws = torch.empty(mp.mla_tree_attention_workspace_size(case.T, case.H, 512), dtype=torch.uint8, device="cuda")
        call = mp.mla_tree_attention_paged_fp8_cache if case.host.dtype == "e4m3" else mp.mla_tree_attention_paged

        def run(case=case, out=out, z=z, ws=ws, call=call):
            call(case.q, case.iro, case.mask, case.scale, 512, cache_of(case), 1, out, ws, lse=z)
        ref = attend(case)
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        runs.append((graph, torch.cuda.Stream(), out, z, ref, run))   # (run holds the graph's workspace)
    for _ in range(5):
        for graph, stream, out, *_ in runs:
            out.zero_()
            stream.wait_stream(torch.cuda.current_stream())
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, out, z, ref, _ in runs:
            assert same(out, ref[0]) and same(z, ref[1])


@pytest.mark.parametrize("heads, page_size", [(16, 64), (128, 64), (128, 60)])
def test_far_pages_of_an_e4m3_cache(heads, page_size):
    # page offsets past 2^32 bytes, and past 2^27 floats in the scales
    pages = 130000
    case = AttentionCase(30, [150], [2], heads, page_size=page_size, dtype="e4m3")
    out, z = attend(case)
    pool = torch.zeros((pages, 1, 1, page_size, 1, 576), dtype=torch.uint8, device="cuda")
    scales = torch.ones((pages, 1, 1, page_size, 5), device="cuda")
    far = [pages - 1, 3, pages - 4000]
    for i, f in enumerate(far):
        page = int(case.host.page_table[0, i])
        pool[f, 0] = case.dev.pool[page, 1]
        scales[f, 0] = case.dev.scales[page, 1]
    table = torch.tensor([far], dtype=torch.int32, device="cuda")
    got, gz = torch.empty_like(out), torch.empty_like(z)
    ws = torch.empty(mp.mla_tree_attention_workspace_size(2, heads, 512), dtype=torch.uint8, device="cuda")
    mp.mla_tree_attention_paged_fp8_cache(case.q, case.iro, None, case.scale, 512,
                                          mp.PagedKVCache(pool, table, case.dev.cache_lengths, scales=scales), 0, got,
                                          ws, lse=gz)
    assert same(out, got) and same(z, gz)


def test_far_pages_of_the_page_calls():
    # 8 GiB of pages: copies, forks and compaction across offsets past 2^32 bytes
    ps, pages, layers = 64, 29200, 4
    pool = torch.zeros((pages, layers, 1, ps, 1, 576), dtype=torch.bfloat16, device="cuda")
    far = pages - 1
    g = torch.Generator(device="cuda").manual_seed(1)
    pool[far] = torch.randn((layers, 1, ps, 1, 576), generator=g, device="cuda").to(torch.bfloat16)
    want = pool[far].clone()
    table = torch.tensor([[far], [-1]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([40, 0], dtype=torch.int32, device="cuda")
    cache = mp.PagedKVCache(pool, table, lengths)

    def ids(*a):
        return torch.tensor(a, dtype=torch.int32, device="cuda")
    mp.mla_copy_pages(ids(far), ids(0), cache)
    assert same(pool[0], want)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[far] = 1
    mp.mla_fork_paged(ids(0), ids(1), ids(far - 1), refs, cache)
    assert same(pool[far - 1][:, :, :40], want[:, :, :40]) and bool((pool[far - 1][:, :, 40:] == 0).all())
    mp.mla_compact_paged(ids(3, 9), ids(0, 2, 2), cache)
    want[:, :, 40], want[:, :, 41] = want[:, :, 43].clone(), want[:, :, 49].clone()
    assert same(pool[far], want)
    assert not bool(pool[1:far - 1].view(torch.int16).any())
