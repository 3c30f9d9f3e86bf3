"""The paged K/V cache's operators at the edges of what they accept: rows behind the last request, values near the
largest that the sums hold."""
import math

import numpy as np
import pytest
import torch

import mla_paged_latent_page_amd as mp
import workloads as W
from plain_kv import KvCase, check_kv_attention
from plain_step import i32
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
