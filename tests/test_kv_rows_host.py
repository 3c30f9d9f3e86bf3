"""The checks of tests/kv_rows.py see one row lost, doubled or taken for another: mistakes planted in a plain
form, on the CPU."""
import math

import pytest
import torch

from kv_rows import Rows, check_each_row, check_whole_numbers, whole_numbers
from plain_kv import KvCase


def plain(case, hide=(), twice=(), swap=None):
    """out, lse in the operator's types; rows of the last request that are hidden, doubled, or taken for others."""
    G = case.H // case.KH
    out = torch.zeros((case.T, case.H, case.D), dtype=torch.float64)
    lse = torch.zeros((case.T, case.H), dtype=torch.float64)
    at = 0
    for b, (n, m) in enumerate(zip(case.lens.tolist(), case.new.tolist())):
        if not m:
            continue
        K, V, see = case.rows64(b, 0, range(n + m)), case.rows64(b, 1, range(n + m)), case.seen(b).double()
        if b == len(case.lens) - 1:
            see[:, list(hide)] = 0.0
            see[:, list(twice)] *= 2.0
            if swap:
                V[swap[0]] = V[swap[1]]
        for h in range(case.H):
            s = torch.exp(case.q[at:at + m, h].double() @ K[:, h // G].T * case.scale) * see
            out[at:at + m, h] = s @ V[:, h // G] / s.sum(1, keepdim=True)
            lse[at:at + m, h] = torch.log(s.sum(1))
        at += m
    return out.to(case.q.dtype), lse.float()


def case_of(lens, new, H, KH, D, dtype, **kw):
    return KvCase(1, lens, new, H, KH, D, dtype=dtype, device="cpu", **kw)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("window, sinks", [(0, 0), (90, 5)])
def test_right_results_pass(window, sinks, dtype):
    case = case_of([5, 300], [2, 40], 4, 2, 64, dtype, window=window, sinks=sinks)
    check_each_row(case, plain)
    whole_numbers(case)
    assert check_whole_numbers(case, plain(case)[1]) < 1e-4


def test_one_row_of_33000_is_seen_in_the_lse():
    case = case_of([33000], [1], 1, 1, 64, "bf16")
    rows = Rows(case)
    rows.check_lse(plain(case)[1])
    for kw in (dict(hide=[32999]), dict(hide=[0]), dict(twice=[16400])):
        with pytest.raises(AssertionError, match="lse off"):
            rows.check_lse(plain(case, **kw)[1])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_each_row_is_seen_in_its_column(dtype):
    case = case_of([40, 300], [1, 3], 4, 2, 64, dtype)
    rows = Rows(case)
    for first, row in ((0, 0), (0, 127), (128, 200), (256, 299)):
        rows.plant(first)
        rows.check_out(first, plain(case)[0])
        for kw in (dict(hide=[row]), dict(twice=[row]), dict(swap=(row, (row + 1) % 300)), dict(swap=((row + 1) % 300, row))):
            with pytest.raises(AssertionError, match="of its request"):
                rows.check_out(first, plain(case, **kw)[0])
        rows.plant(first, 0.0)


def test_a_row_of_middling_weight_is_seen_among_9000():
    case = case_of([9000], [2], 2, 1, 64, "bf16")
    whole_numbers(case)
    check_whole_numbers(case, plain(case)[1])
    mean = math.log((case.q[0, 0].double() @ case.rows64(0, 0, range(9001))[:, 0].T * case.scale).exp().mean())
    s = (case.q[0, 0].double() @ case.rows64(0, 0, range(9001))[:, 0].T) * case.scale
    row = int((s > mean).nonzero()[0])
    with pytest.raises(AssertionError, match="lse off"):
        check_whole_numbers(case, plain(case, hide=[row])[1])
