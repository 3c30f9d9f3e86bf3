"""Checks of the paged K/V attention that see each single row, at any length.

With queries of zero every row that a token sees weighs 1, sums of weights are whole numbers, and joining
partial results multiplies by 1: lse is ln(count) and out is (sum of seen V) / count, both to within the last
roundings.  A value of 1 in one column of one row is then 1 / count where the row is seen and 0 elsewhere,
and there is a column of some key head for each of as many rows at a time."""
import math

import torch

from plain_step import HALF_BF16, U32

# Native log2 is off by a unit in its last place, 2^-19 below 2^32; the factor ln 2, the product and the sum
# with the reference round by 2^-24 of at most 12 each: together below ln 2 2^-19 + 3 12 2^-24 < 2^-18.
LOG_ERROR = 2.0 ** -18


class Rows:
    """The rows in use of a KvCase, its values all zero, its queries zero."""

    def __init__(self, case):
        self.case = case
        case.q.zero_()
        at = [(b, n + m) for b, (n, m) in enumerate(zip(case.lens.tolist(), case.new.tolist())) if m]
        where = [case.where(b, range(n)) for b, n in at]
        self.page, self.slot = torch.cat([w[0] for w in where]), torch.cat([w[1] for w in where])
        self.pos = torch.cat([torch.arange(n, device=case.device) for _, n in at])
        self.longest, self.block = max(n for _, n in at), case.KH * case.D
        self.seen = [case.seen(b) for b, _ in at]
        self.count = torch.cat([s.sum(1) for s in self.seen]).double()
        assert float(self.count.max()) < 2 ** 17        # 1 / count is above twice LOG_ERROR
        self.fill(self.page, self.slot, slice(None), slice(None), 0.0)
        if case.dtype == "e4m3":
            case.dev.scales[self.page, case.layer, 1, self.slot] = 1.0

    def fill(self, page, slot, head, col, value):
        pool = self.case.dev.pool
        if self.case.dtype == "e4m3":
            value = 0x38 if value == 1.0 else 0         # the code of 1
        pool[page, self.case.layer, 1, slot, head, col] = value

    def plant(self, first, value=1.0):
        """Row first + i of every request: `value` in column i % D of key head i / D."""
        take = ((self.pos >= first) & (self.pos < first + self.block)).nonzero()[:, 0]
        i, D = self.pos[take] - first, self.case.D
        self.fill(self.page[take], self.slot[take], i // D, i % D, value)

    def want(self, first):
        """What out is with rows planted from `first` on: float64 [tokens, heads, D]."""
        parts = []
        for s in self.seen:
            s = s[:, first:first + self.block]
            parts.append(torch.nn.functional.pad(s, (0, self.block - s.shape[1])))
        case = self.case
        x = torch.cat(parts).double() / self.count[:, None]
        return x.view(-1, case.KH, 1, case.D).expand(-1, -1, case.H // case.KH, -1).reshape(-1, case.H, case.D)

    def check_lse(self, lse):
        off = (lse[:self.count.numel()].double() - torch.log(self.count)[:, None]).abs().max()
        assert float(off) <= LOG_ERROR, f"lse off by {float(off)}, a row is {1 / float(self.count.max())}"

    def check_out(self, first, out):
        """1 / count comes out of a division, a product and one rounding to the output's type."""
        want = self.want(first)
        tol = want * ((4 * U32 if self.case.dtype == "f32" else HALF_BF16) + 4 * U32)
        wrong = ((out[:want.shape[0]].double() - want).abs() > tol).nonzero()
        if wrong.numel():
            t, h, c = wrong[0].tolist()
            row = first + h // (self.case.H // self.case.KH) * self.case.D + c
            raise AssertionError(f"token {t}, head {h}: {float(out[t, h, c])} for row {row} of its request")


def check_each_row(case, attend):
    """attend(case) -> out, lse.  Every row of every request, in as many calls as it takes."""
    rows = Rows(case)
    for first in range(0, rows.longest, rows.block):
        rows.plant(first)
        out, lse = attend(case)
        if first == 0:
            rows.check_lse(lse)
        rows.check_out(first, out)
        rows.plant(first, 0.0)


def whole_numbers(case):
    """Queries and keys of small whole numbers, whose products binary32 sums without an error; scale 1/16."""
    g = torch.Generator(device=case.device).manual_seed(7)
    case.scale = 2.0 ** -4
    case.q.copy_(torch.randint(-1, 2, case.q.shape, generator=g, device=case.device))
    for b, (n, m) in enumerate(zip(case.lens.tolist(), case.new.tolist())):
        if m:
            page, slot = case.where(b, range(n + m))
            k = torch.randint(-2, 3, (n + m, case.KH, case.D), generator=g, device=case.device).float()
            if case.dtype == "e4m3":
                case.dev.pool[page, case.layer, 0, slot] = k.to(torch.float8_e4m3fn).view(torch.uint8)
                case.dev.scales[page, case.layer, 0, slot] = 1.0
            else:
                case.dev.pool[page, case.layer, 0, slot] = k.to(case.dev.pool.dtype)


def check_whole_numbers(case, lse):
    """lse against binary64 where scores are exact.  With A the largest score in base 2, an exponent is off by 2 A 2^-23
    (scale log2 e, rounded twice), A 2^-24 (the reference's) and 2 A 2^-24 (its own rounding), a weight by ln 2 times that and
    2^-23 more.  Sums add one rounding each: 11 in a tile and one a tile, or one for each of the rows that one group of
    lanes of the general form takes (a 16th, with more than 128 columns an 8th), and two for each of 256 shares."""
    ref, zref, _, _ = case.reference()
    live = int(case.new.sum())
    A = 0.0
    for b, (n, m) in enumerate(zip(case.lens.tolist(), case.new.tolist())):
        if m:
            k = case.rows64(b, 0, range(n + m))
            A = max(A, float(k.abs().sum(2).max()) * case.scale * math.log2(math.e))    # |q| is at most 1
    longest = int((case.lens + case.new).max())
    tol = math.log(2) * 7 * A * U32 + 2.0 ** -23 + (11 + longest / (16 if case.D <= 128 else 8) + 512) * U32 + LOG_ERROR
    off = float((lse[:live].double() - zref[:live]).abs().max())
    assert off <= tol, f"lse off by {off}, its bound is {tol}"
    return tol
