"""Plain 64-bit forms of the paged K/V cache's operators and the inputs of their tests.
torch float64 on whatever device the inputs are on; no code of the package."""
import math

import numpy as np
import torch

import workloads as W
from plain_step import HALF_BF16, U32, i32

BF16 = torch.bfloat16


def cast_pool(pool, dtype):
    return pool.view(torch.float8_e4m3fn).float().double() if dtype == "e4m3" else pool.double()


class KvCase:
    """A batch on one device: the pool of workloads.make_paged_cache (poison in every slot behind the
    rows in use, in the other layer and in spare pages), queries, offsets.  ``extra_tokens``: rows of q
    behind the last request."""

    def __init__(self, seed, lens, new, heads, kv_heads, head_dim, *, page_size=16, dtype="bf16", window=0, sinks=0,
                 q_std=1.0, device="cuda", extra_tokens=0):
        rng = np.random.default_rng(seed)
        lens, new = np.asarray(lens, np.int64), np.asarray(new, np.int64)
        cache = W.make_paged_cache(rng, cache_lengths=lens + new, page_size=page_size, num_heads=kv_heads,
                                   head_dim=head_dim, dtype=dtype, num_kv=2)
        cache.cache_lengths = lens.astype(np.uint32)
        self.host, self.dev = cache, W.device_cache(cache, device)
        self.lens, self.new, self.H, self.KH, self.D, self.layer = lens, new, heads, kv_heads, head_dim, 1
        self.window, self.sinks, self.dtype, self.device = window, sinks, dtype, device
        self.T = int(new.sum()) + extra_tokens
        q = rng.standard_normal((self.T, heads, head_dim)).astype(np.float32) * np.float32(q_std)
        self.q = torch.from_numpy(q).to(torch.float32 if dtype == "f32" else BF16).to(device)
        self.iro = i32(np.concatenate([[0], np.cumsum(new)]), device)
        self.scale = head_dim ** -0.5

    def where(self, b, positions):
        """Pool indices (page, slot) of a request's positions."""
        p = np.asarray(positions, np.int64)
        ps = self.host.page_size
        ids = self.host.page_table[b, p // ps].astype(np.int64)
        return torch.from_numpy(ids).to(self.device), torch.from_numpy(p % ps).to(self.device)

    def rows64(self, b, half, positions):
        """float64 [positions, kv_heads, head_dim] keys (0) or values (1)."""
        page, slot = self.where(b, positions)
        rows = cast_pool(self.dev.pool[page, self.layer, half, slot], self.dtype)
        if self.dtype == "e4m3":
            width = self.KH * self.D
            sc = self.dev.scales[page, self.layer, half, slot].double().repeat_interleave(128, dim=1)[:, :width]
            rows = rows * sc.view(rows.shape)
        return rows

    def seen(self, b):
        """bool [new, len + new]: which rows each token sees."""
        n, m = int(self.lens[b]), int(self.new[b])
        p = np.arange(n, n + m)[:, None]
        k = np.arange(n + m)[None, :]
        see = k <= p
        if self.window:
            see &= (p - k < self.window) | (k < self.sinks)
        return torch.from_numpy(see).to(self.device)

    def reference(self):
        """out, lse and a bound of the error of each element of both (float64 tensors).

        Bounds.  A score is a binary32 sum of D products in some order: off by at most
        ds = (D + 8) 2^-24 scale sum |q||k| (the 8 covers the scalings of scores and e4m3
        blocks and the exponential's argument).  Every weight is then off by a factor
        exp(+-2 ds) and the exponential's own error (2^-20 covers its argument in base 2 at
        |s| < 2^4 and its rounding), and rounded to bf16 (not with a binary32 cache); sums of L
        positive weights and of L products in binary32 add L 2^-24 of the sum of magnitudes;
        the result is rounded once to its own type."""
        f32, G = self.dtype == "f32", self.H // self.KH
        out = torch.zeros((self.T, self.H, self.D), dtype=torch.float64, device=self.device)
        lse = torch.full((self.T, self.H), -math.inf, dtype=torch.float64, device=self.device)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        at = 0
        for b, (n, m) in enumerate(zip(self.lens.tolist(), self.new.tolist())):
            if m == 0:
                continue
            hidden = ~self.seen(b)
            count = (~hidden).sum(1).double()[:, None]
            K, V = self.rows64(b, 0, range(n + m)), self.rows64(b, 1, range(n + m))
            # rows that a token does not see must not matter, whatever they hold
            for h in range(self.H):
                k, v, q = K[:, h // G].contiguous(), V[:, h // G].contiguous(), self.q[at:at + m, h].double()
                s = ((q @ k.t().contiguous()) * self.scale).masked_fill(hidden, -math.inf)
                mags = ((q.abs() @ k.abs().t().contiguous()) * abs(self.scale)).masked_fill(hidden, 0.0)
                ds = mags.amax(dim=1) * (self.D + 8) * U32
                z = torch.logsumexp(s, dim=1)
                w = torch.exp(s - torch.where(z == -math.inf, 0.0, z)[:, None])
                o, mag = w @ v, w @ v.abs()
                rel = (2 * ds + 2.0 ** -20)[:, None] + 3 * count * U32 + (0.0 if f32 else HALF_BF16)
                out[at:at + m, h], lse[at:at + m, h] = o, z
                tol[at:at + m, h] = mag * rel + o.abs() * ((2 * U32) if f32 else HALF_BF16) * 1.02 + 1e-30
                ltol[at:at + m, h] = ds + 2.0 ** -20 + 3 * count[:, 0] * U32 + z.abs() * 2 * U32
            at += m
        return out, lse, tol, ltol


def check_kv_attention(case, out, lse):
    ref, zref, tol, ltol = case.reference()
    live = int(case.new.sum())
    got, z = out[:live].double(), lse[:live].double()
    assert bool(torch.isfinite(got).all())
    over = ((got - ref[:live]).abs() - tol[:live]).max() if live else torch.tensor(-1.0)
    assert float(over) <= 0, f"out off by {float(over)} more than its bound"
    empty = torch.isinf(zref[:live])
    assert bool((z[empty] == -math.inf).all()) and bool((got[empty] == 0).all())
    assert bool(((z - zref[:live]).abs()[~empty] <= ltol[:live][~empty]).all())


def rotated(x, table, rope, half):
    """The last `rope` columns of x [T, heads, D] (float64) rotated with table [T, rope] of (cos, sin) pairs;
    also the sum of the magnitudes that enter each output."""
    if rope == 0:
        return x, x.abs()
    from plain_step import rotate
    D = x.shape[-1]
    y, mag = rotate(x[..., D - rope:], table[:, None], half)
    return torch.cat([x[..., :D - rope], y], -1), torch.cat([x[..., :D - rope].abs(), mag], -1)


def quantised(x):
    """Codes (as values), scales of [T, width] float64 rows, per 128 columns, in binary32 as documented."""
    T, width = x.shape
    pad = -width % 128
    y = torch.nn.functional.pad(x.float(), (0, pad)).view(T, -1, 128)
    am = y.abs().amax(2)
    zero = am == 0
    am = torch.where(zero, torch.full_like(am, 448.0), am.clamp_min(448.0 * 2.0 ** -126))
    most = torch.full_like(am, 448.0)     # (by a number, torch multiplies by its reciprocal)
    codes = (y * (most / am)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(T, -1)[:, :width], am / most
