"""Plain 64-bit forms of the speculative-decoding step (rotary positions, tree
attention, page upkeep) and the inputs of its tests.  torch float64 on whatever
device the inputs are on; no code of the package."""
import math

import numpy as np
import torch

import workloads as W

HALF_BF16 = 2.0 ** -8     # half a step of bf16, relative
U32 = 2.0 ** -24          # half a step of binary32, relative


def i32(a, device):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int64).astype(np.uint32)).view(np.int32)).to(device)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def frequencies(dim, theta, scaling="none", factor=1.0, original=0, fast=32.0, slow=1.0):
    out = []
    for j in range(dim // 2):
        f = theta ** (-2.0 * j / dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "by_parts":
            def pair(b):
                return dim * math.log(original / (2 * math.pi * b)) / (2 * math.log(theta))
            lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), dim - 1)
            r = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f / factor * r + f * (1 - r)
        out.append(f)
    return np.array(out)


def rotate(x, table, half):
    """x [..., R] float64, table [..., R] of (cos, sin) pairs; also the sum of the
    magnitudes that enter each output (for error bounds)."""
    c, s = table[..., 0::2], table[..., 1::2]
    if half:
        h = x.shape[-1] // 2
        x0, x1 = x[..., :h], x[..., h:]
    else:
        x0, x1 = x[..., 0::2], x[..., 1::2]
    y0, y1 = x0 * c - x1 * s, x0 * s + x1 * c
    m0, m1 = (x0 * c).abs() + (x1 * s).abs(), (x0 * s).abs() + (x1 * c).abs()
    join = (lambda a, b: torch.cat([a, b], -1)) if half else (lambda a, b: torch.stack([a, b], -1).flatten(-2))
    return join(y0, y1), join(m0, m1)


# ---------------------------------------------------------------------------
# tree attention
# ---------------------------------------------------------------------------
def tree(rng, n):
    """Parents of n drafted tokens: -1 for roots."""
    return [-1 if i == 0 else int(rng.integers(max(-1, i - 5), i)) for i in range(n)]


def ancestors(parents):
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | (1 << i))
    return seen


def mask_tensor(rows, words, device):
    """Integers (one per token) as [T, words] 64-bit words."""
    a = np.array([[(m >> (64 * w)) & 0xFFFFFFFFFFFFFFFF for w in range(words)] for m in rows], np.uint64)
    return torch.from_numpy(a.reshape(len(rows), words).view(np.int64)).to(device)


class AttentionCase:
    """A batch on one device: the pool of workloads.make_paged_cache (poison in every
    slot behind the rows in use, in the other layer and in spare pages), queries, masks."""

    def __init__(self, seed, lens, new, heads, *, page_size=16, K=512, R=64, dtype="bf16", mask="chain",
                 q_std=0.6, device="cuda", words=None, extra_tokens=0):
        rng = np.random.default_rng(seed)
        lens, new = np.asarray(lens, np.int64), np.asarray(new, np.int64)
        D = K + R
        cache = W.make_paged_cache(rng, cache_lengths=lens + new, page_size=page_size, num_heads=1, head_dim=D,
                                   dtype=dtype)
        cache.cache_lengths = lens.astype(np.uint32)
        self.host, self.dev = cache, W.device_cache(cache, device)
        self.lens, self.new, self.H, self.K, self.D, self.layer = lens, new, heads, K, D, 1
        self.T = int(new.sum()) + extra_tokens
        self.device = device
        q = rng.standard_normal((self.T, heads, D)).astype(np.float32) * np.float32(q_std)
        self.q = torch.from_numpy(q).to(torch.float32 if dtype == "f32" else torch.bfloat16).to(device)
        self.iro = i32(np.concatenate([[0], np.cumsum(new)]), device)
        self.scale = (128 + R) ** -0.5
        if mask == "chain":
            self.seen = [[(1 << (i + 1)) - 1 for i in range(n)] for n in new]
            self.mask = None
        else:
            self.seen = [ancestors(tree(rng, int(n))) for n in new]
            if mask == "holes":     # arbitrary bits, some tokens see no drafted row at all
                self.seen = [[int.from_bytes(rng.bytes((n + 7) // 8), "little") & ((1 << n) - 1) if rng.random() < 0.6
                              else 0 for _ in range(n)] for n in new.tolist()]
            words = words or max(1, -(-int(new.max(initial=1)) // 64))
            full = (1 << (64 * words)) - 1
            self.seen = [[m & full for m in r] for r in self.seen]
            # bits past a request's own tokens must not matter
            junk = [[m | (full & ~((1 << max(1, n)) - 1) if n else m) for m in r] for r, n in zip(self.seen, new.tolist())]
            rows = [m for r in junk for m in r] + [0] * extra_tokens
            self.mask = mask_tensor(rows, words, device)

    def rows64(self, b):
        """float64 [len + n, D] rows of request b."""
        ps = self.host.page_size
        L = int(self.lens[b] + self.new[b])
        p = np.arange(L)
        ids = self.host.page_table[b, p // ps].astype(np.int64)
        pool = self.dev.pool[torch.from_numpy(ids).to(self.device), self.layer, 0,
                             torch.from_numpy(p % ps).to(self.device)].reshape(L, self.D)
        if self.host.dtype == "e4m3":
            sc = self.dev.scales[torch.from_numpy(ids).to(self.device), self.layer, 0,
                                 torch.from_numpy(p % ps).to(self.device)].double()
            pool = pool.view(torch.float8_e4m3fn).to(torch.float32).double()
            return pool * sc.repeat_interleave(128, dim=1)[:, :self.D]
        return pool.double()

    def reference(self):
        """out, lse and a bound of the error of each element of both (float64 tensors).

        Bounds.  A score is a binary32 sum of D products in some order: off by at most
        ds = (D + 8) 2^-24 scale sum |q||row| (the 8 covers the scalings of scores and
        e4m3 blocks and the exponential's argument).  Every weight is then off by a factor
        exp(+-2 ds) and the exponential's own error (2^-20 covers its argument in base 2
        at |s| < 2^4 and its rounding), and rounded to bf16 (none of it in a binary32
        cache's path); sums of L positive weights and of L products in binary32 add
        L 2^-24 of the sum of magnitudes; the result is rounded once to its own type."""
        f32 = self.host.dtype == "f32"
        out = torch.zeros((self.T, self.H, self.K), dtype=torch.float64, device=self.device)
        lse = torch.full((self.T, self.H), -math.inf, dtype=torch.float64, device=self.device)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        at = 0
        for b, n in enumerate(self.new.tolist()):
            rows, cached = self.rows64(b), int(self.lens[b])
            L = cached + n
            if n == 0:
                continue
            vis = torch.ones((n, L), dtype=torch.bool)
            for i in range(n):
                for j in range(n):
                    vis[i, cached + j] = bool((self.seen[b][i] >> j) & 1)
            vis = vis.to(self.device)
            for i in range(n):
                r = rows[vis[i]]
                if r.shape[0] == 0:
                    continue
                q = self.q[at + i].double()
                s = (q @ r.t().contiguous()) * self.scale
                ds = ((q.abs() @ r.abs().t().contiguous()) * self.scale).amax(dim=1) * (self.D + 8) * U32
                z = torch.logsumexp(s, dim=1)
                w = torch.exp(s - z[:, None])
                o = w @ r[:, :self.K]
                mag = w @ r[:, :self.K].abs()
                rel = 2 * ds + 2.0 ** -20 + 3 * r.shape[0] * U32 + (0.0 if f32 else HALF_BF16)
                out[at + i], lse[at + i] = o, z
                tol[at + i] = mag * rel[:, None] + o.abs() * ((2 * U32) if f32 else HALF_BF16) * 1.02 + 1e-30
                ltol[at + i] = ds + 2.0 ** -20 + 3 * r.shape[0] * U32 + z.abs() * 2 * U32
            at += n
        return out, lse, tol, ltol


def check_attention(case, out, lse):
    ref, zref, tol, ltol = case.reference()
    live = int(case.new.sum())
    got, z = out[:live].double(), lse[:live].double()
    assert bool(torch.isfinite(got).all())
    over = ((got - ref[:live]).abs() - tol[:live]).max() if live else torch.tensor(-1.0)
    assert float(over) <= 0, f"out off by {float(over)} more than its bound"
    empty = torch.isinf(zref[:live])
    assert bool((z[empty] == -math.inf).all()) and bool((got[empty] == 0).all())
    assert bool(((z - zref[:live]).abs()[~empty] <= ltol[:live][~empty]).all())
