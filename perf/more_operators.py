"""The operators of a model with separate keys and values over the paged K/V cache, as measured cases.

``kv_matmul_paged`` fills the pages of such a cache straight from hidden states.  Where the
keys are rotated, or the cache is e4m3, new tokens' keys and values are rotated, quantised and
placed by a write of their own (``write``); attention of a chunk of new tokens, or of one token
per request, reads the pages, causally, with or without a sliding window and a few first tokens
that stay visible (``attend``); and rows are read back into contiguous buffers (``read``).

Every case is a dict of plain values: ``op`` names the operator, ``layout`` seeds the
ragged sizes (lengths, tokens per request), so that the work of a case does not depend on
the seed its values are drawn from.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128                     # columns of a token row per scale of an e4m3 cache
PAGE_NONE = 0xFFFFFFFF          # an unused page-table entry
CODES_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # A decode step's keys and values, taken out of a fused projection: latency counts.
        dict(name="write_step_e4m3", op="write", requests=64, tokens_lo=1, tokens_hi=1, kv_heads=8, head_dim=128,
             len_lo=100, len_hi=8000, page_size=16, rope=128, half=True, cache="e4m3", fused=True, layout=11),
        # A prefill's tokens, rotated in pairs of neighbours.
        dict(name="write_chunk", op="write", requests=6, tokens_lo=1000, tokens_hi=4000, kv_heads=8, head_dim=128,
             len_lo=1, len_hi=20000, page_size=128, rope=128, half=False, cache="bf16", fused=True, layout=12),
        # A large prefill into an e4m3 cache, half of each head rotated.
        dict(name="write_chunk_e4m3", op="write", requests=5, tokens_lo=5000, tokens_hi=8000, kv_heads=8, head_dim=128,
             len_lo=1, len_hi=9000, page_size=64, rope=64, half=True, cache="e4m3", fused=False, layout=13),
        # Shared prefixes read back for a pass that wants plain tensors.
        dict(name="read_prefix_e4m3", op="read", requests=4, kv_heads=8, head_dim=128, len_lo=4000, len_hi=20000,
             page_size=128, cache="e4m3", layout=21),
        # The newest rows of a small batch.
        dict(name="read_small", op="read", requests=8, kv_heads=4, head_dim=64, len_lo=20, len_hi=300, page_size=16,
             cache="bf16", layout=22),
        # Few requests, one token each, short contexts: latency counts.
        dict(name="attend_step_small", op="attend", requests=4, tokens_lo=1, tokens_hi=1, heads=32, kv_heads=8,
             head_dim=128, len_lo=100, len_hi=1000, page_size=16, window=0, sinks=0, cache="bf16", layout=31),
        # A decode batch with contexts of very different lengths: bound by the reading of the cache.
        dict(name="attend_decode", op="attend", requests=64, tokens_lo=1, tokens_hi=1, heads=64, kv_heads=8,
             head_dim=128, len_lo=1000, len_hi=32000, page_size=128, window=0, sinks=0, cache="bf16", layout=32),
        # Long contexts in an e4m3 cache, one to four new tokens, five query heads to a key head.
        dict(name="attend_long_e4m3", op="attend", requests=6, tokens_lo=1, tokens_hi=4, heads=40, kv_heads=8,
             head_dim=128, len_lo=60000, len_hi=131072, page_size=64, window=0, sinks=0, cache="e4m3", layout=33),
        # Prompt chunks behind cached prefixes: bound by the matrix cores.
        dict(name="attend_chunk", op="attend", requests=5, tokens_lo=1000, tokens_hi=4096, heads=32, kv_heads=8,
             head_dim=128, len_lo=1, len_hi=8000, page_size=128, window=0, sinks=0, cache="bf16", layout=34),
        # The same with a sliding window and first tokens that stay, in an e4m3 cache.
        dict(name="attend_window_e4m3", op="attend", requests=4, tokens_lo=1500, tokens_hi=4096, heads=64, kv_heads=8,
             head_dim=128, len_lo=2000, len_hi=20000, page_size=32, window=2048, sinks=4, cache="e4m3", layout=35),
        # One batch of single tokens and prompt chunks together, heads of 64 columns, seven to a key head.
        dict(name="attend_mixed", op="attend", requests=40, tokens_lo=1, tokens_hi=900, heads=28, kv_heads=4,
             head_dim=64, len_lo=1, len_hi=5000, page_size=16, window=0, sinks=0, cache="bf16", chunks=4, layout=36),
        # A binary32 cache, heads of 80 columns, a window: shapes off the matrix cores.
        dict(name="attend_window_f32", op="attend", requests=8, tokens_lo=1, tokens_hi=8, heads=12, kv_heads=12,
             head_dim=80, len_lo=10, len_hi=3000, page_size=100, window=500, sinks=2, cache="f32", layout=37),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "write", "write", "read"])
    layout = rng.randrange(1 << 30)
    page_size = rng.choice([16, 32, 64, 128, 128, 100])
    if op == "write":
        tokens = _log_int(rng, 1, 4000)
        cache = rng.choice(["bf16", "e4m3", "e4m3"])
        head_dim = rng.choice([64, 128, 128, 128, 112, 256])
        kv_heads = rng.choice([1, 2, 4, 5, 8, 8])
        rope = rng.choice([0, head_dim // 2, head_dim, head_dim])
        return dict(op=op, requests=_log_int(rng, 1, 8), tokens_lo=max(1, tokens // 3), tokens_hi=tokens,
                    kv_heads=kv_heads, head_dim=head_dim, len_lo=1, len_hi=_log_int(rng, 2, 20000), page_size=page_size,
                    rope=rope, half=rng.random() < 0.5, cache=cache, fused=rng.random() < 0.5, layout=layout)
    if op == "read":
        hi = _log_int(rng, 2, 20000)
        return dict(op=op, requests=_log_int(rng, 1, 4 if hi > 4000 else 32), kv_heads=rng.choice([1, 4, 8, 8]),
                    head_dim=rng.choice([64, 128, 128, 112]), len_lo=max(1, hi // rng.choice([1, 5, 50])), len_hi=hi,
                    page_size=page_size, cache=rng.choice(["bf16", "e4m3", "e4m3", "f32"]), layout=layout)
    cache = rng.choice(["bf16", "bf16", "bf16", "e4m3", "e4m3", "f32"])
    heads, kv_heads = rng.choice([(32, 8), (64, 8), (40, 8), (28, 4), (16, 16), (18, 2), (8, 1), (42, 3)])
    case = dict(op=op, requests=_log_int(rng, 1, 96), tokens_lo=1, tokens_hi=1, heads=heads, kv_heads=kv_heads,
                head_dim=rng.choice([64, 128, 128]), len_lo=1, len_hi=_log_int(rng, 2, 100000), page_size=page_size,
                window=0, sinks=0, cache=cache, layout=layout)
    if rng.random() < 0.4:
        case["window"] = _log_int(rng, 1, 8192)
        case["sinks"] = rng.choice([0, 0, 1, 4, rng.randint(2, 200)])
    case["tokens_hi"] = rng.choice([1, 1, rng.randint(2, 16), _log_int(rng, 17, 4096)])
    case["tokens_lo"] = rng.choice([1, max(1, case["tokens_hi"] // 3)])
    case["len_lo"] = max(1, case["len_hi"] // rng.choice([1, 4, 30]))
    if rng.random() < 0.15 and case["requests"] > 4:
        case["chunks"] = rng.randint(1, 4)
    if cache == "f32" or rng.random() < 0.1:
        case["head_dim"] = rng.choice([64, 80, 112, 128, 256])
    # Shapes off the matrix cores are met in small models and in tests.
    small = cache == "f32" or case["head_dim"] not in (64, 128)
    flops = work(listed()[11])["flops"] * 4 if small else work(listed()[8])["flops"]
    bytes_ = work(listed()[6])["bytes"]
    if small:
        case["len_hi"] = min(case["len_hi"], 4000)
        case["len_lo"] = min(case["len_lo"], case["len_hi"])
    while case["requests"] > 1 and (work(case)["flops"] > flops or work(case)["bytes"] > bytes_ or
                                    case["requests"] * case["len_hi"] > 600000):
        case["requests"] = (case["requests"] + 1) // 2
    while work(case)["flops"] > flops or work(case)["bytes"] > bytes_:
        case["len_hi"] = max(2, case["len_hi"] // 2)
        case["len_lo"] = min(case["len_lo"], case["len_hi"])
        case["tokens_hi"] = max(1, case["tokens_hi"] * 3 // 4)
        case["tokens_lo"] = min(case["tokens_lo"], case["tokens_hi"])
    if "chunks" in case:
        case["chunks"] = min(case["chunks"], case["requests"])
    return case


# ---------------------------------------------------------------------------
# ragged sizes of a case (from its layout number alone)
# ---------------------------------------------------------------------------
def _lengths(case):
    """Cached tokens and new tokens of each request."""
    r = np.random.default_rng(case["layout"])
    lo, hi = case["len_lo"], case["len_hi"]
    lens = np.round(np.exp(r.uniform(math.log(lo), math.log(hi + 1), case["requests"]))).astype(np.int64)
    lens = np.clip(lens, lo, hi)
    if case["op"] == "read":
        # rows of each request, from a start inside it
        first = r.integers(0, lens, size=case["requests"], endpoint=True) // 4
        return lens, first
    new = r.integers(case["tokens_lo"], case["tokens_hi"], size=case["requests"], endpoint=True)
    if "chunks" in case:       # all the others have one token
        new[r.permutation(case["requests"])[case["chunks"]:]] = 1
    return lens, new


_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def _row_bytes(case):
    """Bytes of a token's keys and values."""
    width = case["kv_heads"] * case["head_dim"]
    return 2 * (width * _BYTES[case["cache"]] + (4 * -(-width // BLOCK) if case["cache"] == "e4m3" else 0))


def work(case):
    lens, new = _lengths(case)
    width = case["kv_heads"] * case["head_dim"]
    if case["op"] == "read":
        rows = int((lens - new).sum())
        out = 2 * width * (2 if case["cache"] == "e4m3" else _BYTES[case["cache"]])
        return dict(bytes=rows * (_row_bytes(case) + out), flops=2 * rows * width if case["cache"] == "e4m3" else 0)
    T = int(new.sum())
    if case["op"] == "write":
        rope = case["rope"]
        return dict(bytes=T * (2 * width * 2 + _row_bytes(case) + rope * 4),
                    flops=T * case["kv_heads"] * 3 * rope + (4 * T * width if case["cache"] == "e4m3" else 0))
    H, D, window, sinks = case["heads"], case["head_dim"], case["window"], case["sinks"]
    pairs = rows = 0
    for n, m in zip(lens.tolist(), new.tolist()):
        p = np.arange(n, n + m, dtype=np.int64)
        low = np.maximum(p + 1 - window, 0) if window else np.zeros_like(p)
        pairs += int((p + 1 - low + np.minimum(sinks, low)).sum())
        rows += n + m - int(low[0]) + min(sinks, int(low[0])) if m else 0
    eb = 4 if case["cache"] == "f32" else 2
    return dict(bytes=rows * _row_bytes(case) + 2 * T * H * D * eb + T * H * 4, flops=4 * D * H * pairs)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 29)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int64).astype(np.uint32)).view(np.int32)).cuda()


def _normal(g, shape, dtype=torch.float32):
    """Normal values made in pieces, so that a large pool never exists in 32 bits."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for lo in range(0, flat.numel(), 1 << 27):
        hi = min(lo + (1 << 27), flat.numel())
        flat[lo:hi] = torch.randn(hi - lo, generator=g, device="cuda")
    return out


def _pool(g, case, pages):
    """[pages, 1, 2, page_size, kv_heads, head_dim] keys and values about N(0, 1), and an e4m3 pool's scales."""
    shape = (pages, 1, 2, case["page_size"], case["kv_heads"], case["head_dim"])
    if case["cache"] != "e4m3":
        return _normal(g, shape, torch.float32 if case["cache"] == "f32" else torch.bfloat16), None
    pool = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    flat = pool.view(-1)
    for lo in range(0, flat.numel(), 1 << 27):
        hi = min(lo + (1 << 27), flat.numel())
        v = torch.randn(hi - lo, generator=g, device="cuda") * 130.0
        flat[lo:hi] = v.clamp_(-CODES_MAX, CODES_MAX).to(torch.float8_e4m3fn)
    blocks = -(-case["kv_heads"] * case["head_dim"] // BLOCK)
    scales = torch.rand((*shape[:4], blocks), generator=g, device="cuda")
    return pool, scales * 0.004 + 0.006


def _table(r, pages_needed, spare=2):
    pages = int(sum(pages_needed)) + spare
    perm = r.permutation(pages)
    table = np.full((len(pages_needed), max(1, max(pages_needed))), PAGE_NONE, np.int64)
    at = 0
    for b, n in enumerate(pages_needed):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pages


def _freqs(rows, dim):
    """A [rows, dim] table of (cos, sin) pairs, base 10000."""
    j = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    ang = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2.0 * j / dim)
    return torch.stack([ang.cos(), ang.sin()], dim=2).reshape(rows, dim).float()


def prepare(case, seed):
    op, g, r = case["op"], _gen(seed), np.random.default_rng(int(seed) + 303)
    lens, new = _lengths(case)
    ps, KH, D = case["page_size"], case["kv_heads"], case["head_dim"]
    s = dict(case=case, lens=lens, new=new)
    if op == "read":
        table, pages = _table(r, [-(-int(n) // ps) for n in lens])
        s["pool"], s["scales"] = _pool(g, case, pages)
        rows = lens - new
        s["M"] = M = int(rows.sum())
        dt = torch.float32 if case["cache"] == "f32" else torch.bfloat16
        s.update(table=_i32(table), lengths=_i32(lens), first=_i32(new), offsets=_i32(np.concatenate([[0], np.cumsum(rows)])),
                 k_out=torch.empty((M, KH, D), dtype=dt, device="cuda"),
                 v_out=torch.empty((M, KH, D), dtype=dt, device="cuda"))
        return _with_cache(s)
    T = s["T"] = int(new.sum())
    table, pages = _table(r, [-(-int(n + m) // ps) for n, m in zip(lens, new)])
    s.update(table=_i32(table), lengths=_i32(lens), offsets=_i32(np.concatenate([[0], np.cumsum(new)])))
    if op == "write":
        if case["fused"]:      # keys and values behind eight times as many query columns
            qkv = _normal(g, (T, 10 * KH, D), torch.bfloat16)
            s["k"], s["v"] = qkv[:, 8 * KH:9 * KH], qkv[:, 9 * KH:]
        else:
            s["k"], s["v"] = _normal(g, (T, KH, D), torch.bfloat16), _normal(g, (T, KH, D), torch.bfloat16)
        dt = torch.float8_e4m3fn if case["cache"] == "e4m3" else torch.bfloat16
        s["pool"] = torch.zeros((pages, 1, 2, ps, KH, D), dtype=torch.uint8 if case["cache"] == "e4m3" else dt,
                                device="cuda").view(dt)
        s["scales"] = None
        if case["cache"] == "e4m3":
            s["scales"] = torch.zeros((pages, 1, 2, ps, -(-KH * D // BLOCK)), device="cuda")
        s["freqs"] = _freqs(int((lens + new).max()) + 1, case["rope"]) if case["rope"] else None
        return _with_cache(s)
    s["pool"], s["scales"] = _pool(g, case, pages)
    dt = torch.float32 if case["cache"] == "f32" else torch.bfloat16
    s.update(q=_normal(g, (T, case["heads"], D), dt), scale=D ** -0.5,
             out=torch.empty((T, case["heads"], D), dtype=dt, device="cuda"),
             lse=torch.empty((T, case["heads"]), device="cuda"))
    s = _with_cache(s)
    if own:
        import mla_paged_latent_page_amd as mp
        size = mp.kv_attention_workspace_size(T, case["heads"], KH, D)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def _with_cache(s):
    if own:
        import mla_paged_latent_page_amd as mp
        s["cache"] = mp.PagedKVCache(s["pool"], s["table"], s["lengths"], scales=s["scales"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import mla_paged_latent_page_amd as mp
    case = s["case"]
    e4m3 = case["cache"] == "e4m3"
    if case["op"] == "write":
        call = mp.kv_write_paged_fp8 if e4m3 else mp.kv_write_paged
        call(s["k"], s["v"], s["offsets"], s["cache"], 0, freqs_cis=s["freqs"],
             layout="half" if case["half"] else "interleaved")
        return (s["pool"], s["scales"]) if e4m3 else s["pool"]
    if case["op"] == "read":
        call = mp.kv_gather_paged_fp8_cache if e4m3 else mp.kv_gather_paged
        call(s["offsets"], s["first"], s["M"], s["cache"], 0, s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    call = mp.kv_attention_paged_fp8_cache if e4m3 else mp.kv_attention_paged
    call(s["q"], s["offsets"], s["scale"], s["cache"], 0, s["out"], s["workspace"], window=case["window"],
         sinks=case["sinks"], lse=s["lse"])
    return s["out"], s["lse"]


def _slots(s, b, positions):
    """Pool indices (page, slot) of a request's positions."""
    ps = s["case"]["page_size"]
    return s["table"][b].long()[positions // ps], positions % ps


def _rotate(x, cos, sin, half):
    """Rotate the pairs of the last axis: (2j, 2j+1), or (j, j + dim/2) in the half layout."""
    if half:
        x0, x1 = x.chunk(2, dim=-1)
        return torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], dim=-1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], dim=-1).flatten(-2)


def _rows(s, b, half, lo, hi):
    """Float rows [hi - lo, kv_heads, head_dim] of the keys (0) or values (1) of a request's positions."""
    case = s["case"]
    page, slot = _slots(s, b, torch.arange(lo, hi, device="cuda"))
    rows = s["pool"][page, 0, half, slot].float()
    if s["scales"] is None:
        return rows
    width = case["kv_heads"] * case["head_dim"]
    sc = s["scales"][page, 0, half, slot].repeat_interleave(BLOCK, dim=1)[:, :width]
    return rows * sc.view(rows.shape)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "write":
        return _write_plain(s)
    if case["op"] == "read":
        at = 0
        for b, (n, first) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
            for half, out in ((0, s["k_out"]), (1, s["v_out"])):
                out[at:at + n - first] = _rows(s, b, half, first, n).to(out.dtype)
            at += n - first
        return s["k_out"], s["v_out"]
    return _attend_plain(s)


def _write_plain(s):
    case = s["case"]
    KH, D, rope = case["kv_heads"], case["head_dim"], case["rope"]
    at = 0
    for b, (n, m) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        pos = torch.arange(n, n + m, device="cuda")
        page, slot = _slots(s, b, pos)
        k, v = s["k"][at:at + m].float(), s["v"][at:at + m].float()
        at += m
        if rope:
            tab = s["freqs"][pos]
            rot = _rotate(k[..., D - rope:], tab[:, None, 0::2], tab[:, None, 1::2], case["half"])
            k = torch.cat([k[..., :D - rope], rot], dim=-1)
        for half, x in ((0, k), (1, v)):
            if s["scales"] is None:
                s["pool"][page, 0, half, slot] = x.to(torch.bfloat16)
                continue
            width = KH * D
            x = torch.nn.functional.pad(x.reshape(m, width), (0, -width % BLOCK)).view(m, -1, BLOCK)
            top = x.abs().amax(dim=2)
            most = torch.full_like(top, CODES_MAX)     # (by a number, torch multiplies by its reciprocal)
            safe = torch.where(top == 0, most, top)
            codes = (x * (most / safe)[..., None]).view(m, -1)[:, :width].to(torch.float8_e4m3fn)
            s["pool"].view(torch.uint8)[page, 0, half, slot] = codes.view(torch.uint8).view(m, KH, D)
            s["scales"][page, 0, half, slot] = safe / most
    return s["pool"] if s["scales"] is None else (s["pool"], s["scales"])


def _attend_plain(s):
    case = s["case"]
    H, KH, D, window, sinks = case["heads"], case["kv_heads"], case["head_dim"], case["window"], case["sinks"]
    G = H // KH
    at = 0
    for b, (n, m) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        # A window leaves only part of a long context to be read.
        low = max(0, n + 1 - window) if window else 0
        if low <= sinks:
            low = 0
        spans = ([(0, sinks)] if low and sinks else []) + [(low, n + m)]
        pos = torch.cat([torch.arange(x, y, device="cuda") for x, y in spans])
        k = torch.cat([_rows(s, b, 0, x, y) for x, y in spans]).permute(1, 2, 0).contiguous()
        v = torch.cat([_rows(s, b, 1, x, y) for x, y in spans]).permute(1, 0, 2).contiguous()
        block = max(1, (1 << 31) // (H * pos.numel()))
        for i in range(0, m, block):
            j = min(m, i + block)
            q = s["q"][at + i:at + j].float().view(j - i, KH, G, D).permute(1, 0, 2, 3).reshape(KH, -1, D)
            score = torch.bmm(q, k).view(KH, j - i, G, -1) * s["scale"]
            p = torch.arange(n + i, n + j, device="cuda")[:, None]
            seen = pos <= p
            if window:
                seen &= (pos > p - window) | (pos < sinks)
            score.masked_fill_(~seen[None, :, None], -math.inf)
            top = score.amax(dim=3, keepdim=True)
            w = score.sub_(top).exp_()
            total = w.sum(dim=3, keepdim=True)
            lse = (torch.log(total) + top)[..., 0]
            o = torch.bmm(w.view(KH, -1, pos.numel()), v).view(KH, j - i, G, D) / total
            s["out"][at + i:at + j] = o.permute(1, 0, 2, 3).reshape(j - i, H, D).to(s["out"].dtype)
            s["lse"][at + i:at + j] = lse.permute(1, 0, 2).reshape(j - i, H)
        at += m
    return s["out"], s["lse"]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _values64(s, b, half, index):
    """float64 [len(index), kv_heads * head_dim] values of a request's positions."""
    case = s["case"]
    ps, width = case["page_size"], case["kv_heads"] * case["head_dim"]
    flat = (s["table"][b].long()[index // ps] * 2 + half) * ps + index % ps
    rows = s["pool"].view(-1, width)[flat].double()
    if s["scales"] is not None:
        col = torch.arange(width, device="cuda") // BLOCK
        rows *= s["scales"].view(-1, s["scales"].shape[-1])[flat].double()[:, col]
    return rows


def exact(case, seed):
    s = prepare(case, seed)
    KH, D, ps = case["kv_heads"], case["head_dim"], case["page_size"]
    if case["op"] == "read":
        k, v = s["k_out"].double(), s["v_out"].double()
        ends = np.cumsum(s["lens"] - s["new"])
        for b, end in enumerate(ends.tolist()):
            index = torch.arange(int(s["new"][b]), int(s["lens"][b]), device="cuda")
            k[end - len(index):end] = _values64(s, b, 0, index).view(-1, KH, D)
            v[end - len(index):end] = _values64(s, b, 1, index).view(-1, KH, D)
        return k, v
    if case["op"] == "write":
        width, rope, half = KH * D, case["rope"], case["half"]
        pool = s["pool"].double().view(-1, width)
        scales = None if s["scales"] is None else s["scales"].double().view(-1, s["scales"].shape[-1])
        ends = np.cumsum(s["new"])
        for b, end in enumerate(ends.tolist()):
            m = int(s["new"][b])
            where = int(s["lens"][b]) + torch.arange(m, device="cuda")
            k, v = s["k"][end - m:end].double(), s["v"][end - m:end].double()
            if rope:
                first = D - rope + torch.arange(rope // 2, device="cuda") * (1 if half else 2)
                second = first + (rope // 2 if half else 1)
                tab = s["freqs"].double()[where].view(m, 1, rope // 2, 2)
                z = torch.complex(k[..., first], k[..., second]) * torch.complex(tab[..., 0], tab[..., 1])
                k[..., first], k[..., second] = z.real, z.imag
            for side, x in ((0, k), (1, v)):
                flat = (s["table"][b].long()[where // ps] * 2 + side) * ps + where % ps
                x = x.reshape(m, width)
                if scales is not None:
                    for j in range(scales.shape[1]):
                        part = x[:, j * BLOCK:(j + 1) * BLOCK]
                        step = part.abs().amax(dim=1) / CODES_MAX
                        step = torch.where(step > 0, step, torch.ones_like(step))
                        scales[flat, j] = step
                        x[:, j * BLOCK:(j + 1) * BLOCK] = part / step[:, None]
                pool[flat] = x
        pool = pool.view(s["pool"].shape)
        return pool if scales is None else (pool, scales.view(s["scales"].shape))
    H, window, sinks = case["heads"], case["window"], case["sinks"]
    if work(case)["flops"] > 1.5e13:
        return None
    G = H // KH
    out = torch.zeros((s["T"], H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], H), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["requests"]):
        n, m = int(s["lens"][b]), int(s["new"][b])
        group = max(1, (1 << 27) // (G * (n + m)))
        spot = torch.arange(n + m, device="cuda")
        rows_k, rows_v = _values64(s, b, 0, spot), _values64(s, b, 1, spot)
        for i0 in range(0, m, group):
            i1 = min(m, i0 + group)
            # the positions that some token of the group sees
            low = max(0, n + i0 + 1 - window) if window else 0
            keep = spot[(spot < n + i1) & ((spot >= low) | (spot < sinks))]
            p = n + torch.arange(i0, i1, device="cuda")
            back = p[:, None] - keep[None, :]
            hidden = back < 0
            if window:
                hidden |= (back >= window) & (keep[None, :] >= sinks)
            for h in range(KH):
                col = slice(h * D, (h + 1) * D)
                q = s["q"][at + i0:at + i1, h * G:(h + 1) * G].double().reshape(-1, D) * s["scale"]
                score = torch.matmul(q, rows_k[keep, col].t().contiguous()).view(i1 - i0, G, -1)
                score.masked_fill_(hidden[:, None], -math.inf)
                z = torch.logsumexp(score, dim=2)
                weight = torch.exp(score - z[:, :, None]).view(-1, keep.numel())
                out[at + i0:at + i1, h * G:(h + 1) * G] = torch.matmul(weight, rows_v[keep, col]).view(i1 - i0, G, D)
                lse[at + i0:at + i1, h * G:(h + 1) * G] = z
        at += m
    return out, lse
