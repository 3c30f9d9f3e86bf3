"""The operators of a speculative-decoding step over the paged MLA cache, as measured cases.

A step drafts a tree of tokens per request.  Its queries are rotated at each token's
depth in the tree and its latent rows are rotated and written behind the cached ones
(``rope``, from tables that ``freqs`` builds); attention reads cached and drafted rows
(``attention``); the rows of the accepted tokens are moved together (``compact``); and
requests that branch share their pages (``fork``).

Every case is a dict of plain values: ``op`` names the operator, ``layout`` seeds the
ragged sizes (lengths, tokens per request), so that the work of a case does not depend on
the seed its values are drawn from.
"""
import math

import numpy as np
import torch

own = False

LATENT, ROPE = 512, 64          # the cache row of the workloads: 512 latent + 64 rope columns
ROW = LATENT + ROPE
NOPE = 128                      # non-rope columns of a query head
BLOCK = 128                     # columns per scale of an e4m3 cache
PAGE_NONE = -1                  # 0xFFFFFFFF as int32: an unused page-table entry


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # A decode step's rotations on one of eight tensor-parallel ranks: latency counts.
        dict(name="rope_step", op="rope", requests=16, tokens_lo=1, tokens_hi=8, heads=16, len_lo=100,
             len_hi=8000, page_size=16, half=False, dtype="bf16", layout=11),
        # A prefill chunk of all 128 heads, half layout.
        dict(name="rope_chunk", op="rope", requests=5, tokens_lo=1000, tokens_hi=2100, heads=128, len_lo=1,
             len_hi=20000, page_size=128, half=True, dtype="bf16", layout=12),
        # The rows a growing context adds to a linearly scaled table.
        dict(name="freqs_rows", op="freqs", first=60000, rows=8191, dim=64, scaling="linear", factor=8.0),
        # A whole long-context table, frequencies scaled by parts.
        dict(name="freqs_table", op="freqs", first=0, rows=262144, dim=128, scaling="by_parts", factor=40.0),
        # Few requests, one token each, one rank's 16 heads, short contexts: latency counts.
        dict(name="attend_step_small", op="attention", requests=4, tokens_lo=1, tokens_hi=1, heads=16, len_lo=100,
             len_hi=1000, page_size=16, mask="chain", cache="bf16", layout=21),
        # The 64-request decode batch (lengths up to 4096), one token each, all heads.
        dict(name="attend_decode", op="attention", requests=64, tokens_lo=1, tokens_hi=1, heads=128, len_lo=256,
             len_hi=4096, page_size=128, mask="chain", cache="bf16", layout=22),
        # Drafted trees of 17 to 40 tokens per request, all heads: bound by the matrix cores.
        dict(name="attend_tree", op="attention", requests=12, tokens_lo=17, tokens_hi=40, heads=128, len_lo=1000,
             len_hi=8192, page_size=64, mask="tree", cache="bf16", layout=23),
        # Long contexts in an e4m3 cache, small trees, one rank's 16 heads.
        dict(name="attend_long_e4m3", op="attention", requests=5, tokens_lo=3, tokens_hi=8, heads=16, len_lo=60000,
             len_hi=131072, page_size=128, mask="tree", cache="e4m3", layout=24),
        # Accepted paths of a small batch moved together.
        dict(name="compact_small", op="compact", requests=8, drafted=16, layers=4, page_size=16, cache="bf16",
             len_hi=2000, layout=31),
        # The same for a large batch over many layers of an e4m3 cache and its scales.
        dict(name="compact_batch_e4m3", op="compact", requests=128, drafted=48, layers=24, page_size=64,
             cache="e4m3", len_hi=500, layout=32),
        # Losing beams freed and the winners forked into their place.
        dict(name="fork_beams", op="fork", parents=4, children=12, layers=4, page_size=16, cache="bf16",
             len_hi=1500, layout=41),
        # Parallel samples of long prompts forked, many layers and large pages.
        dict(name="fork_samples", op="fork", parents=16, children=112, layers=16, page_size=128, cache="bf16",
             len_hi=2500, layout=42),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "rope", "freqs", "compact", "fork"])
    layout = rng.randrange(1 << 30)
    page_size = rng.choice([16, 32, 64, 128, 128, 100])
    if op == "rope":
        tokens = _log_int(rng, 1, 2000)
        return dict(op=op, requests=rng.randint(1, 5), tokens_lo=max(1, tokens // 3), tokens_hi=tokens,
                    heads=rng.choice([16, 20, 32, 64, 128]), len_lo=1, len_hi=_log_int(rng, 2, 30000),
                    page_size=page_size, half=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    layout=layout)
    if op == "freqs":
        return dict(op=op, first=rng.choice([0, rng.randrange(100000)]), rows=_log_int(rng, 1, 262144),
                    dim=rng.choice([8, 32, 64, 96, 128]), scaling=rng.choice(["none", "linear", "by_parts"]),
                    factor=rng.uniform(1.0, 40.0))
    if op == "compact":
        return dict(op=op, requests=_log_int(rng, 1, 128), drafted=rng.randint(1, 48), layers=rng.randint(1, 24),
                    page_size=page_size, cache=rng.choice(["bf16", "e4m3", "f32"]), len_hi=_log_int(rng, 2, 300),
                    layout=layout)
    if op == "fork":
        return dict(op=op, parents=rng.randint(1, 16), children=_log_int(rng, 1, 112), layers=rng.randint(1, 12),
                    page_size=page_size, cache=rng.choice(["bf16", "e4m3"]), len_hi=_log_int(rng, 2, 2000),
                    layout=layout)
    mask = rng.choice(["tree", "tree", "chain"])
    case = dict(op=op, requests=_log_int(rng, 1, 96), tokens_lo=1, tokens_hi=1, heads=0, len_lo=1, len_hi=0,
                page_size=page_size, mask=mask, cache=rng.choice(["bf16", "bf16", "e4m3"]), layout=layout)
    case["heads"] = rng.choice([16, 16, 20, 32, 64, 128, 128])
    case["tokens_hi"] = rng.choice([1, rng.randint(2, 16), rng.randint(2, 64)])
    if mask == "chain" and rng.random() < 0.4:
        case["tokens_hi"] = rng.randint(65, 600)
    case["len_hi"] = _log_int(rng, 2, 100000)
    case["len_lo"] = max(1, case["len_hi"] // rng.choice([1, 4, 30]))
    limit = work(listed()[6])["flops"]
    while case["requests"] > 1 and (work(case)["flops"] > limit or case["requests"] * case["len_hi"] > 600000):
        case["requests"] = (case["requests"] + 1) // 2
    while work(case)["flops"] > limit:
        case["len_hi"] = max(2, case["len_hi"] // 2)
        case["len_lo"] = min(case["len_lo"], case["len_hi"])
        case["tokens_hi"] = max(1, case["tokens_hi"] * 3 // 4)
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
    new = r.integers(case["tokens_lo"], case["tokens_hi"], size=case["requests"], endpoint=True)
    return lens, new


def _accepted_counts(case):
    r = np.random.default_rng(case["layout"])
    lens = r.integers(1, case["len_hi"], size=case["requests"], endpoint=True)
    counts = r.integers(0, min(8, (case["drafted"] + 1) // 2), size=case["requests"], endpoint=True)
    return lens, counts


def _fork_sizes(case):
    r = np.random.default_rng(case["layout"])
    lens = r.integers(1, case["len_hi"], size=case["parents"], endpoint=True)
    parent_of = r.integers(0, case["parents"], size=case["children"])
    return lens, parent_of


_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def _row_bytes(cache):
    return ROW * _BYTES[cache] + (4 * -(-ROW // BLOCK) if cache == "e4m3" else 0)


def work(case):
    op = case["op"]
    if op == "rope":
        _, new = _lengths(case)
        T, eb = int(new.sum()), _BYTES[case["dtype"]]
        rows = 2 * T * case["heads"] * (NOPE + ROPE) * eb + 2 * T * ROW * 2
        return dict(bytes=rows + T * ROPE * 4 + T * 4, flops=T * (case["heads"] * 3 * ROPE + 4 * LATENT + 3 * ROPE))
    if op == "freqs":
        return dict(bytes=case["rows"] * case["dim"] * 4, flops=case["rows"] * case["dim"] // 2 * 40)
    if op == "attention":
        lens, new = _lengths(case)
        H, T = case["heads"], int(new.sum())
        pairs = int((lens * new).sum()) + T
        return dict(bytes=int((lens + new).sum()) * _row_bytes(case["cache"]) + T * H * (ROW + LATENT) * 2 + T * H * 4,
                    flops=2 * H * pairs * (ROW + LATENT))
    if op == "compact":
        _, counts = _accepted_counts(case)
        # the first accepted token stays where it is, the later ones move
        moved = int(np.maximum(counts - 1, 0).sum()) * case["layers"]
        return dict(bytes=2 * moved * _row_bytes(case["cache"]) + int(counts.sum()) * 4, flops=0)
    lens, parent_of = _fork_sizes(case)
    ps = case["page_size"]
    pages = -(-lens // ps)
    partial = int((lens % ps)[parent_of].sum()) * case["layers"]
    entries = int(pages[parent_of].sum())
    # per shared page: two table entries and a count each for fork and free
    return dict(bytes=2 * partial * _row_bytes(case["cache"]) + entries * 4 * 8, flops=0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int64).astype(np.uint32)).view(np.int32)).cuda()


def _normal(g, shape, dtype=torch.float32, std=1.0):
    """Normal values made in pieces, so that a large pool never exists in 32 bits."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for lo in range(0, flat.numel(), 1 << 27):
        hi = min(lo + (1 << 27), flat.numel())
        flat[lo:hi] = torch.randn(hi - lo, generator=g, device="cuda") * std
    return out


def _pool(g, cache, pages, layers, page_size):
    """[pages, layers, 1, page_size, 1, 576] rows about N(0, 1), and an e4m3 pool's scales."""
    shape = (pages, layers, 1, page_size, 1, ROW)
    if cache == "f32":
        return _normal(g, shape), None
    if cache == "bf16":
        return _normal(g, shape, torch.bfloat16), None
    pool = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    flat = pool.view(-1)
    for lo in range(0, flat.numel(), 1 << 27):
        hi = min(lo + (1 << 27), flat.numel())
        v = torch.randn(hi - lo, generator=g, device="cuda") * 100.0
        flat[lo:hi] = v.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    scales = torch.rand((pages, layers, 1, page_size, -(-ROW // BLOCK)), generator=g, device="cuda")
    return pool, scales * 0.004 + 0.008


def _table(r, pages_needed, spare):
    pages = int(sum(pages_needed)) + spare
    perm = r.permutation(pages)
    table = np.full((len(pages_needed), max(1, max(pages_needed))), 0xFFFFFFFF, np.int64)
    at = 0
    for b, n in enumerate(pages_needed):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pages, perm[at:]


def _trees(r, new):
    """Parent of each drafted token (-1: the cached context), and its depth."""
    parents, depths = [], []
    for n in new:
        par, dep = [], []
        for i in range(int(n)):
            p = -1 if i == 0 else int(r.integers(max(-1, i - 6), i))
            par.append(p)
            dep.append(0 if p < 0 else dep[p] + 1)
        parents.append(par)
        depths.append(dep)
    return parents, depths


def _mask_words(parents, words):
    rows = []
    for par in parents:
        seen = []
        for i, p in enumerate(par):
            seen.append((seen[p] if p >= 0 else 0) | (1 << i))
        rows += [[(m >> (64 * w)) & 0xFFFFFFFFFFFFFFFF for w in range(words)] for m in seen]
    return torch.from_numpy(np.array(rows, np.uint64).reshape(len(rows), words).view(np.int64)).cuda()


def _freqs(rows, dim):
    """A [rows, dim] table of (cos, sin) pairs, base 10000."""
    j = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    ang = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2.0 * j / dim)
    return torch.stack([ang.cos(), ang.sin()], dim=2).reshape(rows, dim).float()


def prepare(case, seed):
    op, g, r = case["op"], _gen(seed), np.random.default_rng(int(seed) + 101)
    s = dict(case=case)
    if op == "freqs":
        # the theta of a deployment and the amplitude that long contexts are scaled by
        s.update(theta=10000.0 * (1.0 + 0.25 * float(r.random())), amplitude=1.0 + 0.3 * float(r.random()),
                 out=torch.empty((case["rows"], case["dim"]), device="cuda"))
        return s
    if op == "rope":
        lens, new = _lengths(case)
        T, H = int(new.sum()), case["heads"]
        ps = case["page_size"]
        table, pages, _ = _table(r, [-(-int(l + n) // ps) for l, n in zip(lens, new)], 2)
        _, depths = _trees(r, new)
        pos = np.concatenate([l + np.array(d, np.int64) for l, d in zip(lens, depths)])
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        pool = torch.zeros((pages, 1, 1, ps, 1, ROW), dtype=torch.bfloat16, device="cuda")
        s.update(q=_normal(g, (T, H, NOPE + ROPE), dt), q_out=torch.empty((T, H, NOPE + ROPE), dtype=dt, device="cuda"),
                 x=_normal(g, (T, ROW), torch.bfloat16), gamma=torch.rand(LATENT, generator=g, device="cuda") + 0.5,
                 freqs=_freqs(int((lens + new).max()) + 1, ROPE), positions=_i32(pos), pool=pool, table=_i32(table),
                 lengths=_i32(lens), offsets=_i32(np.concatenate([[0], np.cumsum(new)])), lens=lens, new=new, T=T)
        return _with_cache(s)
    if op == "attention":
        lens, new = _lengths(case)
        T, H, ps = int(new.sum()), case["heads"], case["page_size"]
        table, pages, _ = _table(r, [-(-int(l + n) // ps) for l, n in zip(lens, new)], 2)
        pool, scales = _pool(g, case["cache"], pages, 1, ps)
        mask = None
        if case["mask"] == "tree":
            mask = _mask_words(_trees(r, new)[0], -(-int(new.max()) // 64))
        s.update(q=_normal(g, (T, H, ROW), torch.bfloat16, 0.6), pool=pool, scales=scales, table=_i32(table),
                 lengths=_i32(lens), offsets=_i32(np.concatenate([[0], np.cumsum(new)])), lens=lens, new=new, T=T,
                 mask=mask, scale=(NOPE + ROPE) ** -0.5,
                 out=torch.empty((T, H, LATENT), dtype=torch.bfloat16, device="cuda"),
                 lse=torch.empty((T, H), device="cuda"))
        s = _with_cache(s)
        if own:
            import mla_paged_latent_page_amd as mp
            size = mp.mla_tree_attention_workspace_size(T, H, LATENT)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return s
    if op == "compact":
        lens, counts = _accepted_counts(case)
        ps = case["page_size"]
        table, pages, _ = _table(r, [-(-int(l + case["drafted"]) // ps) for l in lens], 2)
        pool, scales = _pool(g, case["cache"], pages, case["layers"], ps)
        picks = []
        for c in counts:
            # the first drafted token, then a path through the later ones; no row that is moved lies
            # where another one goes, so that a second pass on the same pool changes nothing
            rest = r.permutation(case["drafted"] - int(c))[:max(0, int(c) - 1)] + int(c)
            picks.append(np.sort(np.concatenate([[0], rest]))[:int(c)].astype(np.int64))
        s.update(pool=pool, scales=scales, table=_i32(table), lengths=_i32(lens), lens=lens, picks=picks,
                 accepted=_i32(np.concatenate(picks + [np.zeros(0, np.int64)])),
                 offsets=_i32(np.concatenate([[0], np.cumsum(counts)])))
        return _with_cache(s)
    # fork: the slots after the parents hold the children of the step before, which are freed
    lens, parent_of = _fork_sizes(case)
    ps, P, C = case["page_size"], case["parents"], case["children"]
    need = [-(-int(l) // ps) for l in lens]
    table, pages, spare = _table(r, need, C + 3)
    fresh = spare[:C]
    full = np.full((P + C, table.shape[1]), 0xFFFFFFFF, np.int64)
    full[:P] = table
    all_lens = np.concatenate([lens, lens[parent_of]])
    refs = np.zeros(pages, np.int64)
    for p in range(P):
        refs[table[p, :need[p]]] += 1
    for c, p in enumerate(parent_of):
        shared = int(lens[p]) // ps
        full[P + c, :shared] = table[p, :shared]
        refs[table[p, :shared]] += 1
        if int(lens[p]) % ps:
            full[P + c, shared] = fresh[c]
            refs[fresh[c]] += 1
    pool, scales = _pool(g, case["cache"], pages, case["layers"], ps)
    s.update(pool=pool, scales=scales, table=_i32(full), lengths=_i32(all_lens), parents=_i32(parent_of),
             children=_i32(np.arange(P, P + C)), new_pages=_i32(fresh), refs=_i32(refs),
             free_list=torch.full((pages,), PAGE_NONE, dtype=torch.int32, device="cuda"),
             free_count=torch.zeros(1, dtype=torch.int32, device="cuda"),
             lens=lens, parent_of=parent_of, fresh=fresh)
    return _with_cache(s)


def _with_cache(s):
    if own:
        import mla_paged_latent_page_amd as mp
        s["cache"] = mp.PagedKVCache(s["pool"], s["table"], s["lengths"], scales=s.get("scales"))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import mla_paged_latent_page_amd as mp
    case = s["case"]
    op = case["op"]
    if op == "rope":
        layout = "half" if case["half"] else "interleaved"
        mp.mla_rope_q(s["q"], s["positions"], s["freqs"], s["q_out"], d_nope=NOPE, layout=layout)
        mp.mla_write_latent_paged_at(s["x"], s["offsets"], s["positions"], s["gamma"], 1e-6, s["freqs"], LATENT,
                                     s["cache"], 0, layout=layout)
        return s["q_out"], s["pool"]
    if op == "freqs":
        mp.mla_rope_freqs(s["out"], theta=s["theta"], first_position=case["first"], scaling=case["scaling"],
                          factor=case["factor"], original_max_position=4096, beta_fast=32.0, beta_slow=1.0,
                          amplitude=s["amplitude"])
        return s["out"]
    if op == "attention":
        call = mp.mla_tree_attention_paged if s["scales"] is None else mp.mla_tree_attention_paged_fp8_cache
        call(s["q"], s["offsets"], s["mask"], s["scale"], LATENT, s["cache"], 0, s["out"], s["workspace"],
             lse=s["lse"])
        return s["out"], s["lse"]
    if op == "compact":
        mp.mla_compact_paged(s["accepted"], s["offsets"], s["cache"])
        return (s["pool"],) if s["scales"] is None else (s["pool"], s["scales"])
    s["free_count"].zero_()   # the pages listed by the step before have been taken
    mp.mla_free_paged(s["children"], s["refs"], s["free_list"], s["free_count"], s["cache"])
    mp.mla_fork_paged(s["parents"], s["children"], s["new_pages"], s["refs"], s["cache"])
    out = (s["pool"], s["table"], s["lengths"], s["refs"], s["free_list"], s["free_count"])
    return out if s["scales"] is None else out + (s["scales"],)


def _rows_of(s, b, positions):
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


def _frequencies(case, theta):
    """The rotation frequencies in 64 bits: theta^(-2j/dim), divided by the factor (linear),
    or divided only where fewer than beta_slow turns fit the original 4096 positions, kept
    where more than beta_fast do, and mixed linearly in j between (by parts)."""
    dim = case["dim"]
    j = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    f = theta ** (-2.0 * j / dim)
    if case["scaling"] == "none":
        return f
    if case["scaling"] == "linear":
        return f / case["factor"]

    def pair_with(turns):
        return dim * math.log(4096 / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))
    low, high = max(math.floor(pair_with(32.0)), 0), min(math.ceil(pair_with(1.0)), dim - 1)
    ramp = ((j - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return f / case["factor"] * ramp + f * (1.0 - ramp)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        table = s["freqs"][s["positions"].long()]
        cos, sin = table[:, 0::2], table[:, 1::2]
        q = s["q"].float()
        rot = _rotate(q[..., NOPE:], cos[:, None], sin[:, None], case["half"])
        s["q_out"].copy_(torch.cat([q[..., :NOPE], rot], dim=-1))
        x = s["x"].float()
        lat = x[:, :LATENT]
        lat = s["gamma"] * lat / torch.sqrt((lat * lat).mean(dim=1, keepdim=True) + 1e-6)
        rows = torch.cat([lat, _rotate(x[:, LATENT:], cos, sin, case["half"])], dim=1).to(torch.bfloat16)
        at = 0
        for b, n in enumerate(s["new"]):
            pos = torch.arange(int(s["lens"][b]), int(s["lens"][b]) + int(n), device="cuda")
            page, slot = _rows_of(s, b, pos)
            s["pool"][page, 0, 0, slot, 0] = rows[at:at + int(n)]
            at += int(n)
        return s["q_out"], s["pool"]
    if op == "freqs":
        pos = torch.arange(case["first"], case["first"] + case["rows"], dtype=torch.float64, device="cuda")
        ang = pos[:, None] * _frequencies(case, s["theta"])
        s["out"].copy_((torch.stack([ang.cos(), ang.sin()], dim=2) * s["amplitude"]).flatten(1))
        return s["out"]
    if op == "attention":
        at = 0
        for b, n in enumerate(s["new"]):
            n, L = int(n), int(s["lens"][b]) + int(n)
            page, slot = _rows_of(s, b, torch.arange(L, device="cuda"))
            rows = s["pool"][page, 0, 0, slot, 0].float()
            if s["scales"] is not None:
                sc = s["scales"][page, 0, 0, slot]
                rows = rows * sc.repeat_interleave(BLOCK, dim=1)[:, :ROW]
            q = s["q"][at:at + n].float().reshape(-1, ROW)
            score = (q @ rows.t() * s["scale"]).view(n, case["heads"], L)
            score[:, :, L - n:].masked_fill_(~_draft_mask(s, at, n)[:, None], -math.inf)
            top = score.amax(dim=2, keepdim=True)
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            p = torch.exp(score - top)
            total = p.sum(dim=2, keepdim=True)
            s["lse"][at:at + n] = (torch.log(total) + top)[:, :, 0]
            p = p / torch.where(total == 0, torch.ones_like(total), total)
            o = p.view(n * case["heads"], L) @ rows[:, :LATENT]
            s["out"][at:at + n] = o.view(n, case["heads"], LATENT).to(torch.bfloat16)
            at += n
        return s["out"], s["lse"]
    if op == "compact":
        for b, picks in enumerate(s["picks"]):
            if len(picks) == 0:
                continue
            src = torch.from_numpy(picks).cuda() + int(s["lens"][b])
            dst = torch.arange(len(picks), device="cuda") + int(s["lens"][b])
            for pool in (s["pool"], s["scales"]):
                if pool is not None:
                    raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
                    raw[_at(s, b, dst)] = raw[_at(s, b, src)]
        return (s["pool"],) if s["scales"] is None else (s["pool"], s["scales"])
    return _fork_plain(s)


def _at(s, b, positions):
    """Index of the token rows of every layer: [tokens, layers, ...]."""
    page, slot = _rows_of(s, b, positions)
    layer = torch.arange(s["case"]["layers"], device="cuda")
    return page[:, None], layer[None, :], 0, slot[:, None]


def _draft_mask(s, at, n):
    """Which of a request's n drafted tokens each of them sees."""
    i = torch.arange(n, device="cuda")
    if s["mask"] is None:
        return i[:, None] >= i[None, :]
    words = s["mask"][at:at + n]
    return (words[:, i // 64] >> (i % 64)) & 1 != 0


def _fork_plain(s):
    case = s["case"]
    ps, P = case["page_size"], case["parents"]
    table, refs, lengths = s["table"], s["refs"], s["lengths"]
    s["free_count"].zero_()
    # free: one reference less for every page of the freed requests; pages left with none are listed in order
    kids = s["children"].long()
    rows, lens = table[kids], lengths[kids].long()
    held = torch.arange(table.shape[1], device="cuda")[None, :] < (-(-lens // ps))[:, None]
    ids = rows[held].long()
    before = refs.clone()
    refs.index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    freed = torch.nonzero((refs == 0) & (before > 0)).flatten()
    s["free_list"][:freed.numel()] = freed.int()
    s["free_count"] += freed.numel()
    table[kids] = torch.where(held, torch.full_like(rows, PAGE_NONE), rows)
    lengths[kids] = 0
    # fork: whole pages are shared, the partly filled last one is copied
    for c, p in enumerate(s["parent_of"]):
        n = int(s["lens"][p])
        shared, part = n // ps, n % ps
        table[P + c, :shared] = table[p, :shared]
        refs[table[p, :shared].long()] += 1
        if part:
            src, dst = table[p, shared].long(), int(s["fresh"][c])
            table[P + c, shared] = dst
            refs[dst] = 1
            for pool in (s["pool"], s["scales"]):
                if pool is not None:
                    raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
                    raw[dst, :, :, :part] = raw[src, :, :, :part]
        lengths[P + c] = n
    out = (s["pool"], table, lengths, refs, s["free_list"], s["free_count"])
    return out if s["scales"] is None else out + (s["scales"],)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op in ("compact", "fork"):
        return None   # copies and whole numbers: nothing is computed
    s = prepare(case, seed)
    if op == "freqs":
        out = torch.empty((case["rows"], case["dim"]), dtype=torch.float64, device="cuda")
        p = case["first"] + torch.arange(case["rows"], dtype=torch.float64, device="cuda")
        turns = [case["dim"] * math.log(4096 / (t * math.tau)) / (2 * math.log(s["theta"])) for t in (32.0, 1.0)]
        lo, hi = max(math.floor(turns[0]), 0), min(math.ceil(turns[1]), case["dim"] - 1)
        for j in range(case["dim"] // 2):
            f = math.exp(-2.0 * j / case["dim"] * math.log(s["theta"]))
            if case["scaling"] == "linear":
                f /= case["factor"]
            elif case["scaling"] == "by_parts":
                mix = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
                f = f * (mix / case["factor"] + 1.0 - mix)
            out[:, 2 * j] = s["amplitude"] * torch.cos(p * f)
            out[:, 2 * j + 1] = s["amplitude"] * torch.sin(p * f)
        return out
    if op == "rope":
        dim, half = ROPE, case["half"]
        first = torch.arange(dim // 2, device="cuda") * (1 if half else 2)
        second = first + (dim // 2 if half else 1)
        tab = s["freqs"].double()[s["positions"].long()].view(s["T"], dim // 2, 2)
        turn = torch.complex(tab[..., 0], tab[..., 1])

        def turned(v):
            z = torch.complex(v[..., first], v[..., second]) * (turn if v.dim() == 2 else turn[:, None])
            w = torch.empty_like(v)
            w[..., first], w[..., second] = z.real, z.imag
            return w
        q = s["q"].double()
        q[..., NOPE:] = turned(q[..., NOPE:].clone())
        x = s["x"].double()
        x[:, LATENT:] = turned(x[:, LATENT:].clone())
        rms = x[:, :LATENT].square().sum(dim=1).div(LATENT).add(1e-6).rsqrt()
        x[:, :LATENT] *= rms[:, None] * s["gamma"].double()
        pool = s["pool"].double()
        offs = np.concatenate([[0], np.cumsum(s["new"])])
        for b in range(case["requests"]):
            n = int(s["new"][b])
            where = int(s["lens"][b]) + torch.arange(n, device="cuda")
            flat = s["table"][b].long()[where // case["page_size"]] * case["page_size"] + where % case["page_size"]
            pool.view(-1, ROW)[flat] = x[int(offs[b]):int(offs[b]) + n]
        return q, pool
    # attention, one request and a group of its tokens at a time
    if work(case)["flops"] > 2e13:
        return None
    out = torch.zeros((s["T"], case["heads"], LATENT), dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    flat_pool = s["pool"].view(-1, ROW)
    at = 0
    for b in range(case["requests"]):
        n, cached = int(s["new"][b]), int(s["lens"][b])
        spot = torch.arange(cached + n, device="cuda")
        flat = s["table"][b].long()[spot // case["page_size"]] * case["page_size"] + spot % case["page_size"]
        if s["scales"] is None:
            rows = flat_pool[flat].double()
        else:
            col = torch.arange(ROW, device="cuda") // BLOCK
            rows = flat_pool[flat].double() * s["scales"].view(-1, s["scales"].shape[-1])[flat].double()[:, col]
        group = max(1, (1 << 27) // (case["heads"] * (cached + n)))
        for i0 in range(0, n, group):
            i1 = min(n, i0 + group)
            score = torch.matmul(s["q"][at + i0:at + i1].double().reshape(-1, ROW) * s["scale"], rows.t().contiguous())
            score = score.view(i1 - i0, case["heads"], cached + n)
            for i in range(i0, i1):
                if s["mask"] is None:
                    hidden = list(range(i + 1, n))
                else:
                    words = [int(w) & 0xFFFFFFFFFFFFFFFF for w in s["mask"][at + i].tolist()]
                    hidden = [k for k in range(n) if not words[k // 64] >> (k % 64) & 1]
                if hidden:
                    score[i - i0][:, torch.tensor([cached + k for k in hidden], device="cuda")] = -math.inf
            z = torch.logsumexp(score, dim=2)
            lse[at + i0:at + i1] = z
            weight = torch.exp(score - z.clamp_min(-1e300)[:, :, None])
            out[at + i0:at + i1] = torch.matmul(weight.view(-1, cached + n), rows[:, :LATENT]).view(
                i1 - i0, case["heads"], LATENT)
        at += n
    return out, lse
