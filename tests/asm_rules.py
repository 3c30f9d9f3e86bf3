"""Rules over the generated code of a kernel, for what the compiler cannot see in inline assembly.  Each
follows every path through the branches and returns the places that break it, as (line, text) pairs.

Wait states: one per instruction, N + 1 for s_nop N."""
import functools
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

from mla_paged_latent_page_amd import build as B

VMEM = ("global_", "buffer_", "flat_", "scratch_")


class Line:
    """One instruction (or the label of a branch target, opcode "label")."""

    def __init__(self, number, op, rest, inline):
        self.number, self.op, self.rest, self.inline = number, op, rest, inline
        self.succ, self.pred = [], []

    def __repr__(self):
        return f"({self.number}: {self.op} {self.rest})"

    @property
    def states(self):
        return int(self.rest, 0) + 1 if self.op == "s_nop" else 0 if self.op == "label" else 1

    @property
    def operands(self):
        return [x.strip() for x in re.findall(r"[^,\[]+(?:\[[^\]]*\])?", self.rest)]


def kernels(text):
    """{kernel: its lines, linked to the ones that can follow}."""
    out, code, inline = {}, None, False
    for number, line in enumerate(text.splitlines(), 1):
        m = re.match(r"^(_Z\w+):", line)
        if m:
            code = out[m[1]] = []
            continue
        if code is None:
            continue
        if line.startswith(".Lfunc_end"):
            code = None
            continue
        m = re.match(r"^(\.LBB\w+):", line)
        if m:
            code.append(Line(number, "label", m[1], False))
            continue
        if "#ASMSTART" in line or "#ASMEND" in line:
            inline = "#ASMSTART" in line
            continue
        op, _, rest = line.split(";")[0].strip().partition(" ")
        if re.match(r"^(s|v|ds|global|buffer|flat|scratch)_", op):
            code.append(Line(number, op, rest.strip(), inline))
    out = {k: v for k, v in out.items() if any(x.op == "s_endpgm" for x in v)}
    for code in out.values():
        at = {x.rest: x for x in code if x.op == "label"}
        for x, after in zip(code, code[1:] + [None]):
            assert x.op not in ("s_setpc_b64", "s_swappc_b64", "s_call_b64")   # paths that could not be followed
            if x.op == "s_branch" or x.op.startswith("s_cbranch"):
                x.succ.append(at[x.rest])
            if x.op not in ("s_branch", "s_endpgm") and after is not None:
                x.succ.append(after)
        for x in code:
            for y in x.succ:
                y.pred.append(x)
    return out


def _generated(src):
    r = subprocess.run([B.HIPCC, *B.FLAGS, "-I", os.path.join(B.ROOT, "include"), "--offload-device-only", "-S", "-o", "-",
                        src], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return kernels(r.stdout)


@functools.lru_cache(maxsize=None)
def generated():
    """{source file: its kernels} of the package, compiled with the package's flags."""
    src = B.sources()
    with ThreadPoolExecutor(max_workers=8) as ex:
        return dict(zip(map(os.path.basename, src), ex.map(_generated, src)))


def loads_into_lds(code):
    return [x for x in code if "load_lds" in x.op or x.op.startswith("buffer_load") and re.search(r"\blds\b", x.rest)]


def m0_just_written(code):
    """Loads into LDS with a write of m0, which holds their destination, as the instruction before: one wait state has to
    lie between them."""
    def before(x, seen):
        for y in x.pred:
            if y.op != "label":
                yield y
            elif y not in seen:
                yield from before(y, seen | {y})
    return [(x, y) for x in loads_into_lds(code) for y in before(x, frozenset())
            if y.op.startswith(("s_", "v_")) and y.operands[:1] == ["m0"]]


def pending_stores(code, written_waits=False):
    """Barriers that a wave can reach with a store into LDS still in flight.

    LDS operations end in order: a wait for at most N of them ends every store with N or more behind it.
    ``written_waits``: only the waits written in the source count, at barriers written there, so that the
    result does not rest on what the compiler happens to wait for."""
    NONE = 1 << 30
    least = {code[0]: NONE}       # LDS operations behind the last store in flight, the least over all paths
    todo = [code[0]]
    while todo:
        x = todo.pop()
        behind = least[x]
        if x.op.startswith("ds_"):
            if not re.match(r"ds_(read|bpermute|permute|swizzle)", x.op):
                behind = 0
            elif behind != NONE:
                behind += 1
        elif x.op == "s_waitcnt" and (x.inline or not written_waits):
            m = re.search(r"lgkmcnt\((\d+)\)", x.rest)
            if m and behind >= int(m[1]):
                behind = NONE
        for y in x.succ:
            if behind < least.get(y, NONE + 1):
                least[y] = behind
                todo.append(y)
    return [x for x in code if x.op == "s_barrier" and (x.inline or not written_waits) and least.get(x, NONE) != NONE]


def scalars(text):
    """Names of the scalar registers that an operand (or operand list) holds."""
    out = set()
    for lo, hi in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out.update(range(int(lo), int(hi) + 1))
    out.update(int(n) for n in re.findall(r"\bs(\d+)\b", text))
    return out | ({"vcc"} if re.search(r"\bvcc", text) else set())


def written_by_vector(x):
    """Scalar registers that a vector instruction writes."""
    if x.op.startswith(("v_readfirstlane", "v_readlane", "v_cmp_")):
        return scalars(x.operands[0])
    if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale|v_mad_[ui]64", x.op):
        return scalars(x.operands[1])
    return set()


def written_by_scalar(x):
    if not x.op.startswith("s_") or x.op.startswith(("s_cmp", "s_bitcmp", "s_cbranch", "s_waitcnt", "s_nop", "s_barrier")):
        return set()
    return scalars(x.operands[0]) if x.operands else set()


def scalars_just_written(code, states=5):
    """Memory instructions that read a scalar register which a vector instruction wrote less than 5 wait states before."""
    bad = []
    for x in code:
        if not x.op.startswith(VMEM) or not scalars(x.rest):
            continue
        todo, had = [(y, 0, frozenset(scalars(x.rest))) for y in x.pred], set()
        while todo:
            y, waited, regs = todo.pop()
            if waited >= states or (y, waited, regs) in had:
                continue
            had.add((y, waited, regs))
            if written_by_vector(y) & regs:
                bad.append((x, y))
                continue
            regs -= written_by_scalar(y)
            if regs:
                todo += [(z, waited + y.states, regs) for z in y.pred]
    return bad
