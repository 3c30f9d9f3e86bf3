"""The matrix instructions that tree_attention_mfma.hip issues from inline assembly, in the
generated code: the compiler does not know them as such, so it inserts no waits for them and may
place copies of their sums anywhere.  Checked for each one whose result is in ordinary registers
(8 passes; wait states: one per instruction, N + 1 for s_nop N):

  * for 12 wait states nothing touches its result, except a matrix instruction that takes exactly
    that result as its addend (and, if it writes any of it, all of it);
  * its operands were not written by a vector instruction in the 2 wait states before it."""
import os
import re
import subprocess

import pytest

from mla_paged_latent_page_amd import build as B

RESULT_WAIT, OPERAND_WAIT = 12, 2


def registers(text):
    """Numbers of the ordinary vector registers an operand (or operand list) names."""
    out = set()
    for lo, hi in re.findall(r"\bv\[(\d+):(\d+)\]", text):
        out.update(range(int(lo), int(hi) + 1))
    out.update(int(n) for n in re.findall(r"\bv(\d+)\b", text))
    return out


def instructions(text):
    """(kernel, opcode, operands) of each instruction; opcode "label" for a branch target."""
    kernel = None
    for line in text.splitlines():
        m = re.match(r"^(_Z\w*tree_attention_mfma\w*):", line)
        if m:
            kernel = m[1]
        if kernel is None:
            continue
        if re.match(r"^\.LBB\w+:", line):
            yield kernel, "label", ""
            continue
        code = line.split(";")[0].strip()
        if not code or code.startswith("."):
            continue
        op, _, rest = code.partition(" ")
        yield kernel, op, rest
        if op == "s_endpgm":
            kernel = None


def states(op, rest):
    return int(rest) + 1 if op == "s_nop" else 0 if op == "label" else 1


def split(rest):
    return [x.strip() for x in re.findall(r"[^,\[]+(?:\[[^\]]*\])?", rest)]


def violations(stream):
    bad, seen = [], 0
    stream = list(stream)
    for i, (kernel, op, rest) in enumerate(stream):
        if not op.startswith("v_mfma"):
            continue
        dst, a, b, c = split(rest)[:4]
        if not dst.startswith("v"):
            continue
        seen += 1
        result = registers(dst)
        # operands
        waited = 0
        for k in range(i - 1, -1, -1):
            if waited >= OPERAND_WAIT or stream[k][0] != kernel:
                break
            o, r = stream[k][1], stream[k][2]
            if o.startswith("v_") and not o.startswith("v_mfma") and not o.startswith("v_cmp"):
                if registers(split(r)[0]) & (registers(a) | registers(b)):
                    bad.append((kernel, i, "operand just written", o, r, rest))
            waited += states(o, r)
        # result
        waited = 0
        for k in range(i + 1, len(stream)):
            if waited >= RESULT_WAIT or stream[k][0] != kernel:
                break
            o, r = stream[k][1], stream[k][2]
            if o in ("s_branch", "s_cbranch_scc0", "s_cbranch_scc1", "s_cbranch_vccz", "s_cbranch_vccnz",
                     "s_cbranch_execz", "s_cbranch_execnz", "s_endpgm", "label"):
                bad.append((kernel, i, "result open at a branch", o, r, rest))
                break
            touched = registers(r) & result
            if touched:
                if o.startswith("v_mfma"):
                    d2, a2, b2, c2 = split(r)[:4]
                    if (registers(a2) | registers(b2)) & result or registers(c2) != result or \
                            (registers(d2) & result and registers(d2) != result):
                        bad.append((kernel, i, "result misused", o, r, rest))
                    break      # the next one of the chain is checked by itself
                bad.append((kernel, i, "result touched", o, r, rest))
                break
            waited += states(o, r)
    return bad, seen


def test_the_rules_see_mistakes():
    head = "_Z1tree_attention_mfma1:\n"
    chain = " v_mfma_f32_32x32x16_bf16 v[0:15], v[16:19], v[20:23], 0\n" \
            " v_mfma_f32_32x32x16_bf16 v[0:15], v[24:27], v[20:23], v[0:15]\n"
    ok = head + chain + " s_nop 13\n v_mov_b32_e32 v30, v0\n s_endpgm\n"
    assert violations(instructions(ok)) == ([], 2)
    for text in (chain + " s_nop 9\n v_mov_b32_e32 v30, v0\n s_endpgm\n",
                 chain + " v_mov_b64_e32 v[40:41], v[2:3]\n s_nop 13\n s_endpgm\n",
                 chain + " s_cbranch_scc1 .LBB0_1\n s_endpgm\n",
                 " v_mov_b32_e32 v17, v1\n" + chain + " s_nop 13\n s_endpgm\n",
                 " v_mfma_f32_32x32x16_bf16 v[0:15], v[16:19], v[20:23], 0\n"
                 " v_mfma_f32_32x32x16_bf16 v[8:23], v[24:27], v[28:31], v[0:15]\n s_nop 13\n s_endpgm\n"):
        assert violations(instructions(head + text))[0]


def test_generated_code(tmp_path):
    if not os.path.exists(B.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "k.s"
    src = os.path.join(B.SRC_DIR, "tree_attention_mfma.hip")
    r = subprocess.run([B.HIPCC, *B.FLAGS, "-I", os.path.join(B.ROOT, "include"), "--offload-device-only", "-S", "-o",
                        str(out), src], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = out.read_text()
    bad, seen = violations(instructions(text))
    assert seen >= 4 * 2 * 36          # four variants, a first tile and a loop of 36 products each
    assert not bad, bad[:3]
