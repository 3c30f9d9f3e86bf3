"""Waits that inline assembly needs, in the generated code of the kernels that use it (tests/asm_rules.py)."""
import os

import pytest

from asm_rules import generated, kernels, loads_into_lds, m0_just_written, pending_stores, scalars_just_written
from mla_paged_latent_page_amd import build as B

needs_hipcc = pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="no hipcc")


def one(text):
    (code,) = kernels("_Z1k:\n" + text + "\ts_endpgm\n.Lfunc_end0:\n").values()
    return code


def written(text):
    return "\t;;#ASMSTART\n" + text + "\t;;#ASMEND\n"


STORE, READ = "\tds_write_b128 v0, v[4:7]\n", "\tds_read_b128 v[8:11], v1\n"
BARRIER8 = written("\ts_waitcnt lgkmcnt(8)\n\ts_barrier\n")


@pytest.mark.parametrize("text, any_wait, written_wait", [
    (STORE + BARRIER8, 1, 1),                                                    # the wait is missing
    (STORE + 7 * READ + BARRIER8, 1, 1),
    (STORE + 8 * READ + BARRIER8, 0, 0),                                         # reads behind it push it out
    (STORE + written("\ts_waitcnt lgkmcnt(0)\n") + BARRIER8, 0, 0),
    (STORE + "\ts_waitcnt lgkmcnt(0)\n" + BARRIER8, 0, 1),                       # a wait of the compiler's
    (STORE + "\ts_waitcnt vmcnt(0)\n" + BARRIER8, 1, 1),
    (STORE + "\ts_cbranch_vccz .LBB0_1\n" + 8 * READ + ".LBB0_1:\n" + BARRIER8, 1, 1),     # one path lacks them
    (".LBB0_1:\n" + BARRIER8 + STORE + "\ts_cbranch_scc1 .LBB0_1\n", 1, 1),      # round a loop
    (STORE + "\ts_waitcnt lgkmcnt(0)\n\ts_barrier\n", 0, 0),                     # __syncthreads
])
def test_pending_stores_are_seen(text, any_wait, written_wait):
    assert len(pending_stores(one(text))) == any_wait
    assert len(pending_stores(one(text), written_waits=True)) == written_wait


LOAD = "\tglobal_load_lds_dwordx4 v4, s[2:3]\n"


@pytest.mark.parametrize("text, bad", [
    ("\ts_mov_b32 m0, s1\n" + LOAD, 1),
    ("\ts_add_u32 m0, m0, 0x400\n" + LOAD, 1),
    ("\ts_mov_b32 m0, s1\n\tbuffer_load_dwordx4 v1, s[8:11], s4 offen lds\n", 1),
    ("\ts_mov_b32 m0, s1\n.LBB0_1:\n" + LOAD, 1),
    ("\ts_cbranch_scc1 .LBB0_1\n\ts_mov_b32 m0, s1\n.LBB0_1:\n" + LOAD, 1),
    ("\ts_mov_b32 m0, s1\n\ts_nop 0\n" + LOAD, 0),
    ("\ts_mov_b32 m0, s1\n\ts_mov_b64 exec, 0xffff\n" + LOAD, 0),
    ("\ts_mov_b32 m0, s1\n\tbuffer_load_dwordx4 v[4:7], v1, s[8:11], s4 offen\n", 0),     # into registers
])
def test_m0_just_written_is_seen(text, bad):
    assert len(m0_just_written(one(text))) == bad


@needs_hipcc
def test_m0_is_written_ahead_of_the_loads_that_use_it():
    seen = set()
    for source, found in generated().items():
        for name, code in found.items():
            if loads_into_lds(code):
                seen.add(source)
            bad = m0_just_written(code)
            assert not bad, (source, name, bad[:3])
    assert {"absorb.hip", "decompress_bf16_ring.hip", "decompress_fp8_ring.hip", "decompress_small.hip",
            "kv_attention_mfma.hip", "kv_matmul_ring.hip", "tree_attention_mfma.hip"} <= seen


ADDRESS = "\tv_readfirstlane_b32 s2, v9\n"


@pytest.mark.parametrize("text, bad", [
    (ADDRESS + LOAD, 1),
    (ADDRESS + "\ts_nop 3\n" + LOAD, 1),
    (ADDRESS + "\ts_nop 4\n" + LOAD, 0),
    (ADDRESS + 4 * "\tv_mov_b32_e32 v1, v2\n" + LOAD, 1),
    (ADDRESS + 5 * "\tv_mov_b32_e32 v1, v2\n" + LOAD, 0),
    (ADDRESS + "\ts_add_u32 s2, s2, s5\n" + LOAD, 0),            # read and written by a scalar instruction since
    (ADDRESS + "\ts_add_u32 s3, s2, s5\n" + LOAD, 1),
    ("\tv_readlane_b32 s3, v9, 4\n" + LOAD, 1),
    ("\tv_readlane_b32 s4, v9, 4\n" + LOAD, 0),
    ("\tv_cmp_eq_u32_e64 s[2:3], v1, v2\n" + LOAD, 1),
    ("\tv_readlane_b32 s11, v9, 4\n\tbuffer_load_dwordx4 v1, s[8:11], s4 offen lds\n", 1),
    ("\tv_readlane_b32 s4, v9, 4\n\tbuffer_load_dwordx4 v1, s[8:11], s4 offen lds\n", 1),
    (".LBB0_1:\n" + LOAD + ADDRESS + "\ts_cbranch_scc1 .LBB0_1\n", 1),
])
def test_scalars_just_written_are_seen(text, bad):
    assert len(scalars_just_written(one(text))) == bad


@needs_hipcc
def test_scalar_operands_of_memory_instructions_have_arrived():
    for source, found in generated().items():
        for name, code in found.items():
            bad = scalars_just_written(code)
            assert not bad, (source, name, bad[:3])


@needs_hipcc
def test_no_store_into_lds_is_pending_at_a_barrier():
    for source, found in generated().items():
        for name, code in found.items():
            assert not pending_stores(code), (source, name)
    main = {k: v for k, v in generated()["kv_attention_mfma.hip"].items() if "kv_attention_mfma" in k}
    assert len(main) == 8
    for name, code in main.items():
        assert sum(x.op.startswith("ds_write") for x in code) > 10 and sum(x.op == "s_barrier" for x in code) > 8
        bad = pending_stores(code, written_waits=True)
        assert not bad, (name, bad[:3])
