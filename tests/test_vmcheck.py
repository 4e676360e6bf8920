"""The build's check of registers named while their loads are in flight
(weight_only_int4_02_amd/vmcheck.py), on hand-written gfx9 assembly: each
case is a hazard the check must report or a correct wait it must accept."""
from weight_only_int4_02_amd import vmcheck


def found(body: str):
    asm = "_Zkern:\n" + body.strip("\n") + "\n.Lfunc_end0:\n"
    return vmcheck.check_asm(asm).get("_Zkern", [])


def early(body: str):
    asm = "_Zkern:\n" + body.strip("\n") + "\n.Lfunc_end0:\n"
    return vmcheck.check_asm_sgprs(asm).get("_Zkern", [])


def test_a_descriptor_reloaded_right_before_its_load_is_reported():
    # as the compiler reloads scalar registers that it keeps in lanes of a
    # vector register, and does not see that the inline load reads them
    body = """
    v_readlane_b32 s14, v205, 18
    v_readlane_b32 s15, v205, 19
    {}
    ;;#ASMSTART
    buffer_load_ushort v183, v2, s[12:15], 0 offen
    ;;#ASMEND
    s_endpgm
"""
    f = early(body.format(""))
    assert len(f) == 1 and f[0][2] == [("s", 14), ("s", 15)]
    assert early(body.format("s_nop 3"))[0][2] == [("s", 15)]   # four wait states; s14 has its five
    assert early(body.format("s_nop 4")) == []
    # the compiler's own form: one each for the instructions between
    assert early(body.format("s_nop 1\n    v_mov_b32 v1, v2\n    s_add_i32 s3, s3, 1\n    s_nop 0")) == []
    # a scalar instruction's write in between takes the register over
    assert [r for x in early(body.format("s_mov_b32 s15, 0x20000")) for r in x[2]] == [("s", 14)]


def test_scalar_wait_states_over_branches_and_other_writers():
    f = early("""
    s_cbranch_scc0 .LBB0_2
    v_readfirstlane_b32 s5, v1
    s_branch .LBB0_3
.LBB0_2:
    s_mov_b32 s5, 0
.LBB0_3:
    buffer_load_dwordx4 v[4:7], v1, s[8:11], s5 offen
    s_endpgm
""")
    assert len(f) == 1 and f[0][2] == [("s", 5)]
    assert early("""
    v_cmp_eq_u32_e64 s[8:9], v1, v2
    buffer_load_dword v4, v1, s[8:11], 0 offen
    s_endpgm
""")[0][2] == [("s", 8), ("s", 9)]
    # a scalar operand of a compare is read, not written
    assert early("""
    v_cmp_eq_u32_e32 vcc, s5, v2
    v_mov_b32_e32 v9, s6
    buffer_load_dword v4, v1, s[8:11], s5 offen
    s_endpgm
""") == []


def test_a_matrix_instruction_right_after_its_operand_is_reported():
    def mfma(body):
        return vmcheck.check_asm_mfma("_Zkern:\n" + body.strip("\n") + "\n.Lfunc_end0:\n").get("_Zkern", [])

    body = """
    v_pk_mul_f16 v112, v122, v123
    v_pk_mul_f16 v113, v4, v123
    {}
    ;;#ASMSTART
    v_mfma_f32_16x16x32_f16 v[34:37], v[106:109], v[110:113], v[34:37]
    v_mfma_f32_16x16x32_f16 v[30:33], v[102:105], v[110:113], v[30:33]
    ;;#ASMEND
    s_endpgm
"""
    f = mfma(body.format(""))
    # v112 one wait state, v113 none for the first; for the second v113 one
    assert [x[2] for x in f] == [[("v", 112), ("v", 113)], [("v", 113)]]
    assert [x[2] for x in mfma(body.format("v_mul_u32_u24_e32 v3, 0x10001, v3"))] == [[("v", 113)]]
    assert mfma(body.format("s_nop 1")) == [] and mfma(body.format("s_nop 4")) == []
    # a matrix instruction's own result is not a vector write
    assert mfma("""
    v_mfma_f32_16x16x32_f16 v[34:37], v[106:109], v[110:113], v[34:37]
    v_mfma_f32_16x16x32_f16 v[34:37], v[102:105], v[110:113], v[34:37]
    s_endpgm
""") == []


def paths(body: str):
    asm = "_Zkern:\n" + body.strip("\n") + "\n.Lfunc_end0:\n"
    return vmcheck.check_asm_paths(asm).get("_Zkern", [])


LOOP_BEFORE_THE_WAIT = """
    ;;#ASMSTART
    buffer_load_dwordx4 v[4:7], v1, s[8:11], 0 offen
    ;;#ASMEND
    s_cmp_eq_u32 s4, 0
    s_cbranch_scc1 .LBB0_3
.LBB0_1:
    global_load_dword v20, v[10:11], off
    global_load_dword v21, v[10:11], off offset:4
    s_waitcnt vmcnt({})
    {}
    s_cmp_lg_u32 s4, s5
    s_cbranch_scc1 .LBB0_1
.LBB0_3:
    ;;#ASMSTART
    s_waitcnt vmcnt(0)
    ;;#ASMEND
    v_add_u32_e32 v6, v4, v9
    s_endpgm
"""


def test_a_loop_of_other_loads_before_the_wait():
    # the inline load is in flight over a loop whose length nothing bounds: a
    # register of it is named on a path that no queue common to all holds
    use = "v_add_u32_e32 v5, v30, v31"
    assert found(LOOP_BEFORE_THE_WAIT.format(3, use)) == []
    # two loads follow it in the first round: vmcnt(2) completes it, vmcnt(3) does not
    f = paths(LOOP_BEFORE_THE_WAIT.format(3, use))
    assert [x[2] for x in f] == [[("v", 5)]]
    assert paths(LOOP_BEFORE_THE_WAIT.format(2, use)) == []
    assert paths(LOOP_BEFORE_THE_WAIT.format(3, "v_add_u32_e32 v30, v30, v31")) == []


def test_a_wait_on_another_path_of_a_ring_counts():
    # the way round the loop is ruled out by its trip count, which the walk
    # does not know: past a merge with a path that has waited, nothing
    assert paths("""
    ;;#ASMSTART
    buffer_load_dword v4, v1, s[8:11], 0 offen
    ;;#ASMEND
    s_cmp_lt_i32 s4, 1
    s_cbranch_scc1 .LBB0_2
    ;;#ASMSTART
    s_waitcnt vmcnt(0)
    ;;#ASMEND
    v_add_u32_e32 v6, v4, v9
.LBB0_2:
    v_mov_b32_e32 v4, 0
    s_endpgm
""") == []


BRANCH_FLAG = """
    s_cmp_eq_u32 s4, 0
    s_mov_b64 s[12:13], {first}
    s_cbranch_scc1 .LBB0_2
    s_mov_b64 s[12:13], {second}
    ;;#ASMSTART
    buffer_load_dword v4, v1, s[8:11], 0 offen
    ;;#ASMEND
.LBB0_2:
    s_and_b64 vcc, exec, s[12:13]
    s_cbranch_vccz .LBB0_4
    v_mov_b32_e32 v4, 0
.LBB0_4:
    ;;#ASMSTART
    s_waitcnt vmcnt(0)
    ;;#ASMEND
    s_endpgm
"""


def test_branch_flags_keep_paths_apart():
    # the block that writes v4 is taken only where the load was not issued
    assert paths(BRANCH_FLAG.format(first=-1, second=0)) == []
    f = paths(BRANCH_FLAG.format(first=0, second=-1))
    assert [x[2] for x in f] == [[("v", 4)]]


def test_exec_is_zero_only_where_it_was_narrowed():
    body = """
    ;;#ASMSTART
    buffer_load_dword v4, v1, s[8:11], 0 offen
    ;;#ASMEND
    {}
    s_cbranch_execz .LBB0_2
    ;;#ASMSTART
    s_waitcnt vmcnt(0)
    ;;#ASMEND
    s_endpgm
.LBB0_2:
    v_mov_b32_e32 v4, 0
    s_endpgm
"""
    assert paths(body.format("s_mov_b32 s4, 0")) == []
    assert len(paths(body.format("s_and_saveexec_b64 s[4:5], vcc"))) == 1


def test_read_before_wait_is_reported():
    f = found("""
    buffer_load_dwordx4 v[4:7], v1, s[8:11], 0 offen
    v_accvgpr_write_b32 a3, v5
    s_waitcnt vmcnt(0)
    s_endpgm
""")
    assert len(f) == 1 and "v_accvgpr_write_b32" in f[0][1] and ("v", 5) in f[0][2]


def test_read_after_wait_is_accepted():
    assert found("""
    buffer_load_dwordx4 v[4:7], v1, s[8:11], 0 offen
    s_waitcnt vmcnt(0)
    v_accvgpr_write_b32 a3, v5
    s_endpgm
""") == []


def test_partial_wait_completes_the_older_loads_only():
    body = """
    buffer_load_dword v4, v1, s[8:11], 0 offen
    buffer_load_dword v5, v1, s[8:11], 0 offen offset:64
    s_waitcnt vmcnt(1)
    v_add_u32_e32 v6, v4, v4
    {}
    s_waitcnt vmcnt(0)
    s_endpgm
"""
    assert found(body.format("")) == []
    f = found(body.format("v_add_u32_e32 v7, v5, v5"))
    assert len(f) == 1 and ("v", 5) in f[0][2]


def test_buffer_to_lds_copies_count_in_the_counter():
    # the copy is issued after the load: vmcnt(1) leaves the copy pending and
    # completes the load; vmcnt(2) would not
    body = """
    buffer_load_dword v4, v1, s[8:11], 0 offen
    buffer_load_dword v2, s[8:11], 0 offen lds
    s_waitcnt vmcnt({})
    v_add_u32_e32 v6, v4, v4
    s_endpgm
"""
    assert found(body.format(1)) == []
    assert len(found(body.format(2))) == 1


def test_a_second_load_into_a_pending_register_is_reported():
    f = found("""
    buffer_load_dword v4, v1, s[8:11], 0 offen
    buffer_load_dword v4, v1, s[8:11], 0 offen offset:64
    s_waitcnt vmcnt(0)
    s_endpgm
""")
    assert len(f) == 1 and f[0][1].startswith("buffer_load_dword v4")


def test_pending_on_every_path_into_a_block():
    # both branches leave the load pending: the read after the merge counts
    f = found("""
    buffer_load_dword v4, v1, s[8:11], 0 offen
    s_cbranch_scc0 .LBB0_2
    v_mov_b32_e32 v9, 0
    s_branch .LBB0_3
.LBB0_2:
    v_mov_b32_e32 v9, 1
.LBB0_3:
    v_add_u32_e32 v6, v4, v9
    s_waitcnt vmcnt(0)
    s_endpgm
""")
    assert len(f) == 1 and ("v", 4) in f[0][2]


def test_pending_on_one_path_only_is_not_reported():
    # one branch waits: what is pending on every path is checked
    assert found("""
    buffer_load_dword v4, v1, s[8:11], 0 offen
    s_cbranch_scc0 .LBB0_2
    s_waitcnt vmcnt(0)
.LBB0_2:
    v_add_u32_e32 v6, v8, v9
    s_waitcnt vmcnt(0)
    v_add_u32_e32 v6, v4, v9
    s_endpgm
""") == []


def test_a_load_issued_at_the_end_of_a_loop_reaches_its_top():
    # a ring: the first load before the loop, the next one at the end of
    # each iteration; the iteration reads the register before its wait
    f = found("""
    buffer_load_dword v4, v1, s[8:11], 0 offen
.LBB0_1:
    v_add_u32_e32 v6, v4, v6
    buffer_load_dword v4, v1, s[8:11], 0 offen offset:64
    s_cbranch_scc1 .LBB0_1
    s_waitcnt vmcnt(0)
    s_endpgm
""")
    assert [x for x in f if x[1].startswith("v_add_u32")]


def test_the_loop_with_its_wait_is_accepted():
    assert found("""
    buffer_load_dword v4, v1, s[8:11], 0 offen
.LBB0_1:
    s_waitcnt vmcnt(0)
    v_add_u32_e32 v6, v4, v6
    buffer_load_dword v4, v1, s[8:11], 0 offen offset:64
    s_cbranch_scc1 .LBB0_1
    s_waitcnt vmcnt(0)
    s_endpgm
""") == []
