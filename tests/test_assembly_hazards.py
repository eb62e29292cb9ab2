"""Two orders of instructions that the compiler has left in kernels here and that gave wrong values now and then: none
of the kernels with matrix instructions, or with wide stores, has them as built now."""
import concurrent.futures as cf

import pytest

import assembly

SOURCES = ["gdn_linear_state.hip", "gdn_linear_out.hip", "gdn_linear_dq.hip", "gdn_linear_dkv.hip", "gdn_linear.hip", "gdn_matmul.hip",
           "gdn_rms_norm.hip"]


@pytest.fixture(scope="module")
def built():
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(assembly.kernels, SOURCES)))


@pytest.mark.parametrize("source", SOURCES)
def test_no_result_is_read_early_behind_a_branch(source, built):
    assert built[source]
    for name, lines in built[source].items():
        assert not assembly.early_reads(lines), name


@pytest.mark.parametrize("source", SOURCES)
def test_no_stored_data_is_written_again_at_once(source, built):
    for name, lines in built[source].items():
        assert not assembly.overwritten_stores(lines), name


MFMA = "v_mfma_f32_16x16x32_bf16 v[4:7], v[20:23], v[24:27], v[4:7]"


@pytest.mark.parametrize("lines,bad", [
    ([MFMA, "s_cbranch_vccnz .LBB0_1", "v_add_f32_e32 v1, v2, v3", ".LBB0_1:", "v_add_f32_e32 v9, v4, v8"], True),
    ([MFMA, "s_cbranch_vccnz .LBB0_1", "s_endpgm", ".LBB0_1:", "s_nop 6", "v_add_f32_e32 v9, v4, v8"], False),
    ([MFMA, "s_cbranch_vccnz .LBB0_1", "s_endpgm", ".LBB0_1:", "s_nop 5", "v_add_f32_e32 v9, v4, v8"], True),
    ([MFMA, "s_nop 6", "s_branch .LBB0_2", ".LBB0_2:", "global_store_dword v[0:1], v7, off"], False),
    ([MFMA, ".LBB0_3:", "global_store_dword v[0:1], v7, off"], True),
    ([MFMA, ".LBB0_3:", "v_mov_b32_e32 v7, 0", "global_store_dword v[0:1], v7, off"], False),
    ([MFMA, ".LBB0_3:", "v_mfma_f32_16x16x32_bf16 v[4:7], v[20:23], v[24:27], v[4:7]"], False),
])
def test_early_reads_are_found(lines, bad):
    assert bool(assembly.early_reads(lines)) == bad


@pytest.mark.parametrize("lines,bad", [
    (["buffer_store_dwordx4 v[30:33], v2, s[4:7], s0 offen", "v_accvgpr_read_b32 v30, a0"], True),
    (["buffer_store_dwordx4 v[30:33], v2, s[4:7], 0 offen offset:64", "v_accvgpr_read_b32 v30, a0"], False),
    (["buffer_store_dwordx4 v[30:33], v2, s[4:7], s0 offen", "v_mov_b32_e32 v34, v30"], False),
    (["buffer_store_dwordx2 v[30:31], v2, s[4:7], s0 offen", "v_mov_b32_e32 v30, 0"], False),
])
def test_overwritten_stores_are_found(lines, bad):
    assert bool(assembly.overwritten_stores(lines)) == bad
