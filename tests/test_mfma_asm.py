"""The 8-bit tiles' matrix products are inline assembly (int8_gemm.hip): the compiled kernels keep the
distances that the hardware asks for, whatever the compiler's version does around them."""
import subprocess

import pytest

from bit_matmul_amd import build
from tests.mfma_asm import hazards

MFMA = "v_mfma_i32_16x16x64_i8 "


def text(*lines):
    return "kernel:\n" + "\n".join("\t" + x if not x.endswith(":") else x for x in lines) + "\n\ts_endpgm\n"


@pytest.mark.parametrize("lines,products,bad", [
    # one sum after another, in place
    ([MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]", MFMA + "a[0:3], v[8:11], v[4:7], a[0:3]"], 2, 0),
    # a factor written right before, and after two wait states
    (["v_mov_b32_e32 v5, v9", MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]"], 1, 1),
    (["v_mov_b32_e32 v5, v9", "s_add_u32 s0, s0, s1", MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]"], 1, 1),
    (["v_mov_b32_e32 v5, v9", "s_nop 1", MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]"], 1, 0),
    (["v_accvgpr_write_b32 a2, 0", "s_nop 0", MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]"], 1, 1),
    (["v_permlane32_swap_b32 v20, v6", MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]"], 1, 1),
    (["v_cmpx_gt_u32_e32 v20, v21", "s_nop 2", MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]"], 1, 1),
    # a sum read or cleared too early, and late enough
    ([MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]", "s_nop 10", "v_accvgpr_read_b32 v1, a1"], 1, 1),
    ([MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]", "s_nop 10", "s_nop 0", "v_accvgpr_read_b32 v1, a1"], 1, 0),
    ([MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]", "global_store_dwordx4 v[30:31], a[0:3], off"], 1, 1),
    # overlapping, but not the same; a result as a factor
    ([MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]", MFMA + "a[2:5], v[0:3], v[4:7], a[2:5]"], 2, 1),
    ([MFMA + "v[0:3], v[8:11], v[4:7], v[0:3]", MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]"], 2, 1),
    # over a branch and round a loop
    (["v_mov_b32_e32 v5, v9", "s_cbranch_scc1 .LBB0_2", "s_nop 3", ".LBB0_2:", MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]"],
     1, 1),
    ([".LBB0_1:", MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]", "v_mov_b32_e32 v5, v9", "s_cbranch_scc1 .LBB0_1"], 1, 1),
    ([".LBB0_1:", MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]", "s_cbranch_scc1 .LBB0_1", "v_accvgpr_mov_b32 a9, a2"], 1, 1),
    (["s_branch .LBB0_3", ".LBB0_2:", "v_mov_b32_e32 v5, v9", "s_branch .LBB0_4", ".LBB0_3:",
      MFMA + "a[0:3], v[0:3], v[4:7], a[0:3]", ".LBB0_4:"], 1, 0),
])
def test_the_check_sees_planted_mistakes(lines, products, bad):
    n, found = hazards(text(*lines))
    assert n == products and (len(found) > 0) == (bad > 0), found


def test_products_of_the_8_bit_tiles():
    run = subprocess.run([build.HIPCC, *build.COMMON, "--cuda-device-only", "-S", str(build.CSRC / "int8_gemm.hip"),
                          "-o", "-"], capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stderr[-2000:]
    n, found = hazards(run.stdout)
    assert n > 1000                       # (ten tiles, up to 64 products in each 64 bytes of a step)
    assert not found, found[:10]
