"""The 4-bit tiles' matrix products are inline assembly (mx4_gemm.hip): the compiled kernels keep the
distances that the hardware asks for. Beside their factors these products read two registers of scales."""
import subprocess

from bit_matmul_amd import build
from tests import mfma_asm

MFMA = "v_mfma_scale_f32_16x16x128_f8f6f4 "


class _Inst(mfma_asm._Inst):
    def __init__(self, line):
        super().__init__(line)
        if self.op.startswith("v_mfma_scale"):
            ops = [o.strip() for o in line.partition(" ")[2].split(",")]
            self.factors = self.factors | mfma_asm.regs(ops[4]) | mfma_asm.regs(ops[5])


def hazards(asm, monkeypatch):
    monkeypatch.setattr(mfma_asm, "_Inst", _Inst)
    return mfma_asm.hazards(asm)


def text(*lines):
    return "kernel:\n" + "\n".join("\t" + x for x in lines) + "\n\ts_endpgm\n"


def test_the_check_sees_the_scales(monkeypatch):
    p = MFMA + "a[0:3], v[0:3], v[4:7], a[0:3], v8, v9 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
    assert hazards(text(p, p), monkeypatch) == (2, [])
    for r in (1, 4, 8, 9):
        assert len(hazards(text(f"v_mov_b32_e32 v{r}, v20", p), monkeypatch)[1]) == 1
        assert not hazards(text(f"v_mov_b32_e32 v{r}, v20", "s_nop 1", p), monkeypatch)[1]
    assert hazards(text(p, "s_nop 10", "v_accvgpr_read_b32 v1, a1"), monkeypatch)[1]


def test_products_of_the_4_bit_tiles(monkeypatch):
    run = subprocess.run([build.HIPCC, *build.COMMON, "--cuda-device-only", "-S", str(build.CSRC / "mx4_gemm.hip"),
                          "-o", "-"], capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stderr[-2000:]
    n, found = hazards(run.stdout, monkeypatch)
    assert n > 1000                       # (ten tiles, up to 64 products in each 64 bytes of a step)
    assert not found, found[:10]
