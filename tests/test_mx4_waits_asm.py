"""The waits for copies to LDS in the 4-bit kernels of few tokens and of one, read out of the compiled kernels.

Both count their loads by hand: a wavefront waits until no more loads are in flight than were issued behind the
copies that it reads next (loads return in order). A load that the compiler left out, or moved in front of the
copies, would let it read LDS before they land. Along every path of a kernel, where a step's operands are read from
LDS, the copies that may be in flight are those of later steps, and where a stage's next copies are issued, its reads
are done."""
import re
import subprocess

import pytest

from bit_matmul_amd import build
from tests import mfma_asm

COPY, LOAD = "C", "L"


def compiled(name):
    run = subprocess.run([build.HIPCC, *build.COMMON, "--cuda-device-only", "-S", str(build.CSRC / name), "-o", "-"],
                         capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stderr[-2000:]
    return mfma_asm._kernels(run.stdout)


def branches(lines):
    """For each instruction, those that may follow it."""
    at = {line[:-1]: i for i, line in enumerate(lines) if line.endswith(":")}
    out = []
    for i, line in enumerate(lines):
        op, _, rest = line.partition(" ")
        if op == "s_endpgm":
            out.append([])
        elif op == "s_branch":
            out.append([at[rest.strip()]])
        elif op.startswith("s_cbranch"):
            out.append([i + 1, at[rest.strip()]])
        else:
            assert op not in ("s_setpc_b64", "s_swappc_b64", "s_call_b64"), line
            out.append([i + 1])
    return out


def walk(lines, allowed):
    """What is wrong along some path. allowed(products done): copies that may be in flight at a read of LDS."""
    follow, found = branches(lines), set()
    todo, seen = [(0, "", 0, False)], set()
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        assert len(seen) < 2_000_000
        i, flight, products, reading = state
        op, _, rest = lines[i].partition(" ")
        if op.startswith("global_load_lds"):
            flight += COPY
            if reading:
                found.add((i, lines[i], "copies while operands are still read"))
        elif op.startswith(("global_", "flat_", "buffer_", "scratch_")):
            flight += LOAD
        elif op == "s_waitcnt":
            m = re.search(r"vmcnt\((\d+)\)", rest)
            if m:
                flight = flight[len(flight) - min(len(flight), int(m[1])):]
            if "lgkmcnt(0)" in rest:
                reading = False
        elif op.startswith("ds_read"):
            reading = True
            if flight.count(COPY) > allowed(products):
                found.add((i, lines[i], f"{flight.count(COPY)} copies in flight after {products} products"))
        elif op.startswith("v_mfma"):
            products += 1
        # (beyond the copies in flight nothing of the past matters; products count up to the last step's)
        todo += [(j, flight[-64:], min(products, 16), reading) for j in follow[i]]
    return found


def token_steps(name):
    m = re.search(r"mx4_token_kernelILb\dELb\dELb\dELi(\d+)ELi(\d+)EE", name)
    return int(m[2])


def check_token(lines, steps):
    return walk(lines, lambda products: max(0, steps - 1 - products // 4) * 5)


def check_few(lines, copies):
    return walk(lines, lambda products: copies)


STEP = ["ds_read_b128 v[0:3], v9", "ds_read_b128 v[4:7], v9", "s_waitcnt lgkmcnt(0)"] + \
       ["v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[0:3], v[4:7], a[0:3], v8, v9"] * 4
COPIES = ["global_load_lds_dwordx4 v1, s[0:1]"] * 4 + ["global_load_lds_dword v1, s[0:1]"]
ROW, ENDS = ["global_load_dwordx4 v[0:3], v1, s[0:1]"] * 2, ["global_load_dword v4, v1, s[0:1]"] * 2


@pytest.mark.parametrize("lines,good", [
    (ROW + COPIES + COPIES + ENDS + ["s_waitcnt vmcnt(7)"] + STEP + ["s_waitcnt vmcnt(2)"] + STEP, True),
    (ROW + COPIES + COPIES + ENDS + ["s_waitcnt vmcnt(8)"] + STEP + ["s_waitcnt vmcnt(2)"] + STEP, False),
    (ROW + COPIES + COPIES + ENDS[1:] + ["s_waitcnt vmcnt(7)"] + STEP + ["s_waitcnt vmcnt(2)"] + STEP, False),      # one left out
    (ENDS + ROW + COPIES + COPIES + ["s_waitcnt vmcnt(7)"] + STEP + ["s_waitcnt vmcnt(2)"] + STEP, False),          # moved in front
    (COPIES + COPIES + ROW + ENDS + ["s_waitcnt vmcnt(7)"] + STEP + ["s_waitcnt vmcnt(2)"] + STEP, True),           # more behind: stricter
    (ROW + COPIES + COPIES + ENDS + ["s_waitcnt vmcnt(7)"] + STEP + STEP, False),
    (ROW + COPIES + COPIES + ["s_cbranch_scc0 .LBB0_1"] + ENDS + [".LBB0_1:", "s_waitcnt vmcnt(7)"] + STEP, False),  # on one path
    (ROW + COPIES + COPIES + ENDS + ["s_waitcnt vmcnt(7)", STEP[0], COPIES[0]] + STEP, False),
])
def test_the_walk_sees_mistakes(lines, good):
    assert (not check_token(lines + ["s_endpgm"], 2)) == good


def test_one_token():
    kernels = [k for k in compiled("mx4_token.hip") if "mx4_token_kernel" in k[0]]
    assert len(kernels) == 32
    for name, lines in kernels:
        assert not check_token(lines, token_steps(name)), name
        # the row is loaded first: no load of values among the copies, and those of the output's scale and bias behind them
        loads = [COPY if x.startswith("global_load_lds") else LOAD for x in lines if x.startswith("global_load")]
        order = "".join(loads)
        first, last = order.index(COPY), order.rindex(COPY)
        assert order[first:last + 1] == COPY * (5 * token_steps(name)), (name, order)
        assert order[last + 1:] == LOAD * 2, (name, order)


def test_few_tokens():
    kernels = [k for k in compiled("mx4_few.hip") if "mx4_few_kernel" in k[0]]
    assert len(kernels) == 4
    for name, lines in kernels:
        m = re.search(r"mx4_few_kernelILi(\d+)ELi(\d+)EE", name)
        tokens, panels = int(m[1]), int(m[2])
        found = check_few(lines, 4 * panels + tokens // 4 + panels + 1)
        assert not found, (name, found)
        # (one copy fewer, and the wait would be too late for some step: the count is the least that holds)
        assert check_few(lines, 4 * panels + tokens // 4 + panels)
