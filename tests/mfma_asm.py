"""Wait states around matrix products in gfx950 assembly.

Products written as inline assembly are unknown to the compiler, which then
keeps none of the distances that the hardware does not keep by itself:

* 2 wait states from a vector instruction that writes a register to the
  product that reads it, 4 from one that writes the execution mask;
* 12 (an 8-pass product; one of 4 passes needs 8) from a product to anything
  but a product that reads or writes its result;
* none to a product whose addend and result are exactly that result; to one
  that overlaps it otherwise, or reads it as a factor, 12 too.

An instruction is one wait state, `s_nop n` is n + 1. All paths count: the
smallest distances reach a label from every branch to it.
"""
import re

PRODUCT, VALU, EXEC = 12, 2, 4
_RANGE = re.compile(r"^([va])\[(\d+):(\d+)\]$")
_ONE = re.compile(r"^([va])(\d+)$")


def regs(text):
    """The vector registers that an operand names."""
    text = text.strip().split(" ")[0].strip("-|")
    m = _RANGE.match(text)
    if m:
        return frozenset((m[1], i) for i in range(int(m[2]), int(m[3]) + 1))
    m = _ONE.match(text)
    return frozenset({(m[1], int(m[2]))}) if m else frozenset()


def _kernels(asm):
    """[(name, lines)], a line being a label ("x:") or an instruction."""
    out = []
    for line in asm.splitlines():
        line = line.split(";")[0].split("//")[0].strip()
        if line.endswith(":") and not line.startswith("."):
            out.append((line[:-1], []))
        elif out and line and (line.startswith(".LBB") or not line.startswith(".")):
            out[-1][1].append(line)
    return out


class _Inst:
    def __init__(self, line):
        self.text = line
        self.op, _, rest = line.partition(" ")
        ops = [o.strip() for o in rest.split(",")]
        self.product = self.op.startswith("v_mfma")
        self.valu = self.op.startswith("v_") and not self.product
        self.states = int(rest.strip(), 0) + 1 if self.op == "s_nop" else 1
        two = "swap" in self.op                     # writes both operands
        self.dst = regs(ops[0]) | (regs(ops[1]) if two else frozenset()) if self.op.startswith("v_") else frozenset()
        self.exec = self.op.startswith("v_cmpx")
        self.all = frozenset().union(*map(regs, ops)) if ops else frozenset()
        if self.product:
            self.factors, self.addend = regs(ops[1]) | regs(ops[2]), regs(ops[3])


def _blocks(lines):
    """{label: ([instructions], label behind it or None)}, "" first."""
    blocks, order, name, body = {}, [], "", []
    for line in lines + ["end:"]:
        if line.endswith(":"):
            blocks[name] = body
            order.append(name)
            name, body = line[:-1], []
        else:
            body.append(_Inst(line))
    return {name: (blocks[name], behind) for name, behind in zip(order, order[1:] + [None])}


def _step(state, inst, report):
    """state: {("p" or "v", register) or "exec": wait states since; "set": results of products by register}."""
    ages, results = state
    if inst.product:
        for r in inst.factors | inst.addend:
            if ages.get(("v", r), VALU) < VALU:
                report(inst, "a vector instruction has just written", r)
        if ages.get("exec", EXEC) < EXEC:
            report(inst, "the execution mask has just been written", None)
        for r in inst.factors | inst.addend | inst.dst:
            if ages.get(("p", r), PRODUCT) < PRODUCT:
                same = inst.addend == inst.dst == results.get(r) and r not in inst.factors
                if not same:
                    report(inst, "a product's result is not there yet in", r)
    else:
        for r in inst.all:
            if ages.get(("p", r), PRODUCT) < PRODUCT:
                report(inst, "a product's result is not there yet in", r)
    new, res = {}, {}
    for key, age in ages.items():
        limit = EXEC if key == "exec" else PRODUCT if key[0] == "p" else VALU
        if age + inst.states < limit:
            new[key] = age + inst.states
            if key != "exec" and key[0] == "p":
                res[key[1]] = results[key[1]]
    if inst.product:
        for r in inst.dst:
            new[("p", r)] = 0
            res[r] = inst.dst
            new.pop(("v", r), None)
    elif inst.valu:
        for r in inst.dst:
            new[("v", r)] = 0
        if inst.exec:
            new["exec"] = 0
    return new, res


def _join(a, b):
    ages = dict(a[0])
    results = dict(a[1])
    for key, age in b[0].items():
        if key not in ages or age < ages[key]:
            ages[key] = age
    for r, result in b[1].items():
        # (results that differ count as none that a product may continue)
        results[r] = result if results.get(r, result) == result else frozenset()
    return ages, results


def hazards(asm):
    """(number of products, [(kernel, instruction, what, register)])."""
    products, found = 0, {}
    for kernel, lines in _kernels(asm):
        blocks = _blocks(lines)
        if not any(i.product for body, _ in blocks.values() for i in body):
            continue
        products += sum(i.product for body, _ in blocks.values() for i in body)
        before = {"": ({}, {})}
        todo = [""]
        while todo:
            name = todo.pop()
            state = before[name]

            def report(inst, what, reg, name=name):
                found[(kernel, name, id(inst), what)] = (kernel, inst.text, what, reg)
            body, behind = blocks[name]
            ways = []                           # (label, state on the way there)
            for inst in body:
                state = _step(state, inst, report)
                if inst.op.startswith(("s_branch", "s_cbranch")):
                    ways.append((inst.text.split()[1], state))
                if inst.op in ("s_branch", "s_endpgm", "s_setpc_b64"):
                    break
            else:
                ways += [(behind, state)] if behind is not None else []
            for label, state in ways:
                old = before.get(label)
                new = state if old is None else _join(old, state)
                if old != new:
                    before[label] = new
                    todo.append(label)
    return products, list(found.values())
