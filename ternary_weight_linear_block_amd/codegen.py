"""What the generated gfx950 code of a kernel has to hold where the compiler cannot see to it.

attention.hip has its products for 256-wide heads on accumulation registers written out, and it
and others their loads to LDS.  The compiler keeps the distances that an instruction needs
from the one before it only where it knows both.  The build reads the assembly that it
assembles and stops where a distance is too short, so that no library with wrong results
comes of another compiler.
"""
from __future__ import annotations

import re

# States between two instructions (an instruction is one, s_nop n is n + 1).
RESULT = 19   # from a written-out product to another operation on what it adds to; the compiler keeps 12 behind its own
OPERAND = 2   # from a vector operation to a product that reads what it wrote
ADDRESS = 5   # from a vector operation that writes a scalar register to a load that takes its address from it


def registers(text):
    """The accumulation ('a'), vector ('v') and scalar ('s') registers that an operand text names."""
    out = set()
    for kind, first, last in re.findall(r"\b([avs])\[(\d+):(\d+)\]", text):
        out |= {(kind, r) for r in range(int(first), int(last) + 1)}
    return out | {(kind, int(r)) for kind, r in re.findall(r"\b([avs])(\d+)\b", text)}


def functions(text):
    """name -> body of each function of an assembly text."""
    return {m.group(1): m.group(2) for m in re.finditer(r"^(_Z\w+):[^\n]*\n(.*?)^\.Lfunc_end", text, re.S | re.M)}


class _Block:
    """Instructions that run one after the other: (name, registers of the first operand, of the others, states, line)
    each, the labels behind them and whether the next block is too."""

    def __init__(self):
        self.code, self.targets, self.falls = [], [], True


def _blocks(body):
    blocks, at = [_Block()], {}
    for raw in body.splitlines():
        line = raw.split(";")[0].strip()
        label = re.match(r"(\.?\w+):$", line)
        if label:
            blocks.append(_Block())
            at[label.group(1)] = len(blocks) - 1
            continue
        if not line or line.startswith("."):
            continue
        name, _, operands = line.partition(" ")
        first, _, rest = operands.partition(",")
        states = int(operands) + 1 if name == "s_nop" else 1
        blocks[-1].code.append((name, registers(first), registers(rest), states, line))
        if name.startswith(("s_branch", "s_cbranch", "s_endpgm")):
            if "branch" in name:
                blocks[-1].targets.append(operands.strip())
            blocks[-1].falls = name.startswith("s_cbranch")
            blocks.append(_Block())
        elif name.startswith(("s_setpc", "s_swappc", "s_call")):
            raise RuntimeError(f"{line}: calls are not followed here")
    return blocks, at


def _is_product(name, first):
    return name.startswith("v_mfma") and any(kind == "a" for kind, _ in first)


def _run(block, products, writes, found):
    """Ages in states of what products and vector operations wrote, from a block's start to its end; what is used too
    early goes to `found`."""
    for name, first, rest, states, line in block.code:
        product = _is_product(name, first)
        late = (rest - first if product else first | rest) & products.keys()
        if product:
            late |= {r for r in first | rest if writes.get(r, OPERAND) < OPERAND}
            if len({products.get(r) for r in first}) > 1:  # sums that another product shares in part
                late |= first & products.keys()
        elif name.startswith("global_load_lds"):
            late |= {r for r in first | rest if r[0] == "s" and r in writes}
        if late:
            found.add(line)
        products = {r: t + states for r, t in products.items() if t + states < RESULT}
        writes = {r: t + states for r, t in writes.items() if t + states < (ADDRESS if r[0] == "s" else OPERAND)}
        if product:
            products.update((r, 0) for r in first)
        elif name.startswith("v_") and not name.startswith("v_mfma"):
            writes.update((r, 0) for r in first)
        else:  # a scalar register written again is no longer the vector operation's
            writes = {r: t for r, t in writes.items() if r not in first or not name.startswith("s_")}
    return products, writes


def _younger(a, b):
    out = dict(a)
    for r, t in b.items():
        out[r] = min(t, out.get(r, t))
    return out


def check(text):
    """Raises where a function of an assembly text keeps one of the distances above too short, on any way through its
    branches and loops.  Returns the number of written-out products and of loads to LDS that it looked at."""
    seen_products = seen_loads = 0
    for function, body in functions(text).items():
        if "global_load_lds" not in body and not re.search(r"^\s*v_mfma\S* a\[", body, re.M):
            continue
        blocks, at = _blocks(body)
        start, found, todo = [({}, {}) for _ in blocks], set(), set(range(len(blocks)))
        while todo:
            i = min(todo)
            todo.remove(i)
            end = _run(blocks[i], *start[i], found)
            for j in [at[t] for t in blocks[i].targets] + [i + 1] * (blocks[i].falls and i + 1 < len(blocks)):
                met = tuple(_younger(a, b) for a, b in zip(start[j], end))
                if met != start[j]:
                    start[j] = met
                    todo.add(j)
        if found:
            raise RuntimeError(f"{function}: too close behind what an instruction needs:\n" + "\n".join(sorted(found)[:10]))
        seen_products += sum(_is_product(name, first) for b in blocks for name, first, *_ in b.code)
        seen_loads += body.count("global_load_lds")
    return seen_products, seen_loads
