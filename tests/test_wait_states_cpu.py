"""Wait states of the built kernels that the hardware does not keep by itself.

A vector instruction that writes a scalar register needs five wait states
before a vector memory instruction that reads it.  The compiler sees to it
between its own instructions, but it does not look into an ``asm`` statement,
so the machine code of the whole library is looked through."""
import os
import re
import shutil
import subprocess

import pytest

import gated_deltanet_tree_gdn_amd as gdn

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
WAITS = 5  # between the two, each instruction one, s_nop n: n + 1
MEMORY = ("buffer_", "global_", "flat_", "scratch_", "tbuffer_")


def scalars(operand):
    """The numbers of the scalar registers that an operand names; vcc as -1."""
    if operand.startswith("vcc"):
        return {-1}
    m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]", operand)
    if not m:
        return set()
    return {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))


def parse(text):
    """Functions of a disassembly: name -> list of (address, mnemonic, operands, target of a branch)."""
    functions, code = {}, None
    for line in text.splitlines():
        m = re.match(r"[0-9a-f]+ <(\S+)>:$", line)
        if m:
            code = functions.setdefault(m[1], [])
            continue
        m = re.match(r"\s+([a-z]\w+)\s*(.*?)\s*// ([0-9A-F]+):", line)
        if not m or code is None:
            continue
        target = re.search(r"<\S+\+0x([0-9a-f]+)>|<(\S+)>$", line) if m[1].startswith(("s_branch", "s_cbranch")) else None
        at = int(m[3], 16)
        start = code[0][0] if code else at
        to = None if target is None else start + int(target[1] or "0", 16)
        operands = [x.split()[0] for x in m[2].split(",") if x.split()]
        code.append((at, m[1], operands, to))
    return functions


def written(name, operands):
    """Scalar registers that a vector instruction writes."""
    if not name.startswith("v_") or not operands:
        return set()
    out = scalars(operands[0])
    if ("_co_" in name or name.startswith("v_div_scale")) and len(operands) > 1:
        out = out | scalars(operands[1])
    return out


def too_early(code):
    """(address of the load, of the vector write) of every pair that is too close, on any way through the branches, in order."""
    came, bad = {}, set()
    for i, (_, _, _, to) in enumerate(code):
        if to is not None:
            came.setdefault(to, []).append(i)
    for i, (at, name, operands, _) in enumerate(code):
        if not name.startswith(MEMORY):
            continue
        reads = set().union(*map(scalars, operands))
        todo, seen = [(i, 0, reads)] if reads else [], set()
        while todo:
            j, waits, live = todo.pop()
            before = list(came.get(code[j][0], []))
            if j > 0 and code[j - 1][1] not in ("s_branch", "s_endpgm", "s_setpc_b64"):
                before.append(j - 1)
            for p in before:
                _, n, ops, _ = code[p]
                if live & written(n, ops):
                    bad.add((at, code[p][0]))
                    continue
                left = live - scalars(ops[0]) if n.startswith("s_") and ops and not n.startswith(("s_cmp", "s_bitcmp")) else live
                more = waits + (int(ops[0], 0) + 1 if n == "s_nop" else 1)
                if left and more < WAITS and (p, more, frozenset(left)) not in seen:
                    seen.add((p, more, frozenset(left)))
                    todo.append((p, more, left))
    return sorted(bad)


SAMPLE = """
0000000000001000 <kernel>:
\tv_readlane_b32 s6, v2, 0                                   // 000000001000: D2890006
\ts_mov_b32 m0, s5                                           // 000000001008: BEFC0005
\ts_nop {0}                                                  // 00000000100C: BF800000
\tbuffer_load_dwordx4 v1, s[92:95], s6 offen lds             // 000000001010: E05D1000
\ts_cbranch_scc0 65530                                       // 000000001018: BF84FFFA <kernel+0x{1}>
\ts_endpgm                                                   // 00000000101C: BF810000
"""


@pytest.mark.parametrize("nop,found", [(0, 1), (2, 1), (3, 0)])
def test_the_search_itself(nop, found):
    """straight on, and from the branch behind it to the load as well"""
    for target in ("0", "10"):
        assert len(too_early(parse(SAMPLE.format(nop, target))["kernel"])) == found


def test_a_way_back_to_the_load():
    text = SAMPLE.format(3, "10").replace("s_cbranch_scc0", "s_branch").replace("s_nop 3", "v_readlane_b32 s6, v2, 1")
    text = text.replace("s_mov_b32 m0, s5", "s_branch 2").replace("BEFC0005", "BF820002 <kernel+0x10>")
    # the load is reached from the branch at 8 and from its own loop; what stands before it counts, reached or not
    assert [(a - 0x1000, b - 0x1000) for a, b in too_early(parse(text)["kernel"])] == [(0x10, 0), (0x10, 0xc)]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump not installed")
def test_scalar_operands_of_loads_have_arrived(tmp_path):
    if not os.path.exists(gdn.LIB_PATH):
        pytest.fail("libgdn_tree.so is not built: run __graft_entry__.build()")
    lib = shutil.copy(gdn.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    images = [f for f in sorted(os.listdir(tmp_path)) if "gfx950" in f]
    kernels, bad = 0, []
    for image in images:
        text = subprocess.run([OBJDUMP, "-d", str(tmp_path / image)], check=True, capture_output=True, text=True).stdout
        for name, code in parse(text).items():
            kernels += 1
            bad += [f"{name}: load at {a:x}, written at {b:x}" for a, b in too_early(code)]
    assert kernels > 50
    assert not bad, "\n".join(bad)
