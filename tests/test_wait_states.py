"""The instruction set's software wait states around loads written in inline assembly
(CPU only: compiles each source to gfx950 assembly and follows its control flow).

Two rules of the gfx9 family are software's to keep, and the compiler keeps them only for
instructions of its own, not inside an asm block:

  - a scalar write of M0 stands at least one wait state before a load into LDS, which
    takes its LDS address from M0;
  - a vector instruction's write of a scalar register (v_readfirstlane and the like, vector
    compares) stands at least five wait states before a vector memory instruction that
    reads that register.

An instruction in between is one wait state, s_nop N is N + 1 of them.  A load that is too
early may use the register's old value: its data would land in another part of the LDS, or
come from another tile's addresses."""
import os
import re
import subprocess

import pytest

from float8_quantization_moe_amd import build as B

VMEM = re.compile(r"^(buffer|global|flat|scratch|tbuffer)_")
TERMINATORS = {"s_endpgm", "s_branch", "s_setpc_b64"}


def instructions(asm):
    """[(opcode, operands)] of the device code and {label: index of the next instruction}."""
    out, labels = [], {}
    for line in asm.splitlines():
        line = re.split(r"\s*(?:;|//)", line, maxsplit=1)[0].strip()
        if not line or line.startswith((".", "#")) and not line.endswith(":"):
            continue
        if line.endswith(":"):
            labels[line[:-1]] = len(out)
            continue
        op, _, rest = line.partition(" " if " " in line and "\t" not in line.split(" ")[0] else "\t")
        out.append((op.strip(), [t.strip() for t in rest.split(",")] if rest.strip() else []))
    return out, labels


def scalars(operand):
    """Names of the scalar registers in an operand: s7, s[4:7], vcc, m0."""
    names = set()
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", operand):
        names |= {f"s{i}" for i in range(int(a), int(b) + 1)}
    names |= {f"s{i}" for i in re.findall(r"\bs(\d+)\b", operand)}
    names |= set(re.findall(r"\b(vcc|m0)\b", operand))
    return names


def predecessors(ins, labels):
    pred = [[] for _ in ins]
    for i, (op, args) in enumerate(ins):
        if op not in TERMINATORS and i + 1 < len(ins):
            pred[i + 1].append(i)
        if (op.startswith("s_cbranch") or op == "s_branch") and args and labels.get(args[0], len(ins)) < len(ins):
            pred[labels[args[0]]].append(i)
    return pred


def too_early(ins, pred, at, limit, conflicts):
    """An instruction for which conflicts() holds less than `limit` wait states before ins[at], on any path."""
    todo, seen = [(p, 0) for p in pred[at]], {}
    while todo:
        i, waited = todo.pop()
        if waited >= limit or seen.get(i, limit) <= waited:
            continue
        seen[i] = waited
        op, args = ins[i]
        if conflicts(op, args):
            return i
        waited += int(args[0], 0) + 1 if op == "s_nop" else 1
        todo += [(p, waited) for p in pred[i]]
    return None


def violations(asm):
    ins, labels = instructions(asm)
    pred = predecessors(ins, labels)
    found = []
    for i, (op, args) in enumerate(ins):
        if not VMEM.match(op):
            continue
        if "lds" in (args[-1].split() if args else []):
            j = too_early(ins, pred, i, 1, lambda o, a: o.startswith("s_") and bool(a) and a[0] == "m0")
            if j is not None:
                found.append((ins[j], ins[i]))
        reads = set().union(*(scalars(a) for a in args)) if args else set()
        if reads:
            j = too_early(ins, pred, i, 5, lambda o, a: o.startswith("v_") and bool(a) and bool(scalars(a[0]) & reads))
            if j is not None:
                found.append((ins[j], ins[i]))
    return found


def test_the_check_sees_what_it_is_for():
    load = "buffer_load_dwordx4 v1, s[4:7], 0 offen lds\n"
    assert violations("\ts_mov_b32 m0, s0\n\t" + load)
    assert violations("L:\n\ts_nop 1\n\t" + load + "\ts_mov_b32 m0, s0\n\ts_cbranch_scc1 L\n") == []
    assert violations("L:\n\t" + load + "\ts_nop 0\n\ts_cbranch_scc1 M\n\ts_mov_b32 m0, s0\n\tM:\n\t" + load)
    assert not violations("\ts_mov_b32 m0, s0\n\ts_nop 0\n\t" + load)
    assert violations("\tv_readfirstlane_b32 s6, v2\n\ts_nop 3\n\t" + load)
    assert not violations("\tv_readfirstlane_b32 s6, v2\n\ts_nop 4\n\t" + load)
    assert not violations("\tv_readfirstlane_b32 s8, v2\n\t" + load)


@pytest.mark.slow
@pytest.mark.parametrize("src", B.SOURCES)
def test_wait_states(src, tmp_path):
    out = str(tmp_path / (src + ".s"))
    cmd = [B.hipcc(), *B.COMMON_FLAGS, *B.DEVICE_FLAGS, "--cuda-device-only", "-S",
           os.path.join(B.CSRC, src), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    found = violations(open(out).read())
    assert not found, f"{src}: {len(found)} loads too early, first {found[:3]}"
