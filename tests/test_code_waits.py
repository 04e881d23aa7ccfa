"""Wait states in the compiled kernels (no GPU): the rules that the hardware leaves to software.

The compiler keeps them for the instructions it writes; an instruction inside an inline assembly
statement is hidden from it, and so is what such an instruction reads and writes.  liblrm.so's own
code objects are disassembled and every path through them is walked backwards from
  - a load into LDS: one wait state after a scalar write of M0;
  - a buffer or global access: five after a vector instruction wrote a scalar register it reads;
  - a DPP instruction: two after a vector instruction wrote the vector register it exchanges.
An instruction is one wait state, s_nop N is N + 1.
"""
import os
import re
import shutil
import subprocess

import pytest

from backward_token_expert_amd import lrm

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def registers(op, kind):
    """Numbers of the `kind` ('s' or 'v') registers that operand `op` names."""
    m = re.fullmatch(r"[-|]*%s(?:\[(\d+):(\d+)\]|(\d+))\|?" % kind, op)
    if not m:
        return frozenset()
    if m[3]:
        return frozenset((int(m[3]),))
    return frozenset(range(int(m[1]), int(m[2]) + 1))


class Ins:
    __slots__ = ("text", "op", "args", "nop", "preds")

    def __init__(self, text):
        self.text = text
        words = text.replace(",", " ").split()
        self.op, self.args = words[0], words[1:]
        self.nop = int(self.args[0], 0) + 1 if self.op == "s_nop" else 1
        self.preds = []

    def writes(self, kind):
        """Registers of `kind` a vector ALU instruction writes (its first operand, the second too
        where that is a carry)."""
        if not self.op.startswith("v_") or not self.args:
            return frozenset()
        out = registers(self.args[0], kind)
        if "_co_" in self.op and len(self.args) > 1:
            out |= registers(self.args[1], kind)
        return out


def functions(text):
    """Lists of instructions with their predecessors, one per function of a disassembly."""
    for part in re.split(r"^<(\S+)>:$", text, flags=re.M)[1:][1::2]:
        code, at, jumps = [], {}, []
        for line in part.splitlines():
            m = re.match(r"\s+(\S.*?)\s*// ([0-9A-F]+): ", line)
            if not m:
                continue
            ins, address = Ins(m[1]), int(m[2], 16)
            at[address] = ins
            if code and code[-1].op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
                ins.preds.append(code[-1])
            if ins.op.startswith(("s_branch", "s_cbranch")):
                words = int(ins.args[0])   # a signed 16-bit distance
                jumps.append((ins, address + 4 + 4 * (words - 65536 * (words > 32767))))
            code.append(ins)
        for ins, target in jumps:
            at[target].preds.append(ins)
        yield code


def nearest(ins, hit, limit):
    """The instruction `hit` accepts on some path to `ins` with fewer than `limit` wait states between
    the two, or None."""
    todo, seen = [(p, 0) for p in ins.preds], set()
    while todo:
        at, states = todo.pop()
        if states >= limit or (id(at), states) in seen:
            continue
        seen.add((id(at), states))
        if hit(at):
            return at
        todo += [(p, states + at.nop) for p in at.preds]
    return None


def m0_rule(ins):
    if ins.op.startswith("buffer_") and "lds" in ins.args:
        return nearest(ins, lambda o: o.op.startswith("s_") and o.args[:1] == ["m0"], 1)


def scalar_rule(ins):
    if ins.op.startswith(("buffer_", "global_", "scratch_", "flat_")):
        used = frozenset().union(*[registers(a, "s") for a in ins.args])
        return nearest(ins, lambda o: o.writes("s") & used, 5) if used else None


def dpp_rule(ins):
    if ins.op.endswith("_dpp"):
        used = registers(ins.args[1], "v")
        return nearest(ins, lambda o: o.writes("v") & used, 2)


RULES = {"m0": m0_rule, "scalar": scalar_rule, "dpp": dpp_rule}


def broken(code, rule):
    """The pairs of instructions in a list of functions that `rule` finds too near."""
    pairs = [(RULES[rule](ins), ins) for function in code for ins in function]
    return [(near.text, ins.text) for near, ins in pairs if near]


# What the check has to find, and to leave alone.
WRONG = [("scalar", "v_readfirstlane_b32 s4, v0\n s_nop 3\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds"),
         ("scalar", "v_cmp_eq_u32_e64 s[6:7], v1, v2\n global_load_dword v1, v2, s[6:7]"),
         ("m0", "s_mov_b32 m0, s9\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds"),
         ("dpp", "v_max_f64 v[2:3], v[4:5], v[6:7]\n s_nop 0\n v_mov_b32_dpp v9, v3 quad_perm:[1,0,3,2]")]
RIGHT = [("scalar", "v_readfirstlane_b32 s4, v0\n s_nop 4\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds"),
         ("scalar", "s_mov_b32 s4, s9\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds"),
         ("scalar", "v_readfirstlane_b32 s8, v0\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds"),
         ("m0", "s_mov_b32 m0, s9\n s_nop 0\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds"),
         ("m0", "s_mov_b32 m0, s9\n buffer_load_dwordx4 v[0:3], v1, s[4:7], 0 offen"),
         ("dpp", "v_max_f64 v[2:3], v[4:5], v[6:7]\n s_nop 1\n v_mov_b32_dpp v9, v3 quad_perm:[1,0,3,2]"),
         ("dpp", "v_max_f64 v[2:3], v[4:5], v[6:7]\n v_mov_b32_dpp v9, v4 quad_perm:[1,0,3,2]")]


def listing(code):
    return functions("<f>:\n" + "\n".join("\t%s    // %012X: 00" % (c.strip(), 4 * i)
                                          for i, c in enumerate(code.split("\n"))))


def test_the_check_itself():
    assert all(len(broken(listing(c), rule)) == 1 for rule, c in WRONG)
    assert not any(broken(listing(c), rule) for rule, c in RIGHT)
    # across a loop's back edge: the write at its end, the use at its start
    loop = ("<f>:\n\tbuffer_load_dwordx4 v1, s[4:7], 0 offen lds    // 000000000000: 00\n"
            "\ts_mov_b32 m0, s9    // 000000000008: 00\n"
            "\ts_branch 65532    // 00000000000C: BF82FFFC\n")
    assert not broken(functions(loop), "m0")            # the branch itself is a wait state
    dpp = ("<f>:\n\tv_mov_b32_dpp v9, v3 quad_perm:[1,0,3,2]    // 000000000000: 00\n"
           "\tv_max_f64 v[2:3], v[4:5], v[6:7]    // 000000000008: 00\n"
           "\ts_cbranch_scc1 65532    // 00000000000C: BF85FFFC\n")
    assert len(broken(functions(dpp), "dpp")) == 1


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """The functions of the library's device code."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    where = tmp_path_factory.mktemp("code")
    shutil.copy(lrm.LIB_PATH, where / "liblrm.so")
    subprocess.run([OBJDUMP, "--offloading", "liblrm.so"], check=True, stdout=subprocess.DEVNULL, cwd=where)
    objects = sorted(f for f in os.listdir(where) if "amdgcn" in f)
    assert objects
    return [f for o in objects for f in functions(subprocess.run(
        [OBJDUMP, "-d", "--no-leading-addr", o], check=True, cwd=where, capture_output=True, text=True).stdout)]


@pytest.mark.parametrize("rule", sorted(RULES))
def test_compiled_kernels_keep_the_wait_states(code, rule):
    assert sum("lds" in ins.args for function in code for ins in function) > 1000   # the loads are there
    found = broken(code, rule)
    assert not found, f"{len(found)} of too few wait states, the first: {found[:4]}"
