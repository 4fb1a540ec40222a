"""The wait states around the weight gradient's MFMAs, which sit in inline asm
that the compiler does not look into, followed along every path through the
code: branches, loops back to their start, and what comes after the first of a
kernel's ends.  Two rules of gfx950's matrix instructions are looked for:
  * a vector instruction writes a register -> an MFMA reads it (as A, B or the
    accumulator that it adds to): two wait states between them;
  * a 16x16x32 MFMA writes its accumulator -> anything that is no MFMA touches
    it: eight.
And one of the LDS-DMA, in inline asm too: a vector instruction writes a scalar
register -> a buffer load takes its descriptor from it: five.

The kernels are compiled to assembly (under a minute, no GPU); with
TSGEMM_STRESS_TEST=1 those of the race-detection build too."""

import os
import re
import subprocess

import pytest

from persistent_tile_scheduled_amd import _build

OPERANDS, RESULT, DESCRIPTOR = 2, 8, 5

_REGS = re.compile(r"(?<![\w.])([avs])(?:(\d+)|\[(\d+):(\d+)\])(?![\w\[])")


def _registers(text):
    out = set()
    for kind, one, low, high in _REGS.findall(text):
        out |= {(kind, i) for i in range(int(low or one), int(high or one) + 1)}
    return out


class Instruction:
    def __init__(self, line):
        self.text = line
        self.op, _, rest = line.partition(" ")
        operands = [o.strip() for o in rest.split(",")]
        self.mfma = self.op.startswith("v_mfma")
        self.states = int(operands[0]) + 1 if self.op == "s_nop" else 1
        self.uses = _registers(rest)
        # vector instructions that write two registers
        first = 2 if "swap" in self.op else 1
        self.writes = _registers(",".join(operands[:first])) if self.op.startswith("v_") else set()
        # an accumulator's in-place operand included
        self.reads = _registers(",".join(operands[1:]))
        self.load = self.op.startswith("buffer_load")
        self.goes_on = self.op not in ("s_branch", "s_endpgm", "s_setpc_b64")
        self.target = operands[0] if self.op == "s_branch" or self.op.startswith("s_cbranch") else None


def kernels(asm):
    """{kernel: (instructions, successors)} of the weight gradient's kernels."""
    found = {}
    for name, body in re.findall(r"^(_ZN3tsg12wgrad_kernel\w+):[^\n]*\n(.*?)^\.Lfunc_end", asm, re.S | re.M):
        code, labels = [], {}
        for line in body.split("\n"):
            line = line.split(";")[0].strip()
            if not line:
                continue
            label = re.fullmatch(r"(\.?\w+):", line)
            if label:
                labels[label.group(1)] = len(code)
            elif line[0] != ".":
                code.append(Instruction(line))
        after = []
        for i, c in enumerate(code):
            nexts = [i + 1] if c.goes_on and i + 1 < len(code) else []
            if c.target is not None:
                nexts.append(labels[c.target])
            after.append(nexts)
        found[name] = (code, after)
    return found


def _follow(code, after, start, states, harm):
    """Instructions reached from `start` with fewer than `states` wait states in
    between for which harm(instruction, registers) holds; the registers are
    those that start wrote and nothing has written since."""
    found, least = [], {}
    todo = [(n, 0, frozenset(code[start].writes)) for n in after[start]]
    while todo:
        i, gone, live = todo.pop()
        if gone >= states or not live or least.get((i, live), states) <= gone:
            continue
        least[(i, live)] = gone
        if harm(code[i], live):
            found.append(code[i].text)
        rest = live - code[i].writes if not code[i].mfma else live
        todo += [(n, gone + code[i].states, frozenset(rest)) for n in after[i]]
    return found


def hazards(asm):
    """{kernel: [(writer, instruction too near)]}"""
    out = {}
    for name, (code, after) in kernels(asm).items():
        out[name] = []
        for i, c in enumerate(code):
            near = []
            if c.mfma:
                near = _follow(code, after, i, RESULT, lambda o, live: not o.mfma and live & o.uses)
            elif c.writes:
                near = _follow(code, after, i, OPERANDS, lambda o, live: o.mfma and live & o.reads)
                if any(kind == "s" for kind, _ in c.writes):
                    near += _follow(code, after, i, DESCRIPTOR, lambda o, live: o.load and live & o.uses)
            out[name] += [(c.text, n) for n in near]
    return out


_KERNEL = "_ZN3tsg12wgrad_kernelX: ; @k\n%s\n.Lfunc_end0:\n"
_MFMA = " v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n"


@pytest.mark.parametrize("body,count", [
    # an accumulator cleared too late, and in time
    (" v_accvgpr_write_b32 a2, 0\n" + _MFMA + " s_endpgm\n", 1),
    (" v_accvgpr_mov_b32 a2, a9\n s_nop 0\n" + _MFMA + " s_endpgm\n", 1),
    (" v_accvgpr_write_b32 a2, 0\n s_nop 1\n" + _MFMA + " s_endpgm\n", 0),
    (" v_accvgpr_write_b32 a4, 0\n" + _MFMA + " s_endpgm\n", 0),
    # an operand
    (" v_add_u32_e32 v5, v8, v9\n s_nop 0\n" + _MFMA + " s_endpgm\n", 1),
    # over a branch, and back to a loop's start
    (" v_mov_b32_e32 v0, v9\n s_cbranch_scc1 .LBB0_2\n s_nop 7\n.LBB0_2:\n" + _MFMA + " s_endpgm\n", 1),
    (".LBB0_1:\n" + _MFMA + " s_nop 7\n v_mov_b32_e32 v0, v9\n s_cbranch_scc1 .LBB0_1\n s_endpgm\n", 1),
    # a result, straight on, after the first end, and at a loop's start
    (_MFMA + " s_nop 6\n v_accvgpr_read_b32 v9, a1\n s_endpgm\n", 1),
    (_MFMA + " s_nop 7\n v_accvgpr_read_b32 v9, a1\n s_endpgm\n", 0),
    (" s_cbranch_scc1 .LBB0_3\n s_endpgm\n.LBB0_3:\n" + _MFMA + " global_store_dwordx4 v[8:9], a[0:3], off\n s_endpgm\n", 1),
    (".LBB0_1:\n v_accvgpr_read_b32 v9, a1\n s_nop 7\n" + _MFMA + " s_cbranch_vccnz .LBB0_1\n s_endpgm\n", 1),
    # an MFMA's accumulator as the next one's is no matter
    (_MFMA + _MFMA + " s_endpgm\n", 0),
    # a descriptor
    (" v_readfirstlane_b32 s6, v1\n s_nop 3\n buffer_load_dwordx4 v1, s[4:7], 0 offen sc0 lds\n s_endpgm\n", 1),
    (" v_readfirstlane_b32 s6, v1\n s_nop 4\n buffer_load_dwordx4 v1, s[4:7], 0 offen sc0 lds\n s_endpgm\n", 0),
])
def test_the_search_finds_planted_accesses(body, count):
    assert len(hazards(_KERNEL % body)["_ZN3tsg12wgrad_kernelX"]) == count


@pytest.mark.parametrize("stress", [0, 1])
def test_every_path_keeps_the_wait_states(tmp_path, stress):
    if stress and os.environ.get("TSGEMM_STRESS_TEST") != "1":
        pytest.skip("the race-detection build is looked at with TSGEMM_STRESS_TEST=1")
    out = os.path.join(tmp_path, "wgrad.s")
    flags = [f for f in _build.FLAGS if f != "-fPIC"]
    r = subprocess.run([_build.HIPCC] + flags + [f"-DTSG_STRESS={stress}", "--cuda-device-only", "-S",
                                                 os.path.join(_build.CSRC, "tsgemm_wgrad_tu.hip"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(out) as f:
        found = hazards(f.read())
    assert len(found) == 8, sorted(found)
    assert not any(found.values()), {k: (len(v), v[:3]) for k, v in found.items() if v}
