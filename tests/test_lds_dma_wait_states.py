"""The assembly of the kernels with LDS-DMA loads keeps the wait states before such a load that the
compiler adds by itself around its own loads, but cannot see inside inline assembly: one after a scalar
write of M0, the LDS address, and five after a vector instruction that wrote the scalar base.  CPU
only: the sources are compiled to assembly."""

import os
import re
import subprocess

import pytest

from ternary_bit_quantized_amd import build as BUILD

AFTER_M0, AFTER_BASE = 1, 5


def scalar_regs(text):
    out = set()
    for lo, hi, one in re.findall(r"\bs(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        out.update(range(int(lo), int(hi) + 1) if lo else [int(one)])
    return out


def violations(lines):
    """(LDS-DMA loads, those too close to a write of what they use), along every path of the control flow."""
    ins, labels = [], {}
    for line in lines:
        t = line.split(";")[0].strip()
        m = re.match(r"^([.\w$]+):$", t)
        if m:
            labels[m.group(1)] = len(ins)
        elif re.match(r"^[a-z]", t):
            ins.append(t)
    loads, bad = 0, []
    for i, t in enumerate(ins):
        op, _, args = t.partition(" ")
        loads += "load_lds" in op
        first = args.split(",")[0].strip()
        if op.startswith("s_") and first == "m0":
            need, hit = AFTER_M0, lambda u: True
        elif op.startswith("v_") and scalar_regs(first):
            need, hit = AFTER_BASE, lambda u, w=scalar_regs(first): bool(scalar_regs(u) & w)
        else:
            continue
        stack = [(i + 1, 0)]
        while stack:
            j, w = stack.pop()
            while j < len(ins) and w < need:
                u, _, to = ins[j].partition(" ")
                if "load_lds" in u and hit(ins[j]):
                    bad.append("%s ... %s after %d" % (t, ins[j], w))
                if u == "s_endpgm" or u == "s_setpc_b64":
                    break
                if u.startswith("s_cbranch"):
                    stack.append((labels[to.strip()], w + 1))
                w += int(to, 0) + 1 if u == "s_nop" else 1
                j = labels[to.strip()] if u == "s_branch" else j + 1
    return loads, bad


def test_the_check_finds_planted_violations():
    load = "\tglobal_load_lds_dwordx4 v1, s[4:5]"
    assert violations(["\ts_mov_b32 m0, s2", load]) == (1, ["s_mov_b32 m0, s2 ... %s after 0" % load.strip()])
    assert violations(["\ts_add_u32 m0, m0, s2", "\ts_nop 0", load]) == (1, [])
    assert violations(["\ts_add_u32 m0, m0, s2", ".LBB0_1:", load, "\ts_cbranch_scc0 .LBB0_1"])[1]
    assert violations(["\tv_readfirstlane_b32 s5, v2", "\ts_nop 3", load])[1]
    assert violations(["\tv_readfirstlane_b32 s5, v2", "\ts_nop 4", load]) == (1, [])
    assert violations(["\tv_readfirstlane_b32 s6, v2", load]) == (1, [])
    assert violations(["\tv_readfirstlane_b32 s5, v2", "\ts_branch .LBB0_2", "\ts_nop 7", ".LBB0_2:", load])[1]


def sources():
    for name in sorted(os.listdir(BUILD.CSRC)):
        if name.endswith(".hip") and re.search(r"lds_dma16|load_lds", open(os.path.join(BUILD.CSRC, name)).read()):
            yield name


@pytest.mark.parametrize("src", sources())
def test_wait_states_before_lds_dma(src, tmp_path):
    out = str(tmp_path / "k.s")
    r = subprocess.run([BUILD.HIPCC, *BUILD.FLAGS, *BUILD.PER_FILE.get(src, []), "--cuda-device-only", "-S",
                        os.path.join(BUILD.CSRC, src), "-o", out], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    loads, bad = violations(open(out).read().splitlines())
    assert loads > 0 and not bad, "\n".join(bad[:20])
