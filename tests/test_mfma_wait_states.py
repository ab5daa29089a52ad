"""The assembly of the decoder-step kernels keeps the wait states between a matrix instruction and
the first read (or overwrite) of its result by another unit, along every path of the control
flow.  The compiler inserts them within a block, but was seen to leave them out at a branch's
target, which gives wrong results now and then.  CPU only: the sources are compiled to assembly."""

import os
import re
import subprocess

import pytest

from ternary_bit_quantized_amd import build as BUILD

# From a 16x16 matrix instruction of 8 passes (the only ones in these files) to a VALU, LDS or memory access
# of its result: the compiler itself keeps 8 wait states.
NEED = 8
REG = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")
OTHER = ("v_", "ds_", "global_", "buffer_", "scratch_", "flat_")


def regs(text):
    out = set()
    for kind, lo, hi, one in REG.findall(text):
        out.update((kind, i) for i in (range(int(lo), int(hi) + 1) if lo else [int(one)]))
    return out


def functions(text):
    name, body = None, []
    for line in text.splitlines():
        m = re.match(r"^(_Z\w+):", line)
        if m:
            name, body = m.group(1), []
        elif name and line.startswith(".Lfunc_end"):
            yield name, body
            name = None
        elif name:
            body.append(line)


def violations(body):
    ins, labels = [], {}
    for line in body:
        m = re.match(r"^(\.LBB\w+):", line)
        if m:
            labels[m.group(1)] = len(ins)
            continue
        t = line.split(";")[0].strip()
        if re.match(r"^[a-z]", t):
            ins.append(t)
    count, bad = 0, []
    for i, t in enumerate(ins):
        if not t.startswith("v_mfma"):
            continue
        count += 1
        dst = regs(t.split(",")[0])
        seen, stack = {}, [(i + 1, 0)]
        while stack:
            j, w = stack.pop()
            while j < len(ins) and w < NEED and seen.get(j, NEED) > w:
                seen[j] = w
                u, op = ins[j], ins[j].split()[0]
                if op == "s_nop":
                    w += int(u.split()[1], 0)
                elif op == "s_branch":
                    j = labels[u.split()[1]] - 1
                elif op.startswith("s_cbranch"):
                    stack.append((labels[u.split()[1]], w + 1))
                elif op == "s_endpgm" or (op.startswith("v_mfma") and regs(u.split(",")[0]) == dst):
                    break
                elif op.startswith(OTHER) and not op.startswith("v_mfma") and regs(u) & dst:
                    bad.append("%s ... %s after %d" % (t, u, w))
                    break
                w += 1
                j += 1
    return count, bad


def test_the_check_finds_a_planted_violation():
    body = ["\tv_mfma_f32_16x16x32_f16 v[0:3], v[4:7], v[8:11], v[0:3]", "\ts_cbranch_vccnz .LBB0_1", "\ts_nop 7",
            ".LBB0_1:", "\tv_add_f32_e32 v12, v1, v13", "\ts_endpgm"]
    assert violations(body)[0] == 1 and len(violations(body)[1]) == 1
    body[1], body[2] = "\ts_nop 6", "\ts_nop 0"
    assert violations(body) == (1, [])


@pytest.mark.parametrize("src", ["attn_shared.hip", "moe_layer.hip"])
def test_wait_states(src, tmp_path):
    out = str(tmp_path / "k.s")
    r = subprocess.run([BUILD.HIPCC, *BUILD.FLAGS, *BUILD.PER_FILE.get(src, []), "--cuda-device-only", "-S",
                        os.path.join(BUILD.CSRC, src), "-o", out], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    total, bad = 0, []
    for name, body in functions(open(out).read()):
        n, b = violations(body)
        total += n
        bad += ["%s: %s" % (name, x) for x in b]
    assert total > 0 and not bad, "\n".join(bad[:20])


def masked_loops(body):
    """(number, lane mask changes) of the shortest cycles of the control flow through a row minimum (row_ror):
    with lanes masked it misses what is in another pass of the loop."""
    blocks, names = [[]], {}
    for line in body:
        t = line.split(";")[0].strip()
        if re.match(r"^\.LBB\w+:$", t):
            blocks.append([])
            names[t[:-1]] = len(blocks) - 1
        elif re.match(r"^[a-z]", t):
            blocks[-1].append(t)
            if t.startswith("s_cbranch"):
                blocks.append([])
    nexts = []
    for i, b in enumerate(blocks):
        last = b[-1] if b else ""
        to = [names[last.split()[1]]] if re.match(r"^s_c?branch", last) else []
        if not last.startswith(("s_branch", "s_endpgm")) and i + 1 < len(blocks):
            to.append(i + 1)
        nexts.append(to)
    loops, changes = 0, []
    for start, b in enumerate(blocks):
        if not any("row_ror" in x for x in b):
            continue
        came, queue = {}, [start]
        while queue and start not in came:
            at = queue.pop(0)
            for to in nexts[at]:
                if to not in came:
                    came[to] = at
                    queue.append(to)
        if start in came:
            loops += 1
            at = start
            while True:
                changes += [x for x in blocks[at] if re.match(r"^s_\w+ exec,|^s_\w+_saveexec", x)]
                at = came[at]
                if at == start:
                    break
    return loops, changes


def test_a_masked_loop_is_found():
    loop = [".LBB0_1:", "\tv_min_i32_dpp v1, v1, v1 row_ror:8 row_mask:0xf bank_mask:0xf", "\ts_cbranch_scc0 .LBB0_1"]
    assert masked_loops(loop) == (1, [])
    loop[2:2] = ["\ts_andn2_b64 exec, exec, s[2:3]"]
    assert len(masked_loops(loop)[1]) == 1


def test_the_loop_over_limits_has_all_its_lanes(tmp_path):
    out = str(tmp_path / "k.s")
    r = subprocess.run([BUILD.HIPCC, *BUILD.FLAGS, "--cuda-device-only", "-S", os.path.join(BUILD.CSRC, "attn_shared.hip"), "-o", out],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    kernels = 0
    for name, body in functions(open(out).read()):
        if "attn_rows" in name:
            loops, bad = masked_loops(body)
            kernels += 1
            assert loops >= 1 and not bad, (name, loops, bad[:3])
    assert kernels
