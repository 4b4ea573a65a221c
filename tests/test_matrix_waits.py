"""CPU: in the assembly of every kernel, the wait states between a matrix instruction and the first other use of its
result, along every path.  hipcc 7.2 counts them along one of two ways that meet again, which may be the longer one."""
import concurrent.futures
import os
import re
import subprocess

import pytest

from scale_gla_layer_amd import build as libbuild


def _no_compiler():
    try:
        return not libbuild.hipcc()
    except RuntimeError:
        return True


def _registers(text):
    out = set()
    for kind, a, b in re.findall(r"\b([va])\[(\d+):(\d+)\]", text):
        out |= {(kind, i) for i in range(int(a), int(b) + 1)}
    return out | {(kind, int(i)) for kind, i in re.findall(r"\b([va])(\d+)\b", text)}


def _needed(op):
    """Passes of the instruction, and 2 (fp32 operands) or 3."""
    wide = "_32x32x" in op
    return (16 if wide else 8) + 2 if re.search(r"x[24]_?f32", op) else (8 if wide else 4) + 3


def _instructions(body):
    ops, labels = [], {}
    for line in body.split("\n"):
        line = line.split(";")[0].strip()
        g = re.match(r"(\.LBB\S+):", line)
        if g:
            labels[g.group(1)] = len(ops)
        elif line and not line.startswith(".") and not line.endswith(":"):
            op, _, rest = line.partition(" ")
            ops.append((op, [x.strip() for x in re.split(r",(?![^\[]*\])", rest)]))
    return ops, labels


def _next(ops, labels, i):
    op, args = ops[i]
    if op in ("s_endpgm", "s_setpc_b64"):
        return []
    if op == "s_branch":
        return [labels[args[0]]]
    return [i + 1, labels[args[0]]] if op.startswith("s_cbranch") else [i + 1]


def early_uses(assembly):
    """(matrix instructions, [what reads or writes a result too early])"""
    count, found = 0, []
    for f in re.finditer(r"^(\S+):\s*; @", assembly, re.M):
        body = assembly[f.end():]
        ops, labels = _instructions(body[:body.index(".Lfunc_end")])
        for i, (op, args) in enumerate(ops):
            if "mfma" not in op:
                continue
            count += 1
            result, need, seen = _registers(args[0]), _needed(op), {}
            todo = [(j, 0) for j in _next(ops, labels, i)]
            while todo:
                j, waits = todo.pop()
                if j >= len(ops) or waits >= need or seen.get(j, need) <= waits:
                    continue
                seen[j] = waits
                use, x = ops[j]
                if "mfma" in use:
                    if (_registers(x[1]) | _registers(x[2])) & result:
                        found.append(f"{f.group(1)}: {op} {args} -> {use} {x}: {waits} of {need}")
                        continue
                    if (_registers(x[0]) | _registers(x[3])) & result:
                        continue  # sums go from one to the next by themselves
                elif use.startswith(("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")) and _registers(" ".join(x)) & result:
                    found.append(f"{f.group(1)}: {op} {args} -> {use} {x}: {waits} of {need}")
                    continue
                step = int(x[0], 0) + 1 if use == "s_nop" else 1
                todo += [(k, waits + step) for k in _next(ops, labels, j)]
    return count, found


def test_planted():
    """Two ways to a reader, of which the shorter one has too few wait states."""
    text = """k: ; @k
    v_mfma_f32_32x32x16_bf16 v[0:15], v[16:19], v[20:23], v[0:15]
    s_cbranch_vccnz .LBB0_1
    s_nop 7
.LBB0_1:
    s_nop %d
    v_mov_b32_e32 v30, v15
    s_endpgm
.Lfunc_end0:"""
    assert len(early_uses(text % 2)[1]) == 1 and not early_uses(text % 9)[1]


@pytest.mark.skipif(_no_compiler(), reason="needs hipcc")
def test_every_kernel(tmp_path):
    def assembly(source):
        out = str(tmp_path / source.replace(".hip", ".s"))
        flags = [f for f in libbuild.FLAGS if f != "--hip-link"]
        r = subprocess.run([libbuild.hipcc(), *flags, "-S", "--cuda-device-only", "-o", out, os.path.join(libbuild.CSRC, source)],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return early_uses(open(out).read())

    sources = [s for s in libbuild.SOURCES if s.endswith(".hip")]
    with concurrent.futures.ThreadPoolExecutor(8) as pool:
        results = dict(zip(sources, pool.map(assembly, sources)))
    assert sum(n for n, _ in results.values()) > 1000
    assert not any(f for _, f in results.values()), "\n".join(x for _, f in results.values() for x in f)
