"""The matrix instructions of the pipelined microscaled kernels are inline
assembly, outside the compiler's hazard checks, and their operands come from
LDS reads (codes, scales) or, in the weight gradient, from conversions placed
ahead of them.  This disassembles the built library's device code (our own
build, gfx950) and holds every one of them to test_mfma_hazards' distances,
the scale operands included: no vector-ALU write of a source in the 4 wait
states before it, no other access to its result in the 20 after it."""
import os
import re
import shutil
import subprocess

import pytest

from tests.test_mfma_hazards import AFTER, BEFORE, LIB, OBJDUMP, _parse, _regs, _wait_states

MNEMONIC = re.compile(r"v_mfma_(scale_f32_16x16x128_f8f6f4|f32_16x16x32_bf16)\b")


def findings(ins):
    bad = []
    for i, (op, args) in enumerate(ins):
        if not MNEMONIC.match(op):
            continue
        dst = _regs(args[0])
        # (the last operand carries the modifiers behind it)
        srcs = set().union(*[_regs(a.split()[0]) for a in args[1:6]])
        ws = 0
        for k in range(i - 1, -1, -1):
            o, a = ins[k]
            ws += _wait_states(o, a)
            if ws > BEFORE:
                break
            if o.startswith(("v_mfma", "ds_", "buffer_", "global_", "scratch_", "s_")):
                continue
            if a and _regs(a[0]) & srcs:
                bad.append((i, "write before", o, a))
        ws = 0
        for k in range(i + 1, len(ins)):
            o, a = ins[k]
            ws += _wait_states(o, a)
            if ws > AFTER:
                break
            if o.startswith("v_mfma"):
                continue
            if a and set().union(*[_regs(x) for x in a]) & dst:
                bad.append((i, "access after", o, a))
                break
    return bad


def test_scanner_sees_scales_and_results():
    op = "v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[8:11], v[4:7], a[0:3], v90, v89 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
    tail = "\ns_nop 7\ns_nop 7\ns_nop 7\nv_accvgpr_read_b32 v1, a0"
    assert findings(_parse(op + tail)) == []
    assert findings(_parse("v_and_b32 v89, 1, v2\n" + op + tail))[0][1] == "write before"
    assert findings(_parse("v_and_b32 v5, 1, v2\n" + op + tail))[0][1] == "write before"
    assert findings(_parse("ds_read_u8 v89, v2\n" + op + tail)) == []
    assert findings(_parse(op + "\nv_accvgpr_read_b32 v1, a0"))[0][1] == "access after"


@pytest.mark.skipif(not os.path.exists(LIB) or not os.path.exists(OBJDUMP),
                    reason="needs the built library and ROCm's llvm-objdump")
def test_pipelined_kernels_keep_hazard_distances(tmp_path):
    lib = tmp_path / "libgemm.so"
    shutil.copy(LIB, lib)
    subprocess.run([OBJDUMP, "--offloading", str(lib)], cwd=tmp_path, check=True, capture_output=True)
    checked = {"matmul_pipe": 0, "wgrad_pipe": 0}
    for obj in sorted(p for p in os.listdir(tmp_path) if "amdgcn-amd-amdhsa--gfx950" in p):
        path = str(tmp_path / obj)
        syms = subprocess.run([OBJDUMP, "-t", path], check=True, capture_output=True, text=True).stdout
        names = sorted(set(re.findall(r"(_ZN\S*2mx\S*(?:matmul|wgrad)_pipe\S*Tile\S*)$", syms, re.M)))
        names = [n for n in names if not n.endswith(".kd")]
        if not names:
            continue
        dis = subprocess.run([OBJDUMP, "-d", "--disassemble-symbols=" + ",".join(names), path],
                             check=True, capture_output=True, text=True).stdout
        for m in re.finditer(r"^[0-9a-f]+ <(\S+)>:\n(.*?)(?=\n[0-9a-f]+ <|\Z)", dis, re.S | re.M):
            ins = _parse(m.group(2))
            assert any(MNEMONIC.match(op) for op, _ in ins), m.group(1)
            bad = findings(ins)
            assert not bad, (m.group(1), bad[:3])
            checked["matmul_pipe" if "matmul_pipe" in m.group(1) else "wgrad_pipe"] += 1
    # Each output type's tiles, with and without the epilogue.
    assert all(n >= 12 for n in checked.values()), checked
