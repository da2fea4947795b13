"""How the pipelined microscaled kernels are spread over the library's code
objects.  The compiler's time for a file grows faster than the number of its
large kernels (one 15 s, two 39 s, four 115 s, two dozen 20 minutes), so an
object holds the two of one type and tile.  CPU only."""
import collections
import os
import re
import shutil
import subprocess

import pytest

from dense_gemm_row_amd import build
from tests.test_mfma_hazards import LIB, OBJDUMP


@pytest.mark.skipif(not os.path.exists(LIB) or not os.path.exists(OBJDUMP),
                    reason="needs the built library and ROCm's llvm-objdump")
def test_pipelined_kernels_are_compiled_apart(tmp_path):
    lib = tmp_path / "libgemm.so"
    shutil.copy(LIB, lib)
    subprocess.run([OBJDUMP, "--offloading", str(lib)], cwd=tmp_path, check=True, capture_output=True)
    found = collections.Counter()
    for obj in sorted(p for p in os.listdir(tmp_path) if "amdgcn-amd-amdhsa--gfx950" in p):
        syms = subprocess.run([OBJDUMP, "-t", str(tmp_path / obj)], check=True, capture_output=True, text=True).stdout
        names = {n for n in re.findall(r"(_ZN\S*2mx\S*(?:matmul|wgrad)_pipe\S*Tile\S*)$", syms, re.M) if "." not in n}
        assert len(names) <= 2, (obj, sorted(names))
        found["matmul"] += sum("matmul_pipe" in n for n in names)
        found["wgrad"] += sum("wgrad_pipe" in n for n in names)
    # Three types, two tiles, with and without the epilogue; the product with
    # two widths of its scale copies.
    assert found == {"matmul": 24, "wgrad": 12}


def test_objects_have_names_of_their_own():
    stems = [stem for _, stem, _ in build.OBJECTS + build.PROBE_OBJECTS]
    assert len(set(stems)) == len(stems)
    assert {src for src, _, _ in build.OBJECTS} == set(build.SOURCES) | set(build.PARTS)
    csrc = {f for f in os.listdir(build.CSRC) if f.endswith(".hip")}
    assert csrc == set(build.SOURCES) | set(build.PARTS) | set(build.PROBE_SOURCES)
