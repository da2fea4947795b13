"""The host code of the grouped and 4-bit products leaves no integer's range at
the ends of the documented sizes.  (tests/experts_far_sizes.py, in a child
process: an overflow ends it.)"""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_integer_overflows_at_far_sizes(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    res = subprocess.run([sys.executable, "-m", "tests.experts_far_sizes", str(tmp_path)], cwd=ROOT, capture_output=True, text=True,
                         timeout=600)
    assert res.returncode == 0, (res.stdout.splitlines()[-1:], res.stderr[-2000:])
    assert res.stdout.splitlines()[-1] == "every call returned"
