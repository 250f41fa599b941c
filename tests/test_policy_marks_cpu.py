"""Which tokens of a lane count (ew_policy_marks.h), on the CPU under
UndefinedBehaviorSanitizer: a shift by 32 bits and more is undefined, also where
its result is 0 on the GPU."""
import os
import shutil
import subprocess

import pytest

from memory_bound_elementwise_amd import build as libbuild
from tests.conftest import ROOT


def test_counted_tokens(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("g++ is needed")
    exe = str(tmp_path / "marks")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    "-I", libbuild.CSRC, "-o", exe,
                    os.path.join(ROOT, "tests", "c_abi", "ew_policy_marks.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "0 wrong\n", r.stdout + r.stderr
