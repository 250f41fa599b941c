"""The row operators' host code under AddressSanitizer and
UndefinedBehaviorSanitizer: randomised calls with fabricated addresses
(tests/c_abi/ew_rows_fuzz.c), no GPU visible, so that none is launched."""
import os
import re
import shutil
import subprocess

import pytest

from memory_bound_elementwise_amd import build as libbuild
from tests.conftest import ROOT

CLANG = "/opt/rocm/llvm/bin/clang"
SRC = os.path.join(ROOT, "tests", "c_abi", "ew_rows_fuzz.c")
# host-side instrumentation only: each sanitizer flag is preceded by -Xarch_host
HOST_SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer", "-Xarch_host", "-g"]  # noqa: E501


@pytest.fixture(scope="module")
def fuzz_exe(tmp_path_factory):
    if not os.path.exists(CLANG) or not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("the ROCm clang and hipcc are needed")
    d = tmp_path_factory.mktemp("rows_san")
    lib = libbuild.build(extra_flags=HOST_SAN, out=str(d / "libew_san.so"))
    exe = str(d / "ew_rows_fuzz")
    subprocess.run([CLANG, "-std=c11", "-O1", "-g", "-Wall", "-Wextra", "-Werror",
                    "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
                    "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"),
                    "-o", exe, SRC, lib, "-L/opt/rocm/lib", "-lamdhip64",
                    f"-Wl,-rpath,{d}:/opt/rocm/lib"], check=True)
    return exe


@pytest.mark.parametrize("seed", [1, 2])
def test_row_operators_host_code_is_clean_under_sanitizers(fuzz_exe, seed):
    env = dict(os.environ)
    env.update({
        "ASAN_OPTIONS": "detect_leaks=0:verify_asan_link_order=0:abort_on_error=0:halt_on_error=1",
        "UBSAN_OPTIONS": "print_stacktrace=1:halt_on_error=1",
        "HIP_VISIBLE_DEVICES": "-1", "ROCR_VISIBLE_DEVICES": "-1",
    })
    r = subprocess.run([fuzz_exe, "150000", str(seed)], capture_output=True, text=True,
                       timeout=600, env=env)
    if r.returncode == 77:
        pytest.skip("a GPU is visible")
    out = r.stdout + r.stderr
    assert r.returncode == 0 and " 0 failures" in r.stdout, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    counts = {k: int(v) for k, v in re.findall(r"([A-Z_]+) (\d+)", r.stdout)}
    for name in ("OK", "INVALID_ARG", "MISALIGNED", "OVERLAP", "NO_DEVICE"):
        assert counts[name] > 0, r.stdout
