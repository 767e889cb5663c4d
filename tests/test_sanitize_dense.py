"""The dense operators' argument checks (csrc/abi_dense.cpp against stub
launchers) under AddressSanitizer and UndefinedBehaviorSanitizer: host code
alone, built with g++; no GPU code is compiled or run."""
import os
import shutil
import subprocess

import pytest

from test_sanitize import HERE, ROCM, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "lib", "libamdhip64.so")),
                    reason="needs g++ and the HIP runtime library")
def test_abi_dense_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "abi_dense_san")
    csrc = os.path.join(ROOT, "dropless_moe_expert_amd", "csrc")
    subprocess.check_call(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROCM, "include"),
                           "-I" + os.path.join(ROOT, "include"), "-I" + csrc, os.path.join(csrc, "abi_dense.cpp"),
                           os.path.join(HERE, "abi_dense_checks.cpp"), "-L" + os.path.join(ROCM, "lib"), "-lamdhip64",
                           "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-o", exe])
    assert "ok: 0 checks failed" in _run(exe, tmp_path)
