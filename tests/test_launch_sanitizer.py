"""The adapters' extents, workspaces and launch shapes under UndefinedBehaviorSanitizer, at the ends of the ranges that
the C ABI takes (host code of mx_adapters.hip; CPU only)."""
import os
import shutil
import subprocess

import pytest

from mx_block_scaled_x128_amd.build import ARCH

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mx_block_scaled_x128_amd", "csrc")


def test_extents_under_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    sanitizer = ["-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined"]
    common = [hipcc, "--offload-arch=" + ARCH, "-O1", "-std=c++17", "-I", CSRC, "-I", os.path.join(ROOT, "include")]
    objects = []
    for src, extra in ((os.path.join(CSRC, "mx_adapters.hip"), ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]),
                       (os.path.join(ROOT, "tests", "sanitize", "launch_driver.cpp"), [])):
        objects.append(str(tmp_path / (os.path.basename(src) + ".o")))
        subprocess.run(common + sanitizer + extra + ["-c", src, "-o", objects[-1]], check=True, capture_output=True)
    exe = str(tmp_path / "launch_driver")
    subprocess.run([hipcc] + sanitizer + objects + ["-o", exe], check=True, capture_output=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and "runtime error" not in run.stderr, run.stderr[-4000:]
    assert "all checks passed" in run.stdout
