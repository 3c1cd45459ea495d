"""The cache calls' host checks built with AddressSanitizer and
UndefinedBehaviorSanitizer and driven with the ends of every field (CPU only)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_kv_checks_at_the_ends_of_every_field(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    out = str(tmp_path / "kv_host_check")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"),
           os.path.join(ROOT, "tests", "kv_host_check.cpp"),
           os.path.join(ROOT, "verify_nvfp4_w4a16_amd", "csrc", "host", "kv_shapes.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "host ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
