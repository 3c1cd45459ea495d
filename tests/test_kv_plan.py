"""The cache attention's launch layout and workspace, and the cache kernels' page
and row arithmetic, built with AddressSanitizer and UndefinedBehaviorSanitizer
and driven with the ends of every field, the widest windows and starts in any
order among them (CPU only)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20            # an aligned address that no call here reaches


def _run_check(tmp_path, name, sources, done):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    out = str(tmp_path / name)
    host = os.path.join(ROOT, "verify_nvfp4_w4a16_amd", "csrc", "host")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", name + ".cpp"),
           *(os.path.join(host, s) for s in sources), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and done in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])


def test_kv_plan_at_the_ends_of_every_field(tmp_path):
    _run_check(tmp_path, "kv_plan_check", ["kv_shapes.cpp", "kv_plan.cpp"], "plan ok")


def test_pages_and_rows_of_starts_in_any_order(tmp_path):
    _run_check(tmp_path, "kv_index_check", [], "index ok")


@pytest.mark.parametrize("max_kv,new", [(777, 1), (2048, 1), (65536, 1), (65536, 12), (65536, 40), (131072, 300)])
def test_a_window_that_no_sequence_fills_takes_the_workspace_of_none(max_kv, new):
    import verify_nvfp4_w4a16_amd as nv
    serving = pytest.importorskip("verify_nvfp4_w4a16_amd.serving")
    lib = serving._kv()

    def need(window):
        cache = serving._Cache(A, 4096, 8, 128, 1.0, 1.0)
        seqs = serving._Seqs(A, A, A, 2048, 3, 3 * new)
        queries = serving._Queries(A, 4096, 128, 32, new, max_kv, window, 0.1, 0.0, 1)
        n = ctypes.c_int64(-1)
        assert lib.nvfp4_kv_attention_workspace(cache, seqs, queries, n) == nv.OK
        return n.value

    none = need(0)
    for window in (max_kv, max_kv + 1, (1 << 31) - 1, 1 << 31, 1 << 62, (1 << 63) - 1 - new, (1 << 63) - 1):
        assert need(window) == none, window
