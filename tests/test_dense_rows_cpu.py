"""Where dense attention finds a token's row (dense_common.cuh) on the CPU: the
header's own source, compiled for the host by tests/dense_rows_emu.cpp, reads
nothing outside the block table and names no row outside the cache."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "query_aware_kv_ts_b200", "csrc", "dense_common.cuh")
HARNESS = os.path.join(ROOT, "tests", "dense_rows_emu.cpp")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_no_row_outside_the_table_and_the_cache(tmp_path):
    with open(HEADER) as f:
        src = f.read()
    start = src.index("// The pool's page with token i")
    body = src.index("dense_row(const DenseArgs &a, int b, int64_t off, int64_t i)\n{", start)
    (tmp_path / "rows.inc").write_text(src[start:src.index("\n}\n", body) + 3])
    exe = tmp_path / "dense_rows_emu"
    subprocess.run(["g++", "-std=c++20", "-O1", "-I", str(tmp_path), HARNESS, "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip().endswith(" 0 failures"), r.stdout
