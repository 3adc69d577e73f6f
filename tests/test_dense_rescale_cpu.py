"""The rescaling of a row of the accumulator in tensor memory (dense_tc.cu) on
the CPU: the kernel's own source, compiled for the host by
tests/dense_rescale_emu.cpp against a tensor memory whose stores become visible
when they are waited for.  A tile that is done again rescales twice."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNEL = os.path.join(ROOT, "query_aware_kv_ts_b200", "csrc", "dense_tc.cu")
HARNESS = os.path.join(ROOT, "tests", "dense_rescale_emu.cpp")


def rescale_source(src: str) -> str:
    start = src.index("// O of this thread's row times f.")
    return src[start:src.index("// ---- the softmax of one stream", start)]


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
@pytest.mark.parametrize("waits", [True, False])
def test_two_rescales_in_turn(tmp_path, waits):
    """(Without the wait for the stores the second one reads the old values:
    the model tells.)"""
    with open(KERNEL) as f:
        src = rescale_source(f.read())
    assert src.count("tmem_wait_st();") == 1
    (tmp_path / "rescale.inc").write_text(src if waits else src.replace("tmem_wait_st();", ""))
    exe = tmp_path / "dense_rescale_emu"
    subprocess.run(["g++", "-std=c++20", "-O1", "-Wno-unknown-pragmas", "-I", str(tmp_path), HARNESS, "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.stdout.strip() == "1024 values, %d failures" % (0 if waits else 192), r.stdout
    assert r.returncode == (0 if waits else 1)
