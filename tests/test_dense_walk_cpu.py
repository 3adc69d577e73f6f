"""The division of dense attention's work over blocks (dense_common.cuh) on the
CPU: the header's own source, compiled for the host by
tests/dense_walk_emu.cpp, on random batches and grids.  Every tile of every
item is taken once, and the pieces of an item that blocks share are the ones
its join reads.  Needs no GPU (the GPU tests run the same source there)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "query_aware_kv_ts_b200", "csrc", "dense_common.cuh")
HARNESS = os.path.join(ROOT, "tests", "dense_walk_emu.cpp")


def walk_source(src: str) -> str:
    """From the tile's constant to the end of the walk, without the warp-wide
    search for the next sequence (the harness has its own)."""
    start = src.index("constexpr int kDenseTile")
    search = src.index("// The first sequence from b on that has items")
    place = src.index("// A place on the line")
    end = src.index("// The block's part, found by one warp")
    return src[start:search] + src[place:end]


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_every_tile_once_and_every_join(tmp_path):
    with open(HEADER) as f:
        (tmp_path / "walk.inc").write_text(walk_source(f.read()))
    exe = tmp_path / "dense_walk_emu"
    subprocess.run(["g++", "-std=c++20", "-O2", "-I", str(tmp_path), HARNESS, "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert r.stdout.strip().endswith("12000 cases, 0 failures")
