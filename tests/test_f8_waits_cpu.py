"""The counts by which the e4m3 products wait for their loads, played on the CPU for every form
that the sources launch: what is read next has landed."""

import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "decode_matmul_amd", "csrc")


def source(file):
    """A source without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())


@pytest.fixture(scope="module")
def play(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("waits") / "play")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, os.path.join(HERE, "play_waits.cpp"), "-o", exe],
                   check=True)

    def answers(lines):
        r = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, check=True, timeout=60)
        return r.stdout.splitlines()

    return answers


def tiles():
    """(stages, loads of x and of W a wave sends for a slab, early) of every form of f8_gemm.hip."""
    found = set()
    for args in re.findall(r"launch<EXACT, ([^>]*)>\(a, s\)", source("f8_gemm.hip")):
        BM, BN, WM, WN, KD, KG, NS = (int(v) for v in args.split(", ")[:7])
        for exact in (True, False):
            early = NS == 2 and KD == 1 and KG == 1 and BM // WM // 16 >= 4 and not exact
            found.add((NS, KD * BM // 8 // (WM * WN), KD * BN // 8 // (WM * WN), early))
    return sorted(found)


def test_tiles(play):
    forms = tiles()
    assert {f[0] for f in forms} == {2, 3, 4} and {f[3] for f in forms} == {False, True}
    assert play([f"tile {n} {x} {w} {int(early)} -1" for n, x, w, early in forms]) == ["ok"] * len(forms)


def test_tiles_that_begin_with_more_under_way(play):
    """x of all stages but the first is too much to leave under way with three stages and more."""
    forms = tiles()
    got = play([f"tile {n} {x} {w} {int(early)} {(n - 1) * x}" for n, x, w, early in forms])
    assert [g == "ok" for g in got] == [f[0] == 2 for f in forms]
    assert all(g == "ok" or g.startswith("slab 1 ") for g in got)


def streams():
    """(buffers, waves, loads of a block) of every form of f8_gemv.hip."""
    found = re.findall(r"launch<(\d+), (\d+), (\d+), (\d+), (?:true|false)>\(a, s\)", source("f8_gemv.hip"))
    return sorted({(nbuf, W, 2 * NT + TB // 8) for TB, NT, W, nbuf in (map(int, f) for f in found)})


def test_streams(play):
    forms = streams()
    assert {f[0] for f in forms} == {2, 3} and {f[1] for f in forms} == {4, 8}
    assert play([f"stream {n} {w} {loads} 0" for n, w, loads in forms]) == ["ok"] * len(forms)


def test_streams_whose_next_block_is_not_there(play):
    """The blocks behind the first ones count only where there are any."""
    forms = streams()
    got = play([f"stream {n} {w} {loads} 1" for n, w, loads in forms])
    assert got == [f"block {w} of {w + 1}" for n, w, loads in forms]


def test_the_kernels_wait_by_these_counts():
    assert set(re.findall(r"wait_loads<([^;]*)>\(\)", source("f8_gemv.hip"))) == {"0", "kLoads", "(NBUF - 1) * kLoads"}
    assert "blocks_behind(c, W, NBUF, nb)" in source("f8_gemv.hip")
    assert set(re.findall(r"wait_loads<([^;]*)>\(\)", source("f8_gemm.hip"))) == {"0", "kQueue.begin()", "kQueue.slab()"}
