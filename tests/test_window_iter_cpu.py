"""The windowed walks (csrc/window_iter.cuh), compiled for the host, against
the mask itself: a walk holds every tile with a visible pair once, no tile
without one, in position order, and flags exactly the tiles that need masking."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle.window import allowed

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sequence_exact_attention_gb300", "csrc")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
CAP = 1 << 14


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA headers are not available")
    out = str(tmp_path_factory.mktemp("window") / "libwindow.so")
    cmd = [gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(CUDA, "include"), os.path.join(ROOT, "tests", "window_harness.cpp"),
           os.path.join(CSRC, "plan.cpp"), "-L", os.path.join(CUDA, "lib64"),
           "-Wl,-rpath," + os.path.join(CUDA, "lib64"), "-lcudart", "-o", out]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return ctypes.CDLL(out)


def tiles(S, tile):
    """(index, first position, tokens) of every tile."""
    return [(i, lo, min(tile, S - lo)) for i, lo in enumerate(range(0, S, tile))]


LENGTHS = [1, 5, 130, 777, 1000, 1001, 1300, 2048]
WINDOWS = [(1, 0), (1, 1), (64, 4), (100, 130), (128, 0), (129, 128), (500, 260), (5000, 0), (3, 5000), (128, 129)]


def clamp(w, k, S):
    return min(w, S), min(k, S)


@pytest.mark.parametrize("S", LENGTHS)
@pytest.mark.parametrize("window,n_sink", WINDOWS)
@pytest.mark.parametrize("tile,rows", [(128, 256), (128, 128), (64, 64), (64, 32)])
def test_key_walk(harness, S, window, n_sink, tile, rows):
    w, k = clamp(window, n_sink, S)
    see = allowed(np.arange(S), np.arange(S), w, k)
    every = tiles(S, tile)
    buf = (ctypes.c_int * (3 * CAP))()
    for ti, lo, _ in every:
        if rows > tile and ti % (rows // tile):
            continue
        hi = min(lo + rows, S)
        n = harness.ra_win_walk(S, tile, w, k, ti, rows, buf, CAP)
        assert n >= 0
        walk = [tuple(buf[3 * i:3 * i + 3]) for i in range(n)]
        assert [e[0] for e in walk] == sorted(set(e[0] for e in walk))
        met = {e[0]: e for e in walk}
        for _, klo, kn in every:
            block = see[lo:hi, klo:klo + kn]
            assert (klo in met) == block.any()
            if klo in met:
                assert met[klo][1] == kn
                assert block.all() or met[klo][2] == 2          # masked tiles are flagged
                if kn == tile and hi - lo == rows:
                    assert (met[klo][2] == 1) == block.all()    # and full ones are not


@pytest.mark.parametrize("S", LENGTHS)
@pytest.mark.parametrize("window,n_sink", WINDOWS)
def test_query_walk_and_its_shares(harness, S, window, n_sink):
    w, k = clamp(window, n_sink, S)
    see = allowed(np.arange(S), np.arange(S), w, k)
    every = tiles(S, 128)
    buf = (ctypes.c_int * (4 * CAP))()

    def walk(ti, a, b):
        n = harness.ra_win_qwalk(S, w, k, ti, 2, a, b, buf, CAP)
        return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]

    for ti, lo, n in every:
        whole = walk(ti, 0, S)
        met = {(e[0], e[1]): e for e in whole}
        assert len(met) == len(whole)
        for h in range(2):
            for _, qlo, qn in every:
                block = see[qlo:qlo + qn, lo:lo + n]
                if block.any():
                    assert (h, qlo) in met and met[h, qlo][2] == qn
                    assert block.all() or met[h, qlo][3] == 1
                elif (h, qlo) in met:
                    # a tile with first tokens meets every later tile
                    assert lo < k and met[h, qlo][3] == 1
        for span in (128, 384, 4096):
            cut = [e for s in range(0, S, span) for e in walk(ti, s, min(S, s + span))]
            assert sorted(cut) == sorted(whole)


@pytest.mark.parametrize("S", LENGTHS)
@pytest.mark.parametrize("n_sink", [0, 1, 4, 128, 129, 300, 2000])
def test_tiles_with_first_tokens(harness, S, n_sink):
    k = min(n_sink, S)
    want = [lo for _, lo, _ in tiles(S, 128) if lo < k]
    buf = (ctypes.c_int * CAP)()
    n = harness.ra_win_sink_tiles(S, k, -(-k // 128) + 2, buf)
    assert buf[:n] == want
