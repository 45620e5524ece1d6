"""The windowed walks (csrc/window_iter.cuh), compiled for the host, against
the mask itself: a walk holds every tile with a visible pair once, no tile
without one, in ring order, and flags exactly the tiles that need masking."""

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


def facts(h, S, P, order, tile):
    f = (ctypes.c_int * 3)()
    assert h.ra_win_facts(S, P, order, tile, f) == 0
    return list(f)


def tiles(S, seg_len, n_seg, nt, tile):
    """(segment, index, first position, tokens) of every tile that holds any."""
    for seg in range(n_seg):
        for ti in range(nt):
            lo = seg * seg_len + ti * tile
            n = min(tile, min(seg_len, S - seg * seg_len) - ti * tile)
            if n > 0:
                yield seg, ti, lo, n


SHAPES = [(1, 1, 0), (130, 1, 0), (777, 1, 0), (1000, 4, 1), (1001, 3, 0), (2048, 2, 1), (700, 8, 1), (5, 4, 1),
          (1300, 1, 1)]
WINDOWS = [(1, 0), (1, 1), (64, 4), (100, 130), (128, 0), (129, 128), (500, 260), (5000, 0), (3, 5000)]


def clamp(w, k, S):
    return min(w, S), min(k, S)


@pytest.mark.parametrize("S,P,order", SHAPES)
@pytest.mark.parametrize("window,n_sink", WINDOWS)
@pytest.mark.parametrize("tile,rows", [(128, 256), (128, 128), (64, 64)])
def test_key_walk(harness, S, P, order, window, n_sink, tile, rows):
    w, k = clamp(window, n_sink, S)
    seg_len, n_seg, nt = facts(harness, S, P, order, tile)
    see = allowed(np.arange(S), np.arange(S), w, k)
    every = list(tiles(S, seg_len, n_seg, nt, tile))
    buf = (ctypes.c_int * (5 * CAP))()
    for seg, ti, lo, _ in every:
        if ti % (rows // tile):
            continue
        hi = min(lo + rows, min((seg + 1) * seg_len, S))
        n = harness.ra_win_walk(S, P, order, tile, w, k, seg, ti, rows, buf, CAP)
        assert n >= 0
        walk = [tuple(buf[5 * i:5 * i + 5]) for i in range(n)]
        met = {e[2]: e for e in walk}
        assert len(met) == n
        for _, _, klo, kn in every:
            block = see[lo:hi, klo:klo + kn]
            assert (klo in met) == block.any()
            if klo in met:
                assert met[klo][3] == kn
                assert block.all() or met[klo][4] == 2          # masked tiles are flagged
                if kn == tile and hi - lo == rows:
                    assert (met[klo][4] == 1) == block.all()    # and full ones are not
        owner = seg if order == 0 or seg < P else 2 * P - 1 - seg
        assert [e[0] for e in walk] == sorted(e[0] for e in walk)
        assert all(e[1] == (owner - e[0]) % P for e in walk)


@pytest.mark.parametrize("S,P,order", SHAPES)
@pytest.mark.parametrize("window,n_sink", WINDOWS)
def test_query_walk_and_its_shares(harness, S, P, order, window, n_sink):
    w, k = clamp(window, n_sink, S)
    seg_len, n_seg, nt = facts(harness, S, P, order, 128)
    see = allowed(np.arange(S), np.arange(S), w, k)
    every = list(tiles(S, seg_len, n_seg, nt, 128))
    buf = (ctypes.c_int * (4 * CAP))()

    def walk(seg, ti, a, b):
        n = harness.ra_win_qwalk(S, P, order, w, k, seg, ti, 2, a, b, buf, CAP)
        return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]

    for seg, ti, lo, n in every:
        whole = walk(seg, ti, 0, S)
        met = {(e[0], e[1]): e for e in whole}
        assert len(met) == len(whole)
        for h in range(2):
            for _, _, qlo, qn in every:
                block = see[qlo:qlo + qn, lo:lo + n]
                if block.any():
                    assert (h, qlo) in met and met[h, qlo][2] == qn
                    assert block.all() or met[h, qlo][3] == 1
                elif (h, qlo) in met:
                    # a tile with first tokens meets every later tile
                    assert lo < k and met[h, qlo][3] == 1
        for span in (128, 384, 4096):
            cut = [e for s in range(0, S, span) for e in walk(seg, ti, s, min(S, s + span))]
            assert sorted(cut) == sorted(whole)


@pytest.mark.parametrize("S,P,order", SHAPES)
@pytest.mark.parametrize("n_sink", [0, 1, 4, 128, 129, 300, 2000])
def test_tiles_with_first_tokens(harness, S, P, order, n_sink):
    k = min(n_sink, S)
    seg_len, n_seg, nt = facts(harness, S, P, order, 128)
    want = sorted(lo for _, _, lo, _ in tiles(S, seg_len, n_seg, nt, 128) if lo < k)
    most = min(n_seg * nt, -(-k // 128) + n_seg + 1)       # the bound that packed batches use
    buf = (ctypes.c_int * CAP)()
    n = harness.ra_win_sink_tiles(S, P, order, k, most, buf)
    assert buf[:n] == want
