"""Host checks of the TMA views of the int8 x int8 products: every in-bounds element of
every box that a kernel places lies inside its tensor, and every row that a kernel keeps is
the one its epilogue assumes (see test_tma_views.py, whose box walk this uses)."""
import os
import shutil
import subprocess

import pytest

from test_tma_views import CSRC, CUDA_INC, ROOT, box_rows, read_views

# (E, n, K): n weight rows of K per expert; single experts, partial 128- and 256-row tiles,
# K that ends inside a box
SIZES = [(1, 32, 16), (1, 64, 128), (3, 96, 144), (2, 160, 272), (5, 288, 704), (4, 1408, 2816), (2, 320, 4096)]


@pytest.fixture(scope="module")
def views_bin(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA_INC, "cuda.h")):
        pytest.skip("needs g++ and the CUDA headers")
    out = str(tmp_path_factory.mktemp("views8") / "tma_views8")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, "-I", CUDA_INC,
                        os.path.join(ROOT, "tests", "tma_views8_main.cpp"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


@pytest.mark.parametrize("E,n,K", SIZES)
def test_int8_weight_views(views_bin, E, n, K):
    v = read_views(views_bin, E, n, K)
    total = E * n * K
    for name, view in v.items():
        assert view["elem"] == 1 and view["dims"][0] == K and view["box"][0] == 128, name
        assert all(s % 16 == 0 for s in view["strides"]) and all(1 <= b <= 256 for b in view["box"]), name
    for chunked in (False, True):
        I = n // 2
        row = lambda g, j: g * n + ((j % 2) * I + j // 2 if chunked else j)
        sfx = "_chunked" if chunked else ""
        for g in range(E):
            for w0 in range(0, (n + 255) // 256 * 256, 128):
                # fragment order: box row 32 Q + 8 q + j = row w0 + 32 Q + 4 j + q
                at = [0, 0, 0, 0, g * (I // 8) + w0 // 32] if chunked else [0, 0, 0, w0 // 32, g]
                seen = set()
                for i, off in box_rows(v["quads" + sfx], at):
                    assert off + K <= total
                    j = w0 + 32 * (i // 32) + 4 * (i % 8) + (i % 32) // 8
                    if j < n:
                        assert off == row(g, j) * K
                        seen.add(j)
                assert seen == set(range(w0, min(w0 + 128, n)))
                # pair order: box row i = row w0 + i
                if w0 >= n:
                    continue
                seen = set()
                for i, off in box_rows(v["pairs" + sfx], [0, 0, w0 // 2, g]):
                    assert off + K <= total
                    assert off == row(g, w0 + i) * K
                    seen.add(w0 + i)
                assert seen == set(range(w0, min(w0 + 128, n)))
