"""Which kernel and tile the INT8 product takes (csrc/int8_tiles.h), compiled for the host: the
GPU tests' products have to reach every one of them, and every way in which it stores its results."""
import itertools
import os
import shutil
import subprocess

import pytest

from precision_quantization_block_amd import _build
from test_gpu_int8_layer_edges import PRODUCTS

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "csrc", "int8_tiles_check.cpp")
KERNELS = ("ring", "deep", "tile")


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("tiles") / "tiles")
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{_build.CSRC}", SRC, "-o", exe], check=True)

    def run(shapes):
        text = "".join("%d %d %d\n" % s for s in shapes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        rows = [[int(x) for x in line.split()] for line in out.splitlines()]
        return [((KERNELS[r[0]], r[1], r[2]), bool(r[3])) for r in rows]
    return run


def test_the_gpu_tests_reach_every_kernel(choose):
    """Of each kernel: rows of whole lines and others, more rows than channels and fewer."""
    assert len({p[:3] for p in PRODUCTS}) == len(PRODUCTS) == 9 + 1 + 2
    for *kernel, shapes in PRODUCTS:
        got = choose(shapes)
        assert [k for k, _ in got] == [tuple(kernel)] * len(shapes)
        assert [along for _, along in got] == [m > n for m, n, _ in shapes]
        seen = {(n % 64 == 0, m > n) for m, n, _ in shapes}
        assert seen == set(itertools.product((False, True), repeat=2)), kernel


@pytest.mark.parametrize("edge,grid", [(128, 512), (256, 256)])
def test_the_gpu_tests_reach_what_staying_workgroups_do(edge, grid):
    """With rows of whole lines: one, two, an odd and an even number of blocks of K of several tiles in
    turn, the last rows inside a wave's part of a tile."""
    shapes = [p for *kernel, products in PRODUCTS if kernel == ["tile", edge, edge] for p in products if p[1] % 64 == 0]
    for m, n, _ in shapes:
        assert -(-m // edge) * -(-n // edge) > grid and m % 16
    blocks = {-(-k // 128) for _, _, k in shapes}
    assert {1, 2} <= blocks and any(b > 2 and b % 2 for b in blocks) and any(b > 2 and b % 2 == 0 for b in blocks)


def test_every_shape_has_a_kernel(choose):
    """The largest and smallest sizes that the product accepts, too."""
    sizes = (1, 16, 100, 4096, 70000, 1 << 20, (1 << 30) - 1)
    shapes = [(m, n, k) for m in sizes for n in sizes for k in (0, 16, 4096, 131056)
              if -(-m // 128) * -(-n // 128) < 1 << 23]
    rings = [(16, 16), (16, 32), (32, 16), (32, 32), (32, 64), (64, 32), (64, 64), (128, 64), (64, 128)]
    known = {("ring", *r) for r in rings} | {("deep", 128, 64), ("tile", 128, 128), ("tile", 256, 256)}
    for shape, (kernel, _) in zip(shapes, choose(shapes)):
        assert kernel in known, shape
        tiles = -(-shape[0] // kernel[1]) * -(-shape[1] // kernel[2])
        assert kernel[0] == "tile" or tiles < 1 << 22, shape      # a grid of 512 threads each stays below 2^32
