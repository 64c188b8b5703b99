"""Host-side parts of the paged cache's binding (CPU only)."""
import itertools
import os
import subprocess
import sys

from precision_quantization_block_amd import pqb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rows_that_meet_a_block():
    """Against the sets of bytes, for blocks before, inside, between and behind the rows."""
    for size, gap, count in itertools.product((1, 4, 7), (0, 1, 5, 30), (1, 2, 3, 5)):
        step, base = size + gap, 200
        rows = {base + t * step + i for t in range(count) for i in range(size)}
        for other in range(base - count * size - 3, base + count * step + 3):
            want = not rows.isdisjoint(range(other, other + count * size))
            assert pqb._rows_meet(base, step, size, count, other) == want, (size, gap, count, other)


def test_import_without_torchs_gpu_names():
    """A torch built without GPU support lacks them; what runs on the host works with it."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import precision_quantization_block_amd as pqb\n"
            "print(pqb.query_sizes('fp8_e4m3', '1x128', 1, 128, 256)['codes'], pqb.PLAN_FLAGS['pages'])\n")
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split() == [str(128 * 256), "1"]
