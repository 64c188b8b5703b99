"""The INT8 product's LDS-DMA loads set m0 from inline assembly, which the compiler is not told
about: sound only while no compiler-generated instruction in the kernel reads or writes m0.
The generated gfx950 assembly is checked for exactly that, and for a wait for the wave's own
LDS reads before every barrier."""
import os
import re
import subprocess
import tempfile

import pytest

from precision_quantization_block_amd import _build

SRC = os.path.join(_build.CSRC, "k_gemm_int8.hip")


@pytest.fixture(scope="module")
def lines():
    if not os.path.exists(_build.HIPCC):
        pytest.skip("hipcc not available")
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k.s")
        flags = [f for f in _build.FLAGS if f != "-fPIC"]
        subprocess.run([_build.HIPCC, *flags, "-S", "--offload-device-only", SRC, "-o", out], check=True, capture_output=True)
        return [ln.strip() for ln in open(out) if not ln.strip().startswith(";")]


def test_only_the_dma_asm_touches_m0(lines):
    uses = [i for i, ln in enumerate(lines) if re.search(r"\bm0\b", ln)]
    assert uses, "expected the DMA sequences to set m0"
    for i in uses:
        assert re.fullmatch(r"s_mov_b32 m0, s\d+", lines[i]), lines[i]
        assert lines[i + 1] == "s_nop 0", lines[i + 1]
        assert re.fullmatch(r"buffer_load_dwordx4 v\d+, s\[\d+:\d+\], s\d+ offen lds", lines[i + 2]), lines[i + 2]


def test_barriers_wait_for_their_waves_lds_reads(lines):
    at = [i for i, ln in enumerate(lines) if ln == "s_barrier"]
    assert at
    for i in at:
        assert lines[i - 1].startswith("s_waitcnt") and "lgkmcnt(0)" in lines[i - 1], lines[i - 1]
