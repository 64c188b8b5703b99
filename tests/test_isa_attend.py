"""The attention kernels' LDS-DMA loads set m0 and name scalar base registers from
inline assembly, which the compiler looks no further into.  That is sound only
while no compiler-generated instruction reads or writes m0, and while no base
register comes from a vector instruction less than five wait states before the
load that reads it (a scalar register written by a vector instruction and read by a
memory instruction needs five).  This test compiles the kernel source to gfx950
assembly with the library's own flags and checks both."""
import os
import re
import subprocess
import tempfile

import pytest

from precision_quantization_block_amd import _build

SRC = os.path.join(_build.CSRC, "k_attend.hip")


@pytest.fixture(scope="module")
def lines():
    if not os.path.exists(_build.HIPCC):
        pytest.skip("hipcc not available")
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k_attend.s")
        flags = [f for f in _build.FLAGS if f != "-fPIC"]
        subprocess.run([_build.HIPCC, *flags, "-S", "--offload-device-only", SRC, "-o", out],
                       check=True, capture_output=True)
        text = [ln.strip() for ln in open(out)]
    return [ln for ln in text if ln and not ln.startswith((";", "."))]


def test_only_the_dma_asm_touches_m0(lines):
    uses = [i for i, ln in enumerate(lines) if re.search(r"\bm0\b", ln)]
    assert uses, "expected the DMA sequences to set m0"
    for i in uses:
        assert re.fullmatch(r"s_mov_b32 m0, s\d+", lines[i]), lines[i]
        assert lines[i + 1] == "s_nop 0", lines[i + 1]
        assert lines[i + 2].startswith("global_load_lds_dword"), lines[i + 2]


def test_dma_bases_are_old_enough(lines):
    seen = 0
    for i, ln in enumerate(lines):
        m = re.match(r"global_load_lds_dwordx4 v\d+, s\[(\d+):(\d+)\]", ln)
        if not m:
            continue
        seen += 1
        base, waited = {int(m.group(1)), int(m.group(2))}, 0
        for prev in reversed(lines[max(0, i - 8):i]):
            if waited >= 5:
                break
            w = re.match(r"v_\S+ s(\d+)|v_\S+ s\[(\d+):(\d+)\]", prev)
            if w:
                lo = int(w.group(1) or w.group(2))
                hi = int(w.group(1) or w.group(3))
                assert not base & set(range(lo, hi + 1)), (prev, ln)
            nop = re.match(r"s_nop (\d+)", prev)
            waited += int(nop.group(1)) + 1 if nop else 1
    assert seen, "expected DMA loads with a scalar base"
