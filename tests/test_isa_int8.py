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


def test_dma_registers_are_old_enough(lines):
    """A scalar register that a vector instruction writes may be read by a memory instruction five wait
    states later at the earliest, and the compiler does not look into the assembly for that: back from each
    load, over every way that leads to it."""
    code = [ln.split(";")[0].strip() for ln in lines]
    code = [ln for ln in code if ln and (not ln.startswith(".") or re.fullmatch(r"\.L\w+:", ln))]
    label = {ln[:-1]: i for i, ln in enumerate(code) if ln.endswith(":")}
    jumps = {}
    for i, ln in enumerate(code):
        m = re.match(r"s_c?branch\S* (\S+)", ln)
        if m and m[1] in label:
            jumps.setdefault(label[m[1]], []).append(i)

    def scalars(text):
        return {r for m in re.finditer(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text)
                for r in (range(int(m[1]), int(m[2]) + 1) if m[1] else (int(m[3]),))}

    loads = [i for i, ln in enumerate(code) if ln.endswith("offen lds")]
    assert len(loads) > 100
    written = 0
    for i in loads:
        need, todo, seen = scalars(code[i].split(",", 1)[1]), [(i - 1, 0)], set()
        while todo:
            j, waited = todo.pop()
            if waited >= 5 or j < 0 or (j, waited) in seen:
                continue
            seen.add((j, waited))
            ln = code[j]
            if ln.endswith(":"):
                todo += [(k, waited) for k in jumps.get(j, ())]
                if not re.match(r"s_branch|s_endpgm|s_setpc", code[j - 1]):
                    todo.append((j - 1, waited))
                continue
            w = re.match(r"v_(?:readf|readl|cmp|div_s|mad_|\S+_co_)\S* (?:v\S+, )?(s\d+|s\[\d+:\d+\])(?:,|$)", ln)
            if w:
                written += 1
                assert not need & scalars(w[1]), (ln, code[i])
            nop = re.match(r"s_nop (\d+)", ln)
            todo.append((j - 1, waited + (int(nop[1]) + 1 if nop else 1)))
    assert written, "expected vector instructions that write scalar registers near some load"
