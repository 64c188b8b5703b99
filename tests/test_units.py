"""The cut of a request into units of tokens (csrc/units.h), compiled for the host and
checked at the largest lengths against 64-bit arithmetic: a wave looks pages up as far
as 256 units ahead, where 32-bit token numbers pass 2^31, and the units of an item come
from a sum that passes 2^31 too."""
import os
import shutil
import subprocess

import pytest

from precision_quantization_block_amd import _build

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "csrc", "units_check.cpp")


def check(header_dir, exe):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    subprocess.run(["g++", "-O1", "-fwrapv", "-std=c++17", f"-I{header_dir}", SRC, "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True)
    return [[int(x) for x in line.split()] for line in out.stdout.splitlines()]


def planted(tmp_path, *changes):
    text = open(os.path.join(_build.CSRC, "units.h")).read()
    for old, new in changes:
        assert text.count(old) == 1
        text = text.replace(old, new)
    (tmp_path / "units.h").write_text(text)
    return check(str(tmp_path), str(tmp_path / "planted"))


def test_units_at_the_largest_lengths(tmp_path):
    (columns, bad), (cuts, bad_cuts) = check(_build.CSRC, str(tmp_path / "units"))
    assert columns > 1_000_000 and bad == 0
    assert cuts > 300 and bad_cuts == 0


def test_the_check_sees_signed_token_numbers(tmp_path):
    out = planted(tmp_path, ("const uint32_t t = (uint32_t)u * kUnit + 16u * (uint32_t)group;",
                             "const int32_t t = u * kUnit + 16 * group;"), ("t < (uint32_t)kv ?", "t < kv ?"))
    assert out[0][1] > 0


def test_the_check_sees_a_share_without_a_bound(tmp_path):
    out = planted(tmp_path, (" : c > kMaxUnits ? kMaxUnits : c;", " : c;"))
    assert out[1][1] > 0
