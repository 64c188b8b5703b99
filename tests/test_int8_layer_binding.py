"""What the INT8 layer refuses, and its host parts, on the CPU: the C entry points are called with
addresses that are never used, since every call here is refused or empty; the binding with CPU
tensors."""
import ctypes
import itertools
import math

import pytest
import torch

import precision_quantization_block_amd as pqb
from precision_quantization_block_amd import pqb as binding

OK, NULL, ENUM, COMBO, SHAPE, ALIGN, VALUE = 0, -1, -2, -3, -4, -5, -9
P = 0x1000000      # an aligned address nobody reads


@pytest.fixture(scope="module")
def L():
    return pqb.lib()


# ---------------------------------------------------------------------------
# gemm_int8
# ---------------------------------------------------------------------------

def gemm(L, m=4, n=8, k=64, out=0, bias=None, c=P, a=None, b=None, sa=None, sb=None):
    A = binding._Int8Mat(P, P, m, k, 1, 0)
    B = binding._Int8Mat(P, P, n, k, 1, 0)
    for mat, changes in ((A, a), (B, b)):
        for f, v in (changes or {}).items():
            setattr(mat, f, v)
    return L.pqb_gemm_int8(ctypes.byref(A), ctypes.byref(B), k, bias, out, c, None)


@pytest.mark.parametrize("want,changes", [
    (ENUM, dict(out=2)), (ENUM, dict(a=dict(reserved=1))), (ENUM, dict(b=dict(per_row=2))),
    (SHAPE, dict(k=8)), (SHAPE, dict(k=-16)), (SHAPE, dict(k=131072)), (SHAPE, dict(m=-1)), (SHAPE, dict(n=1 << 30)),
    (SHAPE, dict(m=1 << 29, n=1 << 29)), (SHAPE, dict(a=dict(stride=48))), (SHAPE, dict(b=dict(stride=72))),
    (SHAPE, dict(b=dict(stride=1 << 23))), (NULL, dict(c=None)), (NULL, dict(a=dict(codes=None))),
    (NULL, dict(b=dict(scales=None))), (ALIGN, dict(c=P + 8)), (ALIGN, dict(a=dict(codes=P + 4))),
    (ALIGN, dict(b=dict(scales=P + 2))), (ALIGN, dict(bias=P + 1)), (OK, dict(m=0)), (OK, dict(n=0)),
    (OK, dict(m=0, c=None, a=dict(codes=None, scales=None)))])
def test_gemm_refusals(L, want, changes):
    assert gemm(L, **changes) == want


def test_gemm_null_operands(L):
    A = binding._Int8Mat(P, P, 1, 16, 1, 0)
    assert L.pqb_gemm_int8(None, ctypes.byref(A), 16, None, 0, P, None) == NULL
    assert L.pqb_gemm_int8(ctypes.byref(A), None, 16, None, 0, P, None) == NULL


# ---------------------------------------------------------------------------
# norm_quant, act_quant
# ---------------------------------------------------------------------------

def norm(L, **changes):
    n = binding._Norm()
    for f in "x residual weight h out scales".split():
        setattr(n, f, P)
    n.rows, n.cols, n.gate_rows = 4, 256, 2
    n.x_stride = n.residual_stride = n.gate_stride = n.h_stride = 256
    n.residual_scale, n.eps, n.fmt, n.gran = 1.0, 1e-6, 6, 1
    for f, v in changes.items():
        setattr(n, f, v)
    return L.pqb_norm_quant(ctypes.byref(n), None)


@pytest.mark.parametrize("want,changes", [
    (ENUM, dict(dtype=2)), (ENUM, dict(kind=2)), (ENUM, dict(reserved=1)), (ENUM, dict(fmt=7)), (ENUM, dict(gran=9)),
    (ENUM, dict(fmt=-2)), (COMBO, dict(fmt=6, gran=2)), (COMBO, dict(fmt=0, gran=0)), (COMBO, dict(fmt=0, gran=3)),
    (COMBO, dict(fmt=1, gran=4)), (COMBO, dict(fmt=3, gran=6)), (COMBO, dict(fmt=6, gran=0)),
    (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=0)), (SHAPE, dict(cols=32776, x_stride=40000, residual_stride=40000, h_stride=40000)),
    (SHAPE, dict(rows=1 << 22)), (SHAPE, dict(rows=1 << 18, cols=32768, x_stride=32768, residual_stride=32768, h_stride=32768)),
    (SHAPE, dict(fmt=0, gran=2, cols=200)), (SHAPE, dict(x_stride=255)), (SHAPE, dict(residual_stride=1 << 40)),
    (SHAPE, dict(h_stride=0)), (SHAPE, dict(gate=P, gate_rows=3)), (SHAPE, dict(gate=P, gate_rows=0)),
    (SHAPE, dict(gate=P, gate_stride=8)), (VALUE, dict(eps=0.0)), (VALUE, dict(eps=-1.0)), (VALUE, dict(eps=float("nan"))),
    (VALUE, dict(eps=2.0)), (VALUE, dict(residual_scale=float("inf"))), (VALUE, dict(residual_scale=float("nan"))),
    (NULL, dict(bias=P)), (NULL, dict(x=None)), (NULL, dict(out=None)), (NULL, dict(scales=None)), (NULL, dict(h=None)),
    (NULL, dict(residual=None)), (ALIGN, dict(x=P + 2)), (ALIGN, dict(scales=P + 2)), (ALIGN, dict(weight=P + 1)),
    (ALIGN, dict(dtype=1, h=P + 1)), (ALIGN, dict(fmt=0, gran=2, x=P + 4)), (ALIGN, dict(fmt=0, gran=2, residual_stride=257)),
    (OK, dict(rows=0)), (OK, dict(rows=0, x=None, out=None, scales=None))])
def test_norm_refusals(L, want, changes):
    assert norm(L, **changes) == want


@pytest.mark.parametrize("want,gate_rows", [(OK, 0), (OK, 1), (OK, 7), (SHAPE, -1)])
def test_norm_of_no_rows_takes_any_gate(L, want, gate_rows):
    assert norm(L, rows=0, gate=P, gate_rows=gate_rows) == want


def test_norm_null(L):
    assert L.pqb_norm_quant(None, None) == NULL


def act(L, gate=P, up=P, dtype=0, rows=4, cols=256, gs=256, us=256, kind=0, fmt=6, gran=1, out=P, scales=P):
    return L.pqb_act_quant(gate, up, dtype, rows, cols, gs, us, kind, fmt, gran, out, scales, None)


@pytest.mark.parametrize("want,changes", [
    (ENUM, dict(dtype=5)), (ENUM, dict(kind=4)), (ENUM, dict(kind=-1)), (ENUM, dict(fmt=99)), (COMBO, dict(fmt=6, gran=2)),
    (COMBO, dict(fmt=2, gran=5)), (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=0)), (SHAPE, dict(cols=32769, gs=40000, us=40000)),
    (SHAPE, dict(gs=255)), (SHAPE, dict(us=255)), (SHAPE, dict(us=1 << 40)), (SHAPE, dict(rows=1 << 22)),
    (SHAPE, dict(fmt=-1, rows=1 << 21, cols=4096, gs=4096, us=4096)), (SHAPE, dict(fmt=0, gran=2, cols=64)),
    (SHAPE, dict(fmt=-1, cols=(1 << 31) - 1, gs=1 << 31, us=1 << 31)),
    (NULL, dict(gate=None)), (NULL, dict(out=None)), (NULL, dict(scales=None)), (ALIGN, dict(gate=P + 2)), (ALIGN, dict(up=P + 1, dtype=1)),
    (ALIGN, dict(scales=P + 1)), (ALIGN, dict(fmt=0, gran=2, up=P + 4)), (ALIGN, dict(fmt=0, gran=2, gs=260)), (OK, dict(rows=0)),
    (OK, dict(rows=0, gate=None, out=None))])
def test_act_refusals(L, want, changes):
    assert act(L, **changes) == want


# ---------------------------------------------------------------------------
# rope
# ---------------------------------------------------------------------------

def rope(L, **changes):
    r = binding._Rope()
    for f in "q k q_out k_out positions angles".split():
        setattr(r, f, P)
    r.tokens, r.q_heads, r.k_heads, r.dim, r.rot = 4, 8, 2, 64, 64
    r.q_stride = r.q_out_stride = 512
    r.k_stride = r.k_out_stride = 128
    r.amplitude = 1.0
    for f, v in changes.items():
        setattr(r, f, v)
    return L.pqb_rope(ctypes.byref(r), None)


@pytest.mark.parametrize("want,changes", [
    (ENUM, dict(dtype=2)), (ENUM, dict(reserved=3)), (SHAPE, dict(tokens=-1)), (SHAPE, dict(tokens=1 << 24)), (SHAPE, dict(dim=1)),
    (SHAPE, dict(dim=1026, q_stride=1 << 20, k_stride=1 << 20, q_out_stride=1 << 20, k_out_stride=1 << 20)), (SHAPE, dict(rot=3)),
    (SHAPE, dict(rot=0)), (SHAPE, dict(rot=66)), (SHAPE, dict(q_heads=0)), (SHAPE, dict(q_heads=8193)), (SHAPE, dict(k_heads=0)),
    (SHAPE, dict(k=None, k_out=None)), (SHAPE, dict(q_stride=511)), (SHAPE, dict(k_out_stride=64)), (SHAPE, dict(batch=-1)),
    (SHAPE, dict(k_stride=1 << 40)), (VALUE, dict(amplitude=float("nan"))), (VALUE, dict(amplitude=float("-inf"))),
    (NULL, dict(q=None)), (NULL, dict(q_out=None)), (NULL, dict(k=None)), (NULL, dict(angles=None)),
    (NULL, dict(positions=None, batch=2)), (NULL, dict(positions=None, batch=2, q_starts=P)), (ALIGN, dict(angles=P + 4)),
    (ALIGN, dict(positions=P + 2)), (ALIGN, dict(q=P + 2)), (ALIGN, dict(dtype=1, k_out=P + 1)), (OK, dict(tokens=0)),
    (OK, dict(positions=None, batch=0))])
def test_rope_refusals(L, want, changes):
    assert rope(L, **changes) == want


def test_rope_null(L):
    assert L.pqb_rope(None, None) == NULL


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------

def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 64)
    c, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: pqb.gemm_int8((c, s), (c, s)), lambda: pqb.norm_quant(x), lambda: pqb.act_quant(x),
                 lambda: pqb.rope(x.view(4, 1, 64), None, torch.zeros(4, dtype=torch.int32), pqb.rope_table(64, device="cpu"))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="int8_sym"):
        pqb.gemm_int8(pqb.Quantized(c.view(-1), s, None, "fp8_e4m3", "row", (1, 4, 64)), (c, s))
    with pytest.raises(ValueError, match="rows, k"):
        pqb.gemm_int8((c.view(-1), s), (c, s))


def test_rows_that_share_memory():
    """Against the sets of bytes, for rows of equal and other strides in one buffer."""
    buf = torch.zeros(64, dtype=torch.int8)

    def rows(at, n, w, stride):
        return buf.as_strided((n, w), (stride, 1), at), {at + i * stride + j for i in range(n) for j in range(w)}

    missed = 0
    for (at, n, w, st), (at2, n2, w2, st2) in itertools.product(
            itertools.product((0, 5), (1, 3), (2, 4), (6, 9)), itertools.product(range(0, 24), (1, 2), (1, 3), (6, 9))):
        (t, own), (o, other) = rows(at, n, w, st), rows(at2, n2, w2, st2)
        meet, said = not own.isdisjoint(other), binding._rows_share(t, st, o, st2)
        assert said or not meet, (at, n, w, st, at2, n2, w2, st2)      # never misses one
        if st == st2 and n > 1 and n2 > 1:                             # one stride: refuses gaps only at the ends
            missed += said != meet
    assert missed < 40


def test_rope_tables():
    """Each scaling against its definition written out pair by pair."""
    make = lambda *a, **k: pqb.rope_table(*a, device="cpu", **k)  # noqa: E731
    plain = [10000.0 ** (-2 * i / 64) for i in range(32)]
    t = make(64)
    assert t.angles.dtype is torch.float64 and t.amplitude == 1.0 and not t.interleaved
    assert t.angles.tolist() == pytest.approx(plain, rel=1e-14)
    assert make(64, scaling="linear", factor=4.0).angles.tolist() == pytest.approx([f / 4 for f in plain], rel=1e-14)
    ntk = make(64, scaling="ntk", factor=8.0, interleaved=True)
    assert ntk.interleaved and ntk.angles[0] == 1.0 and ntk.angles[31].item() == pytest.approx(plain[31] / 8, rel=1e-12)
    got = make(64, scaling="by_turns", factor=8.0, original_length=8192).angles.tolist()
    for f, y in zip(plain, got):
        turns = 8192 * f / (2 * math.pi)
        want = f if turns >= 4 else f / 8 if turns <= 1 else f / 8 + (f - f / 8) * (turns - 1) / 3
        assert y == pytest.approx(want, rel=1e-12)
    y = make(64, scaling="yarn", factor=16.0, original_length=4096)
    assert y.amplitude == pytest.approx(1 + 0.1 * math.log(16))
    first = math.floor(64 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(10000)))
    last = math.ceil(64 * math.log(4096 / (2 * math.pi)) / (2 * math.log(10000)))
    for i, (f, v) in enumerate(zip(plain, y.angles.tolist())):
        share = min(max((i - first) / (last - first), 0), 1)
        assert v == pytest.approx(f * (1 - share) + f / 16 * share, rel=1e-12)
    assert make(64, scaling="yarn", factor=16.0, amplitude=2.0).amplitude == 2.0
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=64, scaling="other"), dict(rotary_dim=64, factor=0.0),
                dict(rotary_dim=2, scaling="ntk"), dict(rotary_dim=64, scaling="yarn", low=5.0, high=2.0)):
        with pytest.raises(ValueError):
            pqb.rope_table(device="cpu", **bad)


@pytest.mark.parametrize("base", [1.0, 0.5])
def test_yarn_needs_angles_that_fall(base):
    """The pair that makes a number of turns is sought by log base."""
    with pytest.raises(ValueError, match="base"):
        pqb.rope_table(64, base, scaling="yarn", factor=4.0, device="cpu")
    assert pqb.rope_table(64, base, scaling="by_turns", factor=4.0, device="cpu").angles.isfinite().all()
