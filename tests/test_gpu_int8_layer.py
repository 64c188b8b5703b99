"""The INT8 layer on the GPU (gemm_int8, norm_quant, act_quant, rope) against plain forms in
64 bits.  What has one right answer in float32 (integer sums and their scales, the residual
stream, an RMS norm's codes) is compared bit for bit; the rest within bounds counted from the
roundings that its header names: u = 2^-24 is half a step of float32, eps / 2 half a step of
the output's type."""
import math

import numpy as np
import pytest
import torch

import precision_quantization_block_amd as pqb

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3, E5M2, I8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.int8
U = 2.0 ** -24
# A row's sum of n <= 32768 squares: 32 of a thread one after the other, 6 + 2 steps over a wave, up to 16
# waves: 56 roundings, and r takes half of their error, one square root, one sum, one quotient.
R_TOL = 34 * U


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def half_step(dtype):
    return 0.0 if dtype is F64 else torch.finfo(dtype).eps / 2


def strided(t, pad, shift=0):
    """t's values in rows `pad` elements further apart, from `shift` elements on."""
    rows, cols = t.shape
    big = torch.full((rows * (cols + pad) + shift + 1,), float("nan") if t.is_floating_point() else 99, dtype=t.dtype,
                     device=t.device)
    v = big[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def close(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (bad.sum().item(), (got.double() - want).abs()[bad][0].item(),
                           (tol.expand_as(want)[bad][0] if torch.is_tensor(tol) else tol))


# ---------------------------------------------------------------------------
# gemm_int8
# ---------------------------------------------------------------------------

def codes(g, rows, k, full=False):
    if full:
        return torch.randint(-128, 128, (rows, k), generator=g, device=DEV).to(I8)
    return (normal(g, rows, k) * 40).round().clamp(-127, 127).to(I8)


def product(a, sa, b, sb, bias, dtype):
    """The definition with an exact sum and float32 roundings one after the other."""
    s = torch.matmul(a.double(), b.double().t())
    assert s.abs().max() < 2 ** 31 if s.numel() else True
    v = s.float() * sa.reshape(-1, 1) * sb.reshape(1, -1)
    return (v if bias is None else v + bias).to(dtype)


def check_gemm(m, n, k, dtype, seed=0, bias=False, full=False, one_scale=(False, False), pads=(0, 0)):
    g = gen(seed)
    a, b = codes(g, m, k, full), codes(g, n, k, full)
    sa = torch.rand(1 if one_scale[0] else m, generator=g, device=DEV) * 0.02 + 1e-3
    sb = torch.rand(1 if one_scale[1] else n, generator=g, device=DEV) * 0.02 + 1e-3
    c = normal(g, n) if bias else None
    want = product(a, sa, b, sb, c, dtype)
    if pads[0]:
        a = strided(a, pads[0])
    if pads[1]:
        b = strided(b, pads[1])
    got = pqb.gemm_int8((a, sa), (b, sb), dtype, bias=c)
    assert got.dtype is dtype and torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 33, 64, 65, 100, 129, 257])
@pytest.mark.parametrize("n,k", [(1, 16), (7, 48), (128, 128), (200, 656), (1001, 2064), (264, 4096)])
def test_gemm_shapes(m, n, k, dtype):
    check_gemm(m, n, k, dtype, seed=m * 7 + n, bias=m % 2 == 1)


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (20, 4100, 1040), (20, 8200, 400), (20, 17000, 272), (60, 4000, 528), (60, 8200, 400),
                                   (60, 16400, 272), (60, 32800, 144), (100, 8200, 400), (100, 16400, 144), (130, 2000, 80), (500, 4100, 272),
                                   (1100, 7000, 144), (2100, 6000, 336), (2500, 5000, 16), (5000, 7000, 272), (300, 70000, 144), (3, 14336, 4096), (64, 1024, 14336), (48, 4100, 131056), (512, 4096, 1040),
                                   (777, 1001, 2064), (1024, 2048, 7168), (2049, 2500, 1536), (4100, 520, 144)])
def test_gemm_large(m, n, k):
    check_gemm(m, n, k, BF, seed=k, bias=n % 2 == 1)


@pytest.mark.parametrize("k", [16, 144, 400, 1040, 2512])
@pytest.mark.parametrize("m,n", [(9, 300), (50, 1005), (10, 4201), (99, 1075), (38, 1418), (367, 180), (20, 4100), (134, 1616), (13, 14400),
                                 (22, 34746), (41, 4100), (302, 1309), (60, 8200), (378, 2048), (64, 16401), (136, 26739), (111, 8201),
                                 (500, 4090), (1000, 4090), (244, 81468), (1300, 7001), (2100, 6001), (2500, 5000)])
def test_gemm_every_tile(m, n, k):
    """Each tile that the launcher takes, twice or more (16 x 16, 16 x 32, 32 x 16, 32 x 32, 32 x 64, 64 x 32, 64 x 64, 64 x 128,
    128 x 64, 128 x 128, 256 x 256), with K ending in every part of a block."""
    check_gemm(m, n, k, BF if k % 32 else F32, seed=m, bias=m % 2 == 1, pads=(0, 16) if k == 400 else (0, 0))


@pytest.mark.parametrize("k", [400, 2512])
@pytest.mark.parametrize("m,n", [(974, 11), (1355, 81), (1319, 55), (1864, 66), (1610, 302), (4734, 40), (2480, 351), (5469, 312), (326, 5439),
                                 (1771, 668), (7040, 316), (8100, 64)])
def test_gemm_more_rows_than_channels(m, n, k):
    """Tiles in the order that shares rows of A (and 128 x 64, either way)."""
    check_gemm(m, n, k, F32 if k == 400 else BF, seed=n, bias=n % 2 == 1)


@pytest.mark.parametrize("m,n,k", [(500, 4090, 4112), (4090, 500, 4368), (300, 4000, 5008)])
def test_gemm_long_rows_few_tiles(m, n, k):
    check_gemm(m, n, k, BF, seed=k, bias=True)
    check_gemm(m, n, k, F32, seed=k, pads=(16, 0))


@pytest.mark.parametrize("m", [1, 40, 300])
def test_gemm_every_code_and_longest_sum(m):
    """Codes down to -128 over the longest k: sums up to 2^31 - 2^18."""
    check_gemm(m, 130, 131056, F32, full=True)
    a = torch.full((m, 131056), -128, dtype=I8, device=DEV)
    one = torch.ones(1, device=DEV)
    got = pqb.gemm_int8((a, one), (a[:1].expand(5, -1).contiguous(), one), F32)
    assert (got == 131056.0 * 16384).all()


@pytest.mark.parametrize("pads", [(16, 0), (0, 48), (4096, 16), (3, 5)])
@pytest.mark.parametrize("m,n,k", [(5, 70, 144), (200, 300, 1040), (40, 264, 4112)])
def test_gemm_strides(m, n, k, pads):
    check_gemm(m, n, k, BF, seed=3, pads=pads)


@pytest.mark.parametrize("one_scale", [(True, False), (False, True), (True, True)])
def test_gemm_scale_per_tensor(one_scale):
    check_gemm(37, 90, 256, F32, one_scale=one_scale, bias=True)


def test_gemm_of_quantized():
    g = gen(1)
    x, w = normal(g, 50, 512).to(BF), normal(g, 96, 512) * 0.02
    for gran in ("row", "tensor"):
        a, b = pqb.quantize(x, "int8_sym", gran), pqb.quantize(w, "int8_sym", "row")
        got = pqb.gemm_int8(a, b, F32)
        want = product(a.codes.view(I8).view(50, 512), a.scales, b.codes.view(I8).view(96, 512), b.scales, None, F32)
        assert torch.equal(got, want)


def test_gemm_empty():
    one = torch.ones(1, device=DEV)
    z = torch.empty(0, 32, dtype=I8, device=DEV)
    a = torch.ones(4, 32, dtype=I8, device=DEV)
    assert pqb.gemm_int8((z, torch.empty(0, device=DEV)), (a, one)).shape == (0, 4)
    assert pqb.gemm_int8((a, one), (z, torch.empty(0, device=DEV))).shape == (4, 0)
    e = torch.empty(3, 0, dtype=I8, device=DEV)
    bias = torch.arange(3.0, device=DEV)
    assert torch.equal(pqb.gemm_int8((e, one), (e, one), F32, bias=bias), bias.expand(3, 3))
    assert torch.equal(pqb.gemm_int8((e, one), (e, one), BF), torch.zeros(3, 3, dtype=BF, device=DEV))


def test_gemm_empty_sums_of_most_rows():
    """2^29 rows of no codes, a column: more tiles than a grid of any ring holds."""
    rows = 2 ** 29
    a, b = torch.empty(rows, 0, dtype=I8, device=DEV), torch.empty(1, 0, dtype=I8, device=DEV)
    one = torch.ones(1, device=DEV)
    got = pqb.gemm_int8((a, one), (b, one), BF, bias=torch.full((1,), 3.0, device=DEV))
    assert got.shape == (rows, 1) and (got == 3).all()


def test_gemm_rows_far_apart():
    """Rows 2^23 bytes apart, which the kernels' offsets do not reach, are copied."""
    g = gen(6)
    big = torch.zeros(40 * 2 ** 23, dtype=I8, device=DEV)
    a = big.view(40, 2 ** 23)[:, :272]
    a.copy_(codes(g, 40, 272))
    b, sa, sb = codes(g, 50, 272), torch.rand(40, generator=g, device=DEV), torch.rand(50, generator=g, device=DEV)
    assert torch.equal(pqb.gemm_int8((a, sa), (b, sb), F32), product(a, sa, b, sb, None, F32))


def test_gemm_output_past_2_31():
    """65600 x 33000 results of 2 bytes; rows on both sides of element 2^31."""
    g = gen(2)
    a, b = codes(g, 65600, 32), codes(g, 33000, 32)
    sa, sb = torch.rand(65600, generator=g, device=DEV), torch.rand(33000, generator=g, device=DEV)
    got = pqb.gemm_int8((a, sa), (b, sb), BF)
    for rows in (slice(0, 3), slice(65070, 65080), slice(65590, 65600)):
        assert torch.equal(got[rows], product(a[rows], sa[rows], b, sb, None, BF))


def test_gemm_into_out():
    g = gen(4)
    a, b = codes(g, 96, 8192), codes(g, 256, 8192)
    sa, sb = torch.rand(96, generator=g, device=DEV), torch.rand(256, generator=g, device=DEV)
    want = product(a, sa, b, sb, None, F32)
    out = torch.empty(96, 256, device=DEV)
    assert pqb.gemm_int8((a, sa), (b, sb), F32, out=out) is out and torch.equal(out, want)
    buf = torch.empty(96 * 256 * 4 + a.numel(), dtype=torch.uint8, device=DEV)
    inside = buf[:a.numel()].view(I8).view(a.shape)
    with pytest.raises(ValueError, match="share memory"):
        pqb.gemm_int8((inside, sa), (b, sb), F32, out=buf[a.numel() - 64:][:96 * 256 * 4].view(F32).view(96, 256))


# ---------------------------------------------------------------------------
# quantized outputs
# ---------------------------------------------------------------------------
FORMS = [(None, None), ("int8_sym", "row"), ("fp8_e4m3", "row"), ("fp8_e4m3", "1x128"), ("fp8_e5m2", "row"),
         ("fp8_e5m2", "1x128")]
TYPE = {"int8_sym": I8, "fp8_e4m3": E4M3, "fp8_e5m2": E5M2}
TOP = {"int8_sym": 127.0, "fp8_e4m3": 448.0, "fp8_e5m2": 57344.0}
STEP = {"fp8_e4m3": (2.0 ** -4, 2.0 ** -10), "fp8_e5m2": (2.0 ** -3, 2.0 ** -17)}   # half a step: relative, least


def per_scale(x, gran):
    """x [rows, cols] as [rows, blocks, values of one scale]."""
    return x.unflatten(1, (-1, 128)) if gran == "1x128" else x[:, None]


def plain_codes(u, fmt, gran):
    """pqb_quantize's codes and scales of float32 u, in float32."""
    b = per_scale(u, gran)
    s = b.abs().amax(2).clamp(min=np.float32(1e-12))
    s = s / torch.full_like(s, TOP[fmt])    # (by a Python number, torch multiplies by the reciprocal)
    q = (b / s[..., None]).reshape(u.shape)
    return q.round().to(I8) if fmt == "int8_sym" else q.to(TYPE[fmt]), s


def check_codes(q, fmt, gran, v, tol, rows, cols):
    """Codes and scales of values that are within tol of v (64 bits)."""
    assert isinstance(q, pqb.Quantized) and (q.fmt, q.gran, q.shape) == (fmt, gran, (1, rows, cols))
    got = q.codes.view(TYPE[fmt]).view(rows, cols).double()
    s = q.scales.view(rows, -1).double()
    want_s = per_scale(v, gran).abs().amax(2).clamp(min=1e-12) / TOP[fmt]
    tol_s = per_scale(tol.expand_as(v), gran).amax(2) / TOP[fmt] + 2 * U * want_s
    close(s, want_s, tol_s)
    wide = s[..., None].expand_as(per_scale(v, gran)).reshape(v.shape)
    # the scale's own error moves a value by its share of the largest; the quotient's rounding by U
    shift = tol_s[..., None].expand_as(per_scale(v, gran)).reshape(v.shape) * got.abs()
    if fmt == "int8_sym":
        close(got * wide, v, wide / 2 + tol + shift + 130 * U * wide)
    else:
        rel, least = STEP[fmt]
        close(got * wide, v, torch.maximum(v.abs() * rel * (1 + 2 * rel), wide * least) + tol + shift + U * v.abs())


# ---------------------------------------------------------------------------
# norm_quant
# ---------------------------------------------------------------------------

def norm64(z, kind, eps):
    z = z.double()
    c = z - z.mean(1, keepdim=True) if kind == "layer" else z
    return c, 1 / torch.sqrt(c.square().mean(1, keepdim=True) + eps)


def check_norm(rows, cols, dtype, fmt, gran, kind="rms", residual=True, scale=1.0, gates=0, post=False, weight=True,
               bias=False, seed=0, pad=0, shift=0, eps=1e-5, size=1.0):
    g = gen(seed)
    mk = lambda *s: normal(g, *s).to(dtype)  # noqa: E731
    x, res = (normal(g, rows, cols) * size).to(dtype), (normal(g, rows, cols) * 3 * size).to(dtype) if residual else None
    w, pw, b = (1 + 0.3 * normal(g, cols)).to(dtype), (1 + 0.3 * normal(g, cols)).to(dtype), mk(cols)
    w, pw, b = w if weight else None, pw if post else None, b if bias else None
    gate = mk(gates, cols) if gates else None
    args = dict(kind=kind, bias=b, eps=eps, residual_scale=scale, post_weight=pw)
    if pad or shift:
        sx, sr, sg = (None if t is None else strided(t, pad, shift) for t in (x, res, gate))
    else:
        sx, sr, sg = x, res, gate
    out, h = pqb.norm_quant(sx, w, fmt, gran, residual=sr, gate=sg, **args)

    # the residual stream
    adds = residual or gates or post
    if not adds:
        assert h is None
        h = x
    else:
        assert h.shape == x.shape and h.dtype is dtype
        gg = gate.repeat_interleave(rows // gates, 0) if gates else None
        if not post:    # float32, rounded operation by operation
            y = x.float() if gg is None else x.float() * gg.float()
            if residual:
                y = y + res.float() * np.float32(scale)
            assert torch.equal(h, y.to(dtype))
        else:
            c, r = norm64(x, kind, eps)
            y = c * r * pw.double()
            err = y.abs() * (R_TOL + 3 * U)
            if kind == "layer":      # the mean's error
                err = err + 64 * U * x.double().abs().mean(1, keepdim=True) * r * pw.double().abs()
            if gg is not None:
                y, err = y * gg.double(), err * gg.double().abs() + (y * gg.double()).abs() * U
            if residual:
                p = res.double() * np.float32(scale)
                y, err = y + p, err + (p.abs() * 2 + y.abs()) * U
            close(h, y, err + (y.abs() + err) * half_step(dtype))

    # the norm of what was written
    c, r = norm64(h, kind, eps)
    ww = 1.0 if w is None else w.double()
    v = c * r * ww
    tol = v.abs() * (R_TOL + 3 * U)
    if kind == "layer":
        tol = tol + 64 * U * h.double().abs().mean(1, keepdim=True) * r * abs(ww)
        if b is not None:
            v = v + b.double()
            tol = tol + v.abs() * U
    if fmt is None:
        assert out.shape == x.shape and out.dtype is dtype
        close(out, v, tol + (v.abs() + tol) * half_step(dtype))
    elif kind == "rms":
        u = h.float() if w is None else h.float() * w.float()
        want, s = plain_codes(u, fmt, gran)
        assert torch.equal(out.codes.view(rows, cols), want.view(torch.uint8))
        close(out.scales.view(rows, -1), s.double() * r, s.double() * r * (R_TOL + U))
    else:
        check_codes(out, fmt, gran, v, tol, rows, cols)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("fmt,gran", FORMS)
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 512), (7, 640), (5, 1024), (9, 2048), (4, 4096), (3, 7168), (2, 12288),
                                       (2, 16384), (2, 32768)])
def test_norm_widths(rows, cols, fmt, gran, kind, dtype):
    check_norm(rows, cols, dtype, fmt, gran, kind, bias=kind == "layer", seed=cols)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("fmt,gran", [f for f in FORMS if f[1] != "1x128"])
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 63, 65, 511, 513, 1005, 1025, 2047, 4095, 4097, 8190, 16383, 32767])
def test_norm_odd_widths(cols, fmt, gran, kind, dtype):
    check_norm(5, cols, dtype, fmt, gran, kind, bias=kind == "layer", seed=cols, eps=1e-2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("base", [0, 504, 4096, 8192, 20480])
def test_norm_ends_of_rows(base, dtype):
    """A last unit of every length; what lies between the rows of h stays as it was."""
    for cols in range(base + 1, base + 17):
        check_norm(3, cols, dtype, "int8_sym", "row", seed=cols, eps=1e-2)
        check_norm(3, cols, dtype, None, None, "layer", bias=True, post=True, seed=cols, eps=1e-2)
        g = gen(cols)
        x, r = normal(g, 3, cols).to(dtype), normal(g, 3, cols).to(dtype)
        wide = torch.full((3, cols + 11), 7.0, dtype=dtype, device=DEV)
        _, h = pqb.norm_quant(x, None, None, residual=r, h_out=wide[:, :cols])
        assert torch.equal(h, (x.float() + r.float()).to(dtype)) and (wide[:, cols:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("parts", [dict(residual=False), dict(residual=False, weight=False), dict(scale=0.22),
                                   dict(gates=1), dict(gates=4), dict(gates=12, scale=0.5), dict(post=True),
                                   dict(post=True, gates=3), dict(post=True, residual=False),
                                   dict(residual=False, gates=2), dict(post=True, gates=12, scale=-1.5)])
@pytest.mark.parametrize("cols,fmt,gran", [(256, None, None), (1280, "fp8_e4m3", "1x128"), (1005, "int8_sym", "row")])
def test_norm_parts(parts, cols, fmt, gran, kind, dtype):
    check_norm(12, cols, dtype, fmt, gran, kind, bias=kind == "layer", seed=cols, **parts)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad,shift", [(8, 0), (64, 8), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("cols,fmt,gran", [(384, "fp8_e4m3", "1x128"), (136, "int8_sym", "row"), (77, None, None)])
def test_norm_strides(pad, shift, cols, fmt, gran, dtype):
    """Rows apart and off their alignment; 1x128 blocks are copied where they have none."""
    check_norm(12, cols, dtype, fmt, gran, gates=3, pad=pad, shift=shift)


@pytest.mark.parametrize("rows", [1, 3, 4, 255, 1000, 4099])
@pytest.mark.parametrize("cols", [64, 256, 1000])
def test_norm_many_rows(rows, cols):
    check_norm(rows, cols, BF, "int8_sym", "row", seed=rows)
    check_norm(rows, cols, F32, None, None, "layer", bias=True, seed=rows)


@pytest.mark.parametrize("fmt,gran", FORMS)
def test_norm_of_zeros_and_extremes(fmt, gran):
    """Rows of zeros, one value among zeros, values near the ends of what the sums hold."""
    x = torch.zeros(6, 256, device=DEV)
    x[1, 100] = 3.0
    x[2] = 1e15
    x[3] = torch.linspace(-1e-20, 1e-20, 256)
    x[4, ::2] = -2.5e17
    w = torch.ones(256, device=DEV)
    out, h = pqb.norm_quant(x, w, fmt, gran, eps=1e-6)
    assert h is None
    c, r = norm64(x, "rms", np.float32(1e-6))
    if fmt is None:
        close(out, c * r, (c * r).abs() * (R_TOL + 3 * U) + 2.0 ** -149)
    else:
        want, s = plain_codes(x, fmt, gran)
        assert torch.equal(out.codes.view(6, 256), want.view(torch.uint8))
        close(out.scales.view(6, -1), s.double() * r, s.double() * r * (R_TOL + U))


def test_norm_in_place_and_empty():
    g = gen(9)
    x, res, w = normal(g, 40, 512).to(BF), normal(g, 40, 512).to(BF), normal(g, 512).to(BF)
    want, h = pqb.norm_quant(x, w, residual=res)
    keep = res.clone()
    got, h2 = pqb.norm_quant(x, w, residual=res, h_out=res)
    assert h2 is res and torch.equal(h2, h) and torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    xx = x.clone()
    got, h3 = pqb.norm_quant(xx, w, residual=keep, h_out=xx)
    assert h3 is xx and torch.equal(xx, h) and torch.equal(got.codes, want.codes)
    # rows of h in the gaps of x's
    both = torch.zeros(40, 1024, dtype=BF, device=DEV)
    both[:, :512] = x
    got, h4 = pqb.norm_quant(both[:, :512], w, residual=keep, h_out=both[:, 512:])
    assert torch.equal(both[:, 512:], h) and torch.equal(both[:, :512], x) and torch.equal(got.codes, want.codes)
    q, h = pqb.norm_quant(x[:0], w, residual=res[:0])
    assert q.codes.numel() == 0 and h.shape == (0, 512)
    y, h = pqb.norm_quant(x.view(4, 10, 512), w, None, residual=keep.view(4, 10, 512))
    assert y.shape == h.shape == (4, 10, 512)


def test_norm_past_2_31():
    rows, cols = 262400, 8192
    x = torch.empty(rows, cols, dtype=BF, device=DEV)
    x.normal_(generator=gen(3))
    res = torch.ones_like(x)
    w = torch.ones(cols, dtype=BF, device=DEV)
    q, h = pqb.norm_quant(x, w, residual=res)
    for at in (slice(0, 2), slice(262142, 262148), slice(rows - 2, rows)):
        hh = (x[at].float() + 1).to(BF)
        assert torch.equal(h[at], hh)
        want, _ = plain_codes(hh.float(), "int8_sym", "row")
        assert torch.equal(q.codes.view(rows, cols)[at], want.view(torch.uint8))


# ---------------------------------------------------------------------------
# act_quant
# ---------------------------------------------------------------------------

# 1 + exp(-z) passes 2^126, whose reciprocal is no normal float32, from z = -126 ln 2 = -87.34 on; a value there
# is at most 87.34 * 2^-126 < 2^-119 (|g| <= |z| down there), and may be 0.
LEAST = 2.0 ** -119


def act64(g, act):
    """Value and its tolerance: the roundings of the formula, times how much it stretches them."""
    g = g.double()
    if act == "silu":
        v = g * torch.sigmoid(g)
        return v, v.abs() * 8 * U
    if act == "gelu_tanh":
        z = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        v = g * torch.sigmoid(z)
        return v, v.abs() * (8 + 5 * z.abs()) * U
    if act == "gelu_erf":
        v = 0.5 * g * torch.special.erfc(-g / math.sqrt(2))
        return v, v.abs() * (16 + 4 * g * g) * U
    v = g.clamp(min=0) ** 2
    return v, v * U


def check_act(rows, cols, dtype, fmt, gran, act="silu", gated=True, seed=0, pad=0, shift=0, size=2.0):
    g = gen(seed)
    gate, up = (normal(g, rows, cols) * size).to(dtype), normal(g, rows, cols).to(dtype)
    v, tol = act64(gate, act)
    if gated:
        v, tol = v * up.double(), tol * up.double().abs() + (v * up.double()).abs() * U
    tol = tol + LEAST
    sg, su = (strided(t, pad, shift) if pad or shift else t for t in (gate, up))
    out = pqb.act_quant(sg, su if gated else None, fmt, gran, act=act)
    if fmt is None:
        assert out.shape == gate.shape and out.dtype is dtype
        close(out, v, tol + (v.abs() + tol) * half_step(dtype))
    else:
        check_codes(out, fmt, gran, v, tol, rows, cols)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu_erf", "relu2"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("fmt,gran", FORMS)
@pytest.mark.parametrize("rows,cols", [(1, 128), (6, 640), (3, 4096), (2, 14336), (2, 28672)])
def test_act(rows, cols, fmt, gran, gated, act, dtype):
    check_act(rows, cols, dtype, fmt, gran, act, gated, seed=cols)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fmt,gran", [f for f in FORMS if f[1] != "1x128"])
@pytest.mark.parametrize("cols", [1, 7, 65, 513, 1285, 2049, 4095, 14337, 32767])
def test_act_odd_widths(cols, fmt, gran, dtype):
    check_act(5, cols, dtype, fmt, gran, "silu", seed=cols)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("base", [0, 2040, 4096, 20480])
def test_act_ends_of_rows(base, dtype):
    """A last unit of every length, and pieces of 2048 with fewer than eight elements."""
    for cols in range(base + 1, base + 17):
        check_act(3, cols, dtype, "fp8_e4m3", "row", seed=cols)
        check_act(3, cols, dtype, None, None, seed=cols)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad,shift", [(8, 0), (384, 8), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("cols,fmt,gran", [(384, "fp8_e4m3", "1x128"), (136, "int8_sym", "row"), (77, None, None)])
def test_act_strides(pad, shift, cols, fmt, gran, dtype):
    check_act(12, cols, dtype, fmt, gran, pad=pad, shift=shift)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu_erf", "relu2"])
def test_act_far_values(act):
    """The whole range of inputs, the largest finite ones among them: no NaN, tails that vanish."""
    top = 1.0e19 if act == "relu2" else 3.0e38
    x = torch.cat([torch.linspace(-200, 200, 4001), torch.tensor([-top, -1e30, -1e10, -88.8, -1e-30, 0.0, -0.0, 1e-30, 1e10, top])])
    x = x.clamp(-top, top).to(DEV).view(1, -1)
    out = pqb.act_quant(x, None, None, act=act)
    v, tol = act64(x, act)
    v, tol = torch.nan_to_num(v, nan=0.0), torch.nan_to_num(tol, nan=0.0, posinf=0.0)
    far = x.double().abs() > 1e9
    v[far] = torch.where(x[far] > 0, (x[far].double() ** 2 if act == "relu2" else x[far].double()), 0.0)
    tol[far] = v[far] * 2 * U
    assert torch.isfinite(out).all()
    close(out, v, tol + LEAST)


def test_act_of_zeros_wide_and_empty():
    z = torch.zeros(3, 256, dtype=BF, device=DEV)
    q = pqb.act_quant(z, z, "fp8_e4m3", "1x128")
    assert not q.codes.any() and (q.scales == np.float32(1e-12) / np.float32(448)).all()
    check_act(3, 70000, BF, None, None)                     # wider than a row with one scale may be
    check_act(3, 65536, BF, "fp8_e4m3", "1x128")
    assert pqb.act_quant(z[:0], z[:0]).codes.numel() == 0
    assert pqb.act_quant(z.view(3, 2, 128), None, None).shape == (3, 2, 128)


def test_act_past_2_31():
    rows, cols = 262400, 8192
    x = torch.empty(rows, cols, dtype=BF, device=DEV)
    x.normal_(generator=gen(3))
    q, y = pqb.act_quant(x, x, "int8_sym"), pqb.act_quant(x, None, None)
    for at in (slice(0, 2), slice(262142, 262148), slice(rows - 2, rows)):
        few, y2 = pqb.act_quant(x[at], x[at], "int8_sym"), pqb.act_quant(x[at], None, None)
        assert torch.equal(q.codes.view(rows, cols)[at].reshape(-1), few.codes) and torch.equal(q.scales[at], few.scales)
        assert torch.equal(y[at], y2)


# ---------------------------------------------------------------------------
# rope
# ---------------------------------------------------------------------------

def turned(x, pos, table):
    """Values in 64 bits, and how far float32 may be off."""
    x = x.double()
    ang = pos.double()[:, None, None] * table.angles
    c, s = ang.cos() * table.amplitude, ang.sin() * table.amplitude
    rot = 2 * table.angles.numel()
    out, tol = x.clone(), torch.zeros_like(x)
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if table.interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., one], x[..., two]
    out[..., one], out[..., two] = a * c - b * s, b * c + a * s
    # cosine and sine within 2^-22, three roundings behind them
    tol[..., one] = tol[..., two] = (a.abs() + b.abs()) * abs(table.amplitude) * (2.0 ** -22 + 3 * U)
    return out, tol


def check_turned(got, x, pos, table):
    want, tol = turned(x, pos, table)
    close(got, want, tol + (want.abs() + tol) * half_step(x.dtype) * (tol > 0))


def check_rope(tokens, hq, hk, dim, rot, dtype, interleaved, seed=0, far=100000, amplitude=1.0, pad=0, shift=0, in_place=False):
    g = gen(seed)
    big = torch.empty(tokens * ((hq + hk) * dim + pad) + shift + 1, dtype=dtype, device=DEV)
    fused = big[shift:shift + tokens * ((hq + hk) * dim + pad)].view(tokens, -1)
    fused.copy_(normal(g, *fused.shape))
    q = fused[:, :hq * dim].unflatten(1, (hq, dim))
    k = fused[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim)) if hk else None
    pos = torch.randint(0, far, (tokens,), generator=g, device=DEV, dtype=torch.int32)
    t = pqb.rope_table(rot, interleaved=interleaved, amplitude=amplitude, device=DEV)
    q0, k0, pad0 = q.clone(), None if k is None else k.clone(), fused[:, (hq + hk) * dim:].clone()
    outs = dict(q_out=q, k_out=k) if in_place else {}
    qo, ko = pqb.rope(q, k, pos, t, **outs)
    check_turned(qo, q0, pos, t)
    if k is None:
        assert ko is None
    else:
        check_turned(ko, k0, pos, t)
    if in_place:
        assert qo is q and ko is k and torch.equal(fused[:, (hq + hk) * dim:], pad0)
    else:
        assert torch.equal(q, q0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 64), (256, 64), (80, 32), (96, 96), (128, 16), (80, 20), (6, 2), (30, 22),
                                     (1024, 512), (128, 20), (96, 24), (80, 40), (77, 30), (3, 2), (129, 128), (100, 100)])
@pytest.mark.parametrize("tokens,hq,hk", [(1, 32, 8), (5, 3, 1), (67, 4, 4), (9, 2, 0)])
def test_rope(tokens, hq, hk, dim, rot, interleaved, dtype):
    check_rope(tokens, hq, hk, dim, rot, dtype, interleaved, seed=dim + tokens)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (128, 8), (1, 0), (0, 1)])
def test_rope_in_place_and_strides(pad, shift, interleaved, dtype):
    for in_place in (True, False):
        check_rope(33, 8, 2, 128, 64, dtype, interleaved, pad=pad, shift=shift, in_place=in_place, amplitude=1.3)


@pytest.mark.parametrize("far", [1, 2, 1 << 20, (1 << 28) - 1])
def test_rope_far_positions(far):
    check_rope(50, 2, 1, 128, 128, F32, False, far=far)
    x = normal(gen(1), 4, 1, 64)
    t = pqb.rope_table(64, device=DEV)
    pos = torch.tensor([-1, -(1 << 27), far, 0], dtype=torch.int32, device=DEV)
    check_turned(pqb.rope(x, None, pos, t)[0], x, pos, t)


@pytest.mark.parametrize("new,cached", [([1] * 40, list(range(40))), ([3, 1, 0, 7, 1], [0, 9, 5, 300, 0]), ([0, 0, 2, 0], [1, 2, 3, 4]),
                                        ([500], [7])])
def test_rope_places_of_a_plan(new, cached):
    """Positions from a step's plan; tokens behind the last request stay as they were."""
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    batch, total = len(new), sum(new)
    table = ints([[8 * b + i for i in range(8)] for b in range(batch)])
    plan = pqb.kv_plan_paged(ints(cached), ints(new), table, ints(list(range(8 * batch, 16 * batch))), ints([0]), 128, total + 5)
    assert plan.status[0] == 0
    g = gen(7)
    q, k = normal(g, total + 5, 4, 64).to(BF), normal(g, total + 5, 2, 64).to(BF)
    t = pqb.rope_table(64, device=DEV)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    pqb.rope(q, k, plan, t, q_out=qo, k_out=ko)
    pos = ints([c + i for c, n in zip(cached, new) for i in range(n)])
    check_turned(qo[:total], q[:total], pos, t)
    check_turned(ko[:total], k[:total], pos, t)
    assert (qo[total:] == 7).all() and (ko[total:] == 7).all()


def test_rope_empty_and_past_2_31():
    t = pqb.rope_table(64, device=DEV)
    x = torch.empty(0, 4, 64, device=DEV)
    assert pqb.rope(x, None, torch.empty(0, dtype=torch.int32, device=DEV), t)[0].shape == (0, 4, 64)
    x = torch.empty(1060000, 32, 64, dtype=BF, device=DEV)
    x.normal_(generator=gen(5))
    pos = torch.arange(1060000, dtype=torch.int32, device=DEV)
    got = pqb.rope(x, None, pos, t)[0]
    for at in (slice(0, 3), slice(1048574, 1048580), slice(1059998, 1060000)):
        check_turned(got[at], x[at], pos[at], t)


# ---------------------------------------------------------------------------
# in use: streams, graphs, and a layer from end to end
# ---------------------------------------------------------------------------

class Layer:
    """A decoder layer on the framework's kernels, W8A8, over a paged cache."""

    def __init__(self, hidden, heads, kv_heads, dim, inner, pages, page, seed):
        g = gen(seed)
        self.h, self.hq, self.hk, self.d, self.page = hidden, heads, kv_heads, dim, page
        self.norms = [(1 + 0.2 * normal(g, hidden)).to(BF) for _ in range(2)]
        mk = lambda n, k: pqb.quantize(normal(g, n, k) / math.sqrt(k), "int8_sym", "row")  # noqa: E731
        self.qkv, self.o = mk((heads + 2 * kv_heads) * dim, hidden), mk(hidden, heads * dim)
        self.gate_up, self.down, self.inner = mk(2 * inner, hidden), mk(hidden, inner), inner
        self.cache = pqb.kv_paged_cache(pages, kv_heads, page, dim, DEV)
        self.table = pqb.rope_table(dim, 500000.0, scaling="by_turns", factor=8.0, device=DEV)

    def step(self, x, plan, block_table, max_q_len):
        q, _ = pqb.norm_quant(x, self.norms[0])
        qkv = pqb.gemm_int8(q, self.qkv).view(-1, self.hq + 2 * self.hk, self.d)
        v = qkv[:, self.hq + self.hk:]
        q, k = pqb.rope(qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hk], plan, self.table)
        pqb.kv_append_paged(k, v, plan.slots, self.cache)
        att = pqb.kv_attend_paged(q, self.cache, block_table, plan.q_starts, plan.kv_lens, max_q_len=max_q_len)
        y = pqb.gemm_int8(pqb.quantize(att.view(-1, self.hq * self.d), "int8_sym", "row"), self.o)
        q, h = pqb.norm_quant(y, self.norms[1], residual=x)
        gu = pqb.gemm_int8(q, self.gate_up)
        y = pqb.gemm_int8(pqb.act_quant(gu[:, :self.inner], gu[:, self.inner:]), self.down)
        return pqb.norm_quant(y, None, None, residual=h)[1]

    def weight(self, q):
        return (q.codes.view(I8).view(q.shape[1:]).double() * q.scales.double()[:, None])

    def plain(self, x, starts, k_past, v_past):
        """The layer in 64 bits without any rounding, one request; returns the output, keys and values."""
        rms = lambda z, w: z * w.double() / torch.sqrt(z.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
        x = x.double()
        qkv = (rms(x, self.norms[0]) @ self.weight(self.qkv).T).view(-1, self.hq + 2 * self.hk, self.d)
        pos = torch.arange(starts, starts + len(x), device=DEV)
        q, k = (turned(t, pos, self.table)[0] for t in (qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hk]))
        k, v = torch.cat((k_past, k)), torch.cat((v_past, qkv[:, self.hq + self.hk:]))
        rep = self.hq // self.hk
        z = torch.einsum("thd,shd->hts", q, k.repeat_interleave(rep, 1)) / math.sqrt(self.d)
        z = z.masked_fill(torch.arange(len(k), device=DEV) > pos[:, None], float("-inf"))
        att = torch.einsum("hts,shd->thd", z.softmax(2), v.repeat_interleave(rep, 1)).reshape(len(x), -1)
        h = x + att @ self.weight(self.o).T
        gu = rms(h, self.norms[1]) @ self.weight(self.gate_up).T
        a = act64(gu[:, :self.inner], "silu")[0] * gu[:, self.inner:]
        return h + a @ self.weight(self.down).T, k, v


def test_decoder_layer_prompts_then_steps():
    """Two prompts and then single tokens through a whole layer, against 64 bits without rounding.  Per
    value, INT8 activations are off by at most 1 / 254 of the row's largest (about 4 times its rms): 1.6% of
    the rms at most, 0.9% rms; E4M3 keys and values by 2^-4 at most, 2.6% rms.  Through four products, attention and
    the residual that is well under 10% of the output's norm."""
    layer = Layer(256, 8, 2, 64, 704, 16, 16, seed=3)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    lens, order = [37, 20], torch.randperm(16, generator=gen(1), device=DEV).to(torch.int32)
    cached, used = ints([0, 0]), ints([0])
    table = torch.zeros(2, 8, dtype=torch.int32, device=DEV)
    past = [(torch.empty(0, 2, 64, dtype=F64, device=DEV),) * 2 for _ in lens]
    g = gen(8)
    for new in (lens, [1, 1], [1, 1], [3, 1]):
        x = normal(g, sum(new) + 2, 256).to(BF)
        plan = pqb.kv_plan_paged(cached, ints(new), table, order, used, 16, sum(new) + 2)
        assert plan.status[0] == 0
        got = layer.step(x, plan, table, max(new))
        at = 0
        for b, n in enumerate(new):
            want, *past[b] = layer.plain(x[at:at + n], int(cached[b]), *past[b])
            off = (got[at:at + n].double() - want).norm() / want.norm()
            assert off < 0.1, (new, b, off.item())
            at += n
        cached, used = plan.kv_lens, plan.free_used


def test_layer_captured_and_replayed():
    """A decode step in a graph: replays advance with the plan, equal to the eager steps, eager work between."""
    def make():
        layer = Layer(256, 8, 2, 64, 704, 24, 16, seed=3)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        return layer, ints([0, 0, 0]), ints([0]), torch.zeros(3, 8, dtype=torch.int32, device=DEV), ints(list(range(24)))

    g = gen(5)
    xs = [normal(g, 3, 256).to(BF) for _ in range(20)]
    one = torch.ones(3, dtype=torch.int32, device=DEV)
    layer, cached, used, table, order = make()
    want = []
    for x in xs:
        plan = pqb.kv_plan_paged(cached, one, table, order, used, 16, 3)
        want.append(layer.step(x, plan, table, 1))
        cached, used = plan.kv_lens, plan.free_used

    layer, cached, used, table, order = make()
    plan = pqb.PagedPlan(torch.empty(3, dtype=torch.int32, device=DEV), torch.empty(4, dtype=torch.int32, device=DEV), cached, used,
                         torch.empty(4, dtype=torch.int32, device=DEV))
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):       # warm up, then back to the start
        layer.step(x, pqb.kv_plan_paged(cached, one, table, order, used, 16, 3, out=plan), table, 1)
        cached.zero_()
        used.zero_()
        table.zero_()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(x, pqb.kv_plan_paged(cached, one, table, order, used, 16, 3, out=plan), table, 1)
    cached.zero_()
    used.zero_()
    table.zero_()
    for i, xi in enumerate(xs):
        x.copy_(xi)
        graph.replay()
        assert torch.equal(out, want[i]), i
        torch.rand(1000, device=DEV).sum()


@pytest.mark.parametrize("m,n,k", [(3, 512, 4096), (96, 256, 8192), (300, 300, 1040)])
def test_two_streams_and_two_graphs(m, n, k):
    """Products that overlap in time, each on its own stream with its own inputs, eager and captured."""
    g = gen(6)
    sets = [(codes(g, m, k), torch.rand(m, generator=g, device=DEV), codes(g, n, k), torch.rand(n, generator=g, device=DEV))
            for _ in range(2)]
    want = [product(*s, None, F32) for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                a, sa, b, sb = sets[i]
                outs[i].append(pqb.gemm_int8((a, sa), (b, sb), F32))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i])
    graphs, res = [], []
    for a, sa, b, sb in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res.append(pqb.gemm_int8((a, sa), (b, sb), F32))
        graphs.append(gr)
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(res[i], want[i]) for i in range(2))
        for r in res:
            r.zero_()
        torch.cuda.synchronize()


def test_results_do_not_change_between_calls():
    g = gen(11)
    x, w = normal(g, 200, 1005), normal(g, 1005)
    first = pqb.norm_quant(x, w, None, kind="layer")[0]
    f2 = pqb.act_quant(x, None, None, act="gelu_erf")
    for _ in range(5):
        assert torch.equal(pqb.norm_quant(x, w, None, kind="layer")[0], first)
        assert torch.equal(pqb.act_quant(x, None, None, act="gelu_erf"), f2)
