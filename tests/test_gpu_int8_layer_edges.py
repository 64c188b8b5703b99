"""The INT8 layer on the GPU where it is easiest to get wrong: far tails and infinities of the
activations, and the large tiles of the product with rows of whole lines, several tiles to a workgroup
and rows that end inside a tile."""
import math

import pytest
import torch

import precision_quantization_block_amd as pqb

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ---------------------------------------------------------------------------
# activations
# ---------------------------------------------------------------------------

def test_gelu_erf_keeps_its_tail():
    """0.5 g erfc(-g / sqrt 2) over all g whose value passes 2^-119, with one tolerance for all of them.
    16 steps of 2^-23 are what an erfc may be off by (OpenCL's bound): 32 U; the product with 0.5 g, the
    correction for the rounding of g / sqrt 2 and what it neglects: U each, one over.  (That rounding alone,
    left uncorrected, reaches g^2 U: 76 measured at g = -9, 47 at -6.)"""
    g = torch.linspace(-12.5, 9.0, 200001, dtype=torch.float64).float().to(DEV)
    got = pqb.act_quant(g.view(1, -1), None, None, act="gelu_erf").view(-1).double()
    want = 0.5 * g.double() * torch.special.erfc(-g.double() / math.sqrt(2))
    off = (got - want).abs() / want.abs().clamp(min=2.0 ** -119) / U
    at = off.argmax()
    assert off[at] <= 36, (g[at].item(), off[at].item())


INF = float("inf")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu_erf", "relu2"])
def test_activations_of_plus_infinity(act, dtype):
    """As the formulas have it, among finite values that they leave alone."""
    x = torch.tensor([[1.0, INF, -2.0, 100.0, 17.5, 3.0e18]], dtype=dtype, device=DEV)
    got = pqb.act_quant(x, None, None, act=act)[0].float()
    alone = pqb.act_quant(x[:, [0, 2, 3, 4, 5]], None, None, act=act)[0].float()
    assert got[1] == INF and torch.equal(got[[0, 2, 3, 4, 5]], alone) and torch.isfinite(alone).all()
    up = torch.full_like(x, -0.5)
    assert pqb.act_quant(x, up, None, act=act)[0, 1] == -INF


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu_erf", "relu2"])
def test_activations_keep_nan(act, dtype):
    """NaN among finite values comes out as NaN, and -inf as 0 times inf (0 for the squared ReLU)."""
    x = torch.tensor([[1.0, float("nan"), -2.0, -INF]], dtype=dtype, device=DEV)
    got = pqb.act_quant(x, None, None, act=act)[0]
    assert got.isnan().tolist() == [False, True, False, act != "relu2"] and (act != "relu2" or got[3] == 0)
    gated = pqb.act_quant(torch.ones_like(x), x, None, act=act)[0]
    assert gated.isnan().tolist() == [False, True, False, False] and gated[3] == -INF


# ---------------------------------------------------------------------------
# norm_quant
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("gates", [0, 1, 3])
def test_norm_of_no_rows_with_a_gate(gates):
    """A batch without tokens, its gates per token (none) or per sequence."""
    x, gate = torch.empty(0, 256, dtype=BF, device=DEV), torch.ones(gates, 256, dtype=BF, device=DEV)
    for fmt in ("int8_sym", None):
        out, h = pqb.norm_quant(x, None, fmt, residual=x, gate=gate)
        assert h.shape == (0, 256) and (out if fmt is None else out.codes).numel() == 0


# ---------------------------------------------------------------------------
# gemm_int8: every tile, both types of result, rows of whole lines and others
# ---------------------------------------------------------------------------

# Kernel ("ring", "deep" or "tile"), its tile, and products that it takes.  Each kernel has rows of C that
# are whole lines (N a multiple of 64) and rows that are not, more rows than channels and fewer; the tiles
# that workgroups take in turn also one, two, an even and an odd number of blocks of K, more tiles than
# workgroups, and rows that end inside a tile, so that whole and partial waves meet in one.
PRODUCTS = [
    ("ring", 16, 16, [(4, 3, 64), (1, 3, 64), (65, 64, 64), (1, 64, 1040)]),
    ("ring", 16, 32, [(388, 307, 64), (1, 4108, 208), (392, 320, 1040), (1, 4160, 64)]),
    ("ring", 32, 16, [(4183, 3, 64), (17, 2103, 336), (337, 192, 64), (17, 2112, 1040)]),
    ("ring", 32, 32, [(4221, 17, 64), (17, 4508, 1040), (403, 320, 336), (17, 4160, 64)]),
    ("ring", 32, 64, [(1613, 294, 1040), (1, 8376, 64), (775, 640, 64), (1, 8320, 336)]),
    ("ring", 64, 32, [(8380, 3, 64), (35, 4100, 1040), (803, 320, 64), (33, 4288, 208)]),
    ("ring", 64, 64, [(8246, 34, 64), (33, 8694, 1040), (1346, 384, 336), (34, 8320, 64)]),
    ("ring", 128, 64, [(8559, 131, 64), (339, 5428, 1040), (8346, 192, 336), (1349, 1472, 64)]),
    ("ring", 64, 128, [(8231, 71, 336), (70, 8501, 64), (1233, 832, 64), (65, 8384, 1040)]),
    ("deep", 128, 64, [(8217, 66, 4368), (65, 8435, 4112), (1218, 832, 4112), (65, 8320, 4368)]),
    ("tile", 128, 128, [(5464, 321, 64), (203, 8398, 336), (8569, 1216, 64), (4619, 2240, 208), (8231, 1856, 1168),
                        (1700, 6080, 128), (1169, 8768, 208), (1166, 8640, 336)]),
    ("tile", 256, 256, [(8318, 5026, 208), (911, 8204, 1040), (8332, 4928, 208), (8485, 2880, 1168), (7193, 3456, 336),
                        (9990, 20032, 128), (3591, 6720, 1168), (3333, 7296, 336)]),
]


def operands(g, m, n, k):
    make = lambda r: (torch.randn((r, k), generator=g, device=DEV) * 40).round().clamp(-128, 127).to(torch.int8)  # noqa: E731
    scales = lambda r: torch.rand(r, generator=g, device=DEV) * 0.02 + 1e-3  # noqa: E731
    return make(m), scales(m), make(n), scales(n), torch.randn(n, generator=g, device=DEV)


def rounded_product(a, sa, b, sb, bias):
    """An exact sum, then float32 roundings one after the other."""
    v = torch.matmul(a.double(), b.double().t()).float().mul_(sa[:, None]).mul_(sb)
    return v if bias is None else v.add_(bias)


@pytest.mark.parametrize("m,n,k", [p for *_, products in PRODUCTS for p in products])
def test_product_of_every_kernel(m, n, k):
    """Both types of result, with and without bias; bit for bit."""
    a, sa, b, sb, bias = operands(gen(m + n), m, n, k)
    for c in (None, bias):
        want = rounded_product(a, sa, b, sb, c)
        assert torch.equal(pqb.gemm_int8((a, sa), (b, sb), F32, bias=c), want)
        want = want.to(BF)
        assert torch.equal(pqb.gemm_int8((a, sa), (b, sb), BF, bias=c), want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n,k", [(4619, 2240, 208), (7193, 3456, 336)])
def test_tiles_in_turn_on_two_streams_and_in_graphs(m, n, k, dtype):
    """Workgroups that store one tile while the next one's blocks arrive, two products at a time."""
    sets = [operands(gen(i), m, n, k) for i in range(2)]
    want = [rounded_product(*s).to(dtype) for s in sets]
    call = lambda s: pqb.gemm_int8(s[:2], s[2:4], dtype, bias=s[4])  # noqa: E731
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        for st, s, w in zip(streams, sets, want):
            with torch.cuda.stream(st):
                outs.append((call(s), w))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in outs)
    graphs = []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(s)
        graphs.append((graph, out))
    for _ in range(4):
        for st, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert torch.equal(out, w)
            out.zero_()
        torch.cuda.synchronize()
