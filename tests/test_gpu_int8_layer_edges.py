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
