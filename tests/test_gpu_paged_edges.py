"""The paged 8-bit KV cache at the ends of what a call may hold: the largest lengths,
values and scores, many requests with everything split, and workspaces in use."""
import numpy as np
import pytest
import torch

import precision_quantization_block_amd as pqb
from oracle import paged
from test_gpu_paged import BF, DEV, F32, filled, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_at_the_largest_length(dtype):
    """The widest table, whose request fills it with one page again and again but for the
    last entry, the only page whose keys count: the others score -128 and the best of
    this one's over 0, so that all 2^31 of them weigh under 2^-100 together."""
    page, dim = 256, 64
    width = (2 ** 31 - 256) // page - 1
    cache, host = filled(np.random.default_rng(26), 2, 1, page, dim, lo=120, hi=120)
    cache.k_codes[0] = host[0][0] = 0xE0            # -32 * 2^-7
    q = torch.ones((1, 1, dim), dtype=dtype)
    table = torch.zeros((1, width), dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    got = pqb.kv_attend_paged(q.to(DEV), cache, table, ints([0, 1]), ints([width * page]), scale=8.0)
    want, bound = paged.attend(q.double().numpy(), *host, np.array([[1]]), [0, 1], [page], True, 8.0, dtype == F32)
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
