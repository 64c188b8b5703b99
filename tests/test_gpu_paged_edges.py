"""The paged 8-bit KV cache at the ends of what a call may hold: the largest lengths,
values and scores, many requests with everything split, and workspaces in use."""
import contextlib

import numpy as np
import pytest
import torch

import precision_quantization_block_amd as pqb
from oracle import paged
from test_gpu_paged import BF, DEV, F32, Server, check_attend, filled, ints, tiles

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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new,kv", [([1, 2, 1], [100, 90, 3000]), ([70, 1, 33], [100, 90, 3000])])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -124, 2.0 ** -127, 2.0 ** -140])
def test_attend_scales_next_to_zero(dtype, new, kv, scale):
    """Products q.k of about 2^121, up to the largest allowed: scale 0 makes all tokens
    alike, and the smallest normal and subnormal scales leave them apart."""
    rng = np.random.default_rng(27)
    for page in (16, 64):
        check_attend(rng, new, kv, 2, 2, 64, page, dtype, scale=scale, qscale=1.5 * 2.0 ** 112, lo=127, hi=127)


def check_values(rng, new, kv, heads, group, dim, page, dtype, v_scale, **more):
    """Attention over positive V of one page exponent (its byte v_scale), within the oracle's bound."""
    counts = [-(-n // page) for n in kv]
    table, pages = tiles(rng, counts, max(counts))
    cache, host = filled(rng, pages, heads, page, dim)
    cache.v_codes &= 0x7F
    cache.v_scales.fill_(v_scale)
    host[1][:], host[3][:] = host[1] & 0x7F, v_scale
    starts = np.concatenate([[0], np.cumsum(new)])
    q = torch.from_numpy(rng.standard_normal((int(starts[-1]), heads * group, dim))).to(dtype)
    got = pqb.kv_attend_paged(q.to(DEV), cache, ints(table), ints(starts), ints(kv), max_q_len=max(new), **more)
    want, bound = paged.attend(q.double().numpy(), *host, table, starts, kv, True, dim ** -0.5, dtype == F32)
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("dtype,dim", [(BF, 64), (BF, 128), (F32, 64), (F32, 256)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("v_scale", [246, 1])
def test_attend_values_at_the_ends_of_float32(dtype, dim, page, v_scale):
    """V of up to 448 * 2^119 = 2.98e38, whose sums pass float32, and of down to 2^-126,
    for which 2^X / l is no normal number: both kernels, whole and split."""
    rng = np.random.default_rng(28)
    check_values(rng, [1, 2, 1], [100, 333, 3], 2, 2, dim, page, dtype, v_scale)
    check_values(rng, [1, 1], [5000, 700], 1, 2, dim, page, dtype, v_scale)
    check_values(rng, [40, 1, 200], [100, 333, 200], 2, 2, dim, page, dtype, v_scale)
    check_values(rng, [20, 33, 1], [5000, 2100, 3000], 1, 2, dim, page, dtype, v_scale)


def check_whole_scores(dtype, dim, page, base, unit, new, kv):
    """Scores unit * (base + a whole number up to 189), exact in float32 and equal for many
    tokens: with unit 1 their differences count, far beyond it the largest of a row alone.
    So, with A = sum p |v| / sum p: p is off by 2^-22 (exp2) and by the rounding of an
    exponent that counts (under 64: 2^-18 and half that from log2(e)); f16 by 2^-11
    (float32: 2^-22); sums by (2 n + 64) 2^-24."""
    rng = np.random.default_rng(29)
    heads, group = 1, 2
    table, pages = tiles(rng, [-(-n // page) for n in kv], -(-max(kv) // page))
    cache, host = filled(rng, pages, heads, page, dim)
    k = np.zeros((pages, heads, page, dim))
    k[..., 0] = 2.0 ** 8 if base else 0
    k[..., 1:22] = rng.integers(0, 4, k[..., 1:22].shape)      # q of 0 .. 3 against them: up to 189
    codes = torch.from_numpy(k).to(torch.float8_e4m3fn).view(torch.uint8)
    cache.k_codes.copy_(codes)
    cache.k_scales.fill_(127)
    host[0][:], host[2][:] = codes.numpy(), 127
    starts = np.concatenate([[0], np.cumsum(new)])
    q = np.zeros((int(starts[-1]), heads * group, dim))
    q[..., 0] = base / 2.0 ** 8
    q[..., 1:22] = rng.integers(0, 4, q[..., 1:22].shape)
    qt = torch.from_numpy(q * unit).to(dtype)
    got = pqb.kv_attend_paged(qt.to(DEV), cache, ints(table), ints(starts), ints(kv), scale=1.0, max_q_len=max(new))
    got = got.double().cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore"):         # the bound for any scores, not used
        want, _ = paged.attend(qt.double().numpy(), *host, table, starts, kv, True, 1.0, dtype == F32)
        host[1] &= 0x7F
        A, _ = paged.attend(qt.double().numpy(), *host, table, starts, kv, True, 1.0, dtype == F32)
    tol = A * (2.0 ** -17 + (2.0 ** -22 if dtype == F32 else 2.0 ** -11) + (2 * max(kv) + 64) * 2.0 ** -24)
    tol += (2.0 ** -24 if dtype == F32 else 2.0 ** -8) * (np.abs(want) + tol)
    assert not np.isnan(got).any() and (np.abs(got - want) <= tol).all()


FEW, MANY, LONG = ([1, 3, 1], [100, 333, 2600]), ([40, 1, 200], [100, 70, 200]), ([20, 33, 2], [2500, 1100, 600])


@pytest.mark.parametrize("dtype,dim", [(BF, 64), (BF, 128), (BF, 192), (BF, 256), (F32, 64), (F32, 128), (F32, 256)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("base", [2.0 ** 9, 2.0 ** 12, 2.0 ** 15])
@pytest.mark.parametrize("new,kv", [FEW, MANY, LONG])
def test_attend_where_one_channel_stands_out(dtype, dim, page, base, new, kv):
    """One product of the sum q.k is up to 2^15 times the others, which alone tell the tokens apart."""
    check_whole_scores(dtype, dim, page, base, 1.0, new, kv)


@pytest.mark.parametrize("dtype,dim", [(BF, 64), (BF, 128), (BF, 192), (BF, 256), (F32, 64), (F32, 128), (F32, 256)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("base,unit", [(2.0 ** 20, 1.0), (2.0 ** 22, 1.0), (0.0, 2.0 ** 24), (2.0 ** 15, 2.0 ** 40),
                                       (0.0, 2.0 ** 110)])
@pytest.mark.parametrize("new,kv", [FEW, MANY, LONG])
def test_attend_scores_far_from_zero(dtype, dim, page, base, unit, new, kv):
    """Scores whose rounding to float32 is coarser than what tells them apart, or that pass
    what an exponent may be: only differences of scores may enter p."""
    check_whole_scores(dtype, dim, page, base, unit, new, kv)


def test_attend_refuses_an_out_that_shares_memory_with_q():
    """The same projection's buffer: parts of it that lie over q's rows are refused, its
    free rows and the gaps between q's rows are not."""
    cache = filled(np.random.default_rng(30), 2, 2, 16, 64)[0]
    buf = torch.randn((12, 8, 64), dtype=BF, device=DEV)
    args = (cache, ints([[0, 1]]), ints([0, 4]), ints([20]))
    q = buf[:4, 2:6]
    want = pqb.kv_attend_paged(q, *args)
    for at in (0, 64, 128, 1920):                                # q's rows end at 384, 896, 1408, 1920
        out = buf.view(-1)[at:at + 1024].view(4, 4, 64)
        with pytest.raises(ValueError) if at < 1920 else contextlib.nullcontext():
            pqb.kv_attend_paged(q, *args, out=out)
    free = buf.view(-1)[4 * 512:4 * 512 + 1024].view(4, 4, 64)
    assert torch.equal(pqb.kv_attend_paged(q, *args, out=free), want)
    wide = torch.randn((2, 12, 64), dtype=BF, device=DEV)        # a gap of 8 heads holds 2 rows of 4
    one = (cache, ints([[0, 1]]), ints([0, 2]), ints([20]))
    got = pqb.kv_attend_paged(wide[:, :4], *one, out=wide.view(-1)[256:768].view(2, 4, 64))
    assert torch.equal(got, pqb.kv_attend_paged(wide[:, :4], *one))


def test_attend_refuses_a_workspace_that_is_no_tensor_there():
    cache = filled(np.random.default_rng(33), 2, 2, 16, 64)[0]
    q = torch.zeros((1, 4, 64), dtype=BF, device=DEV)
    ws = torch.empty((64, 64), dtype=torch.uint8, device=DEV)
    for bad in (1 << 20, ws.data_ptr(), ws.cpu(), ws[:, :32]):
        with pytest.raises(ValueError):
            pqb.kv_attend_paged(q, cache, ints([[0, 1]]), ints([0, 1]), ints([20]), workspace=bad)
    pqb.kv_attend_paged(q, cache, ints([[0, 1]]), ints([0, 1]), ints([20]), workspace=ws)


# ---------------------------------------------------------------------------
# many requests, and workspaces in use
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("batch,hint", [(130, "max"), (200, "max"), (200, None), (200, 1)])
def test_attend_of_many_requests_that_are_cut(dtype, page, batch, hint):
    """More requests than a wave looks at in one round (64): single tokens over thousands
    (cut into items), prompts (wide tiles, some cut along their tokens) and requests
    without queries on both sides of requests 63/64 and 127/128 and behind them."""
    rng = np.random.default_rng(31)
    new = (np.arange(batch) % 3 != 0).astype(int)             # every third has no query
    kv = rng.integers(0, 200, batch)
    for b in (2, 62, 63, 64, 127, 128, 129):
        new[b], kv[b] = 1, 1500 + 7 * b
    for b in (5, 61, 65, 66, 126, batch - 2, batch - 1):
        new[b], kv[b] = 17 + b % 50, 900 + 5 * b
    new[60], kv[60], new[67], kv[67] = 150, 150, 9, 2000
    new[68], kv[68] = 0, 2500
    check_attend(rng, new.tolist(), kv.tolist(), 2, 2, 64, page, dtype, hint=hint)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 64])
def test_attend_of_many_single_tokens_that_are_cut(dtype, page):
    """Decoding alone (the row kernel, its items and their join), over 300 requests."""
    rng = np.random.default_rng(32)
    kv = rng.integers(0, 700, 300)
    kv[[0, 63, 64, 200, 255, 256, 299]] = [3000, 2500, 2600, 5000, 600, 2048, 4097]
    check_attend(rng, [1] * 300, kv.tolist(), 1, 4, 64, page, dtype, spare=3)


class Filled(Server):
    """A server whose requests hold thousands of tokens already."""

    def __init__(self, lens, seed, heads, group, dim, page, width, max_new, dtype):
        super().__init__(len(lens), heads, group, dim, page, width, len(lens) * width, max_new, dtype)
        rng = np.random.default_rng(seed)
        self.cache, self.host = filled(rng, len(lens) * width, heads, page, dim)
        self.new.copy_(ints(lens))
        big = pqb.PagedPlan(ints([0] * sum(lens)), ints([0] * (len(lens) + 1)), self.lens, self.used, ints([0] * 4))
        pqb.kv_plan_paged(self.lens, self.new, self.table, self.free, self.used, page, sum(lens), out=big)
        assert big.status[0].item() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_streams_use_their_workspaces_at_once(dtype):
    """Two servers of other data on two streams: single tokens over thousands and a chunk,
    all cut, so that every call writes and joins parts; each as it does alone."""
    lens, kw = [4000, 2500, 3000], dict(heads=2, group=4, dim=128, page=64, width=80, max_new=64, dtype=dtype)

    def make(k):
        s = Filled(lens, 40 + k, **kw)
        s.qkv.copy_(torch.randn(s.qkv.shape, generator=torch.Generator().manual_seed(50 + k)))
        s.new.copy_(ints([1, 1, 40]))
        return s

    need = pqb.pqb.lib().pqb_kv_attend_workspace_bytes(0 if dtype == F32 else 1, 64, 8, 2, 128, 3, 80, 64, 0)
    assert need > 1 << 20
    servers, streams = [make(0), make(1)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for k, (s, st) in enumerate(zip(servers, streams)):
            with torch.cuda.stream(st):
                s.step()
                outs[k].append(s.out.clone())
    torch.cuda.synchronize()
    for k in range(2):
        alone = make(k)
        for got in outs[k]:
            alone.step()
            assert torch.equal(got, alone.out)
        assert alone.plan.status[0].item() == 0
    assert not torch.equal(outs[0][0], outs[1][0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_replays_cross_into_cuts(dtype):
    """One captured step replayed while lengths pass 512 tokens, where items and tiles
    begin to be cut, and from nothing to a chunk and back; every replay against the plain form."""
    heads, group, dim, page, width = 2, 2, 64, 16, 200
    s = Filled([509, 2000, 30, 511], 60, heads, group, dim, page, width, 64, dtype)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        s.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    rng = np.random.default_rng(61)
    codes = [s.host[0].copy(), np.ascontiguousarray(s.host[1].transpose(0, 1, 3, 2))]
    scales = [s.host[2].copy(), s.host[3].copy()]
    table, free, lens, used = s.table.cpu().numpy(), s.free.cpu().numpy(), s.lens.tolist(), s.used.item()
    hq = heads * group
    for new in ([1, 1, 1, 1], [2, 1, 0, 0], [1, 30, 1, 1], [1, 1, 1, 20], [0, 0, 40, 0], [1, 1, 1, 1], [25, 1, 1, 1]):
        x = torch.from_numpy(rng.standard_normal(tuple(s.qkv.shape))).to(dtype)
        s.qkv.copy_(x)
        s.new.copy_(ints(new))
        s.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        flags, table, slots, starts, lens, used, _ = paged.plan(lens, new, table, free, used, page, 64)
        lens = lens.tolist()
        assert flags == 0 and s.lens.tolist() == lens
        xd = x.double().numpy()
        paged.append(xd[:, hq:hq + heads], slots, codes[0], scales[0])
        paged.append(xd[:, hq + heads:], slots, codes[1], scales[1])
        T = int(starts[-1])
        want, bound = paged.attend(xd[:T, :hq], codes[0], codes[1].transpose(0, 1, 3, 2), *scales,
                                   np.where(table < 0, 0, table), starts, lens, True, dim ** -0.5, dtype == F32)
        got = s.out.double().cpu().numpy()
        assert (got[T:] == 7).all() and (np.abs(got[:T] - want) <= bound).all(), new
