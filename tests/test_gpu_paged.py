"""The paged 8-bit KV cache on the GPU against the plain forms in oracle/paged.py:
plans and appended codes equal in every byte, attention within the bound that its
arithmetic allows (derived in oracle.paged.attend); then steps of plan, append and
attention together, eager and replayed."""
import numpy as np
import pytest
import torch

import precision_quantization_block_amd as pqb
from oracle import paged

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def tiles(rng, counts, width):
    """A block table whose rows hold counts[b] pages of a shuffled pool, and the pool's size."""
    order, at = rng.permutation(sum(counts) + 2), 0
    t = np.full((len(counts), width), -7)
    for b, n in enumerate(counts):
        t[b, :n] = order[at:at + n]
        at += n
    return t, sum(counts) + 2


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

def check_plan(cached, new, table, free, used, page, max_new, in_place=False):
    c, t, f, u = ints(cached), ints(table), ints(free), ints([used])
    out = None
    if in_place:
        out = pqb.PagedPlan(ints(np.full(max_new, 99)), ints(np.full(len(cached) + 1, 99)), c, u, ints([99] * 4))
    p = pqb.kv_plan_paged(c, ints(new), t, f, u, page, max_new, out=out)
    flags, table, slots, starts, kv, used, need = paged.plan(cached, new, np.asarray(table), free, used, page, max_new)
    assert p.status.tolist() == [flags, need, sum(n for n in new if n >= 0) if not flags & 8 else p.status[2].item(), 0]
    for got, want, name in ((t, table, "table"), (p.slots, slots, "slots"), (p.q_starts, starts, "starts"),
                            (p.kv_lens, kv, "kv"), (p.free_used, [used], "used")):
        assert np.array_equal(got.cpu().numpy(), want), name
    return p


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,page,most,spare", [
    (1, 16, 1, 0), (1, 256, 0, 3), (7, 16, 40, 5), (64, 64, 1, 0), (300, 32, 9, 11), (1025, 16, 3, 0),
    (3, 64, 3000, 1), (2500, 128, 2, 4), (9, 16, 2000, 77)])
def test_plan(batch, page, most, spare, in_place):
    rng = np.random.default_rng(batch * 1000 + page)
    cached = rng.integers(0, 4 * page, batch).tolist()
    new = rng.integers(0, most + 1, batch).tolist()
    width = max(-(-(c + n) // page) for c, n in zip(cached, new)) + 2
    table, pages = tiles(rng, [-(-c // page) for c in cached], width)
    free = rng.permutation(pages + sum(new)) + 1000
    check_plan(cached, new, table, free, 3, page, sum(new) + spare, in_place)


def test_plan_without_requests_or_slots():
    p = pqb.kv_plan_paged(ints([]), ints([]), ints(np.zeros((0, 3))), ints([1]), ints([1]), 16, 5)
    assert p.slots.tolist() == [-1] * 5 and p.q_starts.tolist() == [0] and p.status.tolist() == [0] * 4
    check_plan([5, 0], [0, 0], np.array([[1], [2]]), [4], 0, 16, 0)


@pytest.mark.parametrize("max_new", [40, 5000])
@pytest.mark.parametrize("change,flag", [("pages", 1), ("table", 2), ("slots", 4), ("negative", 8), ("used", 8)])
def test_plan_is_all_or_nothing(change, flag, max_new):
    cached, new, table, free, used = [16, 3, 30], [17, 0, 4], np.array([[1, -7, -7], [2, -7, -7], [3, 4, -7]]), [9, 8, 7], 0
    if change == "pages":
        used = 1
    if change == "table":
        new, free = [33, 0, 4], [9, 8, 7, 6]
    if change == "slots":
        new, table = [max_new + 1, 0, 0], np.full((3, max_new // 16 + 4), 1)
        free = list(range(max_new))
    if change == "negative":
        new = [17, -1, 4]
    if change == "used":
        used = -1
    p = check_plan(cached, new, table, free, used, 16, max_new)
    assert p.status[0].item() & flag


def test_plan_with_bad_page_ids_gives_no_slot():
    # a held page that is none, and a free page whose slots pass 2^31
    check_plan([3, 0], [2, 18], np.array([[-5, 0], [0, 0]]), [7, 2 ** 31 - 2], 0, 16, 25)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

class Cache:
    """A cache on the GPU full of one byte, and its plain copy (V token-major)."""

    def __init__(self, pages, heads, page, dim, fill=0xA5):
        self.gpu = pqb.kv_paged_cache(pages, heads, page, dim, DEV)
        for t in (self.gpu.k_codes, self.gpu.v_codes, self.gpu.k_scales, self.gpu.v_scales):
            t.fill_(fill)
        self.k, self.v = (np.full((pages, heads, page, dim), fill, np.uint8) for _ in "kv")
        self.ks, self.vs = (np.full((pages, heads), fill, np.uint8) for _ in "kv")

    def append(self, k, v, slots):
        n = len(k)
        pqb.kv_append_paged(k, v, ints(slots), self.gpu)
        ok = (np.asarray(slots[:n]) >= 0) & (np.asarray(slots[:n]) < self.k.shape[0] * self.k.shape[2])
        z = torch.from_numpy(ok)[:, None, None]
        paged.append(torch.where(z, k.cpu(), 0).double().numpy(), slots[:n], self.k, self.ks)
        paged.append(torch.where(z, v.cpu(), 0).double().numpy(), slots[:n], self.v, self.vs)

    def check(self):
        assert np.array_equal(self.gpu.k_scales.cpu().numpy(), self.ks)
        assert np.array_equal(self.gpu.v_scales.cpu().numpy(), self.vs)
        assert np.array_equal(self.gpu.k_codes.cpu().numpy(), self.k)
        assert np.array_equal(self.gpu.v_codes.cpu().numpy(), self.v.transpose(0, 1, 3, 2))


def values(rng, shape, dtype, spread=3.0):
    """Normal values, each token and head at a magnitude of its own."""
    x = rng.standard_normal(shape) * np.exp2(rng.uniform(-spread, spread, shape[:2] + (1,)))
    return torch.from_numpy(x).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, 1), (128, 64, 3), (192, 32, 2), (256, 256, 1), (128, 128, 2)])
def test_append_steps(dtype, dim, page, heads):
    """Prompts, then chunks of 0 to 70 tokens on whatever the pages hold."""
    rng = np.random.default_rng(dim + page)
    B, width = 5, -(-600 // page)
    table, pages = tiles(rng, [width] * B, width)
    c, lens = Cache(pages, heads, page, dim), [0] * B
    for most in (page + 3, 1, 1, 70, 2, 17):
        new = rng.integers(0, most + 1, B) if most != 1 else np.ones(B, int)
        slots = [table[b, p // page] * page + p % page for b in range(B) for p in range(lens[b], lens[b] + new[b])]
        lens = [a + b for a, b in zip(lens, new)]
        shape = (len(slots), heads, dim)
        c.append(values(rng, shape, dtype), values(rng, shape, dtype), slots)
        c.check()


def test_append_of_many_tokens_and_small_runs():
    """Enough tokens that a workgroup takes a window of them, in runs of 1 to 40."""
    rng = np.random.default_rng(4)
    page, heads, dim, slots = 32, 8, 64, []
    for p in rng.permutation(500):
        o = int(rng.integers(0, page)) if rng.random() < 0.5 else 0
        slots += range(p * page + o, p * page + int(rng.integers(o + 1, page + 1)))
    c = Cache(500, heads, page, dim, fill=0x30)
    for k in range(2):
        c.append(values(rng, (len(slots), heads, dim), BF), values(rng, (len(slots), heads, dim), BF), slots)
        c.check()


def test_append_skips_padding_and_reads_nothing_of_it():
    rng = np.random.default_rng(5)
    c = Cache(4, 2, 16, 64)
    k, v = values(rng, (9, 2, 64), F32), values(rng, (9, 2, 64), F32)
    slots = [-1, 16, 17, 64, 32, 2 ** 31 - 1, -2 ** 31, 0, -1]
    for i, s in enumerate(slots):
        if not 0 <= s < 64:
            k[i], v[i] = float("nan"), float("inf")
    c.append(k, v, slots)
    c.check()
    pqb.kv_append_paged(k[:0], v[:0], ints([]), c.gpu)
    pqb.kv_append_paged(k[:1], v[:1], ints(slots), c.gpu)       # slots may be longer than k
    c.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_of_strided_parts(dtype):
    """k and v inside one projection's rows, and rows that no 16-byte step reaches."""
    rng = np.random.default_rng(6)
    qkv = values(rng, (37, 8, 64), dtype)
    slots = list(range(5, 42))
    for k, v in ((qkv[:, 4:6], qkv[:, 6:8]), (qkv.view(-1)[1:1 + 37 * 128].view(37, 2, 64), qkv[:, 1:3]),
                 (qkv[:, 0:4:2], qkv[:, :2].flip(2))):
        c = Cache(3, 2, 16, 64)
        c.append(k, v, slots)
        c.check()


def test_append_extremes():
    """Zeros, the largest and smallest floats, and scales that rise by over 20."""
    c = Cache(1, 1, 16, 64)
    rows = torch.zeros((16, 1, 64), device=DEV)
    for i, x in enumerate((0.0, 1e-38, 1e-13, 1e-5, 448.0, 449.0, 1e9, 3.3e38)):
        rows[i, 0, ::3], rows[i, 0, 1] = x, -x / 7
        c.append(rows[i:i + 1], rows[i:i + 1] / 3, [i])
        c.check()


# ---------------------------------------------------------------------------
# attend
# ---------------------------------------------------------------------------

def filled(rng, pages, heads, page, dim, lo=117, hi=122):
    """A cache of random codes and scales on the GPU, and the same arrays on the host."""
    def codes():
        x = torch.from_numpy(rng.standard_normal((pages, heads, page, dim)) * 60)
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    k, v = codes(), codes().transpose(2, 3).contiguous()
    ks, vs = (torch.from_numpy(rng.integers(lo, hi + 1, (pages, heads)).astype(np.uint8)) for _ in "kv")
    host = [t.numpy() for t in (k, v, ks, vs)]
    return pqb.PagedKV(*(t.to(DEV) for t in (k, v, ks, vs))), host


def poison(cache, host, table, kv, page):
    """NaN codes behind every request's last token (left out of sight by its length)."""
    for b, n in enumerate(kv):
        if n % page:
            p = table[b, n // page]
            cache.k_codes[p, :, n % page:] = 0x7F
            cache.v_codes[p, :, :, n % page:] = 0xFF


def check_attend(rng, new, kv, heads, group, dim, page, dtype, causal=True, scale=None, hint="max", qscale=1.5,
                 lo=117, hi=122, table=None, spare=0):
    counts = [-(-n // page) for n in kv]
    width = max(counts + [1]) + spare
    if table is None:
        table, pages = tiles(rng, counts, width)
    else:
        pages = max(table.max() // 2, 1)
    cache, host = filled(rng, pages, heads, page, dim, lo, hi)
    starts = np.concatenate([[0], np.cumsum(new)])
    T = int(starts[-1])
    q = torch.from_numpy(rng.standard_normal((T, heads * group, dim)) * qscale).to(dtype)
    if pages > 2:
        poison(cache, host, table, kv, page)
    out = torch.full((T + 2, heads * group, dim), 7.0, dtype=dtype, device=DEV)
    hint = max(new) if hint == "max" else hint
    qd = torch.zeros((T + 2, heads * group, dim), dtype=dtype, device=DEV)
    qd[:T] = q.to(DEV)
    pqb.kv_attend_paged(qd, cache, ints(table), ints(starts), ints(kv), causal=causal, scale=scale, max_q_len=hint,
                        out=out)
    val = 1 / np.sqrt(dim) if scale is None else np.float64(np.float32(scale))
    want, bound = paged.attend(q.double().numpy(), *host, table, starts, kv, causal, val, dtype == F32)
    got = out.double().cpu().numpy()
    assert (got[T:] == 7).all()                       # rows behind the last request
    off = np.abs(got[:T] - want) - bound
    assert not np.isnan(got).any() and (off <= 0).all(), f"{off.max()} over, at {np.unravel_index(off.argmax(), off.shape)}"
    return got[:T]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim,page,heads,group", [
    (64, 16, 1, 1), (64, 32, 2, 4), (128, 64, 2, 4), (128, 16, 1, 8), (192, 64, 1, 3), (256, 128, 2, 2),
    (128, 256, 1, 16), (64, 64, 3, 5)])
def test_attend_single_tokens(dtype, dim, page, heads, group):
    rng = np.random.default_rng(dim + page + group)
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 130, 255, 256, 257, 700, 0]
    check_attend(rng, [1] * len(kv), kv, heads, group, dim, page, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hint", ["max", None, 1])
def test_attend_ragged_queries(dtype, causal, hint):
    """No query, one, a few, more than a tile; fewer tokens than queries (rows that see nothing)."""
    rng = np.random.default_rng(11)
    new, kv = [3, 0, 1, 40, 5, 17, 2, 130], [3, 9, 200, 90, 2, 0, 1000, 131]
    check_attend(rng, new, kv, 2, 3, 64, 32, dtype, causal=causal, hint=hint)


@pytest.mark.parametrize("dtype,dim,heads,group,page", [
    (BF, 128, 2, 4, 64), (BF, 64, 3, 1, 16), (BF, 256, 1, 2, 32), (F32, 128, 1, 2, 64), (BF, 192, 1, 4, 128),
    (F32, 64, 2, 3, 128), (F32, 128, 1, 4, 16), (F32, 256, 1, 2, 32), (F32, 192, 1, 2, 64), (BF, 256, 1, 8, 256)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_prompts(dtype, dim, heads, group, page, causal):
    rng = np.random.default_rng(12)
    check_attend(rng, [300, 1, 65, 129], [300, 77, 400, 500], heads, group, dim, page, dtype, causal=causal)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_splits_long_requests(dtype):
    rng = np.random.default_rng(13)
    check_attend(rng, [1, 1, 1, 6], [9001, 40, 300, 5000], 2, 4, 128, 64, dtype, spare=5)


@pytest.mark.parametrize("dtype,dim", [(BF, 128), (F32, 128), (BF, 256), (F32, 64), (F32, 256)])
@pytest.mark.parametrize("page", [16, 64])
def test_attend_splits_long_prompts(dtype, dim, page):
    """A few rows over many tokens: tiles cut along the tokens, and more units than
    are looked up at a time (64)."""
    rng = np.random.default_rng(23)
    check_attend(rng, [20, 3, 70], [5000, 4500, 4200], 1, 2, dim, page, dtype)
    check_attend(rng, [33], [9000], 1, 1, dim, page, dtype, causal=False, spare=3)


@pytest.mark.parametrize("page", [16, 64])
def test_attend_with_a_wrong_hint_over_many_tokens(page):
    """More rows than the hint allows are not cut: a wave walks over 64 units of its own."""
    rng = np.random.default_rng(25)
    check_attend(rng, [20, 1], [17000, 70], 1, 1, 64, page, BF, hint=1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_of_one_long_row_tile(dtype):
    """Enough heads that nothing is cut: one workgroup walks 150 units."""
    rng = np.random.default_rng(24)
    check_attend(rng, [130] * 10, [9600] + [140] * 9, 16, 1, 64, 64, dtype)


def test_attend_of_many_requests():
    rng = np.random.default_rng(14)
    kv = rng.integers(0, 90, 200).tolist()
    check_attend(rng, rng.integers(0, 3, 200).tolist(), kv, 1, 2, 64, 16, BF, causal=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new", [[1, 1, 2], [90, 70, 65]])
def test_attend_scales_far_apart(dtype, new):
    """Neighbouring pages whose V differ by up to 2^60, and keys that make one token win."""
    rng = np.random.default_rng(15)
    check_attend(rng, new, [100, 333, 90], 2, 2, 64, 16, dtype, lo=90, hi=150, scale=2.0 ** -30)
    check_attend(rng, new, [100, 333, 90], 2, 2, 128, 64, dtype, scale=3.0)
    check_attend(rng, new, [100, 333, 90], 2, 2, 64, 32, dtype, scale=0.0)


def test_attend_leaves_out_pages_that_are_none():
    rng = np.random.default_rng(16)
    table = np.array([[0, 99, 1, -1, 2], [3, 4, 5, 2 ** 30, 1], [77, 77, 77, 77, 77]])
    table_max = np.where(np.abs(table) < 50, table, 0).max()
    for new in ([1, 2, 1], [70, 66, 90]):
        cache, host = filled(rng, int(table_max) + 1, 2, 16, 64)
        kv, starts = [75, 70, 80], np.concatenate([[0], np.cumsum(new)])
        q = torch.from_numpy(rng.standard_normal((int(starts[-1]), 4, 64))).to(BF)
        for causal in (True, False):
            got = pqb.kv_attend_paged(q.to(DEV), cache, ints(table), ints(starts), ints(kv), causal=causal)
            want, bound = paged.attend(q.double().numpy(), *host, table, starts, kv, causal, 0.125, False)
            assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()


def test_attend_cuts_lengths_at_the_table_and_rows_at_q():
    rng = np.random.default_rng(17)
    table, pages = tiles(rng, [2, 2], 2)
    cache, host = filled(rng, pages, 1, 16, 64)
    q = torch.from_numpy(rng.standard_normal((3, 2, 64))).to(F32)
    out = torch.full_like(q, 7.0, device=DEV)
    pqb.kv_attend_paged(q.to(DEV), cache, ints(table), ints([0, 1, 9]), ints([2 ** 31 - 1, -5]), causal=False, out=out)
    want, bound = paged.attend(q.double().numpy(), *host, table, [0, 1, 3], [32, 0], False, 0.125, True)
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


def test_attend_without_pages_or_width():
    q = torch.ones((2, 2, 64), dtype=BF, device=DEV)
    for pages, width in ((0, 3), (2, 0)):
        c = pqb.kv_paged_cache(pages, 1, 16, 64, DEV)
        out = pqb.kv_attend_paged(q, c, ints(np.zeros((1, width))), ints([0, 2]), ints([40]))
        assert (out == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_of_strided_queries(dtype):
    rng = np.random.default_rng(18)
    table, pages = tiles(rng, [7, 4], 7)
    cache, _ = filled(rng, pages, 2, 16, 64)
    qkv = torch.from_numpy(rng.standard_normal((4, 8, 64))).to(dtype).to(DEV)
    args = (cache, ints(table), ints([0, 3, 4]), ints([100, 64]))
    for q in (qkv[:, 2:6], qkv[:, 0:8:2], qkv.view(-1)[1:1025].view(4, 4, 64), qkv[:, :4].flip(2)):
        assert torch.equal(pqb.kv_attend_paged(q, *args), pqb.kv_attend_paged(q.clone(memory_format=torch.contiguous_format), *args))


@pytest.mark.parametrize("new,kv", [([1] * 9, [5000, 30, 2000, 1, 64, 65, 900, 3000, 7]), ([200, 90], [1500, 90])])
def test_attend_repeats_bit_for_bit(new, kv):
    """No sum depends on the order in which workgroups end; a workspace may hold anything."""
    rng = np.random.default_rng(19)
    table, pages = tiles(rng, [-(-n // 32) for n in kv], 200)
    cache, _ = filled(rng, pages, 2, 32, 128)
    q = torch.from_numpy(rng.standard_normal((sum(new), 8, 128))).to(BF).to(DEV)
    ws = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device=DEV)
    args = (q, cache, ints(table), ints(np.concatenate([[0], np.cumsum(new)])), ints(kv))
    first = pqb.kv_attend_paged(*args)
    for _ in range(3):
        assert torch.equal(pqb.kv_attend_paged(*args, workspace=ws), first)


@pytest.mark.parametrize("dtype,dim", [(BF, 64), (BF, 128), (F32, 64), (F32, 256)])
@pytest.mark.parametrize("page", [16, 64])
def test_a_row_that_is_not_finite_spoils_no_other(dtype, dim, page):
    rng = np.random.default_rng(dim + page)
    new, kv, bad = [3, 50, 1], [100, 650, 9], [(1, 1), (10, 0), (40, 3), (53, 2)]
    table, pages = tiles(rng, [-(-n // page) for n in kv], 50)
    cache, host = filled(rng, pages, 2, page, dim)
    starts = np.concatenate([[0], np.cumsum(new)])
    q = torch.from_numpy(rng.standard_normal((sum(new), 4, dim)) * 1.5).to(dtype)
    want, bound = paged.attend(q.double().numpy(), *host, table, starts, kv, True, 1 / np.sqrt(dim), dtype == F32)
    for (t, g), x in zip(bad, (float("nan"), float("inf"), float("-inf"), float("nan"))):
        q[t, g, 5:9] = x
    got = pqb.kv_attend_paged(q.to(DEV), cache, ints(table), ints(starts), ints(kv)).double().cpu().numpy()
    keep = np.ones(got.shape[:2], bool)
    keep[tuple(zip(*bad))] = False
    assert (np.abs(got - want) <= bound)[keep].all()


def test_offsets_past_32_bits():
    """Pages whose codes lie beyond 2^32 bytes: append, then attend, at both ends of the cache."""
    heads, page, dim = 8, 256, 256
    pages = (1 << 32) // (heads * page * dim) + 3
    cache = pqb.kv_paged_cache(pages, heads, page, dim, DEV)
    rng = np.random.default_rng(20)
    ids = np.array([[0, pages - 1, 1, pages - 2]])
    small, host = Cache(4, heads, page, dim), None
    k, v = values(rng, (900, heads, dim), BF, 1.0), values(rng, (900, heads, dim), BF, 1.0)
    pos = np.arange(900)
    pqb.kv_append_paged(k, v, ints(ids[0][pos // page] * page + pos % page), cache)
    small.append(k, v, pos.tolist())
    for i, p in enumerate(ids[0]):
        n = min(page, 900 - i * page)
        assert np.array_equal(cache.k_codes[p, :, :n].cpu().numpy(), small.k[i, :, :n])
        assert np.array_equal(cache.v_codes[p, :, :, :n].cpu().numpy(), small.v[i, :, :n].transpose(0, 2, 1))
    for n in (2, 100):
        q = values(rng, (n, heads, dim), BF, 0.5)
        got = pqb.kv_attend_paged(q, cache, ints(ids), ints([0, n]), ints([900]))
        assert torch.equal(got, pqb.kv_attend_paged(q, small.gpu, ints([[0, 1, 2, 3]]), ints([0, n]), ints([900])))


# ---------------------------------------------------------------------------
# refusals of the binding
# ---------------------------------------------------------------------------

def test_binding_refuses():
    i, t = ints([3]), ints([[0, 0]])
    c = pqb.kv_paged_cache(2, 2, 16, 64, DEV)
    x = torch.zeros((1, 2, 64), dtype=BF, device=DEV)
    s = ints([0, 1])
    bad = [lambda: pqb.kv_plan_paged(i, ints([1, 2]), t, i, i, 16, 4), lambda: pqb.kv_plan_paged(i, i.long(), t, i, i, 16, 4),
           lambda: pqb.kv_plan_paged(i, i, ints([[1, 2], [3, 4]]).t()[:1], i, i, 16, 4),
           lambda: pqb.kv_plan_paged(i, i, t, i, s, 16, 4), lambda: pqb.kv_plan_paged(i, i, t, i, i, 16, -1),
           lambda: pqb.kv_append_paged(x, x.float(), i, c), lambda: pqb.kv_append_paged(x, x[:, :1], i, c),
           lambda: pqb.kv_append_paged(x.half(), x.half(), i, c), lambda: pqb.kv_append_paged(x, x, i[:0], c),
           lambda: pqb.kv_append_paged(x, x.cpu(), i, c), lambda: pqb.kv_append_paged(x[..., :32], x[..., :32], i, c),
           lambda: pqb.kv_append_paged(x, x, i, pqb.PagedKV(c.k_codes, c.k_codes, c.k_scales, c.v_scales)),
           lambda: pqb.kv_append_paged(x, x, i, pqb.PagedKV(c.k_codes, c.v_codes, c.k_scales.float(), c.v_scales)),
           lambda: pqb.kv_attend_paged(x[:, :1], c, t, s, i), lambda: pqb.kv_attend_paged(x, c, t, i, i),
           lambda: pqb.kv_attend_paged(x, c, t, s, i, out=x.float()), lambda: pqb.kv_attend_paged(x, c, t, s, i, out=x), lambda: pqb.kv_attend_paged(x, c, t, s, i, max_q_len=0),
           lambda: pqb.kv_attend_paged(x, c, t.cpu(), s, i)]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {n} was not refused")
    with pytest.raises(pqb.PqbError):
        pqb.kv_plan_paged(i, i, t, i, i, 24, 4)
    with pytest.raises(pqb.PqbError):
        pqb.kv_attend_paged(x, c, t, s, i, scale=-1.0)
    with pytest.raises(pqb.PqbError):      # 2 x 300 x 16 tokens may be split: needs a workspace
        pqb.kv_attend_paged(x, c, ints(np.zeros((1, 300))), s, i, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

class Server:
    """Requests on the GPU: the step a serving program runs, all in place."""

    def __init__(self, batch, heads, group, dim, page, width, pages, max_new, dtype):
        self.cache = pqb.kv_paged_cache(pages, heads, page, dim, DEV)
        for t in (self.cache.k_codes, self.cache.v_codes):
            t.fill_(0x7F)
        self.table, self.free = ints(np.full((batch, width), -1)), ints(np.random.default_rng(0).permutation(pages))
        self.lens, self.used, self.new = ints([0] * batch), ints([0]), ints([0] * batch)
        self.plan = pqb.PagedPlan(ints([0] * max_new), ints([0] * (batch + 1)), self.lens, self.used, ints([0] * 4))
        shape = (max_new, heads * (group + 2), dim)
        self.qkv = torch.zeros(shape, dtype=dtype, device=DEV)
        self.out = torch.zeros((max_new, heads * group, dim), dtype=dtype, device=DEV)
        self.h, self.hq, self.page, self.max_new = heads, heads * group, page, max_new

    def step(self):
        pqb.kv_plan_paged(self.lens, self.new, self.table, self.free, self.used, self.page, self.max_new, out=self.plan)
        q, k, v = self.qkv[:, :self.hq], self.qkv[:, self.hq:self.hq + self.h], self.qkv[:, self.hq + self.h:]
        pqb.kv_append_paged(k, v, self.plan.slots, self.cache)
        pqb.kv_attend_paged(q, self.cache, self.table, self.plan.q_starts, self.lens, out=self.out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("stream", [False, True])
def test_steps_together(dtype, captured, stream):
    """Prompts, chunks and single tokens of four requests, one of which idles now and
    then, checked against the plain forms after every step; captured once and
    replayed with other lengths, or eager; on the default or another stream."""
    B, heads, group, dim, page, width, max_new = 4, 2, 2, 64, 16, 40, 200
    s = Server(B, heads, group, dim, page, width, B * width, max_new, dtype)
    side = torch.cuda.Stream()
    graph = None
    if captured:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):      # the allocator's and the library's first calls
            s.step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
    rng = np.random.default_rng(21)
    host = [np.full((B * width, heads, page, dim), 0x7F, np.uint8) for _ in "kv"]
    scales = [np.zeros((B * width, heads), np.uint8) for _ in "kv"]
    table, free, lens, used = np.full((B, width), -1), s.free.cpu().numpy(), [0] * B, 0
    for new in ([70, 1, 0, 33], [1, 1, 1, 1], [1, 0, 90, 1], [5, 100, 1, 1], [1, 1, 1, 1], [0, 0, 0, 0], [1, 1, 1, 1]):
        x = torch.from_numpy(rng.standard_normal(tuple(s.qkv.shape)) * np.exp2(rng.uniform(-1, 1, (max_new, 1, 1)))).to(dtype)
        s.qkv.copy_(x)
        s.new.copy_(ints(new))
        s.out.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side if stream else torch.cuda.current_stream()):
            graph.replay() if graph else s.step()
        torch.cuda.synchronize()
        flags, table, slots, starts, lens, used, _ = paged.plan(lens, new, table, free, used, page, max_new)
        lens = lens.tolist()
        assert flags == 0 and s.plan.status[0].item() == 0 and s.lens.tolist() == lens and s.used.item() == used
        xd = x.double().numpy()
        hq = heads * group
        paged.append(xd[:, hq:hq + heads], slots, host[0], scales[0])
        paged.append(xd[:, hq + heads:], slots, host[1], scales[1])
        assert np.array_equal(s.cache.k_codes.cpu().numpy(), host[0])
        assert np.array_equal(s.cache.v_codes.cpu().numpy(), host[1].transpose(0, 1, 3, 2))
        T = int(starts[-1])
        want, bound = paged.attend(xd[:T, :hq], host[0], host[1].transpose(0, 1, 3, 2), scales[0], scales[1],
                                   np.where(table < 0, 0, table), starts, lens, True, dim ** -0.5, dtype == F32)
        got = s.out.double().cpu().numpy()
        assert (got[T:] == 7).all() and (np.abs(got[:T] - want) <= bound).all(), new


def test_a_failed_step_changes_nothing():
    s = Server(2, 1, 2, 64, 16, 4, 3, 64, BF)
    s.qkv.normal_()
    s.new.copy_(ints([20, 5]))
    s.step()
    before = [t.clone() for t in (s.cache.k_codes, s.cache.v_codes, s.table, s.lens, s.used, s.out)]
    s.new.copy_(ints([20, 20]))
    s.out.copy_(before[5])
    s.step()
    assert s.plan.status.tolist() == [1, 2, 40, 0]
    for a, b in zip(before, (s.cache.k_codes, s.cache.v_codes, s.table, s.lens, s.used, s.out)):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Two servers' steps on two streams, each with a workspace of its own allocation."""
    servers = [Server(3, 2, 4, 128, 64, 40, 120, 96, BF) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in servers]
    alone = Server(3, 2, 4, 128, 64, 40, 120, 96, BF)
    for s in servers + [alone]:
        torch.manual_seed(3)
        s.qkv.copy_(torch.randn(s.qkv.shape))
        s.new.copy_(ints([40, 30, 20]))
    torch.cuda.synchronize()
    for _ in range(12):
        for s, st in zip(servers, streams):
            with torch.cuda.stream(st):
                s.step()
    torch.cuda.synchronize()
    for _ in range(12):
        alone.step()
    torch.cuda.synchronize()
    assert alone.plan.status.tolist()[0] == 0
    for s in servers:
        assert torch.equal(s.out, alone.out) and torch.equal(s.cache.v_codes, alone.cache.v_codes)


def test_encoder_states():
    """Cross attention: states appended once, then queries of other lengths, not causal."""
    rng = np.random.default_rng(22)
    heads, dim, page, lens = 3, 64, 32, [75, 32, 1]
    table, pages = tiles(rng, [-(-n // page) for n in lens], 3)
    c = Cache(pages, heads, page, dim)
    slots = [table[b, p // page] * page + p % page for b, n in enumerate(lens) for p in range(n)]
    c.append(values(rng, (len(slots), heads, dim), BF), values(rng, (len(slots), heads, dim), BF), slots)
    c.check()
    for new in ([1, 1, 1], [7, 0, 100]):
        starts = np.concatenate([[0], np.cumsum(new)])
        q = torch.from_numpy(rng.standard_normal((sum(new), heads, dim))).to(BF)
        got = pqb.kv_attend_paged(q.to(DEV), c.gpu, ints(table), ints(starts), ints(lens), causal=False)
        want, bound = paged.attend(q.double().numpy(), c.k, c.v.transpose(0, 1, 3, 2), c.ks, c.vs, table, starts, lens,
                                   False, 0.125, False)
        assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
