"""The plain forms of the paged KV cache against values worked out by hand and a
second formulation, and every refusal of the paged entry points (CPU only: each
returns its status before anything reaches the GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import precision_quantization_block_amd as pqb
from oracle import paged
from precision_quantization_block_amd.pqb import _KvPages


def test_e4m3_codes_are_nearest_even():
    v = paged.e4m3_values()
    finite = np.flatnonzero(~np.isnan(v))
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v[finite], t[finite])
    assert np.array_equal(paged.e4m3_codes(v[finite]), finite)
    y = np.random.default_rng(0).uniform(-448, 448, 20000) * np.exp2(-(np.arange(20000) % 20.0))
    y = np.concatenate([y, (v[:0x7E] + v[1:0x7F]) / 2]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(paged.e4m3_codes(y.astype(np.float64)), want)


def test_exponent_is_the_smallest_that_holds():
    for x in (-30, -3, 0, 5, 100):
        assert paged.exponent(448.0 * 2.0 ** x) == x
        assert paged.exponent(np.nextafter(np.float32(448.0 * 2.0 ** x), np.float32(np.inf))) == x + 1
    assert paged.exponent(0.0) == paged.exponent(1e-13) == -48


def test_plan_by_hand():
    # pages of 16; request 0 fills its page and takes one, 1 starts, 2 only waits
    table = np.array([[5, -9, -9], [-9, -9, -9], [7, 8, -9]])
    free = np.array([3, 2, 9, 4])
    flags, t, slots, starts, kv, used, need = paged.plan([15, 0, 20], [2, 17, 0], table, free, 1, 16, 21)
    assert (flags, used, need) == (0, 4, 3)
    assert t.tolist() == [[5, 2, -9], [9, 4, -9], [7, 8, -9]]
    assert slots.tolist() == [5 * 16 + 15, 2 * 16] + [9 * 16 + i for i in range(16)] + [4 * 16, -1, -1]
    assert starts.tolist() == [0, 2, 19, 19] and kv.tolist() == [17, 17, 20]
    assert paged.plan([15], [2], table[:1], free, 4, 16, 9)[0] == 1
    assert paged.plan([15], [40], table[:1], free, 0, 16, 99)[0] == 2
    assert paged.plan([15], [2], table[:1], free, 0, 16, 1)[0] == 4
    assert paged.plan([-1], [2], table[:1], free, 0, 16, 9)[0] == 8


def test_append_rescales_what_the_page_holds():
    codes, scales = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1), np.uint8)
    x = np.full((1, 1, 64), 448.0)
    paged.append(x, np.array([0]), codes, scales)
    assert scales[0, 0] == 127 and (codes[0, 0, 0] == 0x7E).all()
    paged.append(x * 4, np.array([1]), codes, scales)       # X rises by 2
    val = paged.e4m3_values()
    assert scales[0, 0] == 129 and (val[codes[0, 0, 0]] * 4 == 448).all() and (codes[0, 0, 1] == 0x7E).all()
    paged.append(x / 64, np.array([2]), codes, scales)      # and never falls inside a page
    assert scales[0, 0] == 129 and (val[codes[0, 0, 2]] * 4 == 7).all()
    paged.append(x / 64, np.array([0]), codes, scales)      # a page begun anew forgets
    assert scales[0, 0] == 121


def test_attend_against_softmax():
    rng = np.random.default_rng(1)
    kc, vc = rng.integers(0, 0x70, (3, 2, 16, 64)).astype(np.uint8), rng.integers(0, 0x70, (3, 2, 64, 16)).astype(np.uint8)
    sc = np.full((3, 2), 122, np.uint8)
    q, table = rng.standard_normal((5, 4, 64)), np.array([[2, 0, 77], [1, 1, 1]])
    out, bound = paged.attend(q, kc, vc, sc, sc, table, [0, 3, 5], [20, 0], True, 0.1, True)
    val = torch.from_numpy(paged.e4m3_values())
    k = (val[torch.from_numpy(kc[[2, 0]]).long()] / 32).transpose(0, 1).reshape(2, 32, 64)[:, :20]
    v = (val[torch.from_numpy(vc[[2, 0]]).long()] / 32).permute(1, 0, 3, 2).reshape(2, 32, 64)[:, :20]
    for i in range(3):
        for h in range(4):
            p = torch.softmax(torch.from_numpy(q[i, h]) @ k[h // 2, :18 + i].T * 0.1, 0)
            assert np.allclose(out[i, h], (p @ v[h // 2, :18 + i]).numpy(), rtol=1e-12)
    assert (out[3:] == 0).all() and (bound[3:] == 0).all() and (bound[:3] > 0).all()
    # a page id outside the cache hides its tokens: here all but the first 16
    cut, _ = paged.attend(q[:1], kc, vc, sc, sc, np.array([[2, 77, -1]]), [0, 1], [40], False, 0.1, True)
    want, _ = paged.attend(q[:1], kc, vc, sc, sc, np.array([[2, 0, 0]]), [0, 1], [16], False, 0.1, True)
    assert np.allclose(cut, want, rtol=1e-13)


# ---------------------------------------------------------------------------
# refusals (fake addresses: never touched)
# ---------------------------------------------------------------------------

FAKE = ctypes.c_void_p(1 << 20)


def pages(**kw):
    d = dict(k=1 << 20, v=1 << 20, ks=1 << 20, vs=1 << 20, pages=4, heads=2, dim=64, page=16, res=0) | kw
    return ctypes.byref(_KvPages(d["k"], d["v"], d["ks"], d["vs"], d["pages"], d["heads"], d["dim"], d["page"], d["res"]))


def test_status_has_a_text():
    assert pqb.status_string(-9) != "unknown status"


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), -4), (dict(width=-1), -4), (dict(width=1 << 28), -4), (dict(free=-1), -4),
    (dict(max_new=-1), -4), (dict(max_new=1 << 31), -4), (dict(page=24), -4), (dict(page=8), -4),
    (dict(page=512), -4), (dict(cached=None), -1), (dict(status=None), -1), (dict(slots=None), -1),
    (dict(free_pages=None), -1), (dict(table=None), -1), (dict(used=None), -1), (dict(starts=None), -1),
    (dict(table=ctypes.c_void_p((1 << 20) + 2)), -5), (dict(slots=ctypes.c_void_p((1 << 20) + 1)), -5),
    (dict(max_new=1025), -6), (dict(batch=2049), -6), (dict(max_new=1025, ws=None, wsb=1 << 20), -1)])
def test_plan_refuses(kw, status):
    d = dict(cached=FAKE, new=FAKE, batch=3, table=FAKE, width=8, free_pages=FAKE, free=9, used=FAKE, page=16,
             max_new=9, slots=FAKE, starts=FAKE, kv=FAKE, out=FAKE, status=FAKE, ws=FAKE, wsb=0) | kw
    assert pqb.lib().pqb_kv_plan_paged(
        d["cached"], d["new"], d["batch"], d["table"], d["width"], d["free_pages"], d["free"], d["used"], d["page"],
        d["max_new"], d["slots"], d["starts"], d["kv"], d["out"], d["status"], d["ws"], d["wsb"], None) == status


@pytest.mark.parametrize("kw,cache,status", [
    (dict(dtype=2), {}, -2), (dict(), dict(res=1), -2), (dict(), dict(page=48), -4), (dict(), dict(dim=96), -4),
    (dict(), dict(heads=0), -4), (dict(), dict(heads=5000), -4), (dict(), dict(pages=-1), -4),
    (dict(), dict(pages=1 << 27), -4), (dict(tokens=-1), {}, -4), (dict(tokens=1 << 27), {}, -4),
    (dict(kld=64), {}, -4), (dict(vld=64), {}, -4), (dict(vld=1 << 40), {}, -4), (dict(k=None), {}, -1),
    (dict(v=None), {}, -1), (dict(slots=None), {}, -1), (dict(), dict(vs=None), -1),
    (dict(k=ctypes.c_void_p(8)), {}, -5), (dict(kld=132), {}, -5), (dict(), dict(k=8), -5),
    (dict(slots=ctypes.c_void_p(2)), {}, -5), (dict(tokens=0, k=None), {}, 0), (dict(k=None), dict(pages=0), 0)])
def test_append_refuses(kw, cache, status):
    d = dict(k=FAKE, v=FAKE, dtype=1, tokens=3, kld=128, vld=128, slots=FAKE) | kw
    assert pqb.lib().pqb_kv_append_paged(d["k"], d["v"], d["dtype"], d["tokens"], d["kld"], d["vld"], d["slots"],
                                         pages(**cache), None) == status


@pytest.mark.parametrize("kw,cache,status", [
    (dict(dtype=7), {}, -2), (dict(), dict(res=3), -2), (dict(), dict(page=0), -4), (dict(heads=3), {}, -4),
    (dict(heads=0), {}, -4), (dict(rows=-1), {}, -4), (dict(rows=1 << 28), {}, -4), (dict(batch=-1), {}, -4),
    (dict(batch=1 << 20), {}, -4), (dict(width=1 << 27), {}, -4), (dict(ld=255), {}, -4), (dict(ld=260), {}, -5),
    (dict(scale=-1.0), {}, -9), (dict(scale=float("nan")), {}, -9), (dict(scale=float("inf")), {}, -9),
    (dict(q=None), {}, -1), (dict(out=None), {}, -1), (dict(table=None), {}, -1), (dict(starts=None), {}, -1),
    (dict(kv=None), {}, -1), (dict(q=ctypes.c_void_p(8)), {}, -5), (dict(out=ctypes.c_void_p(24)), {}, -5),
    (dict(kv=ctypes.c_void_p(2)), {}, -5), (dict(wsb=0), {}, -6), (dict(ws=None), {}, -1),
    (dict(ws=ctypes.c_void_p(8)), {}, -5), (dict(rows=0, q=None), {}, 0), (dict(batch=0, kv=None), {}, 0)])
def test_attend_refuses(kw, cache, status):
    d = dict(q=FAKE, dtype=1, rows=3, heads=4, ld=256, table=FAKE, width=500, starts=FAKE, kv=FAKE, batch=2,
             scale=0.1, out=FAKE, ws=FAKE, wsb=1 << 40) | kw
    assert pqb.lib().pqb_kv_attend_paged(
        d["q"], d["dtype"], d["rows"], d["heads"], d["ld"], pages(**cache), d["table"], d["width"], d["starts"],
        d["kv"], d["batch"], 1, d["scale"], 0, d["out"], d["ws"], d["wsb"], None) == status


@pytest.mark.parametrize("scale,status", [(2.0 ** 127, 0), (2.5e38, -9), (3e38, -9), (3.4e38, -9), (0.0, 0)])
def test_scale_stays_finite_in_powers_of_two(scale, status):
    """scale * log2(e) is what the kernels multiply by."""
    assert pqb.lib().pqb_kv_attend_paged(FAKE, 1, 0, 2, 128, pages(), FAKE, 1, FAKE, FAKE, 1, 1, scale, 0, FAKE, FAKE,
                                         0, None) == status


def test_null_cache_is_refused():
    L = pqb.lib()
    assert L.pqb_kv_append_paged(FAKE, FAKE, 1, 1, 128, 128, FAKE, None, None) == -1
    assert L.pqb_kv_attend_paged(FAKE, 1, 1, 2, 128, None, FAKE, 1, FAKE, FAKE, 1, 1, 0.1, 0, FAKE, FAKE, 0, None) == -1


def test_workspaces():
    L = pqb.lib()

    def ws(**kw):
        d = dict(dtype=1, rows=64, q_heads=32, heads=8, dim=128, batch=64, width=500, page=64, hint=1) | kw
        return L.pqb_kv_attend_workspace_bytes(*d.values())

    assert ws(width=8) == 0 < ws(width=9)                  # 512 tokens: one item each
    assert ws() <= ws(hint=0) and ws(dtype=0) <= ws(dtype=0, hint=0)
    assert ws(heads=7) == ws(rows=0) == ws(batch=0) == ws(dtype=2) == ws(page=8) == ws(batch=1 << 20) == 0
    assert L.pqb_kv_plan_workspace_bytes(2048, 1024) == 0 and L.pqb_kv_plan_workspace_bytes(7, 1025) == 28


def test_binding_refuses_host_tensors():
    i = torch.zeros(1, dtype=torch.int32)
    c = pqb.PagedKV(*(torch.zeros(s, dtype=torch.uint8) for s in ((1, 1, 16, 64), (1, 1, 64, 16), (1, 1), (1, 1))))
    x = torch.zeros(1, 1, 64)
    for call in (lambda: pqb.kv_plan_paged(i, i, i.view(1, 1), i, i, 16, 1),
                 lambda: pqb.kv_append_paged(x, x, i, c),
                 lambda: pqb.kv_attend_paged(x, c, i.view(1, 1), torch.zeros(2, dtype=torch.int32), i)):
        with pytest.raises(ValueError, match="GPU"):
            call()
