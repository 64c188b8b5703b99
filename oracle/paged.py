"""Plain forms of the paged 8-bit KV cache in 64 bits -- TEST INFRASTRUCTURE ONLY.

Loops over requests, pages and heads in numpy, written from the definitions in
include/pqb.h: the plan in integers, codes and exponents exact, attention in
float64 with the error bound that the engine's arithmetic allows beside it.
"""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes (0x7F and 0xFF are NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(float) - 10))
    v[(c & 0x7F) == 0x7F] = np.nan
    return np.where(c & 0x80, -v, v)


_VAL = e4m3_values()
_POS = _VAL[:0x7F]                       # 0 .. 448, rising with the code


def e4m3_codes(y: np.ndarray) -> np.ndarray:
    """The nearest code of each y (|y| <= 448), ties to the even code, sign kept."""
    a = np.abs(y)
    hi = np.clip(np.searchsorted(_POS, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def exponent(amax: float) -> int:
    """The smallest integer X with max(amax, 1e-12 as float32) <= 448 * 2^X."""
    a = max(float(amax), float(np.float32(1e-12)))
    x = int(np.floor(np.log2(a / 448.0))) - 1
    while a > 448.0 * 2.0 ** x:
        x += 1
    return x


def plan(cached, new, table, free, used, page, max_new):
    """(status flags, table, slots, starts, kv_lens, used, pages needed) after the call."""
    cached, new = [int(c) for c in cached], [int(n) for n in new]
    table, B, width = table.copy(), len(cached), table.shape[1]
    flags = 8 if used < 0 or used > len(free) or any(c < 0 or n < 0 for c, n in zip(cached, new)) else 0
    ok = [(c, n) for c, n in zip(cached, new) if c >= 0 and n >= 0]
    need = sum(-(-(c + n) // page) + (-c // page) for c, n in ok)
    if any(c + n > width * page for c, n in ok):
        flags |= 2
    if sum(n for _, n in ok) > max_new:
        flags |= 4
    if used >= 0 and need > len(free) - used:
        flags |= 1
    slots = np.full(max_new, -1, np.int64)
    if flags:
        return flags, table, slots, np.zeros(B + 1, np.int64), np.array(cached), used, need
    starts, t = [0], 0
    for b, (c, n) in enumerate(ok):
        for j in range(-(-c // page), -(-(c + n) // page)):
            table[b, j] = free[used]
            used += 1
        for pos in range(c, c + n):
            s = int(table[b, pos // page]) * page + pos % page
            slots[t] = s if 0 <= s < 2 ** 31 else -1
            t += 1
        starts.append(t)
    return 0, table, slots, np.array(starts), np.array(cached) + np.array(new), used, need


def append(x, slots, codes, scales):
    """x [T, H, D] float64 into token-major codes [pages, H, page, D] and scale bytes
    [pages, H], both updated in place."""
    pages, H, page, _ = codes.shape
    t = 0
    while t < len(slots):
        s, n = int(slots[t]), 1
        if not 0 <= s < pages * page:
            t += 1
            continue
        p, o = s // page, s % page
        while t + n < len(slots) and o + n < page and slots[t + n] == s + n:
            n += 1
        for h in range(H):
            rows, held = x[t:t + n, h], int(scales[p, h]) - 127
            e = exponent(np.abs(rows).max())
            if o:
                e = max(e, held)
                if e > held:
                    codes[p, h, :o] = e4m3_codes(_VAL[codes[p, h, :o]] * 2.0 ** (held - e))
            codes[p, h, o:o + n] = e4m3_codes(rows * 2.0 ** -e)
            scales[p, h] = e + 127
        t += n


def attend(q, k_codes, v_codes, k_scales, v_scales, table, starts, kv_lens, causal, scale, f32):
    """(out, bound), float64 [T, Hq, D]; rows outside every request are NaN.  `f32`:
    whether q and the output are float32 (else bf16).

    bound, for the engine's float32 evaluation, with A = sum p |v| / sum p:
      scores: products exact, float32 sums over D terms (and over three parts of a
        float32 q), so |ds| <= (3 D + 8) 2^-24 scale sum |k||q|; the exponent's
        argument is rounded twice more, 3 |s - max| 2^-24, and exp2 is within
        2^-22; p moves by at most that factor, above and below the line: 2 ds A;
      p rounded to f16, 2^-11 of itself (float32: remainder kept, 2^-22), and
        2^-34 of the largest below 2^-23; V to 2^-25 of its request's largest
        scale;
      sums over n tokens and at most n / 64 joins and rescalings: (2 n + 64) 2^-24 A;
      the output's rounding, 2^-8 (bf16) or 2^-24 of it."""
    T, Hq, D = q.shape
    pages, H, page, _ = k_codes.shape
    G, out, bound = Hq // H, np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for b in range(len(kv_lens)):
        n, kv = int(starts[b + 1]) - int(starts[b]), min(int(kv_lens[b]), table.shape[1] * page)
        if n <= 0:
            continue
        rows = slice(int(starts[b]), int(starts[b + 1]))
        ids = table[b, :-(-kv // page)].astype(np.int64)
        good = (ids >= 0) & (ids < pages)
        ids = np.where(good, ids, 0)
        usable = np.repeat(good, page)[:kv]
        see = np.broadcast_to(usable, (n, kv)).copy()
        if causal:
            see &= np.arange(kv)[None] <= kv - n + np.arange(n)[:, None]
        for h in range(H):
            k = (_VAL[k_codes[ids, h]] * 2.0 ** (k_scales[ids, h].astype(float) - 127)[:, None, None])
            v = (_VAL[v_codes[ids, h]] * 2.0 ** (v_scales[ids, h].astype(float) - 127)[:, None, None])
            k, v = k.reshape(-1, D)[:kv], v.transpose(0, 2, 1).reshape(-1, D)[:kv]
            k, v = np.where(usable[:, None], k, 0), np.where(usable[:, None], v, 0)
            top = float(np.max(2.0 ** (v_scales[ids, h].astype(float) - 127)[good], initial=0.0))
            for g in range(h * G, (h + 1) * G):
                if kv == 0:
                    out[rows, g], bound[rows, g] = 0, 0
                    continue
                x = q[rows, g]
                s = np.where(see, x @ k.T * scale, -np.inf)
                big = s.max(1, keepdims=True)
                p = np.where(see, np.exp(s - np.where(np.isinf(big), 0, big)), 0)
                total = p.sum(1, keepdims=True)
                safe = np.where(total == 0, 1, total)
                o = p @ v / safe
                u = 2.0 ** -24
                mag = np.abs(x) @ np.abs(k).T * scale
                ds = (3 * D + 8) * u * mag + 3 * u * np.where(see, np.where(np.isinf(big), 0, big) - np.where(see, s, 0), 0) + 2.0 ** -22
                ds = np.expm1(np.where(see, ds, 0))
                A = p @ np.abs(v) / safe
                e = (p * ds) @ np.abs(v) / safe + A * (p * ds).sum(1, keepdims=True) / safe
                e += A * ((2.0 ** -22 if f32 else 2.0 ** -11) + (2 * kv + 64) * u)
                e += 2.0 ** -34 * np.abs(v).sum(0) / safe + 2.0 ** -25 * top
                out[rows, g] = o
                bound[rows, g] = np.where(total == 0, 0, e + (u if f32 else 2.0 ** -8) * (np.abs(o) + e))
    return out, bound
