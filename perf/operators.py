"""Cases of the paged 8-bit KV cache: planning pages, appending tokens, attending.

A request's keys and values live in pages of `page` tokens.  Per page and head
the cache holds E4M3 codes and one power-of-two scale (E8M0 byte X + 127, value
code * 2^X): keys as [pages, heads, page, dim], values transposed inside their
page as [pages, heads, dim, page].  A block table names each request's pages.

  plan    from cached and new lengths: pages from a free list into the block
          table, a slot (page * size + offset) per new token, row offsets and
          lengths of the requests
  append  quantizes new tokens into their slots and keeps each page's scale
  attend  softmax(scale q k^T + mask) v of every new token over its request's
          pages: single tokens, prompts, chunks, and (not causal) queries of
          their own length over an encoder's states
"""
import math

import torch

own = False

PAGE_SCALE_MIN = 1e-12
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 running requests: a token each
        dict(name="plan_step_b64", op="plan", batch=64, q_lo=1, q_hi=1, long=0, ctx_lo=17,
             ctx_hi=8000, page=64),
        # admission: prompts join running requests, odd lengths and small pages
        dict(name="plan_mixed_b777", op="plan", batch=777, q_lo=1, q_hi=1900, long=37, ctx_lo=0,
             ctx_hi=6001, page=16),
        # the token of each of 64 requests, Llama-3.1-8B heads
        dict(name="append_step_b64_bf16", op="append", batch=64, q_lo=1, q_hi=1, long=0,
             ctx_lo=17, ctx_hi=300, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # prompts of one prefill batch
        dict(name="append_prompt_bf16", op="append", batch=4, q_lo=2048, q_hi=8192, long=4,
             ctx_lo=0, ctx_hi=0, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # odd chunks on top of partly filled small pages, float32, 64-wide heads
        dict(name="append_chunk_f32", op="append", batch=13, q_lo=3, q_hi=301, long=5,
             ctx_lo=5, ctx_hi=177, kv_heads=4, dim=64, page=16, dtype="f32"),
        # the smallest call: one token of a young conversation
        dict(name="attend_one_bf16", op="attend", batch=1, q_lo=1, q_hi=1, long=0, ctx_lo=290,
             ctx_hi=290, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16", causal=True),
        # a decode step of 64 ragged requests, Llama-3.1-8B heads
        dict(name="attend_step_b64_bf16", op="attend", batch=64, q_lo=1, q_hi=1, long=0,
             ctx_lo=200, ctx_hi=8191, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
             causal=True),
        # one long document, 32768 cached tokens, 16 query heads over 8
        dict(name="attend_long_bf16", op="attend", batch=1, q_lo=1, q_hi=1, long=0, ctx_lo=32767,
             ctx_hi=32767, heads=16, kv_heads=8, dim=128, page=128, dtype="bf16", causal=True),
        # float32 queries, a few tokens each, 64-wide heads, small pages
        dict(name="attend_few_f32", op="attend", batch=9, q_lo=1, q_hi=5, long=4, ctx_lo=0,
             ctx_hi=1999, heads=12, kv_heads=4, dim=64, page=16, dtype="f32", causal=True),
        # two whole prompts
        dict(name="attend_prompt_bf16", op="attend", batch=2, q_lo=4096, q_hi=4096, long=2,
             ctx_lo=0, ctx_hi=0, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
             causal=True),
        # a 512-token chunk of two prompts beside 14 decoding requests
        dict(name="attend_chunk_mixed_bf16", op="attend", batch=16, q_lo=1, q_hi=512, long=2,
             ctx_lo=1001, ctx_hi=7600, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
             causal=True),
        # a decoder's tokens over an encoder's 1500 states, every head its own keys
        dict(name="attend_cross_bf16", op="attend", batch=8, q_lo=1, q_hi=224, long=6,
             ctx_lo=1500, ctx_hi=1500, heads=20, kv_heads=20, dim=64, page=32, dtype="bf16",
             causal=False),
    ]


def _between(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        batch = _between(rng, 1, 1500)
        return dict(op=op, batch=batch, q_lo=1, q_hi=_between(rng, 1, 2000),
                    long=rng.randint(0, min(batch, 35)), ctx_lo=rng.randint(0, 50),
                    ctx_hi=_between(rng, 51, 9000), page=page)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dim = rng.choice([64, 128, 128, 256])
    if op == "append":
        batch = _between(rng, 1, 96)
        q_hi = _between(rng, 1, max(1, 6000 // batch))
        return dict(op=op, batch=batch, q_lo=rng.randint(1, q_hi), q_hi=q_hi,
                    long=rng.randint(0, batch), ctx_lo=0, ctx_hi=_between(rng, 1, 400),
                    kv_heads=rng.choice([1, 2, 4, 8]), dim=dim, page=page, dtype=dtype)
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 8] if kv_heads < 8 else [1, 2, 4])
    causal = rng.random() < 0.75
    if rng.random() < 0.6:      # single tokens, or a few
        batch = _between(rng, 1, 96)
        ctx_hi = _between(rng, 1, max(2, min(32768, 250000 // batch)))
        q_hi = rng.choice([1, 1, 1, 2, 5])
        long = rng.randint(0, batch)
    else:                       # prompts and chunks
        batch = _between(rng, 1, 4)
        ctx_hi = _between(rng, 1, 2000)
        q_hi = _between(rng, 16, 1100 if dtype == "bf16" and dim < 256 else 700)
        long = rng.randint(1, batch)
    return dict(op=op, batch=batch, q_lo=1, q_hi=q_hi, long=long, ctx_lo=rng.randint(0, ctx_hi),
                ctx_hi=ctx_hi, heads=heads, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype,
                causal=causal)


def lengths(case):
    """(new tokens, cached tokens) of each request: `long` of them, spread over
    the batch, have q_hi new tokens (the last of several q_hi down to q_lo), the
    others q_lo; cached lengths spread over [ctx_lo, ctx_hi]."""
    b = case["batch"]
    new, ctx, seen = [], [], 0
    for i in range(b):
        is_long = (i + 1) * case["long"] // b > seen
        if is_long:
            seen += 1
        spread = (i * 0.6180339887498949 + 0.5) % 1.0
        n = case["q_lo"]
        if is_long:
            n = case["q_hi"] - int((case["q_hi"] - case["q_lo"]) * (seen - 1) // (2 * case["long"]))
        new.append(n)
        ctx.append(case["ctx_lo"] + int(spread * (case["ctx_hi"] - case["ctx_lo"] + 1)))
    return new, ctx


def _kv_lengths(case):
    new, ctx = lengths(case)
    return [c + n for c, n in zip(ctx, new)] if case.get("causal", True) else ctx


def work(case):
    new, ctx = lengths(case)
    total, page = sum(new), case["page"]
    if case["op"] == "plan":
        pages = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
        return {"bytes": 4 * (2 * case["batch"] + total + 2 * case["batch"] + 1 + 2 * pages),
                "flops": 0}
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        row = case["kv_heads"] * case["dim"]
        touched = sum(-(-(c + n) // page) - c // page for c, n in zip(ctx, new))
        return {"bytes": 2 * total * row * (es + 1) + 4 * total + 2 * touched * case["kv_heads"],
                "flops": 0}
    pairs = kv_tokens = 0
    for n, kv in zip(new, _kv_lengths(case)):
        kv_tokens += kv
        pairs += n * kv - (n * (n - 1) // 2 if case["causal"] else 0)
    return {"bytes": 2 * kv_tokens * case["kv_heads"] * case["dim"]
            + 2 * total * case["heads"] * case["dim"] * es,
            "flops": 4 * case["dim"] * case["heads"] * pairs}


# ---------------------------------------------------------------------------
# what a serving program has in hand
# ---------------------------------------------------------------------------

def _device():
    return torch.device("cuda")


def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _table(counts, width, order):
    """Block table [batch, width] with `counts[b]` pages of `order` in turn, 0 behind them."""
    rows, at = [], 0
    for n in counts:
        rows.append(order[at:at + n] + [0] * (width - n))
        at += n
    return rows


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)
    new, ctx = lengths(case)
    batch, page, total = case["batch"], case["page"], sum(new)
    kv = _kv_lengths(case)
    held = [-(-c // page) for c in ctx]
    final = [-(-n // page) for n in kv]
    if case["op"] == "plan":
        ahead = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        width = max(ahead) + 3
        pages = sum(ahead) + 11
        order = torch.randperm(pages, generator=g, device=dev).tolist()
        free = order[sum(held):]
        return dict(case=case, cached=_ints(ctx, dev), new=_ints(new, dev),
                    table=_ints(_table(held, width, order), dev), free=_ints(free, dev),
                    used=_ints([0], dev), max_new=total + 5)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    heads, dim = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        final = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    pages = sum(final) + 2
    order = torch.randperm(pages, generator=g, device=dev).tolist()
    table = _table(final, max(max(final), 1), order)
    shape = (pages, heads, page, dim)
    # cached values: codes of normal values, each page and head with a scale of its own
    k = (torch.randn(shape, generator=g, device=dev) * 60).to(E4M3)
    v = (torch.randn(shape, generator=g, device=dev) * 60).to(E4M3).transpose(2, 3)
    state = dict(
        case=case, k_codes=k.view(torch.uint8), v_codes=v.contiguous().view(torch.uint8),
        k_scales=torch.randint(119, 122, (pages, heads), generator=g, device=dev,
                               dtype=torch.uint8),
        v_scales=torch.randint(119, 122, (pages, heads), generator=g, device=dev,
                               dtype=torch.uint8),
        table=_ints(table, dev))
    if case["op"] == "append":
        slots = [row[(c + i) // page] * page + (c + i) % page
                 for row, c, n in zip(table, ctx, new) for i in range(n)]
        # keys with a constant bias per channel and a little noise, normal values
        bias = torch.randn((heads, dim), generator=g, device=dev) * 2
        kx = bias + torch.randn((total, heads, dim), generator=g, device=dev) * 0.5
        vx = torch.randn((total, heads, dim), generator=g, device=dev)
        state.update(k=kx.to(dtype), v=vx.to(dtype), slots=_ints(slots, dev))
    else:
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        q = torch.randn((total, case["heads"], dim), generator=g, device=dev) * 1.5
        state.update(q=q.to(dtype), starts=_ints(starts, dev), kv=_ints(kv, dev),
                     max_q=max(new), max_kv=max(kv))
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op == "plan":
        return _run_plan(state)
    return _run_append(state) if op == "append" else _run_attend(state)


def _run_plan(s):
    if own:
        import precision_quantization_block_amd as pqb
        p = pqb.kv_plan_paged(s["cached"], s["new"], s["table"], s["free"], s["used"],
                              s["case"]["page"], s["max_new"])
        return dict(table=s["table"], slots=p.slots, starts=p.q_starts, kv=p.kv_lens,
                    used=p.free_used)
    page = s["case"]["page"]
    c, n, table = s["cached"].long(), s["new"].long(), s["table"].clone()
    held, final = (c + page - 1) // page, (c + n + page - 1) // page
    starts = torch.zeros(c.numel() + 1, dtype=torch.int64, device=c.device)
    starts[1:] = n.cumsum(0)
    rank = (final - held).cumsum(0) - (final - held) - held
    col = torch.arange(table.shape[1], device=c.device)
    takes = (col >= held[:, None]) & (col < final[:, None])
    at = (s["used"].long() + rank[:, None] + col).clamp(0, s["free"].numel() - 1)
    table = torch.where(takes, s["free"][at], table)
    t = torch.arange(s["max_new"], device=c.device)
    b = torch.searchsorted(starts[1:], t, right=True).clamp(max=c.numel() - 1)
    pos = c[b] + t - starts[b]
    slot = table[b, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    slots = torch.where(t < starts[-1], slot, -1)
    return dict(table=table, slots=slots.int(), starts=starts.int(), kv=(c + n).int(),
                used=(s["used"].long() + (final - held).sum()).int())


def _pow2(x):
    """2^x of whole x in [-126, 127], by its float32 exponent."""
    return ((x.to(torch.int32) + 127) << 23).view(torch.float32)


def _run_append(s):
    if own:
        import precision_quantization_block_amd as pqb
        cache = pqb.PagedKV(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        pqb.kv_append_paged(s["k"], s["v"], s["slots"], cache)
        codes = (s["k_codes"], s["v_codes"])
        scales = (s["k_scales"], s["v_scales"])
    else:
        kc, ks = _plain_append(s["k"], s["slots"], s["k_codes"], s["k_scales"])
        vc, vs = _plain_append(s["v"], s["slots"], s["v_codes"].transpose(2, 3), s["v_scales"])
        codes, scales = (kc, vc.transpose(2, 3).contiguous()), (ks, vs)
    return dict(k=codes[0].view(E4M3), v=codes[1].view(E4M3), k_scales=scales[0],
                v_scales=scales[1])


def _plain_append(x, slots, codes, scales):
    """Codes [pages, heads, page, dim] and scales after the call."""
    pages, heads, page, dim = codes.shape
    x, at, off = x.float(), slots.long() // page, slots.long() % page
    amax = x.abs().amax(2)
    most = torch.zeros((pages, heads), device=x.device)
    most = most.scatter_reduce(0, at[:, None].expand(-1, heads), amax, "amax")
    first = torch.full((pages,), page, device=x.device)
    first = first.scatter_reduce(0, at, off, "amin")
    bits = most.clamp(min=PAGE_SCALE_MIN).view(torch.int32)
    need = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    old = scales.int() - 127
    touched, fresh = (first < page)[:, None], (first == 0)[:, None]
    exp = torch.where(touched, torch.where(fresh, need, torch.maximum(need, old)), old)
    held = codes.view(E4M3).float() * _pow2((old - exp).clamp(-20, 0))[:, :, None, None]
    before = torch.arange(page, device=x.device) < torch.where(first < page, first, 0)[:, None]
    again = before[:, None, :, None] & (exp > old)[:, :, None, None]
    out = torch.where(again, held.to(E4M3).view(torch.uint8), codes)
    new = (x * _pow2(-exp)[at][:, :, None]).to(E4M3).view(torch.uint8)
    out[at, :, off] = new
    return out, (exp + 127).to(torch.uint8)


def _run_attend(s):
    case = s["case"]
    if own:
        import precision_quantization_block_amd as pqb
        cache = pqb.PagedKV(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        return pqb.kv_attend_paged(s["q"], cache, s["table"], s["starts"], s["kv"],
                                   causal=case["causal"], max_q_len=s["max_q"])
    q, starts, kv = s["q"], s["starts"].long(), s["kv"].long()
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    batch, group = case["batch"], case["heads"] // case["kv_heads"]
    m, width = s["max_q"], -(-max(s["max_kv"], 1) // page)
    table = s["table"][:, :width].long()
    span = width * page
    j = torch.arange(span, device=q.device)
    i = torch.arange(m, device=q.device)
    n = starts[1:] - starts[:-1]
    k = s["k_codes"].view(E4M3)[table].float() * _pow2(s["k_scales"].int() - 127)[table][..., None, None]
    k = k.permute(0, 2, 1, 3, 4).reshape(batch, heads, span, dim)
    v = s["v_codes"].view(E4M3)[table].float() * _pow2(s["v_scales"].int() - 127)[table][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(batch, heads, span, dim)
    rows = (starts[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = q[rows].float().reshape(batch, m, heads, group, dim).permute(0, 2, 3, 1, 4)
    x = x.reshape(batch, heads, group * m, dim)
    p = torch.matmul(x, k.transpose(2, 3)) * (1.0 / math.sqrt(dim))
    limit = kv[:, None].expand(-1, m)
    if case["causal"]:
        limit = torch.minimum(limit, kv[:, None] - n[:, None] + i + 1)
    seen = (j < limit[:, :, None])[:, None, None]
    p = p.reshape(batch, heads, group, m, span).masked_fill(~seen, float("-inf"))
    top = p.amax(4, keepdim=True)
    p = torch.exp(p - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(4, keepdim=True)
    o = torch.matmul(p.reshape(batch, heads, group * m, span), v).reshape(batch, heads, group, m, dim)
    o = o / torch.where(total == 0, 1.0, total)
    t = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(starts[1:], t, right=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, m, heads * group, dim)
    return o[b, t - starts[b]].to(q.dtype)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                 # whole numbers only
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_attend(s)


def _grid64(y):
    """The nearest E4M3 values of y (|y| <= 448), ties to the even one, in 64 bits."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _exact_append(s):
    case, out = s["case"], {}
    page, slots = case["page"], s["slots"].tolist()
    runs, at = [], 0                # (first token, tokens): one page each
    for t in range(1, len(slots) + 1):
        if t == len(slots) or slots[t] != slots[t - 1] + 1 or slots[t] % page == 0:
            runs.append((at, t - at))
            at = t
    if len(runs) * case["kv_heads"] > 20000:
        return None
    for name in "kv":
        held = s[name + "_codes"].view(E4M3).double()
        held = held.transpose(2, 3).clone() if name == "v" else held.clone()
        x, scales = s[name].double(), s[name + "_scales"]
        for t, n in runs:
            p, o = slots[t] // page, slots[t] % page
            amax = x[t:t + n].abs().amax((0, 2)).clamp(min=PAGE_SCALE_MIN)
            need = torch.ceil(torch.log2(amax / 448.0))
            old = scales[p].double() - 127
            exp = need if o == 0 else torch.maximum(need, old)
            if o:
                grown = _grid64(held[p, :, :o] * torch.exp2(old - exp)[:, None, None])
                held[p, :, :o] = torch.where((exp > old)[:, None, None], grown, held[p, :, :o])
            held[p, :, o:o + n] = _grid64(x[t:t + n].transpose(0, 1) * torch.exp2(-exp)[:, None, None])
        out[name] = held if name == "k" else held.transpose(2, 3).contiguous()
    return dict(k=out["k"], v=out["v"], k_scales=None, v_scales=None)


def _exact_attend(s):
    case, q = s["case"], s["q"].double()
    page, group = case["page"], case["heads"] // case["kv_heads"]
    starts, kv, out = s["starts"].tolist(), s["kv"].tolist(), torch.zeros_like(q)
    for b in range(case["batch"]):
        n, length = starts[b + 1] - starts[b], kv[b]
        if n == 0 or length == 0:
            continue
        ids = s["table"][b, :-(-length // page)].long()
        for h in range(case["kv_heads"]):
            k = s["k_codes"][ids, h].view(E4M3).double()
            k = (k * torch.exp2(s["k_scales"][ids, h].double() - 127)[:, None, None]).flatten(0, 1)
            v = s["v_codes"][ids, h].view(E4M3).double().transpose(1, 2)
            v = (v * torch.exp2(s["v_scales"][ids, h].double() - 127)[:, None, None]).flatten(0, 1)
            k, v = k[:length], v[:length]
            for g in range(h * group, (h + 1) * group):
                z = q[starts[b]:starts[b + 1], g] @ k.T / math.sqrt(case["dim"])
                if case["causal"]:
                    row = torch.arange(n, device=q.device)[:, None] + (length - n)
                    z = z.masked_fill(torch.arange(length, device=q.device) > row, float("-inf"))
                out[starts[b]:starts[b + 1], g] = torch.softmax(z, 1) @ v
    return out
