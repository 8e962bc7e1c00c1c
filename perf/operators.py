"""The operators of the 8-bit latent cache, in plain torch and through the framework, with the inputs they meet.

Three operators serve a paged cache of multi-head latent attention held in E4M3 with one power-of-two scale per page
of 64 tokens (all heads share the one latent):

plan    from every request's present and wanted length: the pages it gets from (or gives back to) a ring of free
        pages, its page table, and for every new token its slot and position.
append  the new tokens' latent entries, quantised into their pages. A page's scale is the smallest power of two 2^e
        (-60 <= e <= 60) with amax <= 448 * 2^e; a page that already holds tokens keeps the larger of its scale and
        the new rows', its old codes being rescaled and rounded to nearest even.
attend  softmax(scale * q k^T) v over a request's cached tokens: k = code * page scale (all elements), v = the first
        kv_lora of them. Query i of a request with n queries and length L sees tokens 0..L-1, or, causal,
        0..L-n+i. A query that sees nothing gives 0 and a log-sum-exp of -inf.

`own` is set from outside: False computes the plain form, True calls the framework.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
EMAX = 60                       # scale exponents are clamped to +-EMAX
FULL = {"kv_lora": 512, "d_rope": 64, "heads": 64}      # the full drafter geometry
TINY = {"kv_lora": 64, "d_rope": 16, "heads": 8}        # the tiny one
LATENTS = [(512, 64), (256, 32), (128, 32), (64, 16)]   # the latent widths of the framework


# --- cases -------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one request whose verification accepted a block: eight tokens, at most one new page
        {"name": "plan_bs1", "op": "plan", "bs": 1, "kind": "step", "len_lo": 4090, "len_hi": 4096, "lengths": 1},
        # one decode step of the paged batch: every request grows by one token
        {"name": "plan_bs32", "op": "plan", "bs": 32, "kind": "decode", "len_lo": 1024, "len_hi": 16384, "lengths": 2},
        # a busy server's step: accepted blocks, requests that end and give their pages back, prompts that arrive
        {"name": "plan_mixed_bs500", "op": "plan", "bs": 500, "kind": "mixed", "len_lo": 1, "len_hi": 8192, "lengths": 3},
        # prompts admitted at once: long slot maps
        {"name": "plan_prompts_bs64", "op": "plan", "bs": 64, "kind": "prompts", "len_lo": 1024, "len_hi": 8192,
         "lengths": 4},
        # every layer's entries of one accepted block (block + 1 tokens)
        {"name": "append_block_bs1", "op": "append", "kv_lora": 512, "d_rope": 64, "layers": 5, "bs": 1, "new_lo": 8,
         "new_hi": 8, "len_lo": 4090, "len_hi": 4096, "dtype": "bf16", "lengths": 5},
        # one decode step of the paged batch, every layer
        {"name": "append_decode_bs32", "op": "append", "kv_lora": 512, "d_rope": 64, "layers": 5, "bs": 32, "new_lo": 1,
         "new_hi": 1, "len_lo": 1024, "len_hi": 16384, "dtype": "bf16", "lengths": 6},
        # ragged prompts, one layer at a time as a prefill writes them
        {"name": "append_prompts_bs24", "op": "append", "kv_lora": 512, "d_rope": 64, "layers": 1, "bs": 24, "new_lo": 700,
         "new_hi": 8192, "len_lo": 0, "len_hi": 200, "dtype": "bf16", "lengths": 7},
        # the tiny geometry's step: latency
        {"name": "attend_tiny", "op": "attend", **TINY, "bs": 1, "q_lo": 7, "q_hi": 7, "len_lo": 128, "len_hi": 128,
         "causal": False, "lengths": 8},
        # the drafter's block at the benchmark's context
        {"name": "attend_block_ctx4096", "op": "attend", **FULL, "bs": 1, "q_lo": 7, "q_hi": 7, "len_lo": 4096,
         "len_hi": 4096, "causal": False, "lengths": 9},
        # the same at the long-context workload's length
        {"name": "attend_block_ctx95000", "op": "attend", **FULL, "bs": 1, "q_lo": 7, "q_hi": 7, "len_lo": 95000,
         "len_hi": 95000, "causal": False, "lengths": 10},
        # single-token decode of the paged batch
        {"name": "attend_decode_bs32", "op": "attend", **FULL, "bs": 32, "q_lo": 1, "q_hi": 1, "len_lo": 1024,
         "len_hi": 16384, "causal": True, "lengths": 11},
        # chunks of two prompts, causal, behind their cached prefixes
        {"name": "attend_chunk_bs2", "op": "attend", **FULL, "bs": 2, "q_lo": 700, "q_hi": 1024, "len_lo": 4000,
         "len_hi": 8192, "causal": True, "lengths": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 0.6)), math.log(hi)))))))


_LARGEST = {"plan": 600_000, "append": 60_000_000, "attend": 1.3e12}


def draw(rng):
    while True:
        op = rng.choice(["plan", "append", "attend", "attend"])
        seed = rng.randrange(1 << 20)
        if op == "plan":
            kind = rng.choice(["step", "decode", "mixed", "prompts"])
            hi = _log(rng, 8, 16384)
            c = {"op": op, "bs": _log(rng, 1, 512), "kind": kind, "len_lo": _log(rng, 1, hi), "len_hi": hi, "lengths": seed}
            if c["bs"] * hi <= _LARGEST[op] or kind in ("step", "decode") and c["bs"] * hi <= 8 * _LARGEST[op]:
                return c
        elif op == "append":
            kv, rope = rng.choice(LATENTS[:1] * 2 + LATENTS)
            hi = _log(rng, 1, 4096)
            lh = _log(rng, 1, 8192)
            c = {"op": op, "kv_lora": kv, "d_rope": rope, "layers": rng.choice([1, 2, 5]), "bs": _log(rng, 1, 64),
                 "new_lo": rng.choice([0, 1, max(1, hi // 2)]) if hi > 1 else 1, "new_hi": hi, "len_lo": rng.choice([0, lh // 2]),
                 "len_hi": lh, "dtype": rng.choice(["bf16", "bf16", "fp32"]), "lengths": seed}
            if c["layers"] * c["bs"] * hi * (kv + rope) <= _LARGEST[op]:
                return c
        else:
            kv, rope = rng.choice(LATENTS[:1] * 4 + LATENTS)
            causal = rng.random() < 0.5
            qhi = rng.choice([1, 1, 7, 8, _log(rng, 2, 40), _log(rng, 2, 600)])
            lh = _log(rng, 1, 40000)
            c = {"op": op, "kv_lora": kv, "d_rope": rope, "heads": rng.choice([64, 64, 64, 1, 5, 8, 12, 16, 40, 128]),
                 "bs": _log(rng, 1, 48), "q_lo": rng.choice([0, qhi, max(1, qhi // 2)]) if qhi > 1 else 1, "q_hi": qhi,
                 "len_lo": rng.choice([0, lh // 2, lh]), "len_hi": lh, "causal": causal, "lengths": seed}
            rows = c["bs"] * c["q_hi"] * c["heads"]
            if 2 * rows * lh * (2 * kv + rope) <= _LARGEST[op] and rows * lh <= 6e8 and c["bs"] * lh <= 600_000:
                return c


# --- lengths, which belong to the case ---------------------------------------------------------------------------
def _pages(n):
    return -(-n // PAGE)


def _lengths(case):
    """(present length, wanted length or queries) of every request, as the case has them."""
    rng = random.Random(case["lengths"])
    bs, lo, hi = case["bs"], case["len_lo"], case["len_hi"]
    length = [rng.randint(lo, hi) for _ in range(bs)]
    if case["op"] == "append":
        return length, [n + rng.randint(case["new_lo"], case["new_hi"]) for n in length]
    if case["op"] == "attend":
        return length, [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(bs)]
    kind, want = case["kind"], []
    for b in range(bs):
        if kind == "decode":
            want.append(length[b] + 1)
        elif kind == "step":
            want.append(length[b] + (8 if bs == 1 else rng.randint(1, 8)))
        elif kind == "prompts":
            want.append(length[b])
            length[b] = 0
        else:
            k = rng.random()
            if k < 0.1:                                   # a prompt arrives
                want.append(length[b])
                length[b] = 0
            elif k < 0.2:                                 # the request has ended
                want.append(0)
            elif k < 0.25:                                # its last tokens are taken back
                want.append(max(0, length[b] - rng.randint(1, 100)))
            else:
                want.append(length[b] + rng.randint(1, 8))
    return length, want


def _spans(case):
    """Of an append or a plan: new tokens and touched pages in all."""
    length, want = _lengths(case)
    new = sum(max(0, w - n) for n, w in zip(length, want))
    seg = sum(_pages(w) - n // PAGE for n, w in zip(length, want) if w > n)
    return new, seg


def work(case):
    first, second = _lengths(case)
    bs = case["bs"]
    if case["op"] == "plan":
        new, seg = _spans(case)
        get = sum(max(0, _pages(w) - _pages(n)) for n, w in zip(first, second))
        give = sum(max(0, _pages(n) - _pages(w)) for n, w in zip(first, second))
        # lengths in and out, running sums, the pages that move (read and written), slots and positions, page spans
        return {"bytes": 4 * (3 * bs + bs + 1) + 8 * (get + give) + 8 * new + 4 * seg + 16, "flops": 4 * new}
    if case["op"] == "append":
        new, seg = _spans(case)
        d, size = case["kv_lora"] + case["d_rope"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["layers"] * (new * d * (size + 1) + 4 * seg) + 4 * (new + seg), "flops": 3 * case["layers"] * new * d}
    kv, d, h = case["kv_lora"], case["kv_lora"] + case["d_rope"], case["heads"]
    nbytes, flops = 0, 0
    for n, q in zip(first, second):
        if q == 0:
            continue
        seen = sum(max(0, n - q + i + 1) for i in range(q)) if case["causal"] else q * n
        nbytes += n * d + 4 * _pages(n) + q * h * (2 * d + 2 * kv + 4)
        flops += 2 * seen * h * (d + kv)
    return {"bytes": max(nbytes, 1), "flops": max(flops, 1)}


# --- inputs ------------------------------------------------------------------------------------------------------
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cumulated(v):
    return [0] + [int(x) for x in np.cumsum(v)] if len(v) else [0]


def _cache(case, layers, held, spare, g):
    """Pages of quantised latents for `held` pages a request and `spare` more: codes, scales, page table."""
    d, kv = case["kv_lora"] + case["d_rope"], case["kv_lora"]
    n_pages, width = max(1, sum(held) + spare), max(1, max(held))
    codes = torch.empty(layers, n_pages, PAGE, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(layers, n_pages, dtype=torch.float32, device="cuda")
    for i in range(layers):
        # normalised latents and roped keys: unit normal, a page's scale the least that holds its largest
        for at in range(0, n_pages, 16384):
            x = torch.randn(min(16384, n_pages - at), PAGE, d, device="cuda", generator=g)
            e = _exponent(x.abs().amax((1, 2)))
            codes[i, at:at + 16384] = (x * _power(-e)[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            scales[i, at:at + 16384] = _power(e)
    order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros(case["bs"], width, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")[None]
    start = _ints(_cumulated(held)[:-1])[:, None]
    table = torch.where(at < _ints(held)[:, None], order[(start + at).clamp(max=n_pages - 1)], table).contiguous()
    return codes, scales, table, order


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    first, second = _lengths(case)
    bs = case["bs"]
    if case["op"] == "plan":
        new, seg = _spans(case)
        need = sum(max(0, _pages(w) - _pages(n)) for n, w in zip(first, second))
        held = [_pages(n) for n in first]
        width = max(1, max(max(_pages(w) for w in second), max(held)))
        n_pages = sum(held) + need + 64
        order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
        at = torch.arange(width, device="cuda")[None]
        start = _ints(_cumulated(held)[:-1])[:, None]
        table = torch.where(at < _ints(held)[:, None], order[(start + at).clamp(max=n_pages - 1)], 0).contiguous()
        head, count = seed % n_pages, n_pages - sum(held)
        ring = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        ring[(head + torch.arange(count, device="cuda")) % n_pages] = order[sum(held):]
        room, spans = new + 16, seg + 8
        empty = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"case": case, "length": _ints(first), "want": _ints(second), "table": table.to(torch.int32), "ring": ring,
                "ring_state": _ints([head, count]), "room": room, "spans": spans,
                "out": {"length": empty(bs), "ring_state": empty(2), "cu_new": empty(bs + 1), "slots": empty(room),
                        "positions": empty(room), "seg_row": empty(spans + 1)}}
    if case["op"] == "append":
        new, seg = _spans(case)
        held = [_pages(w) for w in second]
        codes, scales, table, _ = _cache(case, case["layers"], held, 3, g)
        host, slots, rows = table.cpu().numpy(), [], []
        for b, (n, w) in enumerate(zip(first, second)):
            pos = np.arange(n, w)
            rows += list(len(slots) + np.flatnonzero((pos % PAGE == 0) | (pos == n)))
            slots += list(host[b, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE)
        d = case["kv_lora"] + case["d_rope"]
        x = torch.randn(case["layers"], max(new, 1), d, device="cuda", generator=g)
        x = x * torch.exp2(torch.randint(-1, 3, (case["layers"], max(new, 1), 1), device="cuda", generator=g).float())
        return {"case": case, "codes": codes, "scales": scales, "table": table, "slots": _ints(slots or [-1]),
                "seg_row": _ints([int(r) for r in rows] + [new]), "new": new,
                "entries": x.to(torch.bfloat16) if case["dtype"] == "bf16" else x}
    held = [_pages(n) for n in first]
    codes, scales, table, _ = _cache(case, 1, held, 2, g)
    kv, d, h, total = case["kv_lora"], case["kv_lora"] + case["d_rope"], case["heads"], sum(second)
    # scores of a few units' spread, as trained heads have them; one head in eight looks at few tokens
    sharp = torch.where(torch.arange(h, device="cuda") % 8 == 3, 3.0, 1.0)[None, :, None]
    q = (torch.randn(max(total, 1), h, d, device="cuda", generator=g) * sharp).to(torch.bfloat16)
    return {"case": case, "codes": codes, "scales": scales, "table": table, "q": q[:total], "length": _ints(first),
            "cu_q": _ints(_cumulated(second)), "scale": 1.3 / math.sqrt(d), "longest": max(1, max(first)),
            "queries": max(1, max(second)), "o": torch.empty(total, h, kv, dtype=torch.bfloat16, device="cuda"),
            "lse": torch.empty(total, h, dtype=torch.float32, device="cuda")}


# --- one pass ----------------------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _run_own(state)
    return {"plan": _plan, "append": _append, "attend": _attend}[case["op"]](state)


def _own_cache(state):
    """The framework's view of this state's cache: pointers and a workspace, kept as a program keeps them."""
    import mla_block_diffusion_gb300 as M
    case = state["case"]
    if case["op"] == "plan":
        return M.QCache(512, 64, codes=(), scales=(), page_table=state["table"], n_pages=state["ring"].shape[0])
    return M.QCache(case["kv_lora"], case["d_rope"], codes=list(state["codes"]), scales=list(state["scales"]),
                    page_table=state["table"], n_heads=case.get("heads", 0))


def _run_own(state):
    case = state["case"]
    if "cache" not in state:
        state["cache"] = _own_cache(state)
    cache = state["cache"]
    if case["op"] == "plan":
        out = state["out"]
        cache.plan(state["length"], state["want"], state["ring"], state["ring_state"], out["length"], out["ring_state"],
                   out["cu_new"], out["slots"], out["positions"], out["seg_row"])
        return {**out, "table": state["table"], "ring": state["ring"]}
    if case["op"] == "append":
        cache.append(state["entries"], state["slots"], state["seg_row"])
        return {"codes": state["codes"].view(torch.float8_e4m3fn), "scales": state["scales"]}
    cache.attend(0, state["q"], state["cu_q"], state["length"], state["o"], state["lse"], causal=case["causal"],
                 scale=state["scale"])
    return {"o": state["o"], "lse": state["lse"]}


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, clamped; exact (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, e, -EMAX).clamp(-EMAX, EMAX)


def _power(e):
    """2^e in 32 bits, from its exponent field."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _plan(state):
    length, want, table, ring = state["length"].long(), state["want"].long(), state["table"], state["ring"]
    n_pages, width, room, spans = ring.shape[0], table.shape[1], state["room"], state["spans"]
    head, count = state["ring_state"][0].long(), state["ring_state"][1].long()
    dev = ring.device
    held, hold = (length + PAGE - 1) // PAGE, (want + PAGE - 1) // PAGE
    fits = (want >= 0) & (want <= width * PAGE)
    up = fits & (want > length)
    zero = torch.zeros_like(length)
    need, new = torch.where(up, hold - held, zero), torch.where(up, want - length, zero)
    got = up & (need.cumsum(0) <= count) & (new.cumsum(0) <= room)
    need, new = torch.where(got, need, zero), torch.where(got, new, zero)
    down = fits & (want < length)
    give = torch.where(down, held - hold, zero)
    out_length = torch.where(got | (fits & ~up), want, length)
    pad = zero[:1]
    cu_need, cu_new, cu_give = (torch.cat([pad, v.cumsum(0)]) for v in (need, new, give))
    # the pages that requests get, and those that they give back
    at = torch.arange(width, device=dev)[None]
    k = at - held[:, None]
    page = ring[(head + cu_need[:-1, None] + k.clamp(min=0)) % n_pages]
    filled = torch.where((k >= 0) & (k < need[:, None]), page, table)
    k = at - hold[:, None]
    back = (k >= 0) & (k < give[:, None])
    place = torch.where(back, (head + count + cu_give[:-1, None] + k) % n_pages, n_pages)
    ring.copy_(torch.cat([ring, ring[:1]]).scatter(0, place.reshape(-1), table.reshape(-1))[:n_pages])
    table.copy_(filled)
    # the tokens' slots and positions, and the first row of every page that new tokens touch
    total = cu_new[-1]
    i = torch.arange(room, device=dev)
    b = torch.searchsorted(cu_new[1:], i, right=True).clamp(max=length.shape[0] - 1)
    live = i < total
    pos = length[b] + i - cu_new[b]
    slot = filled[b, (pos // PAGE).clamp(0, width - 1)].long() * PAGE + pos % PAGE
    first = length // PAGE
    cu_seg = torch.cat([pad, torch.where(got, hold - first, zero).cumsum(0)])
    s = torch.arange(spans + 1, device=dev)
    b = torch.searchsorted(cu_seg[1:], s, right=True).clamp(max=length.shape[0] - 1)
    k = s - cu_seg[b]
    row = cu_new[b] + torch.where(k == 0, torch.zeros_like(k), (first[b] + k) * PAGE - length[b])
    row = torch.where(s < cu_seg[-1], row, total)
    taken = cu_need[-1]
    after = torch.stack([(head + taken) % n_pages, count - taken + cu_give[-1]])
    whole = lambda v: v.to(torch.int32)  # noqa: E731
    return {"length": whole(out_length), "ring_state": whole(after), "cu_new": whole(cu_new),
            "slots": whole(torch.where(live, slot, -1)), "positions": whole(torch.where(live, pos, -1)),
            "seg_row": whole(row), "table": table, "ring": ring}


def _append(state):
    codes, scales, n = state["codes"], state["scales"], state["new"]
    if n:
        layers, _, _, d = codes.shape
        x, slots, rows = state["entries"][:, :n].float(), state["slots"][:n].long(), state["seg_row"].long()
        pages = slots[rows[:-1]] // PAGE                              # of every touched page
        old = slots[rows[:-1]] % PAGE                                 # tokens that it holds already
        span = torch.searchsorted(rows[1:], torch.arange(n, device=x.device), right=True)
        amax = torch.zeros(layers, pages.shape[0], device=x.device)
        amax = amax.scatter_reduce(1, span[None].expand(layers, n), x.abs().amax(2), "amax")
        _, e_old = torch.frexp(scales[:, pages])
        e = torch.maximum(_exponent(amax), torch.where(old > 0, e_old - 1, -EMAX))
        held = codes[:, pages].view(torch.float8_e4m3fn).float()
        kept = (held * _power(e_old - 1 - e)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        keep = (torch.arange(PAGE, device=x.device) < old[:, None])[None, :, :, None]
        codes[:, pages] = torch.where(keep, kept, codes[:, pages])
        fresh = (x * _power(-e)[:, span][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes.view(layers, -1, d)[:, slots] = fresh
        scales[:, pages] = _power(e)
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}


def _attend(state):
    case, q, cu, length = state["case"], state["q"], state["cu_q"].long(), state["length"].long()
    kv, d, h, bs, most, dev = case["kv_lora"], q.shape[2], q.shape[1], length.shape[0], state["queries"], q.device
    pages = state["table"][:, :_pages(state["longest"])].long()
    k = state["codes"][0][pages].view(torch.float8_e4m3fn).float() * state["scales"][0][pages][:, :, None, None]
    k = k.reshape(bs, -1, d)
    i = torch.arange(most, device=dev)[None]
    n = (cu[1:] - cu[:-1])[:, None]
    live = i < n
    sees = torch.where(live, (length[:, None] - n + i + 1).clamp(min=0) if case["causal"] else length[:, None], 0)
    at = (cu[:-1, None] + i).clamp(max=max(0, q.shape[0] - 1))
    x = q[at].float().reshape(bs, most * h, d) if q.shape[0] else torch.zeros(bs, most * h, d, device=dev)
    s = torch.matmul(x, k.transpose(1, 2)).mul_(state["scale"]).reshape(bs, most, h, -1)
    s = s.masked_fill_((torch.arange(k.shape[1], device=dev) >= sees[:, :, None])[:, :, None], float("-inf"))
    top = s.amax(3, keepdim=True)
    base = torch.where(top == float("-inf"), 0.0, top)
    p = s.sub_(base).exp_()
    total = p.sum(3)
    o = torch.matmul(p.reshape(bs, most * h, -1), k[:, :, :kv]).reshape(bs, most, h, kv)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    lse = base[..., 0] + torch.log(total)
    token = torch.arange(q.shape[0], device=dev)
    b = torch.searchsorted(cu[1:], token, right=True)
    return {"o": o[b, token - cu[b]].to(torch.bfloat16), "lse": lse[b, token - cu[b]]}


# --- the definition in 64 bits -----------------------------------------------------------------------------------
def _e4m3():
    """The value of each of the 256 codes: sign, 4 exponent bits of bias 7, 3 fraction bits; 0x7f and 0xff are NaN."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e.astype(np.float64) - 7))
    v = np.where(c >= 128, -v, v)
    v[(c & 127) == 127] = np.nan
    return v


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "plan":
        return None
    value = torch.from_numpy(_e4m3()).cuda()
    if case["op"] == "append":
        if state["codes"].numel() > 1_200_000_000:
            return None
        held = torch.stack([value[c.int()] for c in state["codes"]])
        scales, entries = state["scales"].double().cpu(), state["entries"].double()
        slots, rows = state["slots"].tolist(), state["seg_row"].tolist()
        steps = torch.tensor([2.0 ** (k - 9) for k in range(15)], dtype=torch.float64, device="cuda")

        def rounded(x):
            """To the nearest E4M3 value, halves to the even one."""
            step = steps[(torch.frexp(x)[1] - 1).clamp(min=-6, max=8) + 6]
            return torch.round(x / step) * step
        for layer in range(held.shape[0]):
            tops = entries[layer].abs().amax(1).tolist()
            for a, z in zip(rows[:-1], rows[1:]):
                page, at = divmod(slots[a], PAGE)
                scale, before = 2.0 ** -EMAX, float(scales[layer, page])
                while max(tops[a:z]) > 448 * scale and scale < 2.0 ** EMAX:
                    scale *= 2
                if at:
                    scale = max(scale, before)
                    held[layer, page, :at] = rounded(held[layer, page, :at] * (before / scale))
                held[layer, page, at:at + z - a] = rounded(entries[layer, a:z] / scale)
                scales[layer, page] = scale
        return {"codes": held, "scales": scales}
    kv, h = case["kv_lora"], case["heads"]
    first, second = _lengths(case)
    if sum(n * q for n, q in zip(first, second)) * h > 2e9:
        return None
    cu = _cumulated(second)
    o = torch.zeros(cu[-1], h, kv, dtype=torch.float64, device="cuda")
    lse = torch.full((cu[-1], h), -math.inf, dtype=torch.float64, device="cuda")
    table = state["table"].cpu()
    for b, (n, count) in enumerate(zip(first, second)):
        keys = [value[state["codes"][0, p].long()] * state["scales"][0, p].double() for p in table[b, :_pages(n)].tolist()]
        if not keys:
            continue
        keys = torch.cat(keys)[:n]
        block = max(1, 100_000_000 // (h * n))                 # queries at a time
        for i in range(0, count, block):
            j = min(count, i + block)
            query = state["q"][cu[b] + i:cu[b] + j].double()
            score = torch.einsum("ihd,kd->ihk", query, keys) * state["scale"]
            if case["causal"]:
                last = n - count + torch.arange(i, j, device="cuda")
                score[(torch.arange(n, device="cuda")[None] > last[:, None])[:, None].expand_as(score)] = -math.inf
            lse[cu[b] + i:cu[b] + j] = torch.logsumexp(score, 2)
            weight = torch.softmax(score, 2).nan_to_num(0.0)
            o[cu[b] + i:cu[b] + j] = torch.einsum("ihk,kd->ihd", weight, keys[:, :kv])
    return {"o": o, "lse": lse}
