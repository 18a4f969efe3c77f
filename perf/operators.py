"""The serving operators over a paged key-value cache, and rotary positions:
what is measured of them, and their plain forms.

Four operators, named in a case's ``"op"``:

* ``decode``  attention of one new token per request over a paged cache
* ``append``  rotary positions of a step's q and k, and k, v written to their pages
* ``rotary``  rotary positions of one tensor, with the gradient
* ``maps``    block tables and slot maps from request lengths

Caches are indexed ``[block, token of the page, head, d]``; ``heads_first``
cases hold them as ``[block, head, token, d]`` in memory (a permuted view).
Lengths follow from the case alone and the seed shuffles them, so that
``work`` is exact.
"""
import math
import random

import torch

own = False

_E4M3_MAX = 448.0


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly spread."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _decode(name, B, hq, hkv, d, page, lo, hi, cache="bf16", heads_first=False, empty=0):
    return {"op": "decode", "B": B, "hq": hq, "hkv": hkv, "d": d, "page": page, "lo": lo, "hi": hi, "cache": cache,
            "heads_first": heads_first, "empty": empty} | ({"name": name} if name else {})


def _append(name, T, hq, hkv, d, page, r, cache="bf16", interleaved=False, heads_first=False, pad=0, k_out=False):
    return {"op": "append", "T": T, "hq": hq, "hkv": hkv, "d": d, "page": page, "r": r, "cache": cache,
            "interleaved": interleaved, "heads_first": heads_first, "pad": pad, "k_out": k_out} | (
                {"name": name} if name else {})


def _rotary(name, B, H, N, d, r, interleaved=False, factor=1.0):
    return {"op": "rotary", "B": B, "H": H, "N": N, "d": d, "r": r, "interleaved": interleaved, "factor": factor} | (
        {"name": name} if name else {})


def _maps(name, B, page, ctx_lo, ctx_hi, new_lo, new_hi, width, pad=0):
    return {"op": "maps", "B": B, "page": page, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "new_lo": new_lo,
            "new_hi": new_hi, "width": width, "pad": pad} | ({"name": name} if name else {})


def listed():
    return [
        # one user's chat turn: a few small launches, where latency is all
        _decode("decode_one", 1, 32, 8, 128, 16, 1000, 1000),
        # a small d = 64 model, one key head per query head, ragged and short, odd lengths
        _decode("decode_short_d64", 9, 12, 12, 64, 16, 1, 2001),
        # a serving batch with grouped heads, ragged lengths, padded up to its graph's size
        _decode("decode_batch", 64, 32, 8, 128, 16, 300, 8192, empty=3),
        # this repository's long decode: 2 sequences of 65536 keys, 32 heads each
        _decode("decode_long", 2, 32, 32, 128, 64, 65536, 65536),
        # a large batch whose cache is held in 8 bits, pages stored head by head
        _decode("decode_e4m3", 128, 64, 8, 128, 64, 777, 8190, cache="e4m3", heads_first=True),
        # the step before decode_batch: one new token per request, padded rows
        _append("append_step", 64, 32, 8, 128, 16, 128, pad=3),
        # a batch of prompts, rotated keys wanted for the prefill attention too
        _append("append_prompts", 16411, 32, 8, 128, 16, 128, k_out=True),
        # prompts into an 8-bit cache, interleaved pairs on half of the head
        _append("append_e4m3", 20000, 64, 8, 128, 64, 64, cache="e4m3", interleaved=True, heads_first=True, pad=100),
        # this repository's ragged training shape, part of the head, interleaved
        _rotary("rotary_ragged", 2, 4, 1000, 64, 32, interleaved=True),
        # this repository's prefill shape, forward and gradient, scaled for long contexts
        _rotary("rotary_prefill", 4, 32, 4096, 128, 128, factor=1.1),
        # one new token for each of 256 requests
        _maps("maps_step", 256, 16, 1, 8191, 1, 1, 513),
        # prompts and running requests in one step (chunked prefill)
        _maps("maps_prompts", 60, 16, 0, 4000, 1, 4096, 600, pad=77),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "rotary", "maps"])
    if op == "decode":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 5, 8, 12, 32])
        hq = hkv * (rng.choice([1, 1, 2]) if hkv >= 12 else rng.choice([1, 2, 3, 4, 7, 8, 16]))
        B = _log(rng, 1, 128)
        room = 128 * 8192 * 8 * 128 // (B * hkv * d)  # keys per request that cost no more than the largest case's
        hi = _log(rng, 1, max(1, min(65536, room // 2)))
        lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
        return _decode(None, B, hq, hkv, d, rng.choice([16, 32, 64, 128]), lo, hi, rng.choice(["bf16", "bf16", "e4m3"]),
                       rng.random() < 0.4, empty=rng.randint(0, max(0, B - 1) // 8))
    if op == "append":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 5, 8, 12])
        T = _log(rng, 1, 16000)
        return _append(None, T, hkv * rng.choice([1, 3, 4, 5]), hkv, d, rng.choice([16, 32, 64, 128]),
                       rng.choice([d, d, d // 2, d // 4]), rng.choice(["bf16", "bf16", "e4m3"]), rng.random() < 0.5,
                       rng.random() < 0.4, rng.randint(0, (T - 1) // 10), rng.random() < 0.5)
    if op == "rotary":
        d = rng.choice([64, 128])
        return _rotary(None, rng.randint(1, 4), rng.choice([1, 3, 4, 8, 16, 32]), _log(rng, 1, 4096), d,
                       rng.choice([d, d, d // 2, d // 4]), rng.random() < 0.5, rng.choice([1.0, 1.0, 1.1, 1.25]))
    page = rng.choice([16, 32, 64, 128])
    ctx, new = _log(rng, 1, 8192), rng.choice([1, _log(rng, 1, 2048)])
    return _maps(None, _log(rng, 1, 256), page, rng.choice([0, 1, ctx // 2]), ctx, rng.randint(0, 1), new,
                 (ctx + new) // page + 1 + rng.randint(0, 9), pad=rng.randint(0, 64))


def _lens(case):
    return [0] * case["empty"] + _spread(case["B"] - case["empty"], case["lo"], case["hi"])


def _shuffled(values, seed):
    values = list(values)
    random.Random(seed).shuffle(values)
    return values


def _int(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _cache(blocks, case, dev):
    """An uninitialised cache, indexed [block, token, head, d] whatever its order in memory."""
    t = torch.float8_e4m3fn if case["cache"] == "e4m3" else torch.bfloat16
    if case["heads_first"]:
        return torch.empty(blocks, case["hkv"], case["page"], case["d"], dtype=t, device=dev).permute(0, 2, 1, 3)
    return torch.empty(blocks, case["page"], case["hkv"], case["d"], dtype=t, device=dev)


def _fill(cache, g, scale):
    """Normal values in units of the head's scale, a block range at a time."""
    step = max(1, (1 << 26) // max(1, cache[0].numel()))
    for at in range(0, cache.shape[0], step):
        part = cache[at:at + step]
        x = torch.randn(part.shape, generator=g, device=cache.device)
        if scale is not None:
            x = (x / scale[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
        part.copy_(x.to(cache.dtype))


def _scales(case, g, dev):
    if case["cache"] != "e4m3":
        return None, None
    return tuple(0.01 + 0.02 * torch.rand(case["hkv"], generator=g, device=dev) for _ in range(2))


def _inv_freq(r, dev):
    """Rotary frequencies of base 500000, the slower ones stretched 8 times for long contexts."""
    f = 500000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    return torch.where(2 * math.pi / f > 8192, f / 8, f).to(dev)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "decode":
        B, hq, hkv, d, page = (case[k] for k in ("B", "hq", "hkv", "d", "page"))
        lens = _shuffled(_lens(case), seed)
        pages = [-(-n // page) for n in lens]
        width = max(1, max(pages))
        blocks = sum(pages) + 3
        order = torch.randperm(blocks, generator=g, device=dev, dtype=torch.int32).cpu()
        table = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
        s["k_scale"], s["v_scale"] = _scales(case, g, dev)
        s["k"], s["v"] = _cache(blocks, case, dev), _cache(blocks, case, dev)
        _fill(s["k"], g, s["k_scale"])
        _fill(s["v"], g, s["v_scale"])
        s["q"] = torch.randn(B, hq, d, generator=g, device=dev).bfloat16()
        s["table"], s["lens"] = table.to(dev), _int(lens, dev)
        s["scale"] = 1.0 / math.sqrt(d)
    elif case["op"] == "append":
        T, hq, hkv, d, page = (case[k] for k in ("T", "hq", "hkv", "d", "page"))
        s["qkv"] = torch.randn(T, hq + 2 * hkv, d, generator=g, device=dev).bfloat16()
        s["q"], s["k"], s["v"] = s["qkv"].split([hq, hkv, hkv], 1)  # the three parts of one projection's output
        blocks = -(-T // page) + 2
        slots = torch.randperm(blocks * page, generator=g, device=dev, dtype=torch.int32)[:T]
        slots[T - case["pad"]:] = -1
        s["slots"] = slots
        s["positions"] = torch.randint(0, 131072, (T,), generator=g, device=dev, dtype=torch.int32)
        s["inv_freq"] = _inv_freq(case["r"], dev)
        s["k_scale"], s["v_scale"] = _scales(case, g, dev)
        s["k_cache"], s["v_cache"] = _cache(blocks, case, dev), _cache(blocks, case, dev)
        _fill(s["k_cache"], g, s["k_scale"])
        _fill(s["v_cache"], g, s["v_scale"])
        s["q_out"] = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.zeros(T, hkv, d, dtype=torch.bfloat16, device=dev) if case["k_out"] else None
    elif case["op"] == "rotary":
        shape = (case["B"], case["H"], case["N"], case["d"])
        s["x"] = torch.randn(shape, generator=g, device=dev).bfloat16()
        s["dy"] = torch.randn(shape, generator=g, device=dev).bfloat16()
        start = torch.randint(0, 131072 - case["N"], (case["B"], 1), generator=g, device=dev, dtype=torch.int32)
        s["positions"] = start + torch.arange(case["N"], device=dev, dtype=torch.int32)
        s["inv_freq"] = _inv_freq(case["r"], dev)
    else:
        B, page, width = case["B"], case["page"], case["width"]
        ctx = _shuffled(_spread(B, case["ctx_lo"], case["ctx_hi"]), seed)
        fresh = _shuffled(_spread(B, case["new_lo"], case["new_hi"]), seed + 1)
        blocks = B * width + 7
        order = torch.randperm(blocks, generator=g, device=dev, dtype=torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        held = -(-_int(ctx, dev) // page)
        have = torch.arange(width, device=dev)[None] < held[:, None]
        n = int(held.sum())
        table[have] = order[:n]
        s["table"], s["unused"] = table, order[n:].contiguous()
        s["context_lens"], s["new_lens"] = _int(ctx, dev), _int(fresh, dev)
        s["T"] = sum(fresh) + case["pad"]
    return s


def _bits(t):
    """A view that can be indexed, of a tensor of 8-bit floats."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _plain_decode(s):
    c = s["case"]
    B, hq, hkv, d = c["B"], c["hq"], c["hkv"], c["d"]
    pages = s["table"].clamp(min=0).long()

    def rows(cache):  # [B, hkv, keys, d] in 32 bits
        x = _bits(cache)[pages].view(cache.dtype).float()
        return x.reshape(B, -1, hkv, d).transpose(1, 2)

    q = s["q"].float().view(B, hkv, hq // hkv, d)
    scores = torch.matmul(q, rows(s["k"]).transpose(2, 3)) * s["scale"]
    if s["k_scale"] is not None:
        scores = scores * s["k_scale"][:, None, None]
    seen = torch.arange(scores.shape[-1], device=q.device) < s["lens"][:, None, None, None]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows(s["v"])) / torch.where(total > 0, total, 1.0)
    if s["v_scale"] is not None:
        o = o * s["v_scale"][:, None, None]
    lse = top + torch.log(total)
    return o.reshape(B, hq, d).bfloat16(), lse.reshape(B, hq)


def _turn(x, cos, sin, interleaved):
    """x [..., d] with its first 2 * cos.shape[-1] values turned, pair by pair."""
    n = cos.shape[-1]
    x1, x2 = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)
    return torch.cat((y, x[..., 2 * n:]), -1)


def _cos_sin(positions, inv_freq, factor=1.0):
    angle = positions.double()[..., None] * inv_freq  # angles of far positions need 64 bits
    return (angle.cos() * factor).float(), (angle.sin() * factor).float()


def _encode(x, scale, dtype):
    if scale is None:
        return x.to(dtype)
    return (x / scale[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(dtype)


def _plain_append(s):
    c = s["case"]
    cos, sin = _cos_sin(s["positions"][:, None], s["inv_freq"])
    q = _turn(s["q"].float(), cos, sin, c["interleaved"])
    k = _turn(s["k"].float(), cos, sin, c["interleaved"])
    valid = s["slots"] >= 0
    slots = s["slots"][valid].long()
    block, token = slots // c["page"], slots % c["page"]
    s["q_out"][valid] = q[valid].bfloat16()
    if s["k_out"] is not None:
        s["k_out"][valid] = k[valid].bfloat16()
    for cache, x, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], s["v"].float(), s["v_scale"])):
        _bits(cache)[block, token] = _bits(_encode(x[valid], scale, cache.dtype))


def _plain_rotary(s):
    c = s["case"]
    cos, sin = _cos_sin(s["positions"][:, None], s["inv_freq"], c["factor"])
    y = _turn(s["x"].float(), cos, sin, c["interleaved"])
    dx = _turn(s["dy"].float(), cos, -sin, c["interleaved"])
    return y.bfloat16(), dx.bfloat16()


def _plain_maps(s):
    c = s["case"]
    page, width, T = c["page"], c["width"], s["T"]
    dev = s["table"].device
    ctx, fresh = s["context_lens"].long(), s["new_lens"].long()
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    cu = torch.cat((zero, fresh.cumsum(0)))
    held = (ctx + page - 1) // page
    need = (((ctx + fresh + page - 1) // page).clamp(max=width) - held).clamp(min=0)
    first = need.cumsum(0) - need
    column = torch.arange(width, device=dev) - held[:, None]
    given = (column >= 0) & (column < need[:, None])
    rank = first[:, None] + column
    got = torch.where(rank < s["unused"].numel(), s["unused"][rank.clamp(0, s["unused"].numel() - 1)], -1)
    s["table"].copy_(torch.where(given, got, s["table"]))
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu, t, right=True) - 1
    real = b < c["B"]
    b = b.clamp(max=c["B"] - 1)
    pos = ctx[b] + t - cu[b]
    entry = s["table"][b, (pos // page).clamp(max=width - 1)].long()
    slots = torch.where(real & (pos < width * page) & (entry >= 0), entry * page + pos % page, -1)
    total = need.sum()
    counts = torch.stack((total.clamp(max=s["unused"].numel()), (total - s["unused"].numel()).clamp(min=0), cu[-1],
                          (ctx + fresh > width * page).sum()))
    return (s["table"], slots.int(), torch.where(real, pos, 0).int(), cu.int(), (ctx + fresh).int(), counts.int())


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import exact_attention_91_gb300 as fa
        c = s["case"]
        if op == "decode":
            return fa.attention_decode_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=s["scale"],
                                             k_scale=s["k_scale"], v_scale=s["v_scale"])
        if op == "append":
            fa.cache_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_cache"],
                            s["v_cache"], interleaved=c["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                            q_out=s["q_out"], k_out=s["k_out"])
        elif op == "rotary":
            y = fa.rotary(s["x"], s["positions"], s["inv_freq"], interleaved=c["interleaved"], factor=c["factor"])
            dx = fa.rotary(s["dy"], s["positions"], s["inv_freq"], interleaved=c["interleaved"], factor=c["factor"],
                           inverse=True)
            return y, dx
        else:
            m = fa.page_maps(s["context_lens"], s["new_lens"], s["table"], s["unused"], c["page"], s["T"])
            return (s["table"], m.slots, m.positions, m.cu_seqlens, m.seq_lens, m.counts)
    elif op == "decode":
        return _plain_decode(s)
    elif op == "append":
        _plain_append(s)
    elif op == "rotary":
        return _plain_rotary(s)
    else:
        return _plain_maps(s)
    out = (s["q_out"], s["k_cache"], s["v_cache"])
    return out if s["k_out"] is None else out + (s["k_out"],)


def work(case):
    elt = 1 if case.get("cache") == "e4m3" else 2
    if case["op"] == "decode":
        keys, hq, hkv, d = sum(_lens(case)), case["hq"], case["hkv"], case["d"]
        pages = sum(-(-n // case["page"]) for n in _lens(case))
        return {"bytes": keys * hkv * d * 2 * elt + case["B"] * (hq * (4 * d + 4) + 4) + 4 * pages,
                "flops": 4 * keys * hq * d}
    if case["op"] == "append":
        n, hq, hkv, d = case["T"] - case["pad"], case["hq"], case["hkv"], case["d"]
        kept = 2 * hq + 2 * hkv * elt + (2 * hkv if case["k_out"] else 0)
        return {"bytes": n * d * (2 * (hq + 2 * hkv) + kept) + 4 * n + 4 * case["T"] + 4 * case["r"],
                "flops": 3 * n * (hq + hkv) * case["r"]}
    if case["op"] == "rotary":
        n = case["B"] * case["H"] * case["N"]
        return {"bytes": 8 * n * case["d"] + 8 * case["B"] * case["N"] + 8 * case["r"], "flops": 6 * n * case["r"]}
    B, page, width = case["B"], case["page"], case["width"]
    fresh = _spread(B, case["new_lo"], case["new_hi"])
    T = sum(fresh) + case["pad"]
    # (how many pages a step takes depends on which request gets which length: the mean)
    return {"bytes": 8 * B + 8 * T + 4 * (B + 1) + 4 * B + 8 * (sum(fresh) / page) + 16, "flops": 4 * T}


def _exact_decode(s):
    c = s["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    o = torch.zeros(c["B"], hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((c["B"], hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        where = torch.arange(n, device=o.device)
        block, token = s["table"][b].long()[where // page], where % page
        for h in range(hkv):
            k, v = ((t.view(torch.uint8) if c["cache"] == "e4m3" else t)[block, token, h].view(t.dtype).double()
                    for t in (s["k"], s["v"]))
            if c["cache"] == "e4m3":
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            mine = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            score = s["q"][b, mine].double() @ k.T * s["scale"]
            lse[b, mine] = torch.logsumexp(score, -1)
            o[b, mine] = torch.exp(score - lse[b, mine, None]) @ v
    return o, lse


def _exact_turn(x, positions, inv_freq, interleaved, factor=1.0, back=False):
    """Each pair as a complex number, multiplied by factor * exp(+-i * angle)."""
    angle = positions.double().unsqueeze(-1) * inv_freq
    z = torch.polar(torch.full_like(angle, factor), -angle if back else angle)
    r = 2 * inv_freq.numel()
    x = x.double()
    pairs = x[..., :r].unflatten(-1, (-1, 2)) if interleaved else x[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    y = x.clone()
    y[..., :r] = turned.flatten(-2) if interleaved else turned.transpose(-1, -2).flatten(-2)
    return y


def _exact_append(s):
    c = s["case"]
    q = _exact_turn(s["q"], s["positions"].unsqueeze(1), s["inv_freq"], c["interleaved"])
    k = _exact_turn(s["k"], s["positions"].unsqueeze(1), s["inv_freq"], c["interleaved"])
    n = c["T"] - c["pad"]
    q[n:] = 0
    slots = s["slots"][:n].long()
    caches = []
    for cache, x, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], s["v"].double(), s["v_scale"])):
        whole = cache.to(torch.float64)
        x = x if scale is None else (x / scale.double()[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
        whole[slots // c["page"], slots % c["page"]] = x[:n]
        caches.append(whole)
    out = (q, caches[0], caches[1])
    if s["k_out"] is None:
        return out
    k[n:] = 0
    return out + (k,)


def _exact_maps(s):
    """The same step taken one token after the other, as a host would."""
    c = s["case"]
    page, width = c["page"], c["width"]
    table, unused = s["table"].tolist(), s["unused"].tolist()
    slots, positions, cu, lens = [], [], [0], []
    taken = missing = beyond = 0
    for row, ctx, fresh in zip(table, s["context_lens"].tolist(), s["new_lens"].tolist()):
        for pos in range(ctx, ctx + fresh):
            column = pos // page
            if column >= width:
                slots.append(-1)
            else:
                if pos % page == 0:
                    if taken < len(unused):
                        row[column] = unused[taken]
                        taken += 1
                    else:
                        row[column] = -1
                        missing += 1
                slots.append(row[column] * page + pos % page if row[column] >= 0 else -1)
            positions.append(pos)
        cu.append(cu[-1] + fresh)
        lens.append(ctx + fresh)
        beyond += ctx + fresh > width * page
    slots += [-1] * c["pad"]
    positions += [0] * c["pad"]
    return tuple(torch.tensor(x, dtype=torch.int32)
                 for x in (table, slots, positions, cu, lens, [taken, missing, cu[-1], beyond]))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(s)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "rotary":
        at = s["positions"].unsqueeze(1)
        return (_exact_turn(s["x"], at, s["inv_freq"], case["interleaved"], case["factor"]),
                _exact_turn(s["dy"], at, s["inv_freq"], case["interleaved"], case["factor"], back=True))
    return _exact_maps(s)
