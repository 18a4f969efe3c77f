"""Attention's backward pass, and attention over a prefix that requests share:
what is measured of them, and their plain forms.

Three operators, named in a case's ``"op"``:

* ``backward``  gradients of attention on [B, H, N, d], from its inputs, O and LSE
* ``varlen``    the same over packed sequences [total, H, d] with their own query
  and key counts
* ``shared``    attention of one new token per request over a paged cache, where
  the requests of a group share the pages of a long prefix

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


def _named(case, name):
    return case | ({"name": name} if name else {})


def _backward(name, B, H, N, d, causal, dlse=False):
    return _named({"op": "backward", "B": B, "H": H, "N": N, "d": d, "causal": causal, "dlse": dlse}, name)


def _varlen(name, B, H, d, causal, q_lo, q_hi, k_lo=0, k_hi=0, dlse=False):
    """Query counts from q_lo to q_hi; key counts from k_hi down to k_lo, or the query counts where k_hi is 0."""
    return _named({"op": "varlen", "B": B, "H": H, "d": d, "causal": causal, "q_lo": q_lo, "q_hi": q_hi,
                   "k_lo": k_lo, "k_hi": k_hi, "dlse": dlse}, name)


def _shared(name, B, groups, hq, hkv, d, page, prefix_lo, prefix_hi, own_lo, own_hi, cache="bf16", heads_first=False,
            empty=0):
    """Groups of B / groups requests: prefixes of prefix_lo to prefix_hi tokens, then own_lo to own_hi of a request's
    own; the last `empty` requests of a group hold nothing (a padded batch)."""
    return _named({"op": "shared", "B": B, "groups": groups, "hq": hq, "hkv": hkv, "d": d, "page": page,
                   "prefix_lo": prefix_lo, "prefix_hi": prefix_hi, "own_lo": own_lo, "own_hi": own_hi, "cache": cache,
                   "heads_first": heads_first, "empty": empty}, name)


def listed():
    return [
        # this repository's tiny shape: one tile, where latency is all
        _backward("bwd_tiny", 1, 1, 128, 64, False),
        # its ragged causal shape, with a loss on LSE too
        _backward("bwd_ragged", 2, 4, 1000, 64, True, dlse=True),
        # its many-heads shape: one wave of short heads
        _backward("bwd_heads", 16, 16, 1024, 128, False),
        # its prefill shape: a training step's layer
        _backward("bwd_prefill", 4, 32, 4096, 128, True),
        # its long sequence
        _backward("bwd_long", 1, 8, 16384, 64, False),
        # a packed training batch of documents
        _varlen("bwd_documents", 12, 16, 128, True, 100, 2048),
        # queries and keys of their own counts, some queries without keys, some sequences without either
        _varlen("bwd_cross", 9, 6, 64, True, 0, 700, 0, 1501, dlse=True),
        # four answers to one question: a few small launches
        _shared("shared_few", 4, 1, 32, 8, 128, 16, 2000, 2000, 1, 40),
        # three prompts of a small d = 64 model, 16 answers each
        _shared("shared_groups", 48, 3, 12, 12, 64, 16, 500, 1501, 1, 300),
        # a serving batch behind one system prompt, padded up to its graph's size
        _shared("shared_batch", 64, 1, 32, 8, 128, 16, 8192, 8192, 1, 512, empty=3),
        # two long documents that are asked about 8 times each
        _shared("shared_long", 16, 2, 32, 8, 128, 64, 65000, 65536, 100, 1000),
        # a large batch whose cache is held in 8 bits, pages stored head by head
        _shared("shared_e4m3", 128, 4, 64, 8, 128, 64, 777, 8190, 1, 800, cache="e4m3", heads_first=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_MOST_FLOPS = 10 * 4 * 32 * (4096 * 4097 // 2) * 128  # the largest listed backward pass's
_MOST_SCORES = 4 * 32 * 4096 * 4096                   # and its scores, all of which the plain form makes


def draw(rng):
    op = rng.choice(["backward", "backward", "varlen", "shared", "shared"])
    if op == "backward":
        d, causal = rng.choice([64, 128]), rng.random() < 0.6
        N = _log(rng, 1, 16384)
        pairs = N * (N + 1) // 2 if causal else N * N
        room = max(1, min(_MOST_FLOPS // (10 * pairs * d), _MOST_SCORES // (N * N), 512))
        B = _log(rng, 1, min(room, 16))
        return _backward(None, B, _log(rng, 1, min(room // B, 32)), N, d, causal, rng.random() < 0.3)
    if op == "varlen":
        d, causal = rng.choice([64, 128]), rng.random() < 0.7
        B, H = rng.randint(1, 16), rng.choice([1, 3, 4, 8, 16])
        hi = _log(rng, 2, int(math.sqrt(_MOST_SCORES / 3 / (B * H))))
        if rng.random() < 0.5:
            return _varlen(None, B, H, d, causal, rng.randint(0, hi), hi, dlse=rng.random() < 0.3)
        k_hi = _log(rng, 1, max(1, min(16384, _MOST_SCORES // 3 // (B * H * hi))))
        return _varlen(None, B, H, d, causal, rng.randint(0, hi), hi, rng.randint(0, k_hi), k_hi,
                       dlse=rng.random() < 0.3)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8, 12])
    hq = hkv * (1 if hkv >= 12 else rng.choice([1, 2, 3, 4, 7, 8, 16]))
    groups = rng.choice([1, 1, 2, 3, 4])
    each = _log(rng, 2, 128 // groups)
    room = 128 * 8192 * 8 * 128 // (groups * each * hkv * d)  # keys per request that cost no more than the largest's
    prefix = _log(rng, 16, max(16, min(65536, room // 2)))
    fresh = _log(rng, 1, max(1, min(1000, room // 4)))
    return _shared(None, groups * each, groups, hq, hkv, d, rng.choice([16, 32, 64, 128]),
                   max(1, int(prefix * rng.uniform(0.3, 1.0))), prefix, rng.randint(1, fresh), fresh,
                   rng.choice(["bf16", "bf16", "e4m3"]), rng.random() < 0.4, empty=rng.randint(0, (each - 1) // 8))


def _counts(case):
    """(queries, keys) of each sequence of a varlen case."""
    nq = _spread(case["B"], case["q_lo"], case["q_hi"])
    nk = _spread(case["B"], case["k_lo"], case["k_hi"])[::-1] if case["k_hi"] else nq
    return list(zip(nq, nk))


def _pairs(nq, nk, causal):
    """Pairs of a query and a key that it sees; the causal mask is aligned at the end."""
    if not causal:
        return nq * nk
    if nq <= nk:
        return nq * (nk - nq) + nq * (nq + 1) // 2
    return nk * (nk + 1) // 2


def _own_lens(case):
    """A request's own tokens, of the requests of one group."""
    each = case["B"] // case["groups"]
    return _spread(each - case["empty"], case["own_lo"], case["own_hi"]) + [0] * case["empty"]


def _prefixes(case):
    return _spread(case["groups"], case["prefix_lo"], case["prefix_hi"])


def _shuffled(values, seed):
    values = list(values)
    random.Random(seed).shuffle(values)
    return values


def _int(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


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


def _forward(q, k, v, seen, scale):
    """O (bf16) and LSE of heads [..., N, d], as the forward pass leaves them."""
    s = torch.matmul(q.float(), k.float().transpose(-1, -2)) * scale
    if seen is not None:
        s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    return torch.matmul(p, v.float()).bfloat16(), lse


def _causal(nq, nk):
    i = torch.arange(nq, device="cuda")[:, None]
    return torch.arange(nk, device="cuda")[None] <= i + (nk - nq)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case, "scale": 1.0 / math.sqrt(case["d"])}
    if case["op"] == "backward":
        B, H, N, d = (case[k] for k in ("B", "H", "N", "d"))
        s["q"], s["k"], s["v"], s["do"] = (_normal(g, B, H, N, d) for _ in range(4))
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, H, N, device=dev)
        seen = _causal(N, N) if case["causal"] else None
        heads = max(1, (1 << 29) // (N * N))
        flat = [s[x].view(B * H, N, d) for x in ("q", "k", "v", "o")] + [s["lse"].view(B * H, N)]
        for h in range(0, B * H, heads):
            q, k, v, o, lse = (x[h:h + heads] for x in flat)
            out = _forward(q, k, v, seen, s["scale"])
            o.copy_(out[0])
            lse.copy_(out[1])
        s["dlse"] = torch.randn(B, H, N, generator=g, device=dev) if case["dlse"] else None
    elif case["op"] == "varlen":
        H, d = case["H"], case["d"]
        counts = _shuffled(_counts(case), seed)
        cu_q, cu_k = [0], [0]
        for nq, nk in counts:
            cu_q.append(cu_q[-1] + nq)
            cu_k.append(cu_k[-1] + nk)
        total_q, total_k = cu_q[-1], cu_k[-1]
        s["q"], s["do"] = (_normal(g, total_q, H, d) for _ in range(2))
        s["k"], s["v"] = (_normal(g, total_k, H, d) for _ in range(2))
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(H, total_q, device=dev)
        for b, (nq, nk) in enumerate(counts):
            if not nq:
                continue
            rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
            q, k, v = (x.transpose(0, 1) for x in (s["q"][rows], s["k"][keys], s["v"][keys]))
            o, lse = _forward(q, k, v, _causal(nq, nk) if case["causal"] else None, s["scale"])
            s["o"][rows] = o.transpose(0, 1)
            s["lse"][:, rows] = lse
        s["cu_q"], s["cu_k"] = _int(cu_q, dev), _int(cu_k, dev)
        s["max_q"], s["max_k"] = max(n for n, _ in counts), max(n for _, n in counts)
        s["dlse"] = torch.randn(H, total_q, generator=g, device=dev) if case["dlse"] else None
    else:
        B, G, hq, hkv, d, page = (case[k] for k in ("B", "groups", "hq", "hkv", "d", "page"))
        each = B // G
        prefixes, lens, pages = _shuffled(_prefixes(case), seed), [], []
        for i, n in enumerate(prefixes):
            lens += [n + m if m else 0 for m in _shuffled(_own_lens(case), seed + i)]
        # a group's whole pages of prefix are its requests' common ones; what begins behind them is each one's own
        common = [n // page for n in prefixes]
        private = [max(0, -(-n // page) - common[b // each]) for b, n in enumerate(lens)]
        width = max(1, max(common[b // each] + n for b, n in enumerate(private)))
        blocks = sum(common) + sum(private) + 3
        order = torch.randperm(blocks, generator=g, device=dev, dtype=torch.int32).cpu()
        table = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(common):
            table[i * each:(i + 1) * each, :n] = order[at:at + n]
            at += n
        for b, n in enumerate(private):
            table[b, common[b // each]:common[b // each] + n] = order[at:at + n]
            at += n
        s["k_scale"], s["v_scale"] = (0.01 + 0.02 * torch.rand(hkv, generator=g, device=dev)
                                      if case["cache"] == "e4m3" else None for _ in range(2))
        s["k"], s["v"] = _cache(blocks, case, dev), _cache(blocks, case, dev)
        _fill(s["k"], g, s["k_scale"])
        _fill(s["v"], g, s["v_scale"])
        s["q"] = _normal(g, B, hq, d)
        s["table"], s["lens"], s["prefix"] = table.to(dev), _int(lens, dev), _int(prefixes, dev)
    return s


def _gradients(do, q, k, v, o, lse, dlse, seen, scale):
    """dq, dk, dv in 32 bits of heads [..., N, d]; `seen`: which keys a query sees, or None for all."""
    do, q, k, v = do.float(), q.float(), k.float(), v.float()
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).sub_(lse[..., None]).exp_()
    if seen is not None:
        p = p.masked_fill_(~seen, 0.0)
    dv = torch.matmul(p.transpose(-1, -2), do)
    delta = (do * o.float()).sum(-1)
    if dlse is not None:
        delta = delta - dlse
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_(delta[..., None]).mul_(p)
    return torch.matmul(ds, k) * scale, torch.matmul(ds.transpose(-1, -2), q) * scale, dv


def _plain_backward(s):
    N = s["case"]["N"]
    seen = _causal(N, N) if s["case"]["causal"] else None
    return tuple(x.bfloat16() for x in _gradients(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["dlse"], seen,
                                                  s["scale"]))


def _plain_varlen(s):
    """The sequences side by side, padded to the longest."""
    def places(cu, most):  # [B, most] rows of the packed tensors, and which of them are the sequence's
        at = cu[:-1, None].long() + torch.arange(most, device=cu.device)
        return at, at < cu[1:, None]

    at_q, have_q = places(s["cu_q"], s["max_q"])
    at_k, have_k = places(s["cu_k"], s["max_k"])

    def heads(x, at, have):  # [B, H, most, ...]
        if not x.shape[0]:
            return x.new_zeros((at.shape[0], x.shape[1], at.shape[1]) + x.shape[2:])
        x = x[at.clamp(max=x.shape[0] - 1)].float()
        return x.masked_fill(~have.view(have.shape + (1,) * (x.dim() - 2)), 0.0).transpose(1, 2)

    nq, nk = (cu[1:].long() - cu[:-1].long() for cu in (s["cu_q"], s["cu_k"]))
    seen = have_q[:, None, :, None] & have_k[:, None, None, :]
    if s["case"]["causal"]:
        i, j = (torch.arange(n, device=nq.device) for n in (s["max_q"], s["max_k"]))
        seen = seen & (j <= i[:, None] + (nk - nq)[:, None, None, None])
    do, q, o = (heads(s[x], at_q, have_q) for x in ("do", "q", "o"))
    k, v = (heads(s[x], at_k, have_k) for x in ("k", "v"))
    lse = heads(s["lse"].T, at_q, have_q)
    dlse = heads(s["dlse"].T, at_q, have_q) if s["dlse"] is not None else None
    dq, dk, dv = _gradients(do, q, k, v, o, lse, dlse, seen, s["scale"])
    return tuple(x.transpose(1, 2)[have].bfloat16() for x, have in ((dq, have_q), (dk, have_k), (dv, have_k)))


def _bits(t):
    """A view that can be indexed, of a tensor of 8-bit floats."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _plain_shared(s):
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


def run(state):
    s, c = state, state["case"]
    if own:
        import exact_attention_91_gb300 as fa
        if c["op"] == "backward":
            return fa.attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], causal=c["causal"],
                                         scale=s["scale"], dlse=s["dlse"])
        if c["op"] == "varlen":
            return fa.attention_backward_varlen(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu_q"],
                                                s["cu_k"], s["max_q"], s["max_k"], causal=c["causal"],
                                                scale=s["scale"], dlse=s["dlse"])
        return fa.attention_decode_shared(s["q"], s["k"], s["v"], s["table"], s["lens"], s["prefix"],
                                          scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["op"] == "backward":
        return _plain_backward(s)
    if c["op"] == "varlen":
        return _plain_varlen(s)
    return _plain_shared(s)


def work(case):
    d = case["d"]
    if case["op"] == "backward":
        n = case["B"] * case["H"] * case["N"]
        pairs = case["B"] * case["H"] * _pairs(case["N"], case["N"], case["causal"])
        return {"bytes": n * (8 * d * 2 + 4 + (4 if case["dlse"] else 0)), "flops": 10 * pairs * d}
    if case["op"] == "varlen":
        H, counts = case["H"], _counts(case)
        nq, nk = sum(n for n, _ in counts), sum(n for _, n in counts)
        pairs = sum(_pairs(a, b, case["causal"]) for a, b in counts)
        return {"bytes": H * (nq * (4 * d * 2 + 4 + (4 if case["dlse"] else 0)) + nk * 4 * d * 2) + 8 * (case["B"] + 1),
                "flops": 10 * H * pairs * d}
    elt = 1 if case["cache"] == "e4m3" else 2
    hq, hkv, page, G, B = (case[k] for k in ("hq", "hkv", "page", "groups", "B"))
    fresh, live = _own_lens(case), B // case["groups"] - case["empty"]
    prefixes = _prefixes(case)
    # a prefix's whole pages once, the rest of it and the own tokens once for each request
    keys = sum(n // page * page + live * (n % page) + sum(fresh) for n in prefixes)
    scores = sum(live * n + sum(fresh) for n in prefixes)
    pages = sum(n // page + sum(-(-(n % page + m) // page) for m in fresh if m) for n in prefixes)
    return {"bytes": keys * hkv * d * 2 * elt + B * (hq * (4 * d + 4) + 4) + 4 * pages + 4 * G,
            "flops": 4 * scores * hq * d}


def _exact_head(do, q, k, v, o, lse, dlse, causal, scale):
    """Gradients of one head in 64 bits, from dP/dS = diag(p) - p p' row by row: row i of dS is p_i * (dp_i - c_i)."""
    do, q, k, v, o, lse = (x.double() for x in (do, q, k, v, o, lse))
    score = torch.einsum("id,jd->ij", q, k) * scale
    if causal:
        i = torch.arange(q.shape[0], device=q.device)
        j = torch.arange(k.shape[0], device=q.device)
        hidden = j[None] - i[:, None] > k.shape[0] - q.shape[0]
        score[hidden] = -math.inf
    p = torch.exp(score - torch.where(lse == -math.inf, math.inf, lse)[:, None])
    c = torch.einsum("id,id->i", do, o)
    if dlse is not None:
        c = c - dlse.double()
    ds = p * (torch.einsum("id,jd->ij", do, v) - c[:, None])
    return (torch.einsum("ij,jd->id", ds, k) * scale, torch.einsum("ij,id->jd", ds, q) * scale,
            torch.einsum("ij,id->jd", p, do))


def _exact_backward(s):
    c = s["case"]
    out = tuple(torch.empty(s["q"].shape, dtype=torch.float64, device="cuda") for _ in range(3))
    for b in range(c["B"]):
        for h in range(c["H"]):
            dlse = None if s["dlse"] is None else s["dlse"][b, h]
            for x, y in zip(out, _exact_head(*(s[n][b, h] for n in ("do", "q", "k", "v", "o", "lse")), dlse,
                                             c["causal"], s["scale"])):
                x[b, h] = y
    return out


def _exact_varlen(s):
    c = s["case"]
    dq, dk, dv = (torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in ("q", "k", "v"))
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(c["B"]):
        i, j = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        if i.start == i.stop or j.start == j.stop:
            continue
        for h in range(c["H"]):
            dlse = None if s["dlse"] is None else s["dlse"][h, i]
            dq[i, h], dk[j, h], dv[j, h] = _exact_head(s["do"][i, h], s["q"][i, h], s["k"][j, h], s["v"][j, h],
                                                       s["o"][i, h], s["lse"][h, i], dlse, c["causal"], s["scale"])
    return dq, dk, dv


def _exact_shared(s):
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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "backward":
        return _exact_backward(s)
    if case["op"] == "varlen":
        return _exact_varlen(s)
    return _exact_shared(s)
