"""The serving operators together, as a server uses them: prompts and new
tokens through page maps, append and decode against 64-bit attention over the
whole history; steps captured into graphs; several streams; chains of dependent
calls whose launches overlap; no device memory taken."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest

from . import serve_oracle as so

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_91_gb300 as fa
    return fa


class Server:
    """Requests over one layer's cache; every token's q, k, v is drawn when it
    is needed and kept, so that the whole history can be recomputed."""

    def __init__(self, fa, B, hq, hkv, d, page=16, width=40, e4m3=False, seed=0):
        self.fa, self.B, self.hq, self.hkv, self.d, self.page = fa, B, hq, hkv, d, page
        self.g = torch.Generator().manual_seed(seed)
        blocks = B * width + 1
        t = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.kc, self.vc = (torch.zeros(blocks, page, hkv, d, device="cuda").to(t) for _ in range(2))
        self.ks = self.vs = torch.full((hkv,), 0.03, device="cuda") if e4m3 else None
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.unused = torch.randperm(blocks, generator=self.g).int().cuda()
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.freq, self.factor = fa.rotary_inv_freq(d, 10000.0, device="cuda")
        self.history = [[] for _ in range(B)]        # per request: (k turned, v) in 64 bits, as the cache should hold them

    def draw(self, T):
        qkv = torch.randn(T, self.hq + 2 * self.hkv, self.d, generator=self.g).bfloat16().cuda()
        return qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hkv], qkv[:, self.hq + self.hkv:]

    def maps(self, fresh, pad=0):
        fresh_t = torch.tensor(fresh, dtype=torch.int32).cuda()
        m = self.fa.page_maps(self.lens, fresh_t, self.table, self.unused, self.page, sum(fresh) + pad)
        counts = m.counts.tolist()
        assert counts[1] == 0 and counts[2] == sum(fresh) and counts[3] == 0
        self.unused = self.unused[counts[0]:].contiguous()
        self.lens = m.seq_lens
        return m

    def append(self, m, q, k, v, **kw):
        return self.fa.cache_append(q, k, v, m.positions, m.slots, self.freq, self.kc, self.vc, factor=self.factor,
                                    k_scale=self.ks, v_scale=self.vs, **kw)

    def remember(self, m, k, v, fresh):
        """The 64-bit keys and values of the step's tokens, from positions counted here."""
        at, ks = 0, so.f64(k)
        for b, n in enumerate(fresh):
            for _ in range(n):
                pos = len(self.history[b])
                assert m.positions[at].item() == pos
                turned, _ = so.turn(ks[at][:, None], np.array([pos]), self.freq.cpu().numpy(), False, self.factor)
                self.history[b].append((turned[:, 0], so.f64(v[at])))
                at += 1

    def attend64(self, b, q, upto):
        """Attention of one turned query [Hq, d] over the first `upto` tokens."""
        k = np.stack([h[0] for h in self.history[b][:upto]])
        v = np.stack([h[1] for h in self.history[b][:upto]])
        G = self.hq // self.hkv
        o, lse = np.zeros((self.hq, self.d)), np.zeros(self.hq)
        for i in range(self.hq):
            s = k[:, i // G] @ q[i] / math.sqrt(self.d)
            lse[i] = s.max() + math.log(np.exp(s - s.max()).sum())
            o[i] = np.exp(s - lse[i]) @ v[:, i // G]
        return o, lse


def _near(o, lse, want, e4m3):
    """q and the cache hold rounded values: each score is off by its two
    roundings (bf16 2^-8 each; e4m3 2^-4 for k), in random directions, so by
    their root mean square over d products at most, times four; O by that and by
    v's own rounding and its own."""
    o_ref, lse_ref = want
    unit = so.E4M3_HALF if e4m3 else so.BF16_HALF
    off = 4 * unit * 3.0                                  # |q||k|/sqrt(d) is about 1 to 3 for normal draws
    assert np.abs(lse - lse_ref).max() <= off
    assert np.abs(o - o_ref).max() <= off * 4             # |v| up to 4


@pytest.mark.parametrize("hq,hkv,d,e4m3", [(4, 4, 64, False), (8, 2, 128, False), (6, 3, 64, True)])
def test_prompts_then_tokens(hq, hkv, d, e4m3):
    fa = _fa()
    s = Server(fa, 4, hq, hkv, d, e4m3=e4m3, seed=d)
    fresh = [37, 1, 130, 16]
    m = s.maps(fresh, pad=5)
    q, k, v = s.draw(sum(fresh) + 5)
    k_out = torch.zeros_like(k)
    q_rot = s.append(m, q, k, v, k_out=k_out)
    s.remember(m, k, v, fresh)
    if hq == hkv:                                         # the prompt's own attention: the packed kernel on the turned q, k
        n = sum(fresh)
        o, lse = fa.attention_forward_varlen(q_rot[:n].contiguous(), k_out[:n].contiguous(), v[:n].contiguous(), m.cu_seqlens,
                                             m.cu_seqlens, max(fresh), causal=True)
        cu = m.cu_seqlens.tolist()
        for b in range(4):
            for i in {0, fresh[b] // 2, fresh[b] - 1}:
                y, _ = so.turn(so.f64(q[cu[b] + i])[:, None], np.array([i]), s.freq.cpu().numpy(), False, s.factor)
                _near(so.f64(o[cu[b] + i]), so.f64(lse[:, cu[b] + i]), s.attend64(b, y[:, 0], i + 1), False)
        # and the last token of each prompt through the paged kernel: the same attention
        last = torch.tensor([c - 1 for c in cu[1:]]).cuda()
        od, ld = fa.attention_decode_paged(q_rot[last].contiguous(), s.kc, s.vc, s.table, s.lens)
        assert (od.float() - o[last].float()).abs().max().item() <= 2 ** -6
        assert (ld - lse[:, last].t()).abs().max().item() <= 1e-3
    for step in range(6):
        fresh = [1, 1, 0 if step % 2 else 1, 1]           # a request that pauses
        m = s.maps(fresh)
        q, k, v = s.draw(sum(fresh))
        q_rot = s.append(m, q, k, v)
        s.remember(m, k, v, fresh)
        rows = [b for b, n in enumerate(fresh) if n]
        full = torch.zeros(4, hq, d, dtype=torch.bfloat16, device="cuda")
        full[rows] = q_rot
        o, lse = fa.attention_decode_paged(full, s.kc, s.vc, s.table, s.lens, k_scale=s.ks, v_scale=s.vs)
        # exactly: against what the cache holds
        want = so.decode(so.f64(full), so.f64(s.kc), so.f64(s.vc), s.table.cpu().numpy(), s.lens.cpu().numpy(),
                         1 / math.sqrt(d), None if s.ks is None else so.f64(s.ks), None if s.vs is None else so.f64(s.vs))
        so.assert_decode(so.f64(o), so.f64(lse), want)
        # and against the whole history in 64 bits
        for j, b in enumerate(rows):
            pos = len(s.history[b]) - 1
            y, _ = so.turn(so.f64(q[j])[:, None], np.array([pos]), s.freq.cpu().numpy(), False, s.factor)
            _near(so.f64(o[b]), so.f64(lse[b]), s.attend64(b, y[:, 0], pos + 1), e4m3)


def _step_buffers(fa, B, hq, hkv, d, page, width, seed):
    g = torch.Generator().manual_seed(seed)
    blocks = B * width
    x = dict(kc=torch.randn(blocks, page, hkv, d, generator=g).bfloat16().cuda(),
             vc=torch.randn(blocks, page, hkv, d, generator=g).bfloat16().cuda(),
             table=torch.full((B, width), -1, dtype=torch.int32).cuda(),
             unused=torch.randperm(blocks, generator=g).int().cuda(),
             lens=torch.zeros(B, dtype=torch.int32).cuda(), ones=torch.ones(B, dtype=torch.int32).cuda(),
             qkv=torch.randn(B, hq + 2 * hkv, d, generator=g).bfloat16().cuda(), freq=fa.rotary_inv_freq(d, device="cuda")[0])
    return x


def _step(fa, x, hq, hkv, page):
    """One captured-able step: nothing is read back, buffers stay in place."""
    B = x["lens"].shape[0]
    m = fa.page_maps(x["lens"], x["ones"], x["table"], x["unused"], page, B)
    q, k, v = x["qkv"].split([hq, hkv, hkv], 1)
    q = fa.cache_append(q, k, v, m.positions, m.slots, x["freq"], x["kc"], x["vc"])
    o, lse = fa.attention_decode_paged(q, x["kc"], x["vc"], x["table"], m.seq_lens)
    return o, lse, m


@pytest.mark.parametrize("width", [6, 400])               # both forms of the decode kernel
def test_a_captured_step_replays_like_the_eager_one(width):
    fa = _fa()
    B, hq, hkv, d, page = 5, 8, 2, 128, 16
    a, b = (_step_buffers(fa, B, hq, hkv, d, page, width, seed=3) for _ in range(2))
    small = fa.fa_decode_paged_workspace(B, hq, hkv, d, fa.CACHE_BF16, page, width,
                                         torch.cuda.get_device_properties(0).multi_processor_count) == 0
    assert small == (width == 6)
    _step(fa, _step_buffers(fa, B, hq, hkv, d, page, width, seed=4), hq, hkv, page)   # the device's first calls
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(fa, a, hq, hkv, page)
    g = torch.Generator().manual_seed(9)
    for step in range(40):
        lens = torch.randint(0, 60, (B,), generator=g).int().cuda() if step % 3 else torch.full((B,), step, dtype=torch.int32).cuda()
        qkv = torch.randn(B, hq + 2 * hkv, d, generator=g).bfloat16().cuda()
        for x in (a, b):
            x["lens"].copy_(lens)
            x["qkv"].copy_(qkv)
            x["table"].fill_(-1)
            held = (lens + page - 1) // page
            ids = torch.arange(B * 4, device="cuda", dtype=torch.int32).view(B, 4)
            x["table"][:, :4] = torch.where(torch.arange(4, device="cuda") < held[:, None], ids + 1, -1)
        graph.replay()
        ref = _step(fa, b, hq, hkv, page)
        torch.cuda.synchronize()
        for u, w in zip((out[0], out[1], *out[2], a["table"], a["kc"], a["vc"]), (ref[0], ref[1], *ref[2], b["table"], b["kc"], b["vc"])):
            assert torch.equal(u, w)


def test_graphs_replayed_on_two_streams_at_once():
    """Each graph has its own workspace: overlapping replays give the bits of
    separate ones."""
    fa = _fa()
    from .test_decode_paged import make
    xs = [make([3000 + 500 * i, 40, 2500, 0, 777], 8, 2, 128, 16, e4m3=bool(i), seed=50 + i) for i in range(2)]

    def run(x):
        return fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"], k_scale=x["ks"], v_scale=x["vs"])

    refs = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for x, s in zip(xs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append([run(x) for _ in range(20)])
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for ref, mine in zip(refs, outs):
        for o, lse in mine:
            assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_calls_on_another_stream():
    """stream=: work is ordered there, what the call allocates is not memory that
    the current stream's work still uses, and is not handed out again while
    either stream may still use it."""
    fa = _fa()
    from .test_decode_paged import make
    x = make([4000, 900, 3333], 8, 2, 128, 16, seed=61)
    ref = fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    kept, dropped = [], 0
    for i in range(20):
        with torch.cuda.stream(side):
            for _ in range(2):
                big = big @ big * 1e-4                      # keeps the side stream busy
        o, lse = fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"], stream=side)
        if i % 2:
            kept.append((o, lse))
        else:
            del o, lse
            dropped += 1
        torch.full((3 << 20,), 7, dtype=torch.uint8, device="cuda")   # takes freed blocks of this stream at once
        freq = fa.rotary_inv_freq(128, device="cuda")[0]
    side.synchronize()
    for o, lse in kept:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    del kept
    for _ in range(10):
        # memory freed on the current stream while its work is still to read it
        held = torch.full_like(ref[0], 3.0)
        torch.cuda._sleep(2000000)
        seen = held.clone()
        del held
        o, lse = fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"], stream=side)
        # a result that the current stream still reads when it is dropped
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(2000000)
        o_seen = o.clone()
        del o, lse
        for _ in range(3):
            p, _ = fa.attention_decode_paged(x["q"] * 2, x["k"], x["v"], x["table"], x["lens"], stream=side)
        torch.cuda.synchronize()
        assert (seen == 3).all() and torch.equal(o_seen, ref[0])
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    want = fa.rotary(x["q"], pos, freq)
    torch.cuda.synchronize()
    got = fa.rotary(x["q"], pos, freq, stream=side)
    out = torch.empty_like(got)
    assert fa.rotary(x["q"], pos, freq, out=out, stream=side) is out
    m = fa.page_maps(x["lens"], pos, x["table"].clone(), pos, 16, 9, stream=side)
    n = fa.page_maps(x["lens"], pos, x["table"].clone(), pos, 16, 9)
    kc, vc = x["k"].clone(), x["v"].clone()
    torch.cuda.synchronize()
    k = x["q"][:, :2]
    qa = fa.cache_append(x["q"], k, k, pos, pos, freq, kc, vc, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(out, want) and torch.equal(qa, want)
    assert all(torch.equal(a, b) for a, b in zip(m, n))


def test_a_chain_of_dependent_calls():
    """Each call reads what the one before it wrote, without a pause between:
    the launches overlap, the results are those of one call after the other."""
    fa = _fa()
    g = torch.Generator().manual_seed(70)
    freq = fa.rotary_inv_freq(128, device="cuda")[0]
    for shape in ((3, 5, 128), (3000, 32, 128)):
        pos = torch.randint(0, 1000, (shape[0],), generator=g).int().cuda()
        x = torch.randn(shape, generator=g).bfloat16().cuda()
        a, b = x.clone(), x.clone()
        for _ in range(30):
            fa.rotary(a, pos, freq, out=a)
            torch.cuda.synchronize()
        for _ in range(30):
            fa.rotary(b, pos, freq, out=b)
        assert torch.equal(a, b)
    # append, then decode that must see the appended key and value, many times over the same slots
    B, hq, hkv, d = 64, 8, 2, 128
    kc, vc = (torch.zeros(B * 2, 16, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(B * 2, dtype=torch.int32, device="cuda").view(B, 2)
    lens = torch.full((B,), 17, dtype=torch.int32, device="cuda")
    slots = table[:, 1] * 16
    pos = torch.full((B,), 16, dtype=torch.int32, device="cuda")
    steps = [torch.randn(B, hq + 2 * hkv, d, generator=g).bfloat16().cuda() for _ in range(30)]

    def chain(sync):
        outs = []
        for t in (table, table.repeat(1, 300)[:, :600]):       # both forms of the decode kernel
            for x in steps:
                q, k, v = x.split([hq, hkv, hkv], 1)
                q = fa.cache_append(q, k, v, pos, slots, freq, kc, vc)
                if sync:
                    torch.cuda.synchronize()
                outs.append(fa.attention_decode_paged(q, kc, vc, t, lens)[0])
                if sync:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    assert all(torch.equal(a, b) for a, b in zip(chain(True), chain(False)))


def test_other_streams_are_waited_for():
    """An early launch overlaps its predecessor on the stream only: work that the
    stream was told to wait for (an event of another stream, a copy) is done
    before the kernel reads."""
    fa = _fa()
    freq = fa.rotary_inv_freq(128, device="cuda")[0]
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    a, b = (torch.zeros(64, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    src = torch.randn(64, 8, 128, device="cuda").bfloat16()
    want = fa.rotary(src, pos, freq)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(40):
        with torch.cuda.stream(main):
            b.zero_()
            fa.rotary(a, pos, freq, out=a)                 # the predecessor on the stream
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
            if i % 2:
                b.copy_(src)
            else:
                fa.rotary(src, torch.zeros_like(pos), freq, out=b)   # position 0: a copy
        main.wait_stream(side)
        with torch.cuda.stream(main):
            y = fa.rotary(b, pos, freq)
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_a_graph_with_branches_between_the_calls():
    """Captured: a call, a branch on another stream that makes the input of the
    next call, and that call after the join."""
    fa = _fa()
    freq = fa.rotary_inv_freq(128, device="cuda")[0]
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    src, a, b = (torch.randn(64, 8, 128, device="cuda").bfloat16() for _ in range(3))
    zero = torch.zeros_like(pos)
    fa.rotary(src, pos, freq)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.zero_()
        fa.rotary(a, zero, freq, out=a)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(100000)
            fa.rotary(src, zero, freq, out=b)
        fa.rotary(a, zero, freq, out=a)
        torch.cuda.current_stream().wait_stream(side)
        y = fa.rotary(b, pos, freq)
        z = fa.rotary(y, pos, freq, inverse=True)
    for _ in range(10):
        src.copy_(torch.randn_like(src))
        graph.replay()
        want = fa.rotary(src, pos, freq)
        assert torch.equal(y, want) and torch.equal(z, fa.rotary(want, pos, freq, inverse=True))


def test_rotary_gradient_in_a_graph():
    fa = _fa()
    from exact_attention_91_gb300 import torch_op  # noqa: F401
    freq = fa.rotary_inv_freq(64, device="cuda")[0]
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    x = torch.randn(2, 3, 33, 64, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn(2, 3, 33, 64, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(torch.ops.fa91.rotary(x, pos, freq), x, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = torch.ops.fa91.rotary(x, pos, freq)
        dx, = torch.autograd.grad(y, x, dy)
    with torch.no_grad():
        x.copy_(torch.randn_like(x))
    dy.copy_(torch.randn_like(dy))
    graph.replay()
    assert torch.equal(y, fa.rotary(x.detach(), pos, freq)) and torch.equal(dx, fa.rotary(dy, pos, freq, inverse=True))


def test_operators_equal_the_functions_and_compile():
    fa = _fa()
    from exact_attention_91_gb300 import torch_op  # noqa: F401
    from .test_decode_paged import make
    x = make([30, 0, 65], 4, 2, 64, 16, e4m3=True, seed=80)
    args = (x["q"], x["k"], x["v"], x["table"], x["lens"], 0.2, x["ks"], x["vs"])
    o, lse = fa.attention_decode_paged(*args[:5], scale=0.2, k_scale=x["ks"], v_scale=x["vs"])
    for f in (torch.ops.fa91.attention_decode_paged, torch.compile(lambda *a: torch.ops.fa91.attention_decode_paged(*a), fullgraph=True)):
        o2, l2 = f(*args)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    ctx, new = x["lens"], torch.tensor([3, 0, 40], dtype=torch.int32).cuda()
    unused = torch.arange(50, 60, dtype=torch.int32).cuda()
    ta, tb = x["table"].clone(), x["table"].clone()
    m = fa.page_maps(ctx, new, ta, unused, 16, 50)
    n = torch.ops.fa91.page_maps(ctx, new, tb, unused, 16, 50)
    assert torch.equal(ta, tb) and all(torch.equal(a, b) for a, b in zip(m, n))
    freq = fa.rotary_inv_freq(64, device="cuda")[0]
    q, k, v = torch.randn(50, 8, 64, device="cuda").bfloat16().split([4, 2, 2], 1)
    kc, vc = (torch.zeros(70, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kd, vd = kc.clone(), vc.clone()
    qa = fa.cache_append(q, k, v, m.positions, m.slots, freq, kc, vc)
    qb = torch.ops.fa91.cache_append(q, k, v, m.positions, m.slots, freq, kd, vd)
    real = m.slots >= 0
    assert torch.equal(qa[real], qb[real]) and torch.equal(kc, kd) and torch.equal(vc, vd) and kc.abs().sum() > 0


def test_calls_leave_device_memory_unchanged():
    fa = _fa()
    from .test_decode_paged import make
    x = make([5000, 700, 3], 8, 2, 128, 16, seed=90)
    o, lse = torch.empty_like(x["q"]), torch.empty(3, 8, device="cuda")
    n = fa.fa_decode_paged_workspace(3, 8, 2, 128, fa.CACHE_BF16, 16, x["table"].shape[1],
                                     torch.cuda.get_device_properties(0).multi_processor_count)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    freq = fa.rotary_inv_freq(128, device="cuda")[0]
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    maps = fa.page_maps(x["lens"], pos, x["table"], pos, 16, 9)

    def calls():
        fa.page_maps(x["lens"], pos, x["table"], pos, 16, 9, out=maps)
        fa.cache_append(x["q"], x["q"][:, :2], x["q"][:, :2], pos, pos, freq, x["k"], x["v"], q_out=o)
        fa.rotary(x["q"], pos, freq, out=o)
        fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"], out=o, lse=lse, workspace=ws)

    calls()
    torch.cuda.synchronize()
    free0, held0 = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
    for _ in range(100):
        calls()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free0 and torch.cuda.memory_allocated() == held0


CHILD = r"""
import torch
import exact_attention_91_gb300 as fa
x = torch.ones(4, 2, 64, device="cuda").bfloat16()
pos = torch.arange(4, dtype=torch.int32, device="cuda")
freq = fa.rotary_inv_freq(64, device="cuda")[0]
fa.load_binding()
out = torch.full_like(x, 7.0)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
status = None
with torch.cuda.graph(g):
    try:
        fa.rotary(x, pos, freq, out=out)
    except fa.FaError as e:
        status = e.status
    out2 = out + 1
assert status == -7, status
g.replay()
torch.cuda.synchronize()
assert (out == 7).all() and (out2 == 8).all()
fa.rotary(x, pos, freq, out=out)                 # the first ordinary call
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = fa.rotary(x, pos, freq)
g.replay()
torch.cuda.synchronize()
assert torch.equal(y, out)
print("first-call-in-capture OK")
"""


def test_a_capture_before_the_first_call_is_refused():
    _fa()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, PYTHONPATH=root + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, env=env, timeout=300, cwd=root)
    assert r.returncode == 0 and "first-call-in-capture OK" in r.stdout, (r.stdout[-2000:], r.stderr[-3000:])


def test_refusals_reach_python_as_errors():
    """What only the C call refuses is raised with its status."""
    fa = _fa()
    from .test_decode_paged import make
    x = make([5], 2, 1, 64, 16, seed=1)
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    freq = fa.rotary_inv_freq(24, device="cuda")[0]
    cases = [
        (-2, lambda: fa.rotary(x["q"], pos, freq)),                                     # 24 is no multiple of 16
        (-9, lambda: fa.rotary(x["q"], pos, None, factor=float("nan"))),
        (-9, lambda: fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"], scale=-1.0)),
        (-10, lambda: fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"], out=x["q"])),
        (-11, lambda: fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"].repeat(1, 9000), x["lens"],
                                                workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))),
        (-2, lambda: fa.cache_append(x["q"], x["q"][:, :1], x["q"][:, :1], pos, pos, None, x["k"][:, :9], x["v"][:, :9])),
        (-2, lambda: fa.page_maps(pos, pos, x["table"], pos, 48, 0)),
        (-10, lambda: fa.page_maps(pos, pos, x["table"], x["table"][0], 16, 0)),
    ]
    for status, f in cases:
        with pytest.raises(fa.FaError) as e:
            f()
        assert e.value.status == status, (status, str(e.value))
    with pytest.raises(ValueError):
        fa.rotary(x["q"], pos.cpu(), None)                                              # another device
    o, lse = fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"])   # and nothing is left behind
    assert torch.isfinite(lse).all()
