"""The differentiable operators as a training step uses them: gradients through autograd against the 64-bit ones, eager,
compiled and captured; several streams; a round trip of sampling (shared prefix) and training (packed backward)."""
import os
import subprocess
import sys

import numpy as np
import pytest

from . import grad_oracle as G

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_91_gb300 as fa
    from exact_attention_91_gb300 import torch_op  # noqa: F401
    return fa


def f64(t):
    return t.detach().cpu().double().numpy()


def rand(*shape, seed, grad=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16().requires_grad_(grad)


def check(x, o, lse, do, dlse, causal, scale):
    """x's gradients against the formula on the O and LSE that the forward pass gave."""
    q, k, v = x
    B, H = q.shape[:2]
    for b in range(B):
        for h in range(H):
            want, bound = G.backward(*(f64(t[b, h]) for t in (do, q, k, v, o, lse)), f64(dlse[b, h]), causal, scale)
            G.assert_gradients([f64(t.grad[b, h]) for t in x], want, bound)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("loss", ["o", "lse", "both"])
def test_autograd(fa, d, causal, loss):
    x = [rand(2, 3, 200, d, seed=i) for i in range(3)]
    do, dlse = rand(2, 3, 200, d, seed=5, grad=False), rand(2, 3, 200, seed=6, grad=False).float()
    if loss == "o":
        dlse = torch.zeros_like(dlse)
    if loss == "lse":
        do = torch.zeros_like(do)
    o, lse = torch.ops.fa91.attention_forward(*x, causal, 0.2)
    total = 0.0
    if loss != "lse":
        total = total + (o.float() * do.float()).sum()
    if loss != "o":
        total = total + (lse * dlse).sum()
    total.backward()
    check(x, o, lse, do, dlse, causal, 0.2)


def test_gradients_that_are_broadcast_or_strided(fa):
    x = [rand(1, 2, 130, 64, seed=i) for i in range(3)]
    o, lse = torch.ops.fa91.attention_forward(*x, True, None)
    o.sum().backward()                                        # an expanded gradient
    check(x, o, lse, torch.ones_like(o), torch.zeros_like(lse), True, 64 ** -0.5)
    for t in x:
        t.grad = None
    o, lse = torch.ops.fa91.attention_forward(*x, True, None)
    w = rand(1, 130, 2, 64, seed=9, grad=False)
    (o.transpose(1, 2) * w).float().sum().backward()          # one with other strides
    check(x, o, lse, w.transpose(1, 2), torch.zeros_like(lse), True, 64 ** -0.5)


def test_only_some_inputs_need_gradients(fa):
    q, k, v = rand(1, 2, 100, 64, seed=1), rand(1, 2, 100, 64, seed=2, grad=False), rand(1, 2, 100, 64, seed=3)
    o, _ = torch.ops.fa91.attention_forward(q, k, v, False, None)
    o.float().square().sum().backward()
    assert k.grad is None and q.grad is not None and v.grad is not None
    o, lse = torch.ops.fa91.attention_forward(q.detach(), k, v.detach(), False, None)
    assert not o.requires_grad and not lse.requires_grad


def test_the_forward_pass_keeps_its_results(fa):
    x = [rand(2, 3, 300, 128, seed=i) for i in range(3)]
    o, lse = torch.ops.fa91.attention_forward(*x, True, None)
    want = fa.attention_forward(*(t.detach() for t in x), causal=True)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_packed_autograd_with_padding(fa):
    lens = [70, 200, 1, 129]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    T = sum(lens) + 50
    x = [rand(T, 2, 64, seed=i) for i in range(3)]
    o, lse = torch.ops.fa91.attention_forward_varlen(*x, cu, cu, max(lens), True, None)
    do = rand(T, 2, 64, seed=8, grad=False)
    (o[:T - 50].float() * do[:T - 50].float()).sum().backward()
    at = cu.tolist()
    for b in range(len(lens)):
        i = slice(at[b], at[b + 1])
        for h in range(2):
            want, bound = G.backward(*(f64(t[i, h]) for t in (do, *x, o)), f64(lse[h, i]), np.zeros(lens[b]), True, 0.125)
            G.assert_gradients([f64(t.grad[i, h]) for t in x], want, bound)
    for t in x:
        assert (t.grad[T - 50:] == 0).all()


def test_compiled(fa):
    def step(q, k, v):
        o, lse = torch.ops.fa91.attention_forward(q, k, v, True, None)
        return (o.float() ** 2).sum() + lse.sum()

    x = [rand(1, 2, 150, 64, seed=i) for i in range(3)]
    step(*x).backward()
    want = [t.grad.clone() for t in x]
    for t in x:
        t.grad = None
    torch.compile(step, fullgraph=True, backend="aot_eager")(*x).backward()
    for t, w in zip(x, want):
        # (the loss's own arithmetic may be fused otherwise: half a step of dO, and what it makes of the gradients)
        assert (t.grad.float() - w.float()).abs().max() <= 2.0 ** -7 * w.float().abs().max()


def test_a_captured_step(fa):
    """Forward and backward pass in a CUDA graph: replays on new inputs give the bits of eager steps."""
    q, k, v, do = (rand(2, 2, 260, 128, seed=i, grad=False) for i in range(4))

    def step():
        x = [t.detach().requires_grad_() for t in (q, k, v)]
        o, lse = torch.ops.fa91.attention_forward(*x, True, None)
        return torch.autograd.grad((o, lse), x, (do, torch.ones_like(lse)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (20, 30):
        for i, t in enumerate((q, k, v, do)):
            t.copy_(rand(2, 2, 260, 128, seed=seed + i, grad=False))
        graph.replay()
        want = step()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert fa.fa_device_status() == (0, 0)


def test_captured_calls_replay_with_their_own_workspaces(fa):
    """Two graphs of backward calls (enough units for the counters), replayed at once on two streams."""
    def make(seed):
        q, k, v, do = (rand(2, 24, 600, 64, seed=seed + i, grad=False) for i in range(4))
        o, lse = fa.attention_forward(q, k, v, causal=True)
        return do, q, k, v, o, lse

    sets = [make(100), make(200)]
    want = [fa.attention_backward(*s, causal=True) for s in sets]
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.attention_backward(*s, causal=True))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        for a, b in zip(got, w):
            assert torch.equal(a, b)


def test_calls_at_once_on_two_streams(fa):
    q, k, v, do = (rand(1, 200, 300, 64, seed=i, grad=False) for i in range(4))
    o, lse = fa.attention_forward(q, k, v)
    want = fa.attention_backward(do, q, k, v, o, lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[fa.attention_backward(do, q, k, v, o, lse, stream=s) for _ in range(3)] for s in streams]
    torch.cuda.synchronize()
    for each in got:
        for r in each:
            for a, b in zip(r, want):
                assert torch.equal(a, b)


def test_sampling_and_training_on_the_samples(fa):
    """Several answers to each of two questions are sampled over a paged cache whose prefix pages they share, one token at
    a time; then the packed answers are trained on. Each step's attention agrees with the row that the packed forward pass
    gives for the same token, and the gradients with the formula's."""
    H, d, page, n = 2, 64, 16, 3
    prompts, steps = [32, 48], 5
    B = 2 * n
    g = torch.Generator(device="cuda").manual_seed(0)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q_all = [new(p + steps, H, d) for p in prompts for _ in range(n)]
    k_all, v_all = ([], [])
    for p in prompts:
        k0, v0 = new(p, H, d), new(p, H, d)
        for _ in range(n):
            k_all.append(torch.cat((k0, new(steps, H, d))))
            v_all.append(torch.cat((v0, new(steps, H, d))))
    width = 6000  # (room for more than 128 MB, so that the shared path runs)
    blocks = 64
    kc, vc = (torch.zeros(blocks, page, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32)
    used = 0
    for i, p in enumerate(prompts):
        common = list(range(used, used + p // page))
        used += len(common)
        for b in range(i * n, (i + 1) * n):
            table[b, :len(common)] = torch.tensor(common)
            table[b, len(common)] = used
            used += 1
    table = table.cuda()
    prefix = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    for i, p in enumerate(prompts):  # the prompts' keys and values, once
        slots = (table[i * n, torch.arange(p, device="cuda") // page] * page + torch.arange(p, device="cuda") % page).int()
        fa.cache_append(q_all[i * n][:p], k_all[i * n][:p], v_all[i * n][:p], torch.arange(p, dtype=torch.int32, device="cuda"),
                        slots, None, kc, vc)
    sampled = []
    for t in range(steps):
        at = [prompts[b // n] + t for b in range(B)]
        slots = torch.tensor([int(table[b, a // page]) * page + a % page for b, a in enumerate(at)], dtype=torch.int32, device="cuda")
        take = lambda xs: torch.stack([x[a] for x, a in zip(xs, at)])  # noqa: E731
        q = fa.cache_append(take(q_all), take(k_all), take(v_all), torch.tensor(at, dtype=torch.int32, device="cuda"), slots,
                            None, kc, vc)
        lens = torch.tensor([a + 1 for a in at], dtype=torch.int32, device="cuda")
        sampled.append(torch.ops.fa91.attention_decode_shared(q, kc, vc, table, lens, prefix))
    lens = [x.shape[0] for x in q_all]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    x = [torch.cat(s).requires_grad_() for s in (q_all, k_all, v_all)]
    o, lse = torch.ops.fa91.attention_forward_varlen(*x, cu, cu, max(lens), True, None)
    at = cu.tolist()
    for t, (so, sl) in enumerate(sampled):
        for b in range(B):
            row = at[b] + prompts[b // n] + t
            # (each rounds its weights and its output to bf16: 2^-8 of what the weights' sum of |v| can be, each)
            most = max(1.0, float(v_all[b].float().abs().max()))
            assert (so[b].float() - o[row].float()).abs().max() <= 4 * 2.0 ** -8 * most
            assert (sl[b] - lse[:, row]).abs().max() <= 2.0 ** -14
    do = new(*o.shape)
    (o.float() * do.float()).sum().backward()
    for b in range(B):
        i = slice(at[b], at[b + 1])
        for h in range(H):
            want, bound = G.backward(*(f64(y[i, h]) for y in (do, *x, o)), f64(lse[h, i]), np.zeros(lens[b]), True, d ** -0.5)
            G.assert_gradients([f64(y.grad[i, h]) for y in x], want, bound)


def test_a_captured_step_that_accumulates_into_its_leaves(fa):
    """The usual recipe: ordinary steps on a side stream, their graphs dropped, then a captured one that accumulates."""
    x = [rand(2, 2, 260, 64, seed=i) for i in range(3)]

    def step():
        o, lse = torch.ops.fa91.attention_forward(*x, True, None)
        (o.float().square().sum() + lse.sum()).backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for t in x:
        t.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (40, 50):
        with torch.no_grad():
            for i, t in enumerate(x):
                t.copy_(rand(2, 2, 260, 64, seed=seed + i, grad=False))
                t.grad.zero_()
        graph.replay()
        y = [t.detach().clone().requires_grad_() for t in x]
        o, lse = torch.ops.fa91.attention_forward(*y, True, None)
        want = torch.autograd.grad(o.float().square().sum() + lse.sum(), y)
        for t, w in zip(x, want):
            assert torch.equal(t.grad, w)


@pytest.mark.parametrize("requests", [8, 400])
def test_captured_shared_decode(fa, requests):
    """Replays of two graphs (own workspaces) on two streams, on lengths, shared lengths and pages set before each replay;
    few requests (a cluster's blocks each) and many (equal runs and a join)."""
    H, d, page, width = 2, 64, 16, 1200
    kc, vc = (rand(1024, page, H, d, seed=s, grad=False) for s in (1, 2))
    q = rand(requests, 8, d, seed=3, grad=False)
    lens, prefix = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (requests, 2))
    table = torch.empty(requests, width, dtype=torch.int32, device="cuda")

    def fill(seed):
        g = torch.Generator().manual_seed(seed)
        p = torch.randint(0, 700, (2,), generator=g)
        t = torch.randint(0, 1024, (requests, width), generator=g)
        for i in range(2):
            rows = slice(i * requests // 2, (i + 1) * requests // 2)
            t[rows, :int(p[i]) // page] = t[rows.start, :int(p[i]) // page]
        table.copy_(t.int())
        prefix.copy_(p.int())
        lens.copy_(torch.randint(0, 900, (requests,), generator=g).int())

    fill(0)
    fa.attention_decode_shared(q, kc, vc, table, lens, prefix)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fa.attention_decode_shared(q, kc, vc, table, lens, prefix))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for seed in (1, 2, 3):
        fill(seed)
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        o, lse = fa.attention_decode_shared(q, kc, vc, table, lens, prefix)
        plain_o, plain_lse = fa.attention_decode_paged(q, kc, vc, table, lens)
        for got_o, got_lse in outs:
            assert torch.equal(got_o, o) and torch.equal(got_lse, lse)
        # (both round their weights and outputs to bf16)
        assert (o.float() - plain_o.float()).abs().max() <= 4 * 2.0 ** -8 * float(vc.float().abs().max())
        seen = plain_lse > -float("inf")
        assert torch.equal(seen, lse > -float("inf")) and (lse - plain_lse)[seen].abs().max() <= 2.0 ** -14
    assert fa.fa_device_status() == (0, 0)


FIRST = r"""
import torch
import exact_attention_91_gb300 as fa
z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
i = lambda *s: torch.ones(*s, dtype=torch.int32, device="cuda")
x = z(1, 2, 64, 64)
lse = torch.zeros(1, 2, 64, device="cuda")
ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
out = [z(1, 2, 64, 64) for _ in range(3)]
cache = z(64, 16, 2, 64)
q, o, table, lens, prefix = z(4, 2, 64), z(4, 2, 64), i(4, 20000), i(4), i(1)
c = fa.FaPagedCache(cache.data_ptr(), cache.data_ptr(), 0, 0, 2048, 128, 64, 2048, 128, 64, fa.CACHE_BF16, 64, 16, 2, 64)
def calls(s):
    p = x.data_ptr()
    return (fa.fa_bwd(p, p, p, p, p, lse.data_ptr(), 0, *(t.data_ptr() for t in out), 1, 2, 64, 64, 0.125, 0,
                      ws.data_ptr(), ws.numel(), s),
            fa.fa_decode_shared(q.data_ptr(), c, table.data_ptr(), lens.data_ptr(), prefix.data_ptr(), o.data_ptr(), 0,
                                4, 2, 1, 20000, 20000, 0.125, ws.data_ptr(), ws.numel(), s))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    print("first", *calls(torch.cuda.current_stream().cuda_stream))
    x.add_(0)
fa.fa_bwd(*[x.data_ptr()] * 5, lse.data_ptr(), 0, *(t.data_ptr() for t in out), 1, 2, 64, 64, 0.125, 0, ws.data_ptr(),
          ws.numel(), None)
# (an ordinary call of one serving entry point stands for all of them)
fa.cache_append(z(1, 2, 64), z(1, 2, 64), z(1, 2, 64), i(1), i(1), None, cache, z(64, 16, 2, 64))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    print("then", *calls(torch.cuda.current_stream().cuda_stream))
graph.replay()
torch.cuda.synchronize()
print(fa.fa_device_status())
"""


def test_captures_before_any_ordinary_call_are_refused(fa):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, PYTHONPATH=root + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "first -7 -7" in r.stdout and "then 0 0" in r.stdout and "(0, 0)" in r.stdout, r.stdout


def test_operators_hold_their_registrations(fa):
    x = [rand(1, 2, 100, 64, seed=i) for i in range(3)]
    y = [t.detach() for t in x]
    o, lse = fa.attention_forward(*y, causal=True)
    cu = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    p = [rand(100, 2, 64, seed=i) for i in range(3)]
    po, pl = fa.attention_forward_varlen(*(t.detach() for t in p), cu, cu, 60, causal=True)
    cache = rand(8, 16, 2, 64, seed=3, grad=False)
    table = torch.zeros(4, 4, dtype=torch.int32, device="cuda")
    lens, prefix = torch.full((4,), 20, dtype=torch.int32, device="cuda"), torch.full((2,), 16, dtype=torch.int32, device="cuda")
    ops = torch.ops.fa91
    for op, args in ((ops.attention_forward, (*x, True, None)),
                     (ops.attention_forward_varlen, (*p, cu, cu, 60, True, None)),
                     (ops.attention_backward, (y[0], *y, o, lse, True, None, lse.clone())),
                     (ops.attention_backward_varlen, (po, *(t.detach() for t in p), po, pl, cu, cu, 60, 60, True, None, None)),
                     (ops.attention_decode_shared, (rand(4, 4, 64, seed=4, grad=False), cache, cache, table, lens, prefix))):
        torch.library.opcheck(op.default, args, test_utils=("test_schema", "test_autograd_registration", "test_faketensor"))
    with pytest.raises(RuntimeError):  # (no second derivatives: an error, not zeros)
        o, _ = ops.attention_forward(*x, True, None)
        g, = torch.autograd.grad(o.float().square().sum(), x[0], create_graph=True)
        g.float().sum().backward()
