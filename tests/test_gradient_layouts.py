"""Gradients as autograd hands them back reach the backward kernels wherever they start: a slice of a larger gradient is
contiguous, but begins at any element."""
import numpy as np
import pytest

from . import grad_oracle as G

torch = pytest.importorskip("torch")


def f64(t):
    return t.detach().cpu().double().numpy()


def test_dense_gradients_start_on_a_boundary():
    from exact_attention_91_gb300 import torch_op
    whole = torch.arange(100).bfloat16()
    for at in range(9):
        part = whole[at:at + 64]
        got = torch_op._dense(part)
        assert got.is_contiguous() and got.data_ptr() % 16 == 0 and torch.equal(got, part)
    assert torch_op._dense(whole) is whole  # (nothing is copied that need not be)
    assert torch_op._dense(torch.ones(()).expand(4, 6)).is_contiguous()
    assert torch_op._dense(torch.empty(0, 2, 64)).shape == (0, 2, 64)


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_91_gb300 as fa
    from exact_attention_91_gb300 import torch_op  # noqa: F401
    return fa


def rand(*shape, seed, grad=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16().requires_grad_(grad)


def joined(*parts):
    """A loss on tensors laid end to end: each gradient is a slice of one, at the offset of its part."""
    flat = torch.cat([p.flatten().float() if p.dtype != torch.bfloat16 else p.flatten() for p in parts])
    w = rand(flat.numel(), seed=99, grad=False)
    return (flat.float() * w.float()).sum(), w


@pytest.mark.gpu
@pytest.mark.parametrize("head", [0, 1, 3, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_equal_lengths(fa, d, head):
    x = [rand(2, 2, 130, d, seed=i) for i in range(3)]
    extra = rand(head, seed=7)
    o, lse = torch.ops.fa91.attention_forward(*x, True, None)
    loss, w = joined(extra, o)
    loss.backward()
    do = w[head:].view_as(o)
    for b in range(2):
        for h in range(2):
            want, bound = G.backward(*(f64(t[b, h]) for t in (do, *x, o, lse)), np.zeros(130), True, d ** -0.5)
            G.assert_gradients([f64(t.grad[b, h]) for t in x], want, bound)


@pytest.mark.gpu
def test_lse_in_a_slice(fa):
    x = [rand(1, 2, 130, 64, seed=i) for i in range(3)]
    extra = rand(3, seed=7).float()
    o, lse = torch.ops.fa91.attention_forward(*x, False, None)
    flat = torch.cat([extra, lse.flatten()])
    w = rand(flat.numel(), seed=9, grad=False).float()
    (flat * w).sum().backward()
    dlse = w[3:].view_as(lse)
    for h in range(2):
        want, bound = G.backward(np.zeros((130, 64)), *(f64(t[0, h]) for t in (*x, o, lse, dlse)), False, 0.125)
        G.assert_gradients([f64(t.grad[0, h]) for t in x], want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("head", [1, 5])
def test_packed(fa, head):
    lens = [70, 200]
    cu = torch.tensor([0, 70, 270], dtype=torch.int32, device="cuda")
    x = [rand(270, 2, 64, seed=i) for i in range(3)]
    extra = rand(head, seed=7)
    o, lse = torch.ops.fa91.attention_forward_varlen(*x, cu, cu, 200, True, None)
    loss, w = joined(extra, o)
    loss.backward()
    do = w[head:].view_as(o)
    for b in range(2):
        i = slice(sum(lens[:b]), sum(lens[:b + 1]))
        for h in range(2):
            want, bound = G.backward(*(f64(t[i, h]) for t in (do, *x, o)), f64(lse[h, i]), np.zeros(lens[b]), True, 0.125)
            G.assert_gradients([f64(t.grad[i, h]) for t in x], want, bound)


@pytest.mark.gpu
def test_compiled(fa):
    """The compiled backward pass is traced once, and meets gradients that start elsewhere."""
    x = [rand(1, 2, 64, 64, seed=i) for i in range(3)]
    step = torch.compile(lambda q, k, v: torch.ops.fa91.attention_forward(q, k, v, True, None)[0], fullgraph=True,
                         backend="aot_eager")
    for head in (0, 3):
        for t in x:
            t.grad = None
        o = step(*x)
        loss, w = joined(rand(head, seed=7), o)
        loss.backward()
        lse = torch.ops.fa91.attention_forward(*(t.detach() for t in x), True, None)[1]
        for h in range(2):
            do = w[head:].view_as(o)
            want, bound = G.backward(*(f64(t[0, h]) for t in (do, *x, o, lse)), np.zeros(64), True, 0.125)
            G.assert_gradients([f64(t.grad[0, h]) for t in x], want, bound)
