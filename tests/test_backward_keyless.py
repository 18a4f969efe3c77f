"""A query that sees no key adds nothing to any gradient and has dQ = 0, whatever the gradient of its LSE (minus
infinity) is: what a loss on LSE leaves there is often no number."""
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


# (queries, keys), causal: the first queries of each see nothing, in whole blocks of 128 and beside others
COUNTS = [(300, 5), (200, 150), (7, 0), (130, 2), (257, 129), (60, 60)]


def make(d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nq, nk = ([c[i] for c in COUNTS] for i in (0, 1))
    cu_q, cu_k = (torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda") for n in (nq, nk))
    new = lambda n: torch.randn(n, 2, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    return (new(sum(nq)), new(sum(nk)), new(sum(nk))), new(sum(nq)), cu_q, cu_k


def check(x, do, cu_q, cu_k, o, lse, dlse, grads, d):
    """The oracle leaves queries without a key out by their LSE; their dLSE enters it as zero."""
    q, k, v = x
    a, b = cu_q.tolist(), cu_k.tolist()
    for s in range(len(COUNTS)):
        i, j = slice(a[s], a[s + 1]), slice(b[s], b[s + 1])
        for h in range(2):
            none = np.isneginf(f64(lse[h, i]))
            assert none.sum() == max(0, COUNTS[s][0] - COUNTS[s][1])
            dl = np.where(none, 0.0, f64(dlse[h, i]))
            want, bound = G.backward(f64(do[i, h]), f64(q[i, h]), f64(k[j, h]), f64(v[j, h]), f64(o[i, h]),
                                     f64(lse[h, i]), dl, True, d ** -0.5)
            got = [f64(grads[0][i, h]), f64(grads[1][j, h]), f64(grads[2][j, h])]
            G.assert_gradients(got, want, bound)
            assert (got[0][none] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("there", [float("-inf"), float("inf"), float("nan"), 3e38])
def test_gradients_of_lse_without_a_key(fa, d, there):
    x, do, cu_q, cu_k = make(d, 1)
    o, lse = fa.attention_forward_varlen(*x, cu_q, cu_k, 300, causal=True)
    dlse = torch.randn(lse.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    dlse[lse == -float("inf")] = there
    grads = fa.attention_backward_varlen(do, *x, o, lse, cu_q, cu_k, 300, 150, causal=True, dlse=dlse)
    check(x, do, cu_q, cu_k, o, lse, dlse, grads, d)
    assert fa.fa_device_status() == (0, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_a_loss_on_the_square_of_lse(fa, d):
    """The usual way to leave out rows without a key: the gradient that comes back for them is 0 times infinity."""
    x, do, cu_q, cu_k = make(d, 3)
    y = [t.requires_grad_() for t in x]
    o, lse = torch.ops.fa91.attention_forward_varlen(*y, cu_q, cu_k, 300, True, None)
    lse.retain_grad()
    z = torch.where(lse > -float("inf"), lse ** 2, 0.0).sum()
    ((o.float() * do.float()).sum() + z).backward()
    assert torch.isnan(lse.grad).any()
    check(x, do, cu_q, cu_k, o, lse, lse.grad, [t.grad for t in y], d)
