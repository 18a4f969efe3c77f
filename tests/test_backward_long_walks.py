"""Backward passes whose units walk hundreds of tiles: ring positions, barrier phases and claims far beyond a few rounds.
Some rows' and some keys' gradients against 64-bit ones."""
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
    return fa


def f64(t):
    return t.detach().cpu().double().numpy()


def some(n, seed):
    """Rows of the first, the last and other blocks of 128."""
    r = np.random.default_rng(seed)
    picked = np.concatenate([[0, 1, 127, 128, n // 2, n - 129, n - 128, n - 1], r.integers(0, n, 24)])
    return np.unique(picked[(picked >= 0) & (picked < n)])


def check_head(monkeypatch, do, q, k, v, o, lse, dlse, got, causal, scale, seed):
    """One head: dQ of some queries over all keys, dK and dV of some keys over all queries. (The oracle takes the mask
    from `visible`.)"""
    nq, nk = len(q), len(k)
    rows, keys = some(nq, seed), some(nk, seed + 1)
    see = lambda i, j: (j[None] <= i[:, None] + nk - nq) if causal else np.ones((len(i), len(j)), bool)  # noqa: E731
    with monkeypatch.context() as m:
        m.setattr(G, "visible", lambda *a: see(rows, np.arange(nk)))
        want, bound = G.backward(do[rows], q[rows], k, v, o[rows], lse[rows], dlse[rows], causal, scale)
        G.assert_gradients([got[0][rows]], want[:1], bound[:1])
        m.setattr(G, "visible", lambda *a: see(np.arange(nq), keys))
        want, bound = G.backward(do, q, k[keys], v[keys], o, lse, dlse, causal, scale)
        # (the sums of dQ are not looked at: here they are over these keys alone)
        assert np.isfinite(got[1]).all() and np.isfinite(got[2]).all()
        for g, w, b in zip(got[1:], want[1:], bound[1:]):
            off = np.abs(g[keys] - w)
            assert (off <= b).all(), float((off / b).max())


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_equal_lengths(fa, monkeypatch, d, causal):
    g = torch.Generator(device="cuda").manual_seed(d)
    q, k, v, do = (torch.randn(1, 3, 16384, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    dlse = torch.randn(1, 3, 16384, generator=g, device="cuda")
    o, lse = fa.attention_forward(q, k, v, causal=causal)
    got = fa.attention_backward(do, q, k, v, o, lse, causal=causal, dlse=dlse)
    assert fa.fa_device_status() == (0, 0)
    for h in (0, 2):
        check_head(monkeypatch, *(f64(t[0, h]) for t in (do, q, k, v, o, lse, dlse)), [f64(t[0, h]) for t in got], causal,
                   d ** -0.5, h)
    for a, b in zip(fa.attention_backward(do, q, k, v, o, lse, causal=causal, dlse=dlse), got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_packed_queries_and_keys_of_their_own_counts(fa, monkeypatch, d, causal):
    counts = [(300, 30001), (20001, 40), (1, 25000), (9000, 9001)]
    g = torch.Generator(device="cuda").manual_seed(d + 1)
    nq, nk = ([c[i] for c in counts] for i in (0, 1))
    at = [np.concatenate([[0], np.cumsum(n)]) for n in (nq, nk)]
    cu = [torch.tensor(a, dtype=torch.int32, device="cuda") for a in at]
    new = lambda n: torch.randn(n, 2, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, do, k, v = new(sum(nq)), new(sum(nq)), new(sum(nk)), new(sum(nk))
    o, lse = fa.attention_forward_varlen(q, k, v, *cu, max(nq), causal=causal)
    got = fa.attention_backward_varlen(do, q, k, v, o, lse, *cu, max(nq), max(nk), causal=causal)
    assert fa.fa_device_status() == (0, 0)
    for b, (n, m) in enumerate(counts):
        i, j = slice(at[0][b], at[0][b + 1]), slice(at[1][b], at[1][b + 1])
        h = b % 2
        check_head(monkeypatch, f64(do[i, h]), f64(q[i, h]), f64(k[j, h]), f64(v[j, h]), f64(o[i, h]), f64(lse[h, i]),
                   np.zeros(n), [f64(got[0][i, h]), f64(got[1][j, h]), f64(got[2][j, h])], causal, d ** -0.5, b)
