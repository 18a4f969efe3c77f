"""Many sequences of at most one tile of queries or keys: work items whose second query tile has no key, or none at all,
run many to a block. Every wait ends, and rows without a key are written."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_91_gb300 as fa
    fa.fa_device_status()
    return fa


def reference(q, k, v, causal, scale):
    """O and LSE in 64 bits; q [.., Nq, d], k, v [.., Nk, d]."""
    s = scale * q.double() @ k.double().transpose(-1, -2)
    if causal:
        s = s.masked_fill(~torch.ones_like(s, dtype=torch.bool).tril(s.shape[-1] - s.shape[-2]), -float("inf"))
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse > -float("inf"), lse, 0.0)[..., None])
    return p @ v.double(), lse


def check(o, lse, want_o, want_lse, v):
    seen = want_lse > -float("inf")
    assert torch.equal(lse > -float("inf"), seen) and (o[~seen] == 0).all()
    assert (lse.double() - want_lse)[seen].abs().max() <= 1e-3
    # (P and O rounded to bf16: half a step each, of at most the largest |v|)
    assert (o.double() - want_o)[seen].abs().max() <= 2 * 2.0 ** -8 * float(v.abs().max())


@pytest.mark.parametrize("B,H,N", [(58, 20, 2), (31, 20, 13), (169, 8, 60), (80, 16, 128), (40, 16, 200)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_equal_lengths(fa, B, H, N, d, causal):
    g = torch.Generator(device="cuda").manual_seed(B + N)
    q, k, v = (torch.randn(B, H, N, d, generator=g, device="cuda").bfloat16() for _ in range(3))
    for _ in range(3):
        o, lse = fa.attention_forward(q, k, v, causal=causal)
        assert fa.fa_device_status() == (0, 0)
        check(o, lse, *reference(q, k, v, causal, d ** -0.5), v)


@pytest.mark.parametrize("lo,hi,klo,khi", [(1, 128, 1, 128), (0, 500, 0, 6), (0, 40, 0, 700), (1, 1, 1, 300)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_packed(fa, lo, hi, klo, khi, d, causal):
    r = np.random.default_rng(hi + khi)
    B, H = 60, 16
    nq, nk = r.integers(lo, hi + 1, B), r.integers(klo, khi + 1, B)
    cu = [torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda") for n in (nq, nk)]
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (torch.randn(int(n.sum()), H, d, generator=g, device="cuda").bfloat16() for n in (nq, nk, nk))
    o, lse = (torch.full_like(t, float("nan")) for t in (q, torch.empty(H, q.shape[0], device="cuda")))
    o, lse = fa.attention_forward_varlen(q, k, v, *cu, int(nq.max()), causal=causal, out=o, lse=lse)
    assert fa.fa_device_status() == (0, 0)
    a, b = (c.tolist() for c in cu)
    for i in range(B):
        qi, ki = slice(a[i], a[i + 1]), slice(b[i], b[i + 1])
        if a[i] == a[i + 1]:
            continue
        if b[i] == b[i + 1]:
            assert (o[qi] == 0).all() and (lse[:, qi] == -float("inf")).all()
            continue
        want = reference(q[qi].transpose(0, 1), k[ki].transpose(0, 1), v[ki].transpose(0, 1), causal, d ** -0.5)
        check(o[qi].transpose(0, 1), lse[:, qi], *want, v[ki])
