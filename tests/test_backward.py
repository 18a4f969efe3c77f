"""Attention's backward pass (equal-length and packed) against 64-bit gradients."""
import ctypes
import shutil

import numpy as np
import pytest

import exact_attention_91_gb300 as fa
from exact_attention_91_gb300 import build as fa_build

from . import grad_oracle as G

torch = pytest.importorskip("torch")
P = 1 << 26  # an aligned fake address; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not fa_build.up_to_date():
        if shutil.which(fa_build.nvcc_path()) is None:
            pytest.skip("nvcc not available to build libfa.so")
        fa_build.build()
    return fa.load_library()


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- without a GPU ----------------------------------------------------------


@pytest.mark.parametrize("nq,nk,causal", [(5, 5, True), (4, 7, True), (7, 4, True), (3, 6, False), (1, 1, True)])
def test_oracle_matches_differences(nq, nk, causal):
    """The formula's gradients of Σ O·dO + Σ LSE·dLSE against central differences."""
    rng = np.random.default_rng(nq * 10 + nk)
    q, k, v, do = (rng.normal(size=(n, 6)) for n in (nq, nk, nk, nq))
    seen = G.visible(nq, nk, causal).any(1)
    dlse = rng.normal(size=nq) * seen
    scale = 0.4

    def loss(q, k, v):
        o, lse = G.forward(q, k, v, causal, scale)
        return (o * do).sum() + (np.where(seen, lse, 0) * dlse).sum()

    o, lse = G.forward(q, k, v, causal, scale)
    grads, _ = G.backward(do, q, k, v, o, lse, dlse, causal, scale)
    for which, x in enumerate((q, k, v)):
        for at in np.ndindex(x.shape):
            h = 1e-5
            args = [q.copy(), k.copy(), v.copy()]
            args[which][at] += h
            up = loss(*args)
            args[which][at] -= 2 * h
            num = (up - loss(*args)) / (2 * h)
            assert abs(num - grads[which][at]) < 1e-7 * (1 + abs(num))


def bwd(dout=P, q=2 * P, k=3 * P, v=4 * P, o=5 * P, lse=6 * P, dlse=7 * P, dq=8 * P, dk=9 * P, dv=10 * P, B=2, H=2,
        N=100, d=64, scale=0.125, ws=11 * P, ws_bytes=2 * 2 * 100 * 4 + 16):
    return fa.fa_bwd(dout, q, k, v, o, lse, dlse, dq, dk, dv, B, H, N, d, scale, True, ws, ws_bytes, None)


COMMON = [
    (dict(dout=0), -1), (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(o=0), -1), (dict(lse=0), -1),
    (dict(dq=0), -1), (dict(dk=0), -1), (dict(dv=0), -1), (dict(B=0), -2), (dict(H=0), -2), (dict(d=96), -3),
    (dict(scale=0.0), -9), (dict(scale=float("nan")), -9), (dict(scale=float("inf")), -9),
    (dict(q=2 * P + 8), -4), (dict(dout=P + 2), -4), (dict(dq=8 * P + 4), -4), (dict(dv=10 * P + 8), -4),
    (dict(lse=6 * P + 2), -4), (dict(dlse=7 * P + 1), -4), (dict(ws=11 * P + 8), -4),
    (dict(dq=2 * P), -10), (dict(dk=8 * P), -10), (dict(dv=5 * P + 16), -10), (dict(dq=P), -10), (dict(ws=6 * P), -10),
    (dict(ws=9 * P + 16), -10), (dict(dk=7 * P), -10), (dict(ws=0), -11), (dict(ws_bytes=800), -11),
]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(N=0), -2), (dict(B=1 << 16, H=1 << 15), -2),
                                              (dict(B=1 << 12, H=1 << 12, N=1 << 20), -2)])
def test_bad_calls_are_rejected(kw, code):
    assert bwd(**kw) == code


def test_a_call_without_a_device_or_a_gradient_of_lse():
    if not torch.cuda.is_available():
        assert bwd() == bwd(dlse=0) == bwd_varlen() == bwd_varlen(dlse=0) == -5


def bwd_varlen(dout=P, q=2 * P, k=3 * P, v=4 * P, o=5 * P, lse=6 * P, dlse=7 * P, dq=8 * P, dk=9 * P, dv=10 * P,
               cu_q=12 * P, cu_k=13 * P, B=2, H=2, total_q=100, total_k=120, max_q=60, max_k=120, d=64, scale=0.125,
               ws=11 * P, ws_bytes=2 * 100 * 4 + 16):
    return fa.fa_bwd_varlen(dout, q, k, v, o, lse, dlse, dq, dk, dv, cu_q, cu_k, B, H, total_q, total_k, max_q, max_k, d,
                            scale, True, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(cu_q=0), -1), (dict(cu_k=0), -1), (dict(total_q=-1), -2), (dict(total_k=-1), -2), (dict(max_q=101), -2),
    (dict(max_k=121), -2), (dict(max_q=-1), -2), (dict(max_k=-1), -2), (dict(cu_q=12 * P + 2), -4),
    (dict(cu_k=13 * P + 1), -4), (dict(dq=12 * P), -10), (dict(dv=13 * P), -10), (dict(ws=12 * P), -10),
    (dict(B=1 << 16, H=1 << 15), -2),
])
def test_bad_packed_calls_are_rejected(kw, code):
    assert bwd_varlen(**kw) == code


def test_workspace_sizes():
    assert fa.fa_bwd_workspace(1000, 3) == 12016
    assert fa.fa_bwd_workspace(1, 1) == 32
    assert fa.fa_bwd_workspace(0, 4) == 16
    for bad in ((-1, 1), (1, 0), (1 << 41, 1)):
        assert fa.fa_bwd_workspace(*bad) == -2


# ---- on the GPU -------------------------------------------------------------


def make(B, H, N, d, causal, seed, scale=None, spread=1.0, dlse=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q, k, v, do = ((torch.randn(B, H, N, d, generator=g, device="cuda") * spread).bfloat16() for _ in range(4))
    scale = scale or d ** -0.5
    o = torch.empty_like(q)
    lse = torch.empty(B, H, N, device="cuda")
    for b in range(B):
        for h in range(H):
            oo, ll = G.forward(*(f64(x[b, h]) for x in (q, k, v)), causal, scale)
            o[b, h] = torch.from_numpy(oo).to("cuda").bfloat16()
            lse[b, h] = torch.from_numpy(ll).to("cuda").float()
    dl = torch.randn(B, H, N, generator=g, device="cuda") if dlse else None
    return dict(dout=do, q=q, k=k, v=v, out=o, lse=lse, causal=causal, scale=scale, dlse=dl)


def check(x, got):
    B, H = x["q"].shape[:2]
    for b in range(B):
        for h in range(H):
            dlse = f64(x["dlse"][b, h]) if x["dlse"] is not None else np.zeros(x["q"].shape[2])
            want, bound = G.backward(*(f64(x[n][b, h]) for n in ("dout", "q", "k", "v", "out", "lse")), dlse,
                                     x["causal"], x["scale"])
            G.assert_gradients([f64(t[b, h]) for t in got], want, bound)
    assert fa.fa_device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 127, 128, 129, 200, 256, 300, 511, 640, 1000])
def test_lengths(N, d, causal):
    x = make(1, 2, N, d, causal, N + d)
    check(x, fa.attention_backward(**x))


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,N,d,causal,kw", [
    (3, 5, 130, 64, True, dict(dlse=True)), (2, 3, 257, 128, True, dict(dlse=True)),
    (2, 17, 129, 64, False, dict(dlse=True)), (1, 40, 100, 128, False, {}),
    (1, 1, 513, 64, True, dict(spread=3.0)), (1, 1, 385, 128, False, dict(spread=3.0)),
    (1, 2, 200, 64, False, dict(scale=1.0)), (1, 2, 200, 128, True, dict(scale=0.01)),
])
def test_batches_scales_and_gradients_of_lse(B, H, N, d, causal, kw):
    x = make(B, H, N, d, causal, 7 * N + H, **kw)
    check(x, fa.attention_backward(**x))


def make_varlen(counts, H, d, causal, seed, pad=0, dlse=False):
    """Packed sequences of (queries, keys); `pad` rows of NaN behind the last."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cu_q, cu_k = (np.concatenate([[0], np.cumsum([c[i] for c in counts])]).astype(np.int32) for i in (0, 1))
    tq, tk = int(cu_q[-1]), int(cu_k[-1])
    rand = lambda n: torch.randn(n + pad, H, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, do, k, v = rand(tq), rand(tq), rand(tk), rand(tk)
    scale = d ** -0.5
    o = torch.zeros_like(q)
    lse = torch.zeros(H, tq + pad, device="cuda")
    for b, (nq, nk) in enumerate(counts):
        for h in range(H):
            i, j = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
            oo, ll = G.forward(f64(q[i, h]), f64(k[j, h]), f64(v[j, h]), causal, scale)
            o[i, h] = torch.from_numpy(oo).to("cuda").bfloat16()
            lse[h, i] = torch.from_numpy(ll).to("cuda").float()
    dl = torch.randn(H, tq + pad, generator=g, device="cuda") if dlse else None
    for t in (q, do, o):
        t[tq:] = float("nan")
    for t in (k, v):
        t[tk:] = float("nan")
    lse[:, tq:] = float("nan")
    at = lambda c: torch.from_numpy(c).cuda()  # noqa: E731
    return dict(dout=do, q=q, k=k, v=v, out=o, lse=lse, cu_seqlens_q=at(cu_q), cu_seqlens_k=at(cu_k),
                max_seqlen_q=max(c[0] for c in counts), max_seqlen_k=max(c[1] for c in counts), causal=causal,
                scale=scale, dlse=dl)


def check_varlen(x, got, skip=()):
    cu_q, cu_k = x["cu_seqlens_q"].tolist(), x["cu_seqlens_k"].tolist()
    for b in range(len(cu_q) - 1):
        if b in skip:
            continue
        i, j = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for h in range(x["q"].shape[1]):
            dlse = f64(x["dlse"][h, i]) if x["dlse"] is not None else np.zeros(i.stop - i.start)
            want, bound = G.backward(f64(x["dout"][i, h]), f64(x["q"][i, h]), f64(x["k"][j, h]), f64(x["v"][j, h]),
                                     f64(x["out"][i, h]), f64(x["lse"][h, i]), dlse, x["causal"], x["scale"])
            G.assert_gradients([f64(got[0][i, h]), f64(got[1][j, h]), f64(got[2][j, h])], want, bound)
    assert fa.fa_device_status() == (0, 0)


COUNTS = [
    [(1, 1)], [(128, 128), (128, 128)], [(5, 300), (300, 5), (0, 7), (7, 0), (0, 0), (1, 129)],
    [(130, 131), (1, 640), (257, 256), (64, 64)], [(700, 3), (3, 700)], [(33, 33)] * 40, [(0, 0), (0, 5)],
]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: str(c[:2]))
def test_packed(counts, d, causal):
    x = make_varlen(counts, 2, d, causal, len(counts) + d, dlse=len(counts) % 2 == 0)
    got = fa.attention_backward_varlen(**x)
    check_varlen(x, got)
    # loose bounds on the counts give the same bits
    again = fa.attention_backward_varlen(**x | dict(max_seqlen_q=x["q"].shape[0], max_seqlen_k=x["k"].shape[0]))
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_padding_rows_are_not_read_and_not_written(d):
    x = make_varlen([(200, 200), (70, 140), (129, 129)], 3, d, True, 5, pad=77, dlse=True)
    outs = [torch.full_like(x[n], 3.0) for n in ("q", "k", "v")]
    got = fa.attention_backward_varlen(**x, dq=outs[0], dk=outs[1], dv=outs[2])
    check_varlen(x, got)
    for t in got:
        assert (t[-77:] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_a_sequence_of_nan_stays_alone(d):
    x = make_varlen([(150, 150), (90, 60), (100, 200)], 2, d, False, 6)
    a, b = x["cu_seqlens_q"].tolist()[1:3]
    c, e = x["cu_seqlens_k"].tolist()[1:3]
    for n in ("q", "dout", "out"):
        x[n][a:b] = float("nan")
    for n in ("k", "v"):
        x[n][c:e] = float("inf")
    check_varlen(x, fa.attention_backward_varlen(**x), skip=(1,))


@pytest.mark.gpu
@pytest.mark.parametrize("d,causal", [(64, True), (128, False)])
def test_repeats_streams_and_given_buffers_give_the_same_bits(d, causal):
    x = make(2, 3, 300, d, causal, 9, dlse=True)
    want = fa.attention_backward(**x)
    side = torch.cuda.Stream()
    ws = torch.full((fa.fa_bwd_workspace(2 * 300, 3),), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.full_like(x["q"], float("nan")) for _ in range(3)]
    for kw in ({}, dict(stream=side), dict(dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)):
        got = fa.attention_backward(**x, **kw)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert got[0] is outs[0] and got[2] is outs[2]


@pytest.mark.gpu
@pytest.mark.parametrize("d,causal", [(64, False), (64, True), (128, False), (128, True)])
def test_more_units_than_sms(d, causal):
    """Units beyond the first of a block, in strides and by the counters; the workspace holds anything before a call."""
    x = make(3, 60, 130, d, causal, 11, dlse=True)
    ws = torch.full((fa.fa_bwd_workspace(3 * 130, 60),), 255, dtype=torch.uint8, device="cuda")
    got = fa.attention_backward(**x, workspace=ws)
    check(x, got)
    ws.fill_(1)
    for a, b in zip(fa.attention_backward(**x, workspace=ws), got):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("d,causal", [(64, False), (64, True), (128, True)])
def test_many_packed_sequences(d, causal):
    """More sequences than a warp has lanes, numbered through all of them, some of them empty; more units than SMs."""
    g = np.random.default_rng(d + causal)
    counts = [(int(a), int(b)) for a, b in zip(g.integers(0, 400, 70), g.integers(0, 300, 70))]
    counts[3], counts[40], counts[69] = (0, 0), (0, 90), (1, 1)
    counts[50] = (1100, 1300)
    x = make_varlen(counts, 4, d, causal, 12, dlse=True, pad=5)
    ws = torch.full((fa.fa_bwd_workspace(x["q"].shape[0], 4),), 255, dtype=torch.uint8, device="cuda")
    got = fa.attention_backward_varlen(**x, workspace=ws)
    check_varlen(x, got)
    for a, b in zip(fa.attention_backward_varlen(**x, workspace=ws), got):
        n = a.shape[0] - 5
        assert torch.equal(a[:n], b[:n])


@pytest.mark.gpu
def test_refusals_of_the_python_functions():
    x = make(1, 2, 64, 64, False, 3)
    with pytest.raises(TypeError):
        fa.attention_backward(**x | dict(q=x["q"].float()))
    with pytest.raises(TypeError):
        fa.attention_backward(**x | dict(lse=x["lse"].double()))
    for bad in (dict(k=x["k"][:, :1]), dict(dout=x["dout"].transpose(1, 2)), dict(lse=x["lse"][:, :1]),
                dict(dout=x["dout"].cpu()), dict(dlse=x["lse"][..., :3])):
        with pytest.raises(ValueError):
            fa.attention_backward(**x | bad)
    with pytest.raises(fa.FaError):
        fa.attention_backward(**x, dq=x["q"])
    with pytest.raises(fa.FaError):
        fa.attention_backward(**x, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fa.FaError):
        fa.attention_backward(**x | dict(scale=-1.0))
