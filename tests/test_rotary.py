"""Rotary positions (fa_rotary, torch.ops.fa91.rotary) against the 64-bit form:
both pair layouts, parts of the head, strides, far positions, the gradient."""
import math

import numpy as np
import pytest

from . import serve_oracle as so

torch = pytest.importorskip("torch")


def _fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_91_gb300 as fa
    return fa


def _check(fa, x, positions, freq, got, **kw):
    """x and got are [B, H, N, d] or [T, H, d]."""
    xs, gs = so.f64(x), so.f64(got)
    pos = positions.cpu().numpy()
    if x.dim() == 3:
        xs, gs = xs.transpose(1, 0, 2)[None], gs.transpose(1, 0, 2)[None]
    pos = pos[:, None] if pos.ndim == 2 else pos
    y, mag = so.turn(xs, pos, np.zeros(0) if freq is None else freq.cpu().numpy(), **kw)
    bound = so.turn_bound(y, mag, float(np.abs(pos.astype(np.float64)).max()))
    bound[mag == 0] = 0.0                                  # copied values are exact
    d = np.abs(gs - y)
    assert np.all(d <= bound), float((d / np.maximum(bound, 1e-300)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,r", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 112), (64, 0)])
def test_layouts_and_parts_of_the_head(interleaved, d, r):
    fa = _fa()
    g = torch.Generator().manual_seed(r)
    freq, _ = fa.rotary_inv_freq(r, device="cuda")
    for shape in ((2, 3, 37, d), (1, 1, 1, d), (3, 9, 5, d)):
        x = torch.randn(shape, generator=g).bfloat16().cuda()
        pos = torch.randint(0, 4096, (shape[0], shape[2]), generator=g).int().cuda()
        for inverse in (False, True):
            y = fa.rotary(x, pos, freq if r else None, interleaved=interleaved, inverse=inverse, factor=1.25)
            _check(fa, x, pos, freq, y, interleaved=interleaved, inverse=inverse, factor=1.25)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 1), (3, 40), (77, 5), (9001, 2)])
def test_token_major(T, H):
    fa = _fa()
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, 128, generator=g).bfloat16().cuda()
    pos = torch.randint(-5, 200000, (T,), generator=g).int().cuda()
    freq, _ = fa.rotary_inv_freq(128, 500000.0, device="cuda")
    _check(fa, x, pos, freq, fa.rotary(x, pos, freq), interleaved=False)


@pytest.mark.gpu
def test_far_and_extreme_positions():
    """Positions up to the int32 limits: the angle stays exact."""
    fa = _fa()
    pos = torch.tensor([0, 1, -1, 10 ** 6, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32).cuda()
    x = torch.ones(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    freq, _ = fa.rotary_inv_freq(64, device="cuda")
    _check(fa, x, pos, freq, fa.rotary(x, pos, freq, interleaved=True), interleaved=True)


@pytest.mark.gpu
def test_strides_and_in_place():
    fa = _fa()
    g = torch.Generator().manual_seed(5)
    freq, _ = fa.rotary_inv_freq(64, device="cuda")
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    qkv = torch.randn(50, 12, 128, generator=g).bfloat16().cuda()
    keep = qkv.clone()
    q = qkv[:, :7]                                          # slices of one projection
    y = fa.rotary(q, pos, freq)
    _check(fa, q, pos, freq, y, interleaved=False)
    fa.rotary(q, pos, freq, out=q)
    assert torch.equal(q, y) and torch.equal(qkv[:, 7:], keep[:, 7:])
    t = torch.randn(2, 50, 3, 128, generator=g).bfloat16().cuda().transpose(1, 2)   # [B, H, N, d] over [B, N, H, d]
    y = fa.rotary(t, pos, freq)
    assert y.is_contiguous()
    _check(fa, t, pos, freq, y, interleaved=False)
    one = torch.randn(1, 1, 50, 128, generator=g).bfloat16().cuda().expand(2, 3, 50, 128)   # a broadcast head
    _check(fa, one, pos, freq, fa.rotary(one, pos, freq), interleaved=False)


@pytest.mark.gpu
def test_special_values_stay_in_their_pair():
    fa = _fa()
    freq, _ = fa.rotary_inv_freq(64, device="cuda")
    pos = torch.tensor([3], dtype=torch.int32).cuda()
    x = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 5] = float("nan")
    y = fa.rotary(x, pos, freq)
    bad = torch.isnan(y[0, 0]).nonzero().flatten().tolist()
    assert bad == [5, 37]


@pytest.mark.gpu
def test_gradient_of_the_operator():
    """torch.ops.fa91.rotary: its gradient is the transposed map (within bf16's
    rounding of the 64-bit one), also of a head that is broadcast, and agrees
    with differences."""
    fa = _fa()
    from exact_attention_91_gb300 import torch_op  # noqa: F401
    g = torch.Generator().manual_seed(6)
    freq, factor = fa.rotary_inv_freq(32, device="cuda")
    pos = torch.arange(100, 140, dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        x = torch.randn(2, 3, 40, 64, generator=g).bfloat16().cuda().requires_grad_()
        dy = torch.randn(2, 3, 40, 64, generator=g).bfloat16().cuda()
        y = torch.ops.fa91.rotary(x, pos, freq, interleaved, False, 1.5)
        y.backward(dy)
        _check(fa, dy, pos, freq, x.grad, interleaved=interleaved, inverse=True, factor=1.5)
        # the map is linear: <dy, R e> - differences of the forward kernel - against <grad, e>
        e = torch.zeros_like(dy)
        e[1, 2, 7, 3] = 1.0
        e[1, 2, 7, 40] = 1.0
        up = torch.ops.fa91.rotary((x + e).detach(), pos, freq, interleaved, False, 1.5)
        diff = so.f64(dy) * (so.f64(up) - so.f64(y))
        step = so.f64((x + e).detach()) - so.f64(x)        # the step that bf16 kept
        err = so.BF16_HALF * (np.abs(so.f64(dy)) * (np.abs(so.f64(up)) + np.abs(so.f64(y)))).max(initial=0) * 4
        assert abs(diff.sum() - (so.f64(x.grad) * step).sum()) <= err + so.BF16_HALF * np.abs(so.f64(x.grad) * step).sum()
        # a key head shared by three query heads
        k = torch.randn(2, 1, 40, 64, generator=g).bfloat16().cuda().requires_grad_()
        y = torch.ops.fa91.rotary(k.expand(2, 3, 40, 64), pos, freq, interleaved, False, 1.5)
        y.backward(dy)
        each = so.turn(so.f64(dy), pos.cpu().numpy(), freq.cpu().numpy(), interleaved, 1.5, True)
        want = each[0].sum(1, keepdims=True)
        size = (np.abs(each[0]) + np.abs(want)).sum(1, keepdims=True)
        assert np.all(np.abs(so.f64(k.grad) - want) <= 4 * so.BF16_HALF * size + 2.0 ** -18 * each[1].sum(1, keepdims=True))


@pytest.mark.gpu
def test_operator_compiles_and_tracks_nothing_else():
    fa = _fa()
    from exact_attention_91_gb300 import torch_op  # noqa: F401
    freq, _ = fa.rotary_inv_freq(64, device="cuda")
    pos = torch.arange(10, dtype=torch.int32, device="cuda")
    x = torch.randn(10, 2, 64, device="cuda").bfloat16()
    y = torch.compile(lambda x: torch.ops.fa91.rotary(x, pos, freq, False, False, 1.0), fullgraph=True)(x)
    assert torch.equal(y, fa.rotary(x, pos, freq)) and not y.requires_grad


def test_operator_fake_shapes():
    from torch._subclasses.fake_tensor import FakeTensorMode

    from exact_attention_91_gb300 import torch_op  # noqa: F401
    with FakeTensorMode():
        x = torch.empty(2, 8, 100, 64, dtype=torch.bfloat16, device="meta")
        pos = torch.empty(100, dtype=torch.int32, device="meta")
        f = torch.empty(32, dtype=torch.float64, device="meta")
        y = torch.ops.fa91.rotary(x, pos, f, False, False, 1.0)
    assert y.shape == x.shape and y.dtype == torch.bfloat16 and y.is_contiguous()


# ---- frequencies (host) ------------------------------------------------------

def test_frequencies_and_scalings():
    import exact_attention_91_gb300 as fa
    f, factor = fa.rotary_inv_freq(64, 10000.0)
    np.testing.assert_allclose(f.numpy(), [10000.0 ** (-2 * i / 64) for i in range(32)], rtol=1e-14)
    assert factor == 1.0 and f.dtype == torch.float64
    lin, _ = fa.rotary_inv_freq(64, 10000.0, {"type": "linear", "factor": 4})
    np.testing.assert_allclose(lin.numpy(), f.numpy() / 4, rtol=1e-15)
    ntk, _ = fa.rotary_inv_freq(64, 10000.0, {"type": "ntk", "factor": 4})
    assert ntk[0] == 1.0 and abs(ntk[-1] / f[-1] - 0.25) < 1e-12
    bands, _ = fa.rotary_inv_freq(128, 500000.0, {"type": "bands", "factor": 8, "original": 8192, "low": 1, "high": 4})
    g, _ = fa.rotary_inv_freq(128, 500000.0)
    turns = 8192 * g / (2 * math.pi)
    np.testing.assert_allclose(bands[turns > 4].numpy(), g[turns > 4].numpy(), rtol=1e-15)
    np.testing.assert_allclose(bands[turns < 1].numpy(), g[turns < 1].numpy() / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((bands[mid] < g[mid]) & (bands[mid] > g[mid] / 8)).all()
    yarn, af = fa.rotary_inv_freq(128, 10000.0, {"type": "yarn", "factor": 16, "original": 4096})
    h, _ = fa.rotary_inv_freq(128, 10000.0)
    assert yarn[0] == h[0] and abs(yarn[-1] * 16 / h[-1] - 1) < 1e-12
    assert abs(af - (0.1 * math.log(16) + 1)) < 1e-12
    assert fa.rotary_inv_freq(128, 1e4, {"type": "yarn", "factor": 16, "original": 4096, "attention_factor": 2})[1] == 2
    assert fa.rotary_inv_freq(0)[0].numel() == 0
    for bad in (dict(rotary_dim=7), dict(rotary_dim=64, base=0.0), dict(rotary_dim=64, scaling={"type": "x", "factor": 2}),
                dict(rotary_dim=64, scaling={"type": "linear", "factor": 0}),
                dict(rotary_dim=64, scaling={"type": "bands", "factor": 2, "original": 0}),
                dict(rotary_dim=64, scaling={"type": "yarn", "factor": 2, "original": 8, "low": 5, "high": 4})):
        with pytest.raises(ValueError):
            fa.rotary_inv_freq(**bad)
