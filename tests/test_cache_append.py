"""Rotary positions with the append to a paged cache (fa_cache_append) against
the 64-bit form: both cache types and orders, padding, slices, in place."""
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


def make(T, hq, hkv, d, page, e4m3, head_first=False, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    blocks = -(-T // page) + 2
    t = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    shape = (blocks, hkv, page, d) if head_first else (blocks, page, hkv, d)
    caches = [torch.randn(shape, generator=g).to(t).cuda() for _ in range(2)]
    if head_first:
        caches = [c.permute(0, 2, 1, 3) for c in caches]
    qkv = torch.randn(T, hq + 2 * hkv, d, generator=g).bfloat16().cuda()
    slots = torch.randperm(blocks * page, generator=g)[:T].int()
    where = torch.randperm(T, generator=g)[:pad]
    slots[where] = -1
    scales = [(0.02 + 0.1 * torch.rand(hkv, generator=g)).cuda() if e4m3 else None for _ in range(2)]
    return dict(qkv=qkv, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], slots=slots.cuda(),
                pos=torch.randint(0, 100000, (T,), generator=g).int().cuda(), kc=caches[0], vc=caches[1],
                ks=scales[0], vs=scales[1])


def check(x, before, freq, interleaved, q_out, k_out=None, factor=1.0):
    """Every value of the caches and outputs, the untouched ones bit for bit."""
    f = np.zeros(0) if freq is None else freq.cpu().numpy()
    pos = x["pos"].cpu().numpy()
    far = float(np.abs(pos).max())
    page = x["kc"].shape[1]
    slots = x["slots"].cpu().numpy()
    real = (slots >= 0) & (slots < x["kc"].shape[0] * page)
    for src, got in ((before["q"], q_out), (before["k"], k_out)):
        if got is None:
            continue
        y, mag = so.turn(so.f64(src).transpose(1, 0, 2), pos, f, interleaved, factor)
        b = so.turn_bound(y, mag, far)
        b[mag == 0] = 0
        d = np.abs(so.f64(got).transpose(1, 0, 2) - y)[:, real]
        assert np.all(d <= b[:, real])
    for cache, old, src, scale, turned in ((x["kc"], before["kc"], before["k"], x["ks"], True),
                                           (x["vc"], before["vc"], before["v"], x["vs"], False)):
        y, mag = so.f64(src).transpose(1, 0, 2), np.zeros(1)
        if turned:
            y, mag = so.turn(y, pos, f, interleaved, factor)
            fine = mag * (2.0 ** -20 + far * 2.0 ** -50)
        else:
            fine = np.zeros_like(y)
        if cache.dtype == torch.float8_e4m3fn:
            s = np.ones(y.shape[0]) if scale is None else so.f64(scale)
            # the reciprocal and the product: 2^-24 each
            y, fine = y / s[:, None, None], fine / s[:, None, None] + np.abs(y / s[:, None, None]) * 2.0 ** -22
            lo, hi = np.clip(y - fine, -448, 448), np.clip(y + fine, -448, 448)
            half = np.maximum(so.E4M3_HALF * np.maximum(np.abs(lo), np.abs(hi)), so.E4M3_TINY)
            lo, hi = lo - half, hi + half
        else:
            half = so.BF16_HALF * np.abs(y)
            lo, hi = y - fine - half, y + fine + half
            if not turned:
                lo = hi = y
        got, was = so.f64(cache), so.f64(old)
        seen = np.zeros(got.shape[:2], bool)
        seen[slots[real] // page, slots[real] % page] = True
        np.testing.assert_array_equal(got[~seen], was[~seen])
        g = got[slots[real] // page, slots[real] % page].transpose(1, 0, 2)
        assert np.all((g >= lo[:, real]) & (g <= hi[:, real]))


def snapshot(x):
    out = {n: x[n].clone() for n in ("q", "k", "v")}
    for n in ("kc", "vc"):
        out[n] = x[n].clone() if x[n].dtype == torch.bfloat16 else x[n].view(torch.uint8).clone().view(x[n].dtype)
    return out


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,r,page,head_first,pad", [
    (1, 1, 1, 64, 64, 16, False, 0),
    (1, 32, 8, 128, 128, 16, False, 0),
    (7, 3, 3, 64, 32, 32, True, 2),
    (50, 10, 2, 128, 128, 64, True, 5),
    (33, 9, 1, 128, 48, 16, False, 33),
    (700, 8, 4, 128, 0, 128, False, 1),
    (6001, 2, 1, 64, 64, 16, False, 100),
])
def test_append(T, hq, hkv, d, r, page, head_first, pad, e4m3, interleaved):
    fa = _fa()
    x = make(T, hq, hkv, d, page, e4m3, head_first, pad, seed=T)
    before = snapshot(x)
    freq = fa.rotary_inv_freq(r, device="cuda")[0] if r else None
    k_out = torch.full((T, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    q_out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    back = fa.cache_append(x["q"], x["k"], x["v"], x["pos"], x["slots"], freq, x["kc"], x["vc"],
                           interleaved=interleaved, factor=1.5, k_scale=x["ks"], v_scale=x["vs"], q_out=q_out, k_out=k_out)
    assert back is q_out
    check(x, before, freq, interleaved, q_out, k_out, factor=1.5)
    gone = x["slots"] < 0                                   # padding: left as it was
    assert (q_out[gone] == 7).all() and (k_out[gone] == 7).all()
    assert torch.equal(x["qkv"], torch.cat([before[n] for n in "qkv"], 1))
    q2 = fa.cache_append(x["q"], x["k"], x["v"], x["pos"], x["slots"], freq, x["kc"], x["vc"],
                         interleaved=interleaved, factor=1.5, k_scale=x["ks"], v_scale=x["vs"])
    assert torch.equal(q2[~gone], q_out[~gone])


def test_in_place_over_slices_of_one_buffer():
    fa = _fa()
    freq = fa.rotary_inv_freq(128, device="cuda")[0]
    x, y = (make(40, 6, 2, 128, 16, False, seed=3) for _ in range(2))
    k_out = torch.empty(40, 2, 128, dtype=torch.bfloat16, device="cuda")
    q = fa.cache_append(x["q"], x["k"], x["v"], x["pos"], x["slots"], freq, x["kc"], x["vc"], k_out=k_out)
    fa.cache_append(y["q"], y["k"], y["v"], y["pos"], y["slots"], freq, y["kc"], y["vc"], q_out=y["q"], k_out=y["k"])
    assert torch.equal(y["q"], q) and torch.equal(y["k"], k_out) and torch.equal(y["v"], x["v"])
    assert torch.equal(x["kc"], y["kc"]) and torch.equal(x["vc"], y["vc"])


def test_slots_outside_the_cache_write_nothing():
    fa = _fa()
    x = make(8, 2, 1, 64, 16, False, seed=4)
    n = x["kc"].shape[0] * 16
    x["slots"] = torch.tensor([n, -1, 2 ** 31 - 1, -2 ** 31, 3, n - 1, n + 1, 17], dtype=torch.int32).cuda()
    before = snapshot(x)
    q_out = torch.full((8, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.cache_append(x["q"], x["k"], x["v"], x["pos"], x["slots"], None, x["kc"], x["vc"], q_out=q_out)
    check(x, before, None, False, q_out)
    assert (q_out[[0, 1, 2, 3, 6]] == 7).all() and torch.equal(q_out[[4, 5, 7]], x["q"][[4, 5, 7]])


def test_e4m3_rounding_saturation_and_nan():
    """Every bf16 value through the 8-bit cache, scale 1 and 0.37."""
    fa = _fa()
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16).reshape(1024, 1, 64).cuda()
    slots = torch.arange(1024, dtype=torch.int32).cuda()
    for scale in (None, 0.37):
        s = None if scale is None else torch.full((1,), scale, device="cuda")
        kc, vc = (torch.zeros(64, 16, 1, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        fa.cache_append(v, v, v, slots, slots, None, kc, vc, k_scale=s, v_scale=s)
        x = so.f64(v).reshape(-1) / (1.0 if s is None else float(s.cpu().double()))
        for c in (kc, vc):
            got = so.f64(c).reshape(-1)
            np.testing.assert_array_equal(np.isnan(got), np.isnan(x))
            ok = ~np.isnan(x)
            with np.errstate(over="ignore"):
                t = np.clip(x[ok], -448, 448)
            half = np.maximum(so.E4M3_HALF * np.abs(t), so.E4M3_TINY) * (1 + 2.0 ** -20)
            assert np.all(np.abs(got[ok] - t) <= half)
            if scale is None:
                # scale 1: torch's own rounding of the clamped value
                w = v.float().clamp(-448, 448).to(torch.float8_e4m3fn)
                np.testing.assert_array_equal(got[ok], so.f64(w).reshape(-1)[ok])


def test_keys_and_values_side_by_side_and_large_offsets():
    """k and v of one tensor, in blocks past 2^31 elements."""
    fa = _fa()
    kv = torch.empty(9000, 2, 16, 64, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    assert kv.numel() > 2 ** 31
    kc, vc = kv[:, 0, :, :2], kv[:, 1, :, 5:7]
    x = make(5, 4, 2, 128, 16, True, seed=6)
    x["slots"] = torch.tensor([8999 * 16 + 15, 8998 * 16, 3, 8999 * 16, 8500 * 16 + 7], dtype=torch.int32).cuda()
    small = dict(x)
    fa.cache_append(x["q"], x["k"], x["v"], x["pos"], x["slots"], None, kc, vc, k_scale=x["ks"], v_scale=x["vs"])
    small["slots"] = torch.arange(5, dtype=torch.int32).cuda()
    fa.cache_append(x["q"], x["k"], x["v"], x["pos"], small["slots"], None, x["kc"], x["vc"], k_scale=x["ks"], v_scale=x["vs"])
    for big, ref in ((kc, x["kc"]), (vc, x["vc"])):
        for i, s in enumerate(x["slots"].tolist()):
            assert torch.equal(big[s // 16, s % 16].view(torch.uint8), ref[0, i].view(torch.uint8))


def test_no_tokens():
    fa = _fa()
    x = make(1, 2, 1, 64, 16, False, seed=7)
    q = fa.cache_append(x["q"][:0], x["k"][:0], x["v"][:0], x["pos"][:0], x["slots"][:0], None, x["kc"], x["vc"])
    assert q.shape == (0, 2, 64)
