"""How many bits a weight keeps on its way into P V of the paged decode. The
values are made to cancel, so that O is next to nothing and what is left of it
is the error of the weights, not bf16's rounding."""
import math

import numpy as np
import pytest

from . import serve_oracle as so
from .test_decode_paged import _fa, call

torch = pytest.importorskip("torch")

LOG2E = np.float32(1.4426950408889634)


def to_bf16(x):
    return torch.as_tensor(np.asarray(x, np.float64)).bfloat16().double().numpy()


def to_e4m3(x):
    return torch.as_tensor(np.asarray(x, np.float64)).float().to(torch.float8_e4m3fn).float().double().numpy()


def two_part_error(p, cut):
    """Relative error of p (fp32) as the sum of two 16-bit values."""
    hi = cut(p)
    return (hi + cut(p - hi) - p) / p


def pick(e4m3):
    """Scores of a tile's keys: one above the others (weight 1), then keys whose
    weights two bf16 parts (one fp16 part) give too large and too small by the
    most, in turn, then keys to cancel with."""
    grid = np.unique((to_e4m3 if e4m3 else to_bf16)(np.linspace(-0.7, -0.02, 4001)))
    p = np.exp2(grid * float(LOG2E)).astype(np.float32).astype(np.float64)
    if e4m3:
        err = (p.astype(np.float16).astype(np.float64) - p) / p
    else:
        err = two_part_error(p, to_bf16)
    order = np.argsort(err)
    high, low = grid[order[::-1][:3]], grid[order[:3]]
    return [0.0, *high, *low, -0.5, -0.25, -0.125, -0.375, -0.4375], err[order[-3]], err[order[2]]


def cancelling_values(scores, d, cut):
    """v [keys, d]: column by column one key of either kind, and four that take up
    what their rounded values leave; 64-bit weights."""
    p = np.exp(np.asarray(scores))
    v = np.zeros((len(scores), d))
    for c in range(d):
        a, b = 1 + c % 3, 4 + c // 3 % 3
        v[a, c] = cut(128.0 * (1 + (c % 8) / 8) * (-1) ** c)
        left = p[a] * v[a, c]
        for key in (b, 7, 8, 9, 10):
            v[key, c] = cut(-left / p[key])
            left += p[key] * v[key, c]
    return v


def test_the_chosen_keys_err():
    """What the cases rest on: two bf16 parts lose 2^-18 of such a weight, one
    fp16 part 2^-12; O cancels."""
    for e4m3, size in ((False, 0.7 * 2.0 ** -18), (True, 0.7 * 2.0 ** -12)):
        scores, high, low = pick(e4m3)
        assert high > size and low < -size
        v = cancelling_values(scores, 128, to_e4m3 if e4m3 else to_bf16)
        p = np.exp(np.asarray(scores))
        assert np.all(np.abs(p @ v) <= 2.0 ** -15 * (p @ np.abs(v)))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,width", [(1, None), (8, None), (9, None), (16, None), (20, None), (3, 5000), (16, 5000)])
def test_weights_keep_the_bits_of_fp32(d, e4m3, hq, width):
    """All keys are of one warp's tile. A weight is off by ex2's 2^-22, the
    exponent's rounding (below 1 in size: 2^-25) and that of scale and log2 e
    (2^-24); a tensor-core step's sum of 16 products by less than 2^-21 of the sum
    of their magnitudes; so O by 2^-20 of A = softmax |v| in all, and by its own
    rounding. (Two bf16 parts: 2^-18.4 of A; one fp16 part: 2^-12.4.)"""
    fa = _fa()
    cut = to_e4m3 if e4m3 else to_bf16
    scores, _, _ = pick(e4m3)
    n, t = len(scores), torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k, v = torch.zeros(2, 16, 1, d), torch.zeros(2, 16, 1, d)
    k[1, :n, 0, 0] = torch.tensor(scores)
    v[1, :n, 0] = torch.from_numpy(cancelling_values(scores, d, cut)).float()
    q = torch.zeros(1, hq, d)
    q[:, :, 0] = 1.0
    table = torch.full((1, width or 1), -1, dtype=torch.int32)
    table[0, 0] = 1
    x = dict(q=q.bfloat16().cuda(), k=k.to(t).cuda(), v=v.to(t).cuda(), table=table.cuda(),
             lens=torch.tensor([n], dtype=torch.int32).cuda(), ks=None, vs=None)
    o, lse = call(fa, x, scale=1.0)
    o_ref, lse_ref, a, _ = so.decode(so.f64(x["q"]), so.f64(x["k"]), so.f64(x["v"]), table.numpy(), [n], 1.0)
    assert np.all(so.BF16_HALF * np.abs(o_ref) <= 2.0 ** -22 * a)        # next to nothing
    bound = 2.0 ** -20 * a + so.BF16_HALF * np.abs(o_ref)
    off = np.abs(so.f64(o) - o_ref)
    assert np.all(off <= bound), float((off / bound).max())
    assert np.all(np.abs(so.f64(lse) - lse_ref) <= 2.0 ** -20)
    assert math.isfinite(off.sum())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 1), (16, 1), (64, 4)])
def test_long_sums_are_rounded_not_cut(d, e4m3, hq, hkv):
    """v is 1 for the first half of 16384 keys and -1 for the second, which has the
    same scores in another order: O is 0, and the sum on its way there climbs to
    half of A = 1 (times the keys' weight) and comes back. As many requests as blocks,
    so that each takes a whole one. Rounded to nearest, at most 1024 additions
    are off by 2^-25 of A each (half a step of a sum below A/2) in either direction:
    2^-21.8 at one sigma of their uniform errors, here 2^-19 (seven). Cut towards
    zero, one step of a matrix instruction loses 2^-25 in the mean, always of the
    same sign: 2^-15 of A and more.

    LSE: a lane adds up its tiles' sums one after the other, each addition off by at
    most 2^-24 of a sum that is half of the last one in the mean, so by tiles·2^-25
    in all; the tile's own sum, the exponential, the logarithm and the rounding of an
    LSE below 16 make up less than 2^-20."""
    fa = _fa()
    n, page = 16384, 64
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(d + hq)
    half = torch.rand(n // 2, generator=g) * -0.7
    scores = torch.cat((half, half[torch.randperm(n // 2, generator=g)]))
    t = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k, v = torch.zeros(n, hkv, d), torch.ones(n, hkv, d)
    k[:, :, 0] = scores[:, None].bfloat16().float()
    v[n // 2:] = -1.0
    k, v = (x.view(n // page, page, hkv, d).to(t).cuda() for x in (k, v))
    q = torch.zeros(B, hq, d)
    q[:, :, 0] = 1.0
    table = torch.arange(n // page, dtype=torch.int32).expand(B, -1).contiguous()       # all over the same pages
    x = dict(q=q.bfloat16().cuda(), k=k, v=v, table=table.cuda(), lens=torch.full((B,), n, dtype=torch.int32).cuda(),
             ks=None, vs=None)
    o, lse = call(fa, x, scale=1.0)
    assert o.float().abs().max().item() <= 2.0 ** -19
    s = so.f64(k).reshape(n, hkv, d)[:, 0, 0]
    tiles = n * d * k.element_size() // 4096
    assert np.abs(so.f64(lse) - math.log(np.exp(s).sum())).max() <= tiles * 2.0 ** -25 + 2.0 ** -20

@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (16, 1), (64, 4)])
@pytest.mark.parametrize("above", [14, 18, 20, 22, 24])
def test_small_weights_beside_a_dominant_one(d, hq, hkv, above):
    """The first key of each warp's run is `above` (natural) higher than the other
    16000, which share one score, and has no value: O is the others' sum alone. A
    weight's parts are fp16, biased by 2^7, the second one scaled by 2^12: its
    rounding is off by at most half of fp16's smallest step, 2^-25-12-7 = 2^-44 of
    the largest weight, and all are equal, so they are off alike. (Not scaled:
    2^-32, a tenth of such a weight at 20 and all of it at 24.)"""
    fa = _fa()
    keys, page = 4096 // d, 64
    n = 4 * keys * (16000 // (4 * keys))
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    k, v = torch.zeros(n, hkv, d), torch.full((n, hkv, d), 2.0)
    first = slice(0, 1) if hkv == 4 else slice(0, 4 * keys, keys)       # four warps share one head's tiles
    k[first, :, 0] = float(above)
    v[first] = 0.0
    k, v = (x.view(n // page, page, hkv, d).to(torch.float8_e4m3fn).cuda() for x in (k, v))
    q = torch.zeros(B, hq, d)
    q[:, :, 0] = 1.0
    table = torch.arange(n // page, dtype=torch.int32).expand(B, -1).contiguous()
    x = dict(q=q.bfloat16().cuda(), k=k, v=v, table=table.cuda(), lens=torch.full((B,), n, dtype=torch.int32).cuda(),
             ks=None, vs=None)
    o, lse = call(fa, x, scale=1.0)
    many = 1 if hkv == 4 else 4
    total = many + (n - many) * math.exp(-above)
    want = 2 * (n - many) * math.exp(-above) / total
    # The exponent is below 2^6 in size: its rounding is 2^-19 of a weight. The row's sum has its full size from the
    # first tile on: each of the others, added to it, is rounded by 2^-24 of it at most, all alike. The LSE: that, and
    # m (below 2^6: 2^-19 with its factor's rounding), its sum with the logarithm (2^-19) and the product with ln 2
    # (2^-19 in all), times ln 2: below 2^-18.
    tiles = n / keys
    bound = so.BF16_HALF * want + 2 * n * 2.0 ** -44 / total + want * (2.0 ** -18 + tiles * 2.0 ** -24)
    off = np.abs(so.f64(o) - want).max()
    assert off <= bound * (1 + so.BF16_HALF), off / bound
    assert np.abs(so.f64(lse) - (above + math.log(total))).max() <= 2.0 ** -18 + tiles * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,width", [(1, None), (8, 3000), (16, None), (20, 3000)])
@pytest.mark.parametrize("size", [2.0 ** -100, 1.0, 2.0 ** 100, 2.0 ** 127])
@pytest.mark.parametrize("below", [1, 13, 16, 20])
def test_small_values_of_q_over_an_e4m3_cache(d, hq, width, size, below):
    """q's largest value meets keys that are zero there; the one that counts is about
    2^below smaller and has all of bf16's bits. Its products are exact; the factor of
    scale and log2 e and the exponent round by 2^-24 of the score each, m and the LSE
    by 2^-23 of it in all; the rest of either as in the tests above."""
    fa = _fa()
    k, v = torch.zeros(2, 16, 1, d), torch.zeros(2, 16, 1, d)
    k[1, 0, 0, 1], k[1, 1, 0, 1] = 448.0, 416.0
    v[1, 0, 0], v[1, 1, 0] = 1.0, 2.0
    q = torch.zeros(1, hq, d, dtype=torch.float64)
    q[:, :, 0] = size
    q[:, :, 1] = size * 2.0 ** -below * (1 + 127 / 128)
    q = q.bfloat16()
    little = q[0, 0, 1].double().item()
    scale = float(np.float32(max(12.0 / (448.0 * little), 2.0 ** -125)))
    table = torch.full((1, width or 1), -1, dtype=torch.int32)
    table[0, 0] = 1
    t = torch.float8_e4m3fn
    x = dict(q=q.cuda(), k=k.to(t).cuda(), v=v.to(t).cuda(), table=table.cuda(),
             lens=torch.tensor([2], dtype=torch.int32).cuda(), ks=None, vs=None)
    o, lse = call(fa, x, scale=scale)
    s = np.array([448.0, 416.0]) * little * scale
    w = np.exp(s - s.max())
    want, size = (w[0] + 2 * w[1]) / w.sum(), s.max() + math.log(w.sum())
    off = s.max() * 2.0 ** -22 + 2.0 ** -20
    assert np.abs(so.f64(o) - want).max() <= want * (so.BF16_HALF + 2 * off)
    assert np.abs(so.f64(lse) - size).max() <= off, np.abs(so.f64(lse) - size).max() / off
