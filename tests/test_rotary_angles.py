"""The angles of the rotary operators: pairs chosen so that a turned value is next
to nothing, and what is left of it is the error of its cos and sin."""
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


PI = 31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679
TURN = 2 * PI * 2 ** 200 // 10 ** 100          # 2 pi, scaled by 2^200


def angle_of(position, freq):
    """position · freq less whole turns, from integers (freq >= 2^-7: a multiple of 2^-60)."""
    x = (position * int(freq * 2.0 ** 60) << 140) % TURN
    return (x if 2 * x < TURN else x - TURN) / 2 ** 200


def nearly_turned_away(c, s):
    """bf16 (x1, x2) with x1 c - x2 s next to nothing: of 128 lengths, the best."""
    best = None
    for m in range(128, 256):
        one = np.full_like(c, m / 128)
        with np.errstate(divide="ignore", invalid="ignore"):
            x1 = np.where(np.abs(s) <= np.abs(c), to_bf16(one * s / c), one)
            x2 = np.where(np.abs(s) <= np.abs(c), one, to_bf16(one * c / s))
        left = np.abs(x1 * c - x2 * s)
        if best is None:
            best = [left, x1, x2]
        else:
            less = left < best[0]
            best = [np.where(less, a, b) for a, b in zip((left, x1, x2), best)]
    return best[1], best[2]


def to_bf16(x):
    return torch.from_numpy(np.nan_to_num(x)).bfloat16().double().numpy()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("span", [64, 131072, 2 ** 31 - 1])
def test_cos_and_sin_are_off_by_little(interleaved, span):
    """cos and sin off by 2^-24 and the angle by |position|·2^-59 + 2^-30, as
    fa.h states; the products and their sum round by 2^-24 of the pair at most."""
    fa = _fa()
    g = np.random.default_rng(span)
    N, d = 2000, 64
    freq = np.sort(g.uniform(0.01, 1.0, 32))
    pos = g.integers(-span if span > 64 else 0, span, N)
    angle = np.array([[angle_of(int(p), float(f)) for f in freq] for p in pos])
    c, s = np.cos(angle), np.sin(angle)
    x1, x2 = nearly_turned_away(c, s)
    x = np.zeros((2, N, d))
    first, second = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    x[0, :, first], x[0, :, second] = x1, x2                              # y1 = x1 c - x2 s
    x[1, :, first], x[1, :, second] = x2, -x1                             # y2 = x2' c + x1' s = -x1 c + x2 s
    y = fa.rotary(torch.from_numpy(x)[None].bfloat16().cuda(), torch.from_numpy(pos).int().cuda(),
                  torch.from_numpy(freq).cuda(), interleaved=interleaved)
    y = so.f64(y)[0]
    want = x1 * c - x2 * s
    size = np.abs(x1) + np.abs(x2)
    off = 2.0 ** -24 + 2.0 ** -30 + np.abs(pos)[:, None] * 2.0 ** -59
    bound = size * off + (np.abs(x1 * c) + np.abs(x2 * s)) * 2.0 ** -25 + so.BF16_HALF * np.abs(want)
    for got, ref in ((y[0][:, first], want), (y[1][:, second], -want)):
        worst = (np.abs(got - ref) / bound).max()
        assert worst <= 1.0, worst
