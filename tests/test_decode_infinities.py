"""Infinities in visible values of the paged decode: O is what the definition
gives, an infinity, and NaN only where two of opposite sign meet."""
import math

import numpy as np
import pytest

from . import serve_oracle as so
from .test_decode_paged import _fa, call, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,width", [(4, 4, None), (8, 1, None), (16, 1, None), (2, 1, 5000), (20, 1, 5000)])
def test_infinite_values_stay_infinite(d, hq, hkv, width):
    fa = _fa()
    lens = [1, 40, 333]
    x = make(lens, hq, hkv, d, 16, seed=d + hq, width=width)
    table = x["table"].cpu()
    plus, minus, both = 3, 5, d - 1                            # columns
    for b, n in enumerate(lens):
        # the key of the largest score (its weight is 1, exactly) and the last one
        s = so.f64(x["q"])[b, 0] @ so.f64(x["k"])[table[b, np.arange(n) // 16].numpy(), np.arange(n) % 16, 0].T
        keys = sorted({int(s.argmax()), n - 1})
        for j in keys:
            page, at = table[b, j // 16].item(), j % 16
            x["v"][page, at, :, plus] = math.inf
            x["v"][page, at, :, minus] = -math.inf
        x["v"][table[b, keys[0] // 16].item(), keys[0] % 16, :, both] = math.inf
        if n > 1:
            other = (keys[0] + 1) % n
            x["v"][table[b, other // 16].item(), other % 16, :, both] = -math.inf
    o, lse = call(fa, x)
    assert torch.isfinite(lse).all()
    assert torch.isposinf(o[..., plus].float()).all() and torch.isneginf(o[..., minus].float()).all()
    assert torch.isnan(o[1:, :, both].float()).all() and torch.isposinf(o[0, :, both].float()).all()
    rest = [c for c in range(d) if c not in (plus, minus, both)]
    want = so.decode(so.f64(x["q"]), so.f64(x["k"]), np.nan_to_num(so.f64(x["v"]), posinf=0.0, neginf=0.0), table.numpy(),
                     lens, 1 / math.sqrt(d))
    so.assert_decode(so.f64(o)[..., rest], so.f64(lse), (want[0][..., rest], want[1], want[2][..., rest], want[3]))
