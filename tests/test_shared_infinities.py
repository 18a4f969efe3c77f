"""Infinities in visible values behind a shared prefix: O is what the definition gives, as of paged decode, for few
requests (clusters) and many (equal runs and a join), in shared and in own keys; who does not see them has none."""
import math

import pytest

import exact_attention_91_gb300 as fa

from . import serve_oracle as so
from .test_decode_shared import call, check, make, want

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("where", ["shared", "own"])
@pytest.mark.parametrize("hq,hkv,d,own", [(8, 2, 64, [5, 40, -30, 300]), (4, 4, 128, [1, 17, None, 200]),
                                          (16, 8, 128, [1 + i % 70 for i in range(40)]), (40, 1, 64, [33] * 140)])
def test_infinite_values_stay_infinite(hq, hkv, d, own, where):
    x = make([320, 144], own, hq, hkv, d, 16, seed=hq + d)
    table, lens = x["table"].cpu().numpy(), x["lens"].cpu().numpy()
    n, plus, minus, both = len(own), 3, 5, d - 1
    clean = want(x)
    v = x["v"].clone()
    hit = []  # requests that see the values (placed in the first group's prefix, or behind it in its first request)
    if where == "shared":
        for at, sign in ((2, 1), (200, -1)):  # (of the prefix's 320 tokens: two of its key tiles)
            v[int(table[0, at // 16]), at % 16, :, both] = sign * math.inf
        v[int(table[0, 200 // 16]), 200 % 16, :, plus] = math.inf
        v[int(table[0, 319 // 16]), 15, :, minus] = -math.inf
        hit = [b for b in range(n) if lens[b] >= 320]
    else:
        last = int(lens[0]) - 1
        assert last >= 320
        v[int(table[0, last // 16]), last % 16, :, plus] = math.inf
        v[int(table[0, last // 16]), last % 16, :, minus] = -math.inf
        v[int(table[0, last // 16]), last % 16, :, both] = -math.inf
        v[int(table[0, 0]), 0, :, both] = math.inf
        hit = [0]
    o, lse = call(dict(x, v=v))
    assert hit and torch.isposinf(o[hit][..., plus].float()).all() and torch.isneginf(o[hit][..., minus].float()).all()
    assert torch.isnan(o[hit][..., both].float()).all()
    assert fa.fa_device_status() == (0, 0)
    # (a request that is shorter than the prefix sees some of them in the marked columns; it is not looked at there)
    # all other columns, and the second group whole, are as without them
    cols = [c for c in range(d) if c not in (plus, minus, both)]
    check((o[..., cols], lse), (clean[0][..., cols], clean[1], clean[2][..., cols], clean[3]))
    check((o[n:], lse[n:]), tuple(t[n:] for t in clean))
