"""A server's decode against its whole history: keys and values kept here in 64 bits,
rounded as the cache holds them, in the order of their positions (without tables,
slots or pages), under the bound of the decode alone. What the append wrote and what
the decode read must then be the same tokens' keys and values, at their scales."""
import math

import numpy as np
import pytest

from . import serve_oracle as so
from .test_serving import Server, _fa

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def held(y, fine, scale, got):
    """y as a cache holds it (its code times its scale): rounded to bf16, or to e4m3 over
    `scale`. Where y is known to `fine` only and that spans a border between two of
    them (or more: a pair turned to next to nothing), the one that the cache holds."""
    def to(z):
        t = torch.from_numpy(z if scale is None else np.clip(z / scale, -448, 448))
        if scale is None:
            return t.bfloat16().double().numpy()
        return t.float().to(torch.float8_e4m3fn).float().double().numpy() * scale
    low, high = to(y - fine), to(y + fine)
    assert np.mean(low != high) < 0.02                     # hardly ever
    return np.clip(got, low, high)


class Recorder(Server):
    """Keeps each request's keys and values as the cache should hold them."""

    def take(self, m, k, v, fresh):
        table = self.table.cpu().numpy()
        kc, vc, ks64, vs64 = so.f64(self.kc), so.f64(self.vc), so.f64(k), so.f64(v)
        s = None if self.ks is None else so.f64(self.ks)[:, None]
        at = 0
        for b, n in enumerate(fresh):
            for _ in range(n):
                pos = len(self.history[b])
                page, row = table[b, pos // self.page], pos % self.page
                turned, mag = so.turn(ks64[at][:, None], np.array([pos]), self.freq.cpu().numpy(), False, self.factor)
                # the angle and cos, sin (2^-24 each), the products and their sum
                fine = mag[:, 0] * (2.0 ** -22 + pos * 2.0 ** -50)
                one = 1.0 if s is None else s
                key = held(turned[:, 0], fine, s, kc[page, row] * one)
                value = held(vs64[at], 0.0, s, vc[page, row] * one)        # a quotient rounded to fp32: no doubt left
                np.testing.assert_array_equal(kc[page, row] * one, key)
                np.testing.assert_array_equal(vc[page, row] * one, value)
                self.history[b].append((key, value))
                at += 1

    def attend(self, b, q, keys=None, values=None):
        """(O, LSE, A, S) of one query [Hq, d] over request b's history."""
        k = np.stack([h[0] for h in self.history[b]]) if keys is None else keys
        v = np.stack([h[1] for h in self.history[b]]) if values is None else values
        n = len(k)
        return so.decode(q[None], k[None], v[None], np.zeros((1, 1), np.int64), [n], 1 / math.sqrt(self.d))


@pytest.mark.parametrize("hq,hkv,d,e4m3,width", [(4, 4, 64, False, 40), (8, 2, 128, False, 3000), (6, 3, 64, True, 40),
                                                 (24, 2, 128, True, 40), (8, 8, 128, True, 3000), (16, 1, 64, False, 40)])
def test_decode_is_attention_over_the_history(hq, hkv, d, e4m3, width):
    fa = _fa()
    s = Recorder(fa, 4, hq, hkv, d, width=width, e4m3=e4m3, seed=d + hq)
    fresh = [37, 1, 130, 16]
    steps = [fresh] + [[1, 1, step % 2, 1] for step in range(5)] + [[0, 3, 20, 1]]
    checked = 0
    for fresh in steps:
        m = s.maps(fresh, pad=2)
        q, k, v = s.draw(sum(fresh) + 2)
        q_rot = s.append(m, q, k, v)
        s.take(m, k, v, fresh)
        ends = np.cumsum(fresh) - 1
        rows = [b for b, n in enumerate(fresh) if n]
        full = torch.zeros(4, hq, d, dtype=torch.bfloat16, device="cuda")
        for b in rows:
            full[b] = q_rot[ends[b]]
            pos = len(s.history[b]) - 1
            y, mag = so.turn(so.f64(q[ends[b]])[:, None], np.array([pos]), s.freq.cpu().numpy(), False, s.factor)
            want = held(y[:, 0], mag[:, 0] * (2.0 ** -22 + pos * 2.0 ** -50), None, so.f64(full[b]))
            np.testing.assert_array_equal(so.f64(full[b]), want)
        o, lse = fa.attention_decode_paged(full, s.kc, s.vc, s.table, s.lens, k_scale=s.ks, v_scale=s.vs)
        for b in rows:
            mine = so.f64(o[b:b + 1]), so.f64(lse[b:b + 1])
            so.assert_decode(*mine, s.attend(b, so.f64(full[b])))
            n = len(s.history[b])
            if n < 4:
                continue
            # and would not be, with two tokens' values or keys exchanged, one left out, or a scale of another size
            k, v = (np.stack([h[i] for h in s.history[b]]) for i in range(2))
            other = list(range(n))
            w = np.argsort(k[:, 0] @ so.f64(full[b])[0])
            other[w[-1]], other[w[0]] = other[w[0]], other[w[-1]]       # a key that counts, one that does not
            for wrong in (dict(values=v[other]), dict(keys=k[other]), dict(keys=k[other][:n - 1], values=v[:n - 1]),
                          dict(values=v * 1.03), dict(keys=k * 1.03)):
                with pytest.raises(AssertionError):
                    so.assert_decode(*mine, s.attend(b, so.f64(full[b]), **wrong))
            checked += 1
    assert checked > 5
