"""Plain 64-bit forms of the serving operators (numpy, one request, token or
page at a time), and the error bounds that the tests hold the kernels to.

Nothing here is shared with the CUDA library or with the plain forms of the
measured cases.
"""
import math

import numpy as np

BF16_HALF = 2.0 ** -8     # largest rounding error of bf16, relative
E4M3_HALF = 2.0 ** -4     # of e4m3, relative, for normal values (2^-6 on)
E4M3_TINY = 2.0 ** -10    # half of e4m3's smallest step


def f64(t):
    """A torch tensor of any float type, exactly, as fp64 numpy."""
    import torch
    return t.detach().cpu().to(torch.float32).numpy().astype(np.float64)


def decode(q, k, v, table, lens, scale, ks=None, vs=None):
    """(O, LSE, A, S): q [B, Hq, d]; k, v [blocks, page, heads, d]; A is
    softmax(s) |v| and S the largest scale·Σ|q||k| of a row's visible keys, which
    scale the error bounds."""
    B, Hq, d = q.shape
    blocks, page, heads, _ = k.shape
    G = Hq // heads
    o, a = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    lse, big = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        pos = np.arange(n)
        block = table[b][pos // page]
        seen = (block >= 0) & (block < blocks)
        block, tok = block[seen], (pos % page)[seen]
        if not len(block):
            continue
        for h in range(heads):
            kk, vv = k[block, tok, h], v[block, tok, h]
            if ks is not None:
                kk = kk * ks[h]
            if vs is not None:
                vv = vv * vs[h]
            for i in range(h * G, (h + 1) * G):
                s = scale * (kk @ q[b, i])
                top = s.max()
                p = np.exp(s - top)
                lse[b, i] = top + math.log(p.sum())
                p /= p.sum()
                o[b, i], a[b, i] = p @ vv, p @ np.abs(vv)
                big[b, i] = scale * (np.abs(kk) @ np.abs(q[b, i])).max()
    return o, lse, a, big


def assert_decode(o, lse, want, one_p=False):
    """A score is off by at most big·2^-19: the products are exact in fp32, and
    the D <= 128 additions and the two factors (q·k's scale and log2 e) lose at
    most 2^-23 of the sum of magnitudes each in ~12 steps. A weight is then off
    by twice that (numerator and denominator), by the exponential (2^-22), the
    two-part rounding of P (2^-16) and the fp32 sums (below 2^-15 for these
    lengths, in units of A); O is rounded to bf16 once. ``one_p`` (9 to 16 query
    heads per key head over an e4m3 cache): P is rounded to fp16 alone, 2^-11."""
    o_ref, lse_ref, a, big = want
    assert o.shape == o_ref.shape and lse.shape == lse_ref.shape
    none = np.isneginf(lse_ref)
    np.testing.assert_array_equal(np.isneginf(lse), none)
    assert np.all(o[none] == 0.0)
    off = big * 2.0 ** -19
    rest = 2.0 ** -14 + (2.0 ** -11 if one_p else 0.0)
    bound = BF16_HALF * np.abs(o_ref) + a * (2 * off[..., None] + rest) * (1 + BF16_HALF) + 2.0 ** -133
    d = np.abs(o - o_ref)
    assert np.all(d <= bound), (float((d / bound).max()), np.unravel_index((d / bound).argmax(), d.shape))
    with np.errstate(invalid="ignore"):
        dl = np.where(none, 0.0, np.abs(lse - lse_ref))
    lb = off + 2.0 ** -18 + np.where(none, 0.0, np.abs(lse_ref)) * 2.0 ** -22
    assert np.all(dl <= lb), float((dl / lb).max())


def turn(x, positions, inv_freq, interleaved, factor=1.0, inverse=False):
    """x [..., n, d] (positions broadcast to [..., n]) with its pairs turned, and
    for each value |x1| + |x2| of its pair (0 where it is copied)."""
    r = 2 * len(inv_freq)
    y, mag = x.copy(), np.zeros_like(x)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        ang = np.asarray(positions, np.float64) * f
        c, s = factor * np.cos(ang), factor * np.sin(ang) * (-1.0 if inverse else 1.0)
        x1, x2 = x[..., a], x[..., b]
        y[..., a], y[..., b] = x1 * c - x2 * s, x2 * c + x1 * s
        mag[..., a] = mag[..., b] = factor * (np.abs(x1) + np.abs(x2))
    return y, mag


def turn_bound(y, mag, positions_max):
    """fp32: the angle (2^-29 and the position's share), sincospi (2^-22 of 1),
    the factor and two products (2^-24 each); then one rounding to bf16."""
    return BF16_HALF * np.abs(y) + mag * (2.0 ** -20 + positions_max * 2.0 ** -50) * (1 + BF16_HALF)


def page_maps(context, fresh, table, unused, page, T):
    """The step taken one token after the other: (table, slots, positions, cu,
    lens, counts)."""
    table = [list(row) for row in table]
    width = len(table[0])
    slots, positions, cu, lens = [], [], [0], []
    taken = missing = beyond = 0
    for row, c, n in zip(table, context, fresh):
        c, n = max(int(c), 0), max(int(n), 0)
        held = -(-c // page)
        for pos in range(c, c + n):
            col = pos // page
            if col < width and col >= held and (pos % page == 0 or pos == c):
                if taken < len(unused):
                    row[col] = int(unused[taken])
                    taken += 1
                else:
                    row[col] = -1
                    missing += 1
            slots.append(row[col] * page + pos % page if col < width and row[col] >= 0 else -1)
            positions.append(pos)
        cu.append(cu[-1] + n)
        lens.append(c + n)
        beyond += c + n > width * page
    total = len(slots)
    slots, positions = (slots + [-1] * T)[:T], (positions + [0] * T)[:T]
    return table, slots, positions, cu, lens, [taken, missing, total, beyond]
