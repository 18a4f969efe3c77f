"""Attention's gradients in 64 bits (numpy, one head at a time), and the error
bounds that the tests hold the backward kernels to. Nothing here is shared with
the CUDA library or with the plain forms of the measured cases.

Bounds, from the inputs as given (bf16 q, k, v, dO, O; fp32 LSE, dLSE). A score
is off by at most 2^-19 of scale·Σ|q||k|: its products are exact in fp32, and the
d <= 128 additions (cut towards zero by the tensor core) and the two factors lose
at most 2^-23 of the magnitudes' sum each in about 12 steps. The exponent adds the
rounding of LSE·log2 e and of the sum, 2^-22 of |LSE| and of |S|, and the exponential
2^-22. So P is off by a relative r = 2^-19 Σ|q||k| scale + 2^-22 (|LSE| + |S| + 1),
doubled for good measure, and by 2^-8 more once it is a bf16 operand. dP is off by
2^-19 Σ|dO||v|, δ by 2^-20 Σ|dO||O| + 2^-23 |dLSE|, and dS is rounded to bf16 too. A
sum of n products in fp32 loses at most n·2^-22 of the magnitudes' sum. The result
is rounded to bf16: 2^-8.
"""
import numpy as np

BF16_HALF = 2.0 ** -8


def visible(nq, nk, causal):
    i, j = np.arange(nq)[:, None], np.arange(nk)[None]
    return (j <= i + nk - nq) if causal else np.ones((nq, nk), bool)


def forward(q, k, v, causal, scale):
    """(O, LSE) of one head."""
    s = np.where(visible(len(q), len(k), causal), scale * (q @ k.T), -np.inf)
    top = s.max(1, initial=-np.inf)
    p = np.exp(s - np.where(np.isfinite(top), top, 0)[:, None])
    total = p.sum(1)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = np.where(total > 0, top + np.log(total), -np.inf)
    return p @ v / np.where(total > 0, total, 1)[:, None], lse


def backward(do, q, k, v, o, lse, dlse, causal, scale):
    """(dq, dk, dv) of one head and their error bounds, all in 64 bits."""
    see = visible(len(q), len(k), causal) & np.isfinite(lse)[:, None]
    s = scale * (q @ k.T)
    lse0 = np.where(np.isfinite(lse), lse, 0.0)
    p = np.where(see, np.exp(np.where(see, s - lse0[:, None], 0)), 0.0)
    delta = (do * o).sum(1) - dlse
    dp = do @ v.T
    ds = p * (dp - delta[:, None])
    dq, dk, dv = scale * (ds @ k), scale * (ds.T @ q), p.T @ do

    r = 2 * (2.0 ** -19 * scale * (np.abs(q) @ np.abs(k).T) + 2.0 ** -22 * (np.abs(lse0)[:, None] + np.abs(s) + 1))
    e_dp = 2.0 ** -19 * (np.abs(do) @ np.abs(v).T)
    e_delta = 2.0 ** -20 * (np.abs(do) * np.abs(o)).sum(1) + 2.0 ** -22 * np.abs(dlse) + 2.0 ** -22 * np.abs(delta)
    e_ds = p * (1 + r) * (e_dp + e_delta[:, None] + (np.abs(dp) + np.abs(delta)[:, None]) * 2.0 ** -22) + r * np.abs(ds)
    e_ds = e_ds * (1 + BF16_HALF) + BF16_HALF * np.abs(ds)
    e_p = p * (r + BF16_HALF * (1 + r))
    n = max(len(q), len(k)) * 2.0 ** -22
    tiny = 1e-30
    b_dv = (e_p + n * p).T @ np.abs(do) + BF16_HALF * np.abs(dv) + tiny
    b_dq = scale * ((e_ds + n * np.abs(ds)) @ np.abs(k)) * 1.01 + BF16_HALF * np.abs(dq) + tiny
    b_dk = scale * ((e_ds + n * np.abs(ds)).T @ np.abs(q)) * 1.01 + BF16_HALF * np.abs(dk) + tiny
    # (the result's own rounding is of the value with its error)
    return (dq, dk, dv), tuple(b * (1 + BF16_HALF) for b in (b_dq, b_dk, b_dv))


def assert_gradients(got, want, bound):
    for name, g, w, b in zip(("dq", "dk", "dv"), got, want, bound):
        assert np.isfinite(g).all(), name
        off = np.abs(g - w)
        worst = float((off / b).max()) if off.size else 0.0
        assert worst <= 1.0, f"{name}: {worst:.3g} of the bound, largest error {off.max():.3g}"
