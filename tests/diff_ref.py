"""The rotated append and differential attention in 64 bits, for the tests, written from
their definitions, and the tolerances that count the kernels' roundings.

A rounding to bf16 is off by at most 2^-8 of the value, to E4M3 by 2^-4 (below its normal
range by half a step, 2^-10 of the scale); fp32 sums are taken to be within 2^-18 of the
sum of magnitudes."""
import math

import numpy as np

from fp8_block_ref import block_scale


# --------------------------------------------------------------------- append --
def bf16_tol(y, tol):
    """How far the bf16 rounding of a number within tol of y may be from y: half a step, 2^-8 of the
    number, or 2^-134 below 2^-126, where bf16's steps stay 2^-133 (2^-126 of 8 bits)."""
    return 2.0 ** -8 * (np.abs(y) + tol) + 2.0 ** -134 + tol


def turn(x, pos, freqs, interleaved):
    """Rows x [n, H, d] turned at positions pos [n]; returns the rows and, elementwise, how far
    fp32 may be off before the final rounding."""
    y, tol = x.copy(), np.zeros_like(x)
    for i, f in enumerate(np.asarray(freqs, np.float64)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(freqs))
        # (the product modulo a turn, in extended precision: 2^-63 of p f)
        angle = np.asarray(pos, np.longdouble) * np.longdouble(f)
        c, s = (np.asarray(g(angle), np.float64)[:, None] for g in (np.cos, np.sin))
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, a] * s + x[:, :, b] * c
        # the angle to 2^-21, sine and cosine to an ulp (2^-23), two products and a sum in fp32
        t = (np.abs(x[:, :, a]) + np.abs(x[:, :, b])) * (2.0 ** -21 + 2.0 ** -23 + 2.0 ** -23)
        tol[:, :, a] = tol[:, :, b] = t
    return y, tol


def check_codes(value, scale, x, tol):
    """One token's E4M3 values [H, d] and scale against x within tol before the rounding."""
    mag = np.abs(x[np.isfinite(x)])
    top = mag.max() if mag.size else 0.0
    off = tol[np.isfinite(x)].max() if mag.size else 0.0
    assert scale in (block_scale(max(top - off, 0.0)), block_scale(top + off)), (scale, top)
    assert np.array_equal(np.isnan(value), ~np.isfinite(x))
    err = np.abs(value * scale - x)
    ok = err <= 2.0 ** -4 * np.abs(x) + scale * 2.0 ** -10 + 2 * tol
    # (the largest value may lie past 448 by what the scale's own maximum was off)
    assert (ok | ~np.isfinite(x)).all(), np.nanmax(err)


# ------------------------------------------------------------------ attention --
def attention(q, k, v, lam, tau, split, pos=None, window=-1, norm_eps=None, weight=None,
              out_scale=1.0):
    """Differential attention of queries q [T, 2 H or H, d] at positions pos [T] (None: the
    last T) over keys k, v [L, H_kv, d], lam [T, H].  Returns out [T, H, d], lse [T, 2 H] and
    the tolerances of both."""
    T, rows, d = q.shape
    L, H_kv, _ = k.shape
    H = rows if split else rows // 2
    G = H // H_kv
    pos = np.arange(L - T, L) if pos is None else np.asarray(pos)
    out, tol = np.zeros((T, H, d)), np.zeros((T, H, d))
    lse, tol_l = np.zeros((T, 2 * H)), np.zeros((T, 2 * H))
    j = np.arange(L)
    seen = j[None] <= pos[:, None]
    if window >= 0:
        seen &= j[None] >= pos[:, None] - window
    for h in range(H):
        kh, vh = k[:, h // G], v[:, h // G]
        o, e = [], []
        for u in (0, 1):
            if split:
                half = slice(u * (d // 2), (u + 1) * (d // 2))
                qu, ku = q[:, h, half], kh[:, half]
            else:
                qu, ku = q[:, 2 * h + u], kh
            x = np.where(seen, tau * (qu @ ku.T), -np.inf)
            m = x.max(1, keepdims=True)
            p = np.exp(x - m)
            total = p.sum(1, keepdims=True)
            w = p / total
            z = (m + np.log(total))[:, 0]
            # the score's products summed in fp32 (2^-20 of the magnitudes covers d = 128
            # terms), its exponent and the logarithm to 2^-20 of the largest |x|
            mags = np.where(seen, tau * (np.abs(qu) @ np.abs(ku).T), 0.0).max(1)
            dx = 2.0 ** -20 * mags + 2.0 ** -20 * (1.0 + np.abs(np.where(seen, x, 0.0)).max(1))
            lse[:, 2 * h + u] = z
            tol_l[:, 2 * h + u] = dx + 2.0 ** -20 * (1.0 + np.abs(z))
            vis = np.where(seen[:, :, None], vh[None], 0.0)  # (unseen rows may hold anything)
            o.append(np.einsum("ts,tsd->td", w, vis))
            # weights in bf16, off by twice the score's error besides
            e.append((2.0 ** -8 + 2 * dx[:, None] + 2.0 ** -18)
                     * np.einsum("ts,tsd->td", w, np.abs(vis)))
        la = lam[:, h, None]
        D = o[0] - la * o[1]
        E = e[0] + np.abs(la) * e[1] + 2.0 ** -22 * (np.abs(o[0]) + np.abs(la * o[1]))
        if norm_eps is not None:
            # |1 / r' - 1 / r| <= dr / (r (r - dr)) with dr <= the root mean square of E
            r = np.sqrt((D ** 2).mean(1, keepdims=True) + norm_eps)
            dr = np.sqrt((E ** 2).mean(1, keepdims=True))
            assert (dr < r).all(), "a test's norm must not rest on the roundings"
            w_ = np.ones(d) if weight is None else weight
            E = np.abs(w_) * (E / (r - dr) + np.abs(D) * dr / (r * (r - dr)))
            D = D / r * w_
            E = E + 2.0 ** -20 * np.abs(D)
        D, E = D * out_scale, E * abs(out_scale)
        out[:, h] = D
        tol[:, h] = E + 2.0 ** -8 * (np.abs(D) + E) + 2.0 ** -130
    return out, lse, tol, tol_l


def default_scale(d, split):
    return 1.0 / math.sqrt(d // 2 if split else d)
