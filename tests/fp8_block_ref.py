"""The block-scaled E4M3 cache in 64 bits, for the tests: quantisation on append,
the values held, and attention over them, written from their definitions with
explicit loops over sequences and blocks.  Also the tolerances of the decode."""
import numpy as np

#: value of every E4M3 code (sign, 4 exponent bits with bias 7, 3 mantissa bits)
E4M3 = np.zeros(256)
for _c in range(256):
    _e, _m = (_c >> 3) & 15, _c & 7
    _v = _m * 2.0 ** -9 if _e == 0 else (8 + _m) * 2.0 ** (_e - 10)
    E4M3[_c] = np.nan if (_c & 127) == 127 else (-_v if _c & 128 else _v)
_POS = E4M3[:127]  # ascending: 0 .. 448


def round_e4m3(x):
    """Nearest E4M3 value (ties to the even code, magnitudes above 448 to 448); NaN stays NaN."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, np.nan_to_num(a), side="left"), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(np.isnan(x), np.nan, np.copysign(np.where(up, _POS[hi], _POS[lo]), x))


def block_scale(amax):
    """The smallest power of two s >= 2^-100 with amax / s <= 448."""
    e = -100
    while amax / 2.0 ** e > 448.0:
        e += 1
    return 2.0 ** e


def append(x_new, values, scales, t_first, block):
    """Append rows x_new [n, H, d] at tokens t_first.. of one sequence whose cache holds the
    E4M3 values `values` [S, H, d] and `scales` [ceil(S / block), H] (both changed in place)."""
    n, H, _ = x_new.shape
    x_new = np.where(np.isfinite(x_new), x_new, np.nan)
    for beta in range(t_first // block, (t_first + n - 1) // block + 1):
        lo, hi = max(beta * block, t_first), min((beta + 1) * block, t_first + n)
        for h in range(H):
            x = x_new[lo - t_first:hi - t_first, h]
            mags = np.abs(x[~np.isnan(x)])
            s = block_scale(mags.max() if mags.size else 0.0)
            if beta * block < t_first:
                old = scales[beta, h]
                if s > old:
                    values[beta * block:t_first, h] = round_e4m3(
                        values[beta * block:t_first, h] * (old / s))
                s = max(s, old)
            values[lo:hi, h] = round_e4m3(x / s)
            scales[beta, h] = s


def attention(q, values_k, scales_k, values_v, scales_v, L, block, tau):
    """Decode of the last T_q queries q [T_q, H_q, d] of a sequence of L tokens; returns O, LSE
    and the tolerances (elementwise for O, per row for LSE) of a kernel that holds q to
    2^-21 of its row's largest magnitude, the weights to 2^-9 of themselves with steps of
    2^-14 at a largest weight of 2^8, everything else in fp32, and O in bf16."""
    T, H_q, d = q.shape
    H = values_k.shape[1]
    G = H_q // H
    blk = np.arange(L) // block
    o = np.zeros((T, H_q, d))
    lse = np.zeros((T, H_q))
    tol_o, tol_l = np.zeros_like(o), np.zeros_like(lse)
    for h in range(H_q):
        kc, vc = values_k[:L, h // G], values_v[:L, h // G]
        sk, sv = scales_k[blk, h // G], scales_v[blk, h // G]
        k, v = kc * sk[:, None], vc * sv[:, None]
        for t in range(T):
            n = L - T + t + 1
            qr = q[t, h]
            x = tau * (k[:n] @ qr)
            m = x.max()
            p = np.exp(x - m)
            w = p / p.sum()
            o[t, h] = w @ v[:n]
            lse[t, h] = m + np.log(p.sum())
            # scores: q to 2^-21 of its largest element, products summed in fp32 (2^-20
            # of the sum of magnitudes covers d = 128 terms of either rounding or
            # truncation), exponent and logarithm to 2^-20 of the largest |x| involved
            dx = tau * (2.0 ** -21 * np.abs(qr).max() * np.abs(k[:n]).sum(1).max()
                        + 2.0 ** -20 * (np.abs(k[:n]) @ np.abs(qr)).max())
            dx += 2.0 ** -20 * (1.0 + np.abs(x).max())
            tol_l[t, h] = dx + 2.0 ** -20 * (1.0 + abs(lse[t, h]))
            mag = w @ np.abs(v[:n])
            # a weight's absolute step: half of 2^-14 of 2^8, at most, of the largest w vs
            small = 2.0 ** -22 * (w * sv[:n]).max() * np.abs(vc[:n]).sum(0)
            tol_o[t, h] = 2.0 ** -8 * np.abs(o[t, h]) + (2.0 ** -9 + 2 * dx + 2.0 ** -18) * mag + small
    return o, lse, tol_o, tol_l
