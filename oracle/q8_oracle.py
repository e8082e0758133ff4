"""Plain fp64 reference of the operators around the 8-bit paged cache, from their
definitions: per-head norms and rotation, e4m3 codes with a power of two per row,
and softmax attention of the newest rows over gathered rows. No code is shared
with the CUDA path. Next to each attention result it gives the sums that an
error bound needs.
"""
from __future__ import annotations

import numpy as np

E_LO, E_HI = -56, 120
NAN_CODE = 0x7F


def _code_values():
    v = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        mag = (8 + f) * 2.0 ** (e - 10) if e else f * 2.0 ** -9
        if e == 15 and f == 7:
            mag = np.nan
        v[c] = -mag if c & 128 else mag
    return v


CODE = _code_values()
_MAG = CODE[:127]                    # values of the codes 0 .. 126, increasing


def norm(x, weight, eps):
    """x [..., D] times weight / root mean square."""
    x = np.asarray(x, np.float64)
    return x * np.asarray(weight, np.float64) / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)


def rope(x, positions, base):
    """Rotate-half form of x [rows, heads, D]; also the size of each element's pair."""
    x = np.asarray(x, np.float64)
    h = x.shape[-1] // 2
    a = (np.asarray(positions, np.float64)[:, None] * base ** (-np.arange(h) / h))[:, None, :]
    z = (x[..., :h] + 1j * x[..., h:]) * np.exp(1j * a)
    size = np.abs(x[..., :h]) + np.abs(x[..., h:])
    return np.concatenate([z.real, z.imag], axis=-1), np.concatenate([size, size], axis=-1)


def exponent(x):
    """Exponent of rows x [..., D]: the least in range that keeps the finite elements within 448 * 2^e."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(axis=-1)
    e = np.full(a.shape, E_LO)
    for k in range(E_LO, E_HI):
        e[a > 448.0 * 2.0 ** k] = k + 1
    return e


def codes(x, e):
    """Nearest e4m3 codes of x * 2^-e, ties to the even code; NaN for what is not finite."""
    y = np.asarray(x, np.float64) * 2.0 ** -np.asarray(e, np.float64)[..., None]
    m = np.where(np.isfinite(y), np.abs(y), 0.0)
    hi = np.searchsorted(_MAG, m).clip(1, 126)
    lo = hi - 1
    up, down = _MAG[hi] - m, m - _MAG[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    c = np.where(np.signbit(y), c | 128, c).astype(np.uint8)
    return np.where(np.isfinite(y), c, NAN_CODE).astype(np.uint8)


def values(c, exp_bytes):
    """What codes [..., D] with exponent bytes [...] stand for."""
    e = np.clip(np.asarray(exp_bytes, np.int64) - 127, E_LO, E_HI)
    return CODE[np.asarray(c, np.uint8)] * 2.0 ** e.astype(np.float64)[..., None]


def attention(q, k, v, n, scale):
    """q [n, Hq, D] over the rows k, v [L, Hkv, D] of one request, the last n of
    them q's own. k or v rows may be NaN where hidden: a row marked by NaN in
    all of k is one no query sees. Returns o, lse and for the error bound
    sum_j p_j |v_j| and max_j |scale| sum_d |q_d k_jd| (over seen keys)."""
    _, hq, D = q.shape
    L, hkv, _ = k.shape
    G = hq // hkv
    o, av = np.zeros((n, hq, D)), np.zeros((n, hq, D))
    lse, big = np.full((n, hq), -np.inf), np.zeros((n, hq))
    hidden = np.isnan(k).all(axis=(1, 2))
    for i in range(n):
        see = np.arange(L) < L - n + i + 1
        see &= ~hidden
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h // G], v[see, h // G]
            s = scale * (kk @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            o[i, h], av[i, h] = (p / l) @ vv, (p / l) @ np.abs(vv)
            lse[i, h] = m + np.log(l)
            big[i, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[i, h]))).max()
    return o, lse, av, big
