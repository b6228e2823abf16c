"""Plain 64-bit references of the 8-bit cache's operators and of the heads' norm and rotation (numpy)."""
from __future__ import annotations

import numpy as np


def _e4m3():
    v = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = np.nan if c & 127 == 127 else m * 2.0**-9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = -x if c & 128 else x
    return v


E4M3 = _e4m3()


def scale_values(b):
    """E8M0 bytes -> powers of two (255: NaN)."""
    b = np.asarray(b).astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, np.where(b == 255, 0, b - 127)))


def values(codes, scale):
    return E4M3[codes] * scale_values(scale)[..., None]


def quantise(x):
    """Codes and scale bytes of rows [..., d] in float64 (bf16 values), by search over the code values."""
    pos = E4M3[:127]  # 0 .. 448, ascending; a code's parity is its mantissa's
    codes = np.empty(x.shape, np.uint8)
    scale = np.empty(x.shape[:-1], np.uint8)
    for i in np.ndindex(*x.shape[:-1]):
        row = x[i]
        if not np.isfinite(row).all():
            codes[i], scale[i] = 0x7F, 255
            continue
        top, e = np.abs(row).max(), -127
        while top > 448.0 * 2.0**e:
            e += 1
        y = np.abs(row) / 2.0**e
        hi = np.searchsorted(pos, y)  # the first code at or above
        lo = np.maximum(hi - 1, 0)
        up, down = pos[hi] - y, y - pos[lo]
        c = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
        codes[i] = np.where(np.signbit(row), c | 128, c)
        scale[i] = e + 127
    return codes, scale


def decode(q, k, v, k_codes_max, lens, table, window, scale, v_scale):
    """q [B, hq, d]; k, v [blocks, hk, bs, d] as values, v_scale their rows' scales, all float64.  Returns out, lse and
    for the bounds sum_j p_j |v_j|, max_j scale sum_d |q_d k_jd| and max_j(p_j 2^e_j) sum_j |v code_j|."""
    B, hq, d = q.shape
    hk, bs = k.shape[1], k.shape[2]
    G = hq // hk
    out, lse = np.zeros((B, hq, d)), np.full((B, hq), -np.inf)
    mass, dot, low = np.zeros((B, hq, d)), np.zeros((B, hq)), np.zeros((B, hq, d))
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        at = np.arange(max(0, n - window) if window else 0, n)
        blk = table[b][at // bs]
        for h in range(hk):
            kk, vv, vs = k[blk, h, at % bs], v[blk, h, at % bs], v_scale[blk, h, at % bs]
            of = slice(h * G, (h + 1) * G)
            s = scale * (q[b, of] @ kk.T)
            m = s.max(axis=1, keepdims=True)
            e = np.exp(s - m)
            tot = e.sum(axis=1, keepdims=True)
            p = e / tot
            lse[b, of] = (m + np.log(tot))[:, 0]
            out[b, of] = p @ vv
            mass[b, of] = p @ np.abs(vv)
            dot[b, of] = scale * (np.abs(q[b, of]) @ np.abs(kk).T).max(axis=1)
            low[b, of] = (p * vs).max(axis=1)[:, None] * (np.abs(vv) / vs[:, None]).sum(axis=0)
    return out, lse, mass, dot, low


def norm_rope(x, gain, pos, freq, axis, rot, interleaved, norm, eps):
    """x [T, heads, d] float64, pos [axes, T]; returns y and, for the bounds, |a| + |b| of each element's pair."""
    T, _, d = x.shape
    if norm:
        x = x / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps)
        if gain is not None:
            x = x * gain
    y, pair = x.copy(), np.abs(x)
    axes = pos.shape[0] if pos is not None else 0
    for i in range(rot // 2):
        ax = int(axis[i]) if axis is not None else 0
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        pair[:, :, a] = pair[:, :, b] = np.abs(x[:, :, a]) + np.abs(x[:, :, b])
        if not 0 <= ax < axes:
            continue
        # the exact product modulo a turn: whole turns taken off in integers of 2^-80 turns
        turns = [_turns(int(p), float(freq[i])) for p in pos[ax]]
        t = 2 * np.pi * np.array(turns)[:, None]
        c, s = np.cos(t), np.sin(t)
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y, pair


_PI = 3141592653589793238462643383279502884197169399375105820974944592307816406286208998628034825342117  # * 10^-96


def _turns(p, f):
    """p * f / (2 pi) modulo 1, from the exact fraction."""
    num, den = f.as_integer_ratio()
    unit = 1 << 80
    x = p * num * 10**96 * unit // (2 * _PI * den)
    return (x % unit) / unit
