"""Plain NumPy float64 definitions of windowed attention, the multi-axis rotary
embedding and block copies -- TEST INFRASTRUCTURE ONLY (see the package's
docstring).  Everything is a direct restatement of the formulas; nothing here
is shared with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def visible_keys(pos: int, window: int, sinks: int) -> np.ndarray:
    """Keys that the row at position pos sees: j <= pos with j > pos - window or
    j < sinks."""
    j = np.arange(pos + 1)
    return j[(j > pos - window) | (j < sinks)]


def window_attention(q, k, v, table, qsl, ctx, scale, window, sinks, block_size):
    """q [T, Hq, d], caches k and v [num_blocks, Hkv, bs, d] (float64 values).
    Returns out [T, Hq, d], lse [T, Hq] and mag [T, Hq, d] = sum_j p_j |v_j|
    (what the rounding of p can cost).  Rows of no request stay NaN."""
    T, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    out = np.full((T, hq, d), np.nan)
    lse = np.full((T, hq), np.nan)
    mag = np.full((T, hq, d), np.nan)
    for b in range(len(ctx)):
        for t in range(qsl[b], qsl[b + 1]):
            j = visible_keys(int(ctx[b]) + t - int(qsl[b]), window, sinks)
            rows = np.asarray(table[b])[j // block_size]
            kk, vv = k[rows, :, j % block_size], v[rows, :, j % block_size]  # [keys, Hkv, d]
            for h in range(hq):
                s = scale * (kk[:, h // g] @ q[t, h])
                m = s.max()
                e = np.exp(s - m)
                z = e.sum()
                lse[t, h] = m + np.log(z)
                out[t, h] = (e / z) @ vv[:, h // g]
                mag[t, h] = (e / z) @ np.abs(vv[:, h // g])
    return out, lse, mag


def rope(x, positions, inv_freq, axis, rot_dim, adjacent, attn_factor=1.0):
    """x [T, H, d] rotated: pair i of a head turned by positions[axis[i]] *
    inv_freq[i] (extended precision, so that far positions keep their angle)."""
    x = np.asarray(x, np.float64).copy()
    axis = np.zeros(rot_dim // 2, int) if axis is None else np.asarray(axis)
    pos = np.asarray(positions)[axis].T.astype(np.longdouble)            # [T, rot_dim / 2]
    two_pi = np.longdouble("6.283185307179586476925286766559005768")
    t = np.fmod(pos * np.asarray(inv_freq, np.longdouble), two_pi)
    c = (np.cos(t) * attn_factor).astype(np.float64)[:, None]
    s = (np.sin(t) * attn_factor).astype(np.float64)[:, None]
    i = np.arange(rot_dim // 2)
    ia, ib = (2 * i, 2 * i + 1) if adjacent else (i, i + rot_dim // 2)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = b * c + a * s
    return x


def copy_blocks(cache, pairs):
    """cache [num_blocks, ...] after the copies (src, dst); negative ids are
    padding.  All reads come from the cache as it was."""
    new = cache.copy()
    for s, t in np.asarray(pairs).reshape(-1, 2):
        if s >= 0 and t >= 0:
            new[t] = cache[s]
    return new
