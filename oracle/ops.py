"""Plain NumPy float64 definitions of windowed, cross and linear attention, the multi-axis
rotary embedding, block copies and the step builder -- TEST INFRASTRUCTURE ONLY (see the package's
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


def cross_attention(q, k, v, table, qsl, lens, scale, block_size):
    """As window_attention, every row with all lens[b] keys (none: out 0, lse -inf)."""
    T, hq, d = q.shape
    g = hq // k.shape[1]
    out = np.full((T, hq, d), np.nan)
    lse = np.full((T, hq), np.nan)
    mag = np.full((T, hq, d), np.nan)
    for b in range(len(lens)):
        j = np.arange(int(lens[b]))
        rows = np.asarray(table[b])[j // block_size]
        kk, vv = k[rows, :, j % block_size], v[rows, :, j % block_size]  # [keys, Hkv, d]
        for t in range(qsl[b], qsl[b + 1]):
            for h in range(hq):
                if len(j) == 0:
                    out[t, h] = mag[t, h] = 0
                    lse[t, h] = -np.inf
                    continue
                s = scale * (kk[:, h // g] @ q[t, h])
                m = s.max()
                e = np.exp(s - m)
                z = e.sum()
                lse[t, h] = m + np.log(z)
                out[t, h] = (e / z) @ vv[:, h // g]
                mag[t, h] = (e / z) @ np.abs(vv[:, h // g])
    return out, lse, mag


def linear_attention(q, k, v, qsl, log_decay, state, state_in, state_out, scale):
    """q [T, Hq, d], k and v [T, Hkv, d], log_decay [Hkv] or [T, Hkv], state [slots, Hkv, d, d].
    Returns out [T, Hq, d] (rows of no request NaN), the new state pool, and the same two
    with every product taken by its absolute value (what rounding can cost)."""
    T, hq, d = q.shape
    hkv = k.shape[1]
    g = np.broadcast_to(log_decay, (T, hkv)) if np.ndim(log_decay) == 1 else np.asarray(log_decay)
    keep = np.exp(np.where(g < 0, g, 0.0).astype(np.float64))
    found = []
    for f in (np.asarray, np.abs):
        out = np.full((T, hq, d), np.nan)
        new = np.array(state, np.float64)
        for b in range(len(state_in)):
            s = f(state[state_in[b]]).astype(np.float64) if state_in[b] >= 0 else \
                np.zeros((hkv, d, d))
            for t in range(qsl[b], qsl[b + 1]):
                s = keep[t][:, None, None] * s + f(k[t])[:, :, None] * f(v[t])[:, None, :]
                for h in range(hq):
                    out[t, h] = scale * (f(q[t, h]) @ s[h // (hq // hkv)])
            if state_out[b] >= 0:
                new[state_out[b]] = s
        found += [out, new]
    return tuple(found)


def build_step(query_lens, cached, table, ring, head, count, num_tokens, block_size):
    """The step builder, row after row: a dict of its outputs, the changed table and ring,
    and the list's head, count and missing blocks."""
    B, width = np.asarray(table).shape
    table, ring = np.array(table), np.array(ring)
    cap = len(ring)
    up = lambda x: -(-x // block_size)  # noqa: E731
    lens = [(max(int(n), 0), int(c)) for n, c in zip(query_lens, cached)]
    bad = any(c < 0 or c + n > width * block_size for n, c in lens) or \
        sum(n for n, _ in lens) > num_tokens or not (0 <= head < cap and 0 <= count <= cap)
    need = 0 if bad else sum(up(c + n) - up(c) for n, c in lens)
    missing = 0 if bad else max(0, need - count)  # (a bad count counts nothing)
    slots, positions = np.full(num_tokens, -1, np.int64), np.zeros(num_tokens, np.int32)
    qsl, ctx, seq, given, taken = [0], [], [], [], 0
    for b in range(B):
        n, c = lens[b] if not bad and not missing else (0, int(cached[b]))
        if query_lens[b] < 0 and not bad and not missing:
            given += [x for x in table[b, :up(c)] if x >= 0]
            c = 0
        for col in range(up(c), up(c + n)) if n else ():
            table[b, col] = ring[(head + taken) % cap]
            taken += 1
        for i in range(n):
            block = table[b, (c + i) // block_size]
            slots[qsl[-1] + i] = -1 if block < 0 else block * block_size + (c + i) % block_size
            positions[qsl[-1] + i] = c + i
        qsl.append(qsl[-1] + n)
        ctx.append(c)
        seq.append(c + n)
    for i, x in enumerate(given):
        ring[(head + count + i) % cap] = x
    state = [head, count, missing, 0] if bad or missing else \
        [(head + taken) % cap, count - taken + len(given), 0, 0]
    i32 = lambda x: np.asarray(x, np.int32)  # noqa: E731
    return {"qsl": i32(qsl), "ctx": i32(ctx), "seq": i32(seq), "slots": slots,
            "positions": positions, "table": i32(table), "ring": i32(ring), "state": i32(state),
            "bad": bad}
