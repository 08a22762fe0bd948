"""Pins of oracle/ops.py (windowed attention, rotary embedding, block copies)
that do not call it to check itself."""
import numpy as np
import pytest

import oracle
from oracle import ops


def random_step(rng, requests, hq, hkv, d, bs):
    lens = [c + n for c, n in requests]
    need = [-(-x // bs) for x in lens]
    perm = rng.permutation(sum(need))
    table = np.full((len(requests), max(need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    qsl = np.concatenate([[0], np.cumsum([n for _, n in requests])]).astype(np.int32)

    def bf16(shape):
        x = rng.standard_normal(shape).astype(np.float32)
        return (x.view(np.uint32) >> 16).astype(np.uint16)
    return (bf16((qsl[-1], hq, d)), bf16((sum(need), hkv, bs, d)), bf16((sum(need), hkv, bs, d)),
            table, qsl, np.array([c for c, _ in requests], np.int32), np.array(lens, np.int32))


def f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def test_wide_window_is_plain_causal_attention():
    rng = np.random.default_rng(1)
    q, k, v, table, qsl, ctx, sl = random_step(rng, [(0, 5), (17, 3), (40, 1)], 4, 2, 8, 16)
    ref_o, ref_l = oracle.attention(q, k, v, table, qsl, ctx, sl, 0.3)
    for window, sinks in ((41, 0), (1000, 7), (1, 41), (20, 30)):
        o, l, _ = ops.window_attention(f64(q), f64(k), f64(v), table, qsl, ctx, 0.3, window, sinks, 16)
        assert np.allclose(o, ref_o, atol=1e-12) and np.allclose(l, ref_l, atol=1e-12)


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (3, 2), (8, 1), (2, 20)])
def test_window_equals_masked_softmax(window, sinks):
    """Against one dense masked softmax per request, written the other way round
    (mask of hidden keys, all keys of the request)."""
    rng = np.random.default_rng(2)
    reqs = [(0, 9), (22, 4)]
    q, k, v, table, qsl, ctx, sl = random_step(rng, reqs, 2, 1, 8, 16)
    o, l, _ = ops.window_attention(f64(q), f64(k), f64(v), table, qsl, ctx, 0.3, window, sinks, 16)
    for b, (c, n) in enumerate(reqs):
        L = c + n
        kk = f64(k)[table[b, :-(-L // 16)], 0].reshape(-1, 8)[:L]
        vv = f64(v)[table[b, :-(-L // 16)], 0].reshape(-1, 8)[:L]
        p, j = c + np.arange(n)[:, None], np.arange(L)
        hidden = (j > p) | ((p - j >= window) & (j >= sinks))
        for h in range(2):
            s = np.where(hidden, -np.inf, 0.3 * f64(q)[qsl[b]:qsl[b + 1], h] @ kk.T)
            w = np.exp(s)
            assert np.allclose(o[qsl[b]:qsl[b + 1], h], w @ vv / w.sum(1, keepdims=True), atol=1e-12)
            assert np.allclose(l[qsl[b]:qsl[b + 1], h], np.log(w.sum(1)), atol=1e-12)


def test_window_of_one_returns_the_rows_own_value():
    rng = np.random.default_rng(3)
    q, k, v, table, qsl, ctx, _ = random_step(rng, [(33, 1)], 1, 1, 8, 16)
    o, l, _ = ops.window_attention(f64(q), f64(k), f64(v), table, qsl, ctx, 0.5, 1, 0, 16)
    blk, off = table[0, 2], 1
    assert np.allclose(o[0, 0], f64(v)[blk, 0, off])
    assert np.allclose(l[0, 0], 0.5 * f64(q)[0, 0] @ f64(k)[blk, 0, off])


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_is_a_complex_rotation_and_keeps_relative_positions(adjacent):
    rng = np.random.default_rng(4)
    inv = 1e4 ** (-np.arange(8) / 8)
    axis = np.array([0, 1, 2, 0, 1, 2, 0, 1])
    x = rng.standard_normal((5, 3, 24))
    pos = rng.integers(-50, 5000, (3, 5))
    y = ops.rope(x, pos, inv, axis, 16, adjacent)
    pairs = (lambda z: z[..., 0:16:2] + 1j * z[..., 1:16:2]) if adjacent else \
        (lambda z: z[..., 0:8] + 1j * z[..., 8:16])
    turn = np.exp(1j * pos[axis].T * inv)[:, None]
    assert np.allclose(pairs(y), pairs(x) * turn, atol=1e-10)
    assert np.array_equal(y[..., 16:], x[..., 16:])
    assert np.allclose(ops.rope(x, np.zeros((3, 5), int), inv, axis, 16, adjacent), x)
    # q.k depends on the difference of the positions alone
    k = rng.standard_normal((5, 3, 24))
    a = (y * ops.rope(k, pos + 11, inv, axis, 16, adjacent)).sum(-1)
    b = (ops.rope(x, pos + 77, inv, axis, 16, adjacent) *
         ops.rope(k, pos + 88, inv, axis, 16, adjacent)).sum(-1)
    assert np.allclose(a, b, atol=1e-9)


def test_rope_keeps_the_angle_of_far_positions():
    """2^31 - 1 positions of a whole number of turns each, and one of a quarter
    turn more."""
    inv = np.full(8, 2 * np.pi)
    x = np.ones((1, 1, 16))
    y = ops.rope(x, np.array([[2 ** 20]]), inv, None, 16, False)
    assert np.allclose(y, x, atol=1e-8)
    y = ops.rope(x, np.array([[1]]), inv / 4, None, 16, False, attn_factor=2.0)
    assert np.allclose(y[..., :8], -2) and np.allclose(y[..., 8:], 2)


def test_copies_read_the_old_cache_and_skip_padding():
    c = np.arange(12).reshape(6, 2)
    new = ops.copy_blocks(c, [(0, 3), (-1, 2), (0, 4), (5, -1)])
    assert np.array_equal(new, c[[0, 1, 2, 0, 0, 5]])
