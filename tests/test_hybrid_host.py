"""pa_build_step, pa_cross_attention and pa_linear_attention without a GPU: their definitions
against closed forms, and the refusals of the C calls."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from oracle import ops


def test_cross_attention_is_softmax_over_all_keys():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(6, 2, 16, 8)), rng.normal(size=(6, 2, 16, 8))
    out, lse, _ = ops.cross_attention(q, k, v, [[4, 1], [5, 0]], [0, 2, 3], [21, 0], 0.3, 16)
    kk = np.concatenate([k[4], k[1][:, :5]], axis=1)
    vv = np.concatenate([v[4], v[1][:, :5]], axis=1)
    for t in range(2):
        for h in range(4):
            s = torch.from_numpy(0.3 * kk[h // 2] @ q[t, h])
            assert np.allclose(out[t, h], torch.softmax(s, 0).numpy() @ vv[h // 2])
            assert np.isclose(lse[t, h], torch.logsumexp(s, 0))
    assert np.all(out[2] == 0) and np.all(np.isneginf(lse[2]))


def test_linear_attention_is_the_decayed_sum():
    """o_t = scale (e^(sum g) q_t S + sum_(j <= t) e^(g_(j+1) + .. + g_t) (q_t k_j) v_j)."""
    rng = np.random.default_rng(1)
    T, hq, hkv, d = 9, 4, 2, 8
    q, k, v = (rng.normal(size=(T, h, d)) for h in (hq, hkv, hkv))
    g, pool = -rng.random((T, hkv)), rng.normal(size=(3, hkv, d, d))
    out, state, _, _ = ops.linear_attention(q, k, v, [0, 2, 9], g, pool, [-1, 1], [0, 2], 0.5)
    for a, b, src, dst in ((0, 2, None, 0), (2, 9, 1, 2)):
        for h in range(hq):
            hk = h // 2
            for t in range(a, b):
                w = lambda j: np.exp(g[j + 1:t + 1, hk].sum())  # noqa: E731
                o = sum(w(j) * (q[t, h] @ k[j, hk]) * v[j, hk] for j in range(a, t + 1))
                if src is not None:
                    o = o + w(a - 1) * q[t, h] @ pool[src, hk]
                assert np.allclose(out[t, h], 0.5 * o)
        for hk in range(hkv):
            end = lambda j: np.exp(g[j + 1:b, hk].sum())  # noqa: E731
            s = sum(end(j) * np.outer(k[j, hk], v[j, hk]) for j in range(a, b))
            if src is not None:
                s = s + end(a - 1) * pool[src, hk]
            assert np.allclose(state[dst, hk], s)
    assert np.array_equal(state[1], pool[1])


def test_build_step_makes_valid_metadata():
    """Its steps pass the host validator, and every block has one owner throughout."""
    rng = np.random.default_rng(2)
    bs, nb, rows, width = 16, 40, 5, 9
    cached, table = np.zeros(rows, np.int32), np.full((rows, width), -1, np.int32)
    ring, head, count = rng.permutation(nb).astype(np.int32), 0, nb
    made = 0
    for _ in range(300):
        n = rng.choice([-1, 0, 1, 7, 30], rows).astype(np.int32)
        r = ops.build_step(n, cached, table, ring, head, count, 100, bs)
        made += r["qsl"][-1] > 0
        pk.pa_validate_metadata(*(torch.from_numpy(r[x]) for x in ("table", "qsl", "ctx", "seq")),
                                num_blocks=nb, block_size=bs,
                                slot_mapping=torch.from_numpy(r["slots"]))
        cached, table, ring = r["seq"], r["table"], r["ring"]
        head, count = int(r["state"][0]), int(r["state"][1])
        owned = [x for b in range(rows) for x in table[b, :-(-cached[b] // bs)]]
        owned += [ring[(head + i) % nb] for i in range(count)]
        assert sorted(owned) == list(range(nb))
    assert made > 100


P = 1 << 20  # an aligned address that is never followed


def build(**kw):
    a = dict(q=P, cached=P, B=2, table=P, width=4, blocks=P, state=P, state_out=P, cap=8, reserved=0,
             nb=8, bs=16, T=4, qsl=P, ctx=P, seq=P, slots=P, pos=P, free=True)
    a.update(kw)
    free = pk.FreeList(a["blocks"], a["state"], a["state_out"], a["cap"], a["reserved"])
    return pk.lib().pa_build_step(a["q"], a["cached"], a["B"], a["table"], a["width"],
                                  ctypes.byref(free) if a["free"] else None, a["nb"], a["bs"],
                                  a["T"], a["qsl"], a["ctx"], a["seq"], a["slots"], a["pos"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), pk.PA_ERR_INVALID_ARG), (dict(T=-1), pk.PA_ERR_INVALID_ARG),
    (dict(B=8193), pk.PA_ERR_UNSUPPORTED), (dict(nb=0), pk.PA_ERR_INVALID_ARG),
    (dict(width=0), pk.PA_ERR_INVALID_ARG), (dict(bs=0), pk.PA_ERR_UNSUPPORTED),
    (dict(bs=24), pk.PA_ERR_UNSUPPORTED), (dict(bs=272), pk.PA_ERR_UNSUPPORTED),
    (dict(bs=256, width=1 << 23), pk.PA_ERR_UNSUPPORTED), (dict(free=False), pk.PA_ERR_INVALID_ARG),
    (dict(cap=0), pk.PA_ERR_INVALID_ARG), (dict(reserved=1), pk.PA_ERR_INVALID_ARG),
    (dict(slots=P + 4), pk.PA_ERR_INVALID_ARG), (dict(q=P + 2), pk.PA_ERR_INVALID_ARG)] +
    [(dict([(x, None)]), pk.PA_ERR_INVALID_ARG) for x in
     ("q", "cached", "table", "blocks", "state", "state_out", "qsl", "ctx", "seq", "slots", "pos")])
def test_build_step_refusals(kw, code):
    assert build(**kw) == code and pk.lib().pa_last_error_message()


def cross(**kw):
    a = dict(q=P, table=P, width=4, qsl=P, lens=P, B=2, T=3, hq=4, scale=0.1, out=P, ws=P,
             bytes=1 << 30, d=64, bs=16)
    a.update(kw)
    kv = pk.KVDesc(P, P, 8, a["bs"], 2, a["d"], 0, 0, None, None)
    return pk.lib().pa_cross_attention(a["q"], ctypes.byref(kv), a["table"], a["width"], a["qsl"],
                                       a["lens"], a["B"], a["T"], a["hq"], a["scale"], a["out"],
                                       None, a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), pk.PA_ERR_INVALID_ARG), (dict(out=None), pk.PA_ERR_INVALID_ARG),
    (dict(table=None), pk.PA_ERR_INVALID_ARG), (dict(qsl=None), pk.PA_ERR_INVALID_ARG),
    (dict(lens=None), pk.PA_ERR_INVALID_ARG), (dict(B=-1), pk.PA_ERR_INVALID_ARG),
    (dict(T=-1), pk.PA_ERR_INVALID_ARG), (dict(hq=3), pk.PA_ERR_INVALID_ARG),
    (dict(hq=512), pk.PA_ERR_UNSUPPORTED), (dict(scale=0.0), pk.PA_ERR_INVALID_ARG),
    (dict(scale=-1.0), pk.PA_ERR_INVALID_ARG), (dict(scale=float("nan")), pk.PA_ERR_INVALID_ARG),
    (dict(scale=float("inf")), pk.PA_ERR_INVALID_ARG), (dict(width=0), pk.PA_ERR_INVALID_ARG),
    (dict(bs=256, width=1 << 23), pk.PA_ERR_UNSUPPORTED), (dict(ws=None), pk.PA_ERR_WORKSPACE),
    (dict(ws=P + 64), pk.PA_ERR_WORKSPACE), (dict(bytes=64), pk.PA_ERR_WORKSPACE),
    (dict(d=96), pk.PA_ERR_UNSUPPORTED), (dict(T=(1 << 30) + 1), pk.PA_ERR_UNSUPPORTED)])
def test_cross_attention_refusals(kw, code):
    assert cross(**kw) == code and pk.lib().pa_last_error_message()


def test_a_windowed_step_still_needs_its_context():
    kv = pk.KVDesc(P, P, 8, 16, 2, 64, 0, 0, None, None)
    assert pk.lib().pa_window_attention(P, ctypes.byref(kv), P, 4, P, None, P, 2, 3, 4, 0.1, 8, 0, P,
                                        None, P, 1 << 30, None) == pk.PA_ERR_INVALID_ARG


def linear(**kw):
    a = dict(q=P, qs=256, k=P, ks=128, v=P, vs=128, qsl=P, B=2, T=3, g=P, si=P, so=P, out=P, ws=P,
             bytes=1 << 30, state=P, slots=4, hq=4, hkv=2, d=64, per_token=1, scale=0.1, desc=True)
    a.update(kw)
    desc = pk.LinearDesc(a["state"], a["slots"], a["hq"], a["hkv"], a["d"], a["per_token"], a["scale"])
    return pk.lib().pa_linear_attention(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qsl"],
                                        a["B"], a["T"], a["g"],
                                        ctypes.byref(desc) if a["desc"] else None, a["si"], a["so"],
                                        a["out"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(desc=False), pk.PA_ERR_INVALID_ARG), (dict(B=-1), pk.PA_ERR_INVALID_ARG),
    (dict(T=-1), pk.PA_ERR_INVALID_ARG), (dict(slots=-1), pk.PA_ERR_INVALID_ARG),
    (dict(hq=3), pk.PA_ERR_INVALID_ARG), (dict(hkv=0), pk.PA_ERR_INVALID_ARG),
    (dict(hq=516, qs=1 << 20), pk.PA_ERR_UNSUPPORTED), (dict(d=32), pk.PA_ERR_UNSUPPORTED),
    (dict(per_token=2), pk.PA_ERR_INVALID_ARG), (dict(scale=float("nan")), pk.PA_ERR_INVALID_ARG),
    (dict(B=1 << 28), pk.PA_ERR_UNSUPPORTED), (dict(qs=248), pk.PA_ERR_INVALID_ARG),
    (dict(ks=132), pk.PA_ERR_INVALID_ARG), (dict(vs=120), pk.PA_ERR_INVALID_ARG),
    (dict(q=P + 8), pk.PA_ERR_INVALID_ARG), (dict(state=P + 8), pk.PA_ERR_INVALID_ARG),
    (dict(g=P + 2), pk.PA_ERR_INVALID_ARG), (dict(ws=None), pk.PA_ERR_WORKSPACE),
    (dict(ws=P + 128), pk.PA_ERR_WORKSPACE), (dict(bytes=8), pk.PA_ERR_WORKSPACE)] +
    [(dict([(x, None)]), pk.PA_ERR_INVALID_ARG) for x in
     ("q", "k", "v", "qsl", "g", "si", "so", "out", "state")])
def test_linear_attention_refusals(kw, code):
    assert linear(**kw) == code and pk.lib().pa_last_error_message()


def test_nothing_to_do():
    assert linear(B=0) == pk.PA_OK and cross(B=0) == pk.PA_OK and cross(T=0) == pk.PA_OK
    size = pk.lib().pa_linear_workspace_size
    assert size(1, 1, 4, 2, 64) > 0 and size(-1, 1, 4, 2, 64) == 0 and size(1, 1, 3, 2, 64) == 0
    assert size(1, 1, 4, 2, 96) == 0
