"""The decays between two tokens of a chunk, one by one.

With q and k the first unit vector, scale 1 and v of token j the unit vector j, element j of token
i's output is e^(g_(j+1) + .. + g_i) itself, once for each pair of tokens.

Tolerance.  It is rounded to bf16 once (as a weight of the chunk; the output that repeats it is
exact): half a step of the value, 2^-8 of its binade at most.  Its relative error in fp32, in powers of
two (times ln 2): with e^(..) = 2^-G, the logarithms' own errors are 2^-23 G, at most 16
roundings of sums up to G 2^-24 G each; where a run of 16 tokens sums up to M (a logarithm counts as
no less than -150), a difference of two such sums is off by at most 16 roundings of 2^-24 M.
Two exponentials and their products add 2^-20."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean

pytestmark = pytest.mark.gpu


def weights(g, group, d):
    """[T, T] of one request of T <= d tokens, the same for every head of the group."""
    T = len(g)
    q = torch.zeros((T, group, d), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((T, 1, d), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros((T, 1, d), dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = k[:, :, 0] = 1
    v[torch.arange(T), 0, torch.arange(T)] = 1
    out = torch.full_like(q, 7)
    one = torch.tensor([-1], dtype=torch.int32, device=DEV)
    state = torch.zeros((1, 1, d, d), device=DEV)
    pk.pa_linear_attention(q, k, v, torch.tensor([0, T], dtype=torch.int32, device=DEV),
                           torch.tensor(g, dtype=torch.float32, device=DEV).view(T, 1).contiguous(),
                           state, one, torch.zeros_like(one), 1.0, out)
    torch.cuda.synchronize()
    assert torch.equal(out, out[:, :1].expand_as(out))
    assert torch.all(out[:, 0, T:] == 0)
    return out[:, 0, :T].double().cpu().numpy(), state[0, 0, 0, :T].double().cpu().numpy()


def patterns(T):
    rng = np.random.default_rng(T)
    small = -1e-3 * rng.random(T)
    clear = np.full(T, -np.inf)
    keep = rng.random(T)
    yield "small", small
    for n in (1, T // 2, T - 16, T - 13):   # cleared tokens first
        yield f"cleared {n}", np.concatenate([clear[:n], small[n:]])
    yield "some cleared", np.where(keep < 0.2, clear, small)
    yield "most cleared", np.where(keep < 0.8, clear, small)
    yield "large", np.where(keep < 0.5, -60.0, small)
    yield "mixed", -np.exp(rng.normal(size=T) * 3 - 2)
    yield "large, then small", np.concatenate([np.full(T // 2, -100.0), 0.1 * small[T // 2:]])


@pytest.mark.parametrize("T,group,d", [(64, 2, 64), (64, 2, 128), (64, 1, 64), (128, 1, 128),
                                       (50, 3, 128), (8, 1, 64)])
def test_weights_between_tokens(T, group, d):
    for name, g in patterns(T):
        got, state = weights(g, group, d)
        g = g.astype(np.float32).astype(np.float64)
        log = np.maximum(g * math.log2(math.e), -150)
        M = np.array([-log[r:r + 16].sum() for r in range(0, T, 16)]).repeat(16)[:T]
        for i in range(T):
            w = np.array([math.exp(math.fsum(g[j + 1:i + 1])) if np.all(np.isfinite(g[j + 1:i + 1]))
                          else 0.0 for j in range(i + 1)])
            step = 2.0 ** (np.floor(np.log2(np.maximum(w, 2.0 ** -126))) - 8)   # half of bf16's
            G = -np.log2(np.maximum(w, 2.0 ** -150))
            exact = math.log(2) * 18 * 2.0 ** -24 * G + 2.0 ** -20
            fp32 = exact + math.log(2) * 16 * 2.0 ** -24 * np.maximum(M[:i + 1], M[i])
            err = np.abs(got[i, :i + 1] - w)
            bound = step + fp32 * w + 2.0 ** -125
            assert np.all(err <= bound), (name, i, np.argmax(err / bound), np.max(err / bound))
            assert np.all(got[i, :i + 1] <= 1) and np.all(got[i, i + 1:] == 0), (name, i)
            if i == T - 1:   # the state keeps them in fp32
                err = np.abs(state - w)
                assert np.all(err <= exact * w + 2.0 ** -125), (name, np.max(err))
    assert_status_clean()
