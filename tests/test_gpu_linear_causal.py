"""An infinity or a NaN in one token of a prompt: no earlier token's output knows of it, nor does
a column that it does not stand in, and every later one does.

The expected outputs are those of the same prompt with a 0 in its place: earlier rows and, for a
value in v, other columns meet no other number.  Rows that were summed up again without the bad
token may differ in the order of fp32 sums and in a weight's rounding to bf16: each is within the
tolerance of test_gpu_linear.py of the definition."""
import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean
from oracle import ops
from test_gpu_linear import Step

pytestmark = pytest.mark.gpu


def definition(s, rows):
    (hq, hkv), d = s.heads, s.d
    rows = rows[:s.total].double().numpy().reshape(s.total, -1, d)
    g = s.g.double().numpy()
    return ops.linear_attention(rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], s.qsl.numpy(),
                                g[:s.total] if g.ndim == 2 else g, s.state.double().numpy(),
                                s.state_in.numpy(), s.state_out.numpy(), s.scale)


def spoil(s, t, x, token, head, bad, column):
    """A device copy of the step's tensors with one element of q, k or v changed."""
    t = {**t, x: t[x].clone(), "state": t["state"].clone(), "out": torch.full_like(t["out"], 7)}
    t[x][token, head, column] = bad
    return t


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (2, 2, 64), (6, 2, 128), (2, 2, 128)])
def test_one_element(hq, hkv, d, bad):
    """Requests of 200 (its chunks' first, inner and last tokens), 70 and 5 tokens; the bad element
    is in one head of the first or the last, in each of v's column slices."""
    s = Step([200, 70, 5], hq, hkv, d, seed=d + hq)
    t = s.to_dev()
    out, state, mag, _ = definition(s, s.fused)
    bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -12) * mag + 1e-30
    group = hq // hkv
    s.call(t)
    clean = t["out"].double().cpu().numpy()
    first = s.to_dev()
    for x, token, column in [("v", 0, 3), ("v", 1, 0), ("v", 63, d - 1), ("v", 64, 17), ("v", 100, 40),
                             ("v", 127, 5), ("v", 128, 33), ("v", 199, 2), ("v", 269, 9), ("v", 271, 1),
                             ("k", 50, 7), ("k", 127, 0), ("k", 199, d - 1), ("q", 90, 11)]:
        b = 0 if token < 200 else 1 if token < 270 else 2
        head = 1 if x != "q" else group
        u = spoil(s, first, x, token, head, bad, column)
        s.call(u)
        got = u["out"].double().cpu().numpy()
        after = u["state"].double().cpu().numpy()
        hit = np.zeros(got.shape, bool)
        if x == "q":
            hit[token, head] = True
        else:
            heads = slice(head * group, (head + 1) * group)
            hit[token:s.qsl[b + 1], heads, column if x == "v" else slice(None)] = True
        what = (x, token, column)
        assert not np.any(np.isfinite(got[hit])), what
        assert np.all(np.isfinite(got[~hit])), (what, np.argwhere(~np.isfinite(got) & ~hit)[:5])
        # (v: a column that the element is not in keeps its bits)
        rest = ~hit
        assert np.all(np.abs(got - out)[rest] <= bound[rest]), what
        same = rest.copy()
        if x == "v":
            same[:, :, column] = False
            assert np.array_equal(got[same], clean[same]), what
        for r in range(3):
            slot = int(s.state_out[r])
            dirty = np.zeros(state[slot].shape, bool)
            if r == b and x == "v":
                dirty[head, :, column] = True
            elif r == b and x == "k":
                dirty[head, column, :] = True
            assert np.array_equal(np.isfinite(after[slot]), ~dirty), what
    assert_status_clean()


def test_many_bad_tokens_and_clusters():
    """Whole tokens of NaN at the end of long prompts (a cluster shares the first), one after the
    other and beside short rows."""
    for lens, hq, hkv in (([900], 4, 2), ([900], 1, 1), ([300, 1, 260, 5], 4, 2), ([130] * 40, 2, 2)):
        s = Step(lens, hq, hkv, 128, seed=len(lens))
        t = s.to_dev()
        out, _, mag, _ = definition(s, s.fused)
        bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -12) * mag + 1e-30
        starts, good = s.qsl.tolist(), np.ones(s.total, bool)
        for b, n in enumerate(lens):
            if n > 100:
                at = starts[b] + n - 77 + b % 9
                good[at:starts[b + 1]] = False
                for x in "qkv":
                    t[x][at:starts[b + 1]] = float("nan")
        s.call(t)
        got = t["out"].double().cpu().numpy()
        assert np.all(np.abs(got - out)[good] <= bound[good])
        assert not np.any(np.isfinite(got[~good]))
        assert_status_clean()


def test_a_prompt_of_nothing_else():
    s = Step([2000], 4, 2, 128, seed=1)
    t = s.to_dev()
    t["v"].fill_(float("inf"))
    s.call(t)
    torch.cuda.synchronize()
    assert not torch.any(torch.isfinite(t["out"]))
    assert_status_clean()
