"""pa_linear_attention within the bounds that its two forms are documented with, each by itself:
the recurrent form rounds nothing but the output, and no form rounds the state.

Tolerances.  Recurrent: the output's rounding to bf16, 2^-8 of its value, and fp32: n tokens back
a term has met at most n + d sums and n decays, each off by 2^-23, and two sums of the four partial
sums of a warp and of the warps (13 more): (2 n + d + 13) 2^-23 of the sums over absolute values.
State of a prompt with one token whose k is not 0: a product of three bf16 parts, which hold the
weighed v's 24 bits, with k is exact but for the three sums (3 x 2^-24); the weight's exponent G (in powers
of two) is off by 18 x 2^-24 G, its exponential by 2^-22 and its product with v by 2^-24; each
later chunk's decay adds 2^-22.  Two parts instead of three would be off by up to 2^-17."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean
from oracle import ops
from test_gpu_linear import Step

pytestmark = pytest.mark.gpu


def definition(s):
    (hq, hkv), d = s.heads, s.d
    rows = s.fused[:s.total].double().numpy().reshape(s.total, -1, d)
    g = s.g.double().numpy()
    return ops.linear_attention(rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], s.qsl.numpy(),
                                g[:s.total] if g.ndim == 2 else g, s.state.double().numpy(),
                                s.state_in.numpy(), s.state_out.numpy(), s.scale)


@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (32, 8, 128), (6, 6, 128), (16, 1, 64), (34, 1, 128)])
@pytest.mark.parametrize("lens", [[1] * 9, [2, 5, 8, 1, 3, 7], [8] * 20, [6, 0, 1, 4, 90, 8]])
def test_recurrent_form_rounds_the_output_alone(lens, hq, hkv, d, decay):
    """Requests of up to 8 tokens, alone and beside a prompt (which is left out of the check)."""
    s = Step(lens, hq, hkv, d, decay=decay, seed=sum(lens) + hq, fresh=(1,))
    t = s.to_dev()
    s.call(t)
    out, state, mag, smag = definition(s)
    got, got_state = t["out"].double().cpu().numpy(), t["state"].double().cpu().numpy()
    for b, n in enumerate(lens):
        if n > 8:
            continue
        rows = slice(int(s.qsl[b]), int(s.qsl[b]) + n)
        fp32 = (2 * n + d + 13) * 2.0 ** -23
        err = np.abs(got - out)[rows]
        bound = 2.0 ** -8 * np.abs(out[rows]) + fp32 * mag[rows] + 1e-30
        assert np.all(err <= bound), (b, np.max(err / bound))
        slot = int(s.state_out[b])
        err = np.abs(got_state[slot] - state[slot])
        assert np.all(err <= 2 * n * 2.0 ** -23 * smag[slot] + 1e-30), (b, n)
    assert_status_clean()


@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (4, 2, 64), (2, 2, 128), (4, 2, 128)])
@pytest.mark.parametrize("T,at", [(9, 0), (64, 5), (128, 100), (300, 130), (40, 38), (700, 690)])
def test_a_prompt_keeps_all_digits_of_its_state(T, at, hq, hkv, d):
    """(700 tokens of these heads: a cluster shares the request.)"""
    s = Step([T], hq, hkv, d, seed=T + d, fresh=(0,))
    s.g = s.g * 0.2
    k = s.fused[:, hq * d:(hq + hkv) * d]
    k[:at] = 0
    k[at + 1:] = 0
    t = s.to_dev()
    s.call(t)
    torch.cuda.synchronize()
    _, state, _, _ = definition(s)
    slot = int(s.state_out[0])
    got, want = t["state"][slot].double().cpu().numpy(), state[slot]
    G = -s.g.double().numpy()[at + 1:].sum(0) / math.log(2)
    tol = math.log(2) * 18 * 2.0 ** -24 * G + 2.0 ** -22 + 4 * 2.0 ** -24 + (T // 64 + 1) * 2.0 ** -22
    err = np.abs(got - want)
    bound = tol[:, None, None] * np.abs(want) + 2.0 ** -120
    assert np.all(err <= bound), np.max(err / bound)
    assert np.max(np.abs(want)) > 2.0 ** -100   # (beside which the 2^-120 is nothing)
    assert_status_clean()


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (2, 2, 128)])
@pytest.mark.parametrize("starts", [[0, 3, 2, 105], [0, 3, 103, 106], [-1, 3, 103, 105],
                                    [0, 3, 2**31 - 1, 105], [0, 50, 40, 105], [0, 3, 3, 105]])
def test_bad_starts_leave_the_other_requests_right(starts, hq, hkv, d):
    """Requests whose rows lie outside the call's are skipped: their rows (where no other request
    has them) and slots keep what stood there, and the others get what they should.  (A row that
    bad starts give to two requests gets either's output.)"""
    s = Step([3, 100, 2], hq, hkv, d, seed=3)
    good = [0 <= starts[b] <= starts[b + 1] <= s.total for b in range(3)]
    t = s.to_dev()
    t["qsl"].copy_(torch.tensor(starts))
    s.call(t)
    torch.cuda.synchronize()
    assert pk.read_device_status(clear=True) == (0 if all(good) else pk.PA_DEV_BAD_METADATA)
    got, got_state = t["out"].double().cpu().numpy(), t["state"].double().cpu().numpy()
    owners = np.zeros(s.total, int)
    for b in range(3):
        if good[b]:
            owners[starts[b]:starts[b + 1]] += 1
    for b in range(3):
        slot = int(s.state_out[b])
        if not good[b]:
            assert np.array_equal(got_state[slot], s.state[slot].double().numpy()), b
            continue
        one = Step([3, 100, 2], hq, hkv, d, seed=3)
        one.qsl = torch.tensor([starts[b], starts[b + 1]], dtype=torch.int32)
        one.state_in, one.state_out = s.state_in[b:b + 1], s.state_out[b:b + 1]
        out, state, mag, smag = definition(one)
        n = starts[b + 1] - starts[b]
        rows = starts[b] + np.flatnonzero(owners[starts[b]:starts[b + 1]] == 1)
        bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -12) * mag + 1e-30
        assert np.all(np.abs(got - out)[rows] <= bound[rows]), b
        tol = (2.0 ** -16 + (2 * n + 2 * d) * 2.0 ** -23) * smag[slot] + 1e-30
        assert np.all(np.abs(got_state[slot] - state[slot]) <= tol), b
    assert np.all(got[owners == 0] == 7)


@pytest.mark.parametrize("far", ["q", "k", "v"])
@pytest.mark.parametrize("hq", [2, 4])
def test_prompts_with_token_rows_far_apart(far, hq):
    """Token rows 2^29 elements (1 GB) apart, read through the prompt kernel's tensor maps."""
    s = Step([11, 1], hq, 2, 64, seed=hq)
    t = s.to_dev()
    rows = torch.empty(((s.total - 1) << 29) + 1024, dtype=torch.bfloat16, device=DEV)
    wide = rows.as_strided(tuple(t[far].shape), (1 << 29, 64, 1))
    wide.copy_(t[far])
    t[far] = wide
    s.call(t)
    s.check(t)
    assert_status_clean()
