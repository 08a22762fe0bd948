"""pa_linear_attention on the GPU against the token-by-token definition in float64.

Tolerances, with mag = the same sums over the absolute values of every factor.
out: rounded to bf16, at most 2^-8 of its value; prompts take the decayed products q k and
the state before a chunk through one rounding to bf16 each, at most 2^-8 of mag together
(they multiply disjoint terms of the sum).  Everything else is fp32: n tokens back, a term
has met at most n + 2 d sums and n decays of relative error 2^-23 (a chunk's decay is one
exponential of a difference of sums of logarithms, off by 2^-23 times the sum's size: the
tests' logarithms stay above -104 a token, and a chunk holds at most 128, where what a sum
of that size still multiplies is below 2^-100): (2 n + 2 d) 2^-23 < 2^-12 of mag for n < 900.
state: fp32 alone, and k times its decay in pieces of bf16 whose rest is below 2^-16 of it."""
import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean
from oracle import ops

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, lens, hq, hkv, d, decay="token", fresh=(), drop=(), in_place=False, seed=0,
                 pad=0, fused=True):
        g = torch.Generator().manual_seed(seed)
        B, self.lens = len(lens), lens
        self.qsl = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
        self.total = int(self.qsl[-1])
        T = self.total + pad
        rows = torch.randn((T, (hq + 2 * hkv) * d), generator=g).to(torch.bfloat16)
        self.fused, self.heads, self.d = rows, (hq, hkv), d
        if decay == "head":
            self.g = torch.log1p(-2.0 ** (-1 - 5 * torch.arange(hkv) / hkv))
        else:
            self.g = -torch.exp(torch.randn((T, hkv), generator=g) * 1.5 - 2)
        self.state = torch.randn((2 * B + 1, hkv, d, d), generator=g)
        slots = torch.randperm(2 * B + 1, generator=g).to(torch.int32)
        self.state_in = slots[:B].clone()
        self.state_out = (slots[:B] if in_place else slots[B:2 * B]).clone()
        for b in fresh:
            self.state_in[b] = -1 - b
        for b in drop:
            self.state_out[b] = -1 - b
        self.scale = d ** -0.5
        self.split = fused

    def to_dev(self):
        t = {x: getattr(self, x).to(DEV) for x in ("qsl", "g", "state", "state_in", "state_out")}
        (hq, hkv), d, fused = self.heads, self.d, self.fused.to(DEV)
        t["q"], t["k"], t["v"] = (x.view(x.shape[0], -1, d) for x in
                                  fused.split([hq * d, hkv * d, hkv * d], dim=1))
        if not self.split:
            t["q"], t["k"], t["v"] = (t[x].contiguous() for x in "qkv")
        t["out"] = torch.full((fused.shape[0], hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
        return t

    def call(self, t, **kw):
        return pk.pa_linear_attention(t["q"], t["k"], t["v"], t["qsl"], t["g"], t["state"],
                                      t["state_in"], t["state_out"], self.scale, t["out"], **kw)

    def check(self, t, state0=None):
        torch.cuda.synchronize()
        (hq, hkv), d = self.heads, self.d
        rows = self.fused[:self.total].double().numpy().reshape(self.total, -1, d)
        g = self.g.double().numpy()
        out, state, mag, smag = ops.linear_attention(
            rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], self.qsl.numpy(),
            g[:self.total] if g.ndim == 2 else g,
            (self.state if state0 is None else state0).double().numpy(), self.state_in.numpy(),
            self.state_out.numpy(), self.scale)
        got, got_state = t["out"].double().cpu().numpy(), t["state"].double().cpu().numpy()
        assert np.all(got[self.total:] == 7)
        got = got[:self.total]
        bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -12) * mag + 1e-30
        assert np.all(np.abs(got - out) <= bound), np.max(np.abs(got - out) / bound)
        written = set(x for x in self.state_out.tolist() if x >= 0)
        n = max(self.lens, default=0)
        for slot in range(len(state)):
            if slot in written:
                tol = (2.0 ** -16 + (2 * n + 2 * d) * 2.0 ** -23) * smag[slot] + 1e-30
                err = np.abs(got_state[slot] - state[slot])
                assert np.all(err <= tol), (slot, np.max(err / tol))
            else:
                assert np.array_equal(got_state[slot], state[slot]), slot


def run(lens, hq, hkv, d, **kw):
    s = Step(lens, hq, hkv, d, **kw)
    t = s.to_dev()
    s.call(t)
    s.check(t)
    assert_status_clean()
    return s, t


@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 385])
def test_lengths(n, d, decay):
    run([n], 4, 2, d, decay=decay, seed=n)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (6, 6), (3, 1), (12, 4), (14, 2), (16, 1), (32, 8),
                                    (128, 1)])
def test_heads(hq, hkv, d):
    run([1, 3, 70, 0, 9, 130], hq, hkv, d, seed=hq, pad=3, fresh=(1,), drop=(2,))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_slots(d, in_place):
    """Fresh and dropped states; requests without tokens copy, clear or keep their slot."""
    run([1, 70, 0, 5, 90, 0, 0, 1, 0], 4, 2, d, in_place=in_place, fresh=(0, 4, 5), drop=(3, 4, 6),
        seed=5, pad=70)


@pytest.mark.parametrize("d", [64, 128])
def test_long_prompts(d):
    """Longer than a segment of the prompt kernels, beside short rows."""
    run([700, 1, 300, 5, 1, 513], 4, 2, d, seed=1)
    run([800], 2, 1, d, seed=2, decay="head", in_place=True)


@pytest.mark.parametrize("d", [64, 128])
def test_decays(d):
    """No decay at all, states cleared in the middle, logarithms that count as 0."""
    lens = [90, 1, 200, 4]
    for values in ([0.0], [0.0, -104.0], [float("-inf"), -0.1, -0.2, -0.05], [-40.0, -1e-3],
                   [0.5, float("nan"), -0.25], [-1000.0, -1e30, -0.01]):
        s = Step(lens, 4, 2, d, seed=len(values))
        pick = torch.randint(len(values), s.g.shape, generator=torch.Generator().manual_seed(1))
        if len(values) == 2:
            pick = (torch.rand(s.g.shape, generator=torch.Generator().manual_seed(2)) < 0.9).long()
            values = values[::-1] if values[0] < -1 else values
            pick = 1 - pick if values[0] > -1 else pick
        s.g = torch.tensor(values)[pick]
        t = s.to_dev()
        s.call(t)
        s.check(t)
    assert_status_clean()


@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [8, 9, 16, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 257, 300, 640])
def test_groups_of_one_head(n, d, decay):
    """Tiles of one head: other chunks than a group's."""
    run([n], 2, 2, d, decay=decay, seed=n)


@pytest.mark.parametrize("d", [64, 128])
def test_groups_of_one_head_side_by_side(d):
    run([700, 1, 300, 5, 1, 513, 128, 0, 129], 3, 3, d, seed=1, pad=5, fresh=(0,), drop=(2,))
    run([800], 1, 1, d, seed=2, decay="head", in_place=True)
    run([(1, 0, 5, 140, 40)[i % 5] for i in range(200)], 2, 2, d, seed=4)
    s = Step([90, 260, 4], 2, 2, d, seed=5, fused=False)
    pick = torch.randint(4, s.g.shape, generator=torch.Generator().manual_seed(1))
    s.g = torch.tensor([float("-inf"), -0.1, -0.2, -0.05])[pick]
    t = s.to_dev()
    t["out"] = torch.full(((t["out"].numel() + 8),), 7.0, dtype=torch.bfloat16,
                          device=DEV)[8:].view(t["out"].shape)   # 16 bytes off the 32
    s.call(t)
    s.check(t)
    assert_status_clean()


def test_many_requests():
    run([1] * 300, 4, 2, 64, seed=3)
    run([(1, 0, 5, 1, 40)[i % 5] for i in range(1300)], 2, 1, 64, seed=4)


def test_steps_carry_their_state():
    """A prompt in chunks and single tokens gives what it gives in one call."""
    s = Step([300], 8, 2, 128, seed=7, in_place=True, fresh=(0,))
    t = s.to_dev()
    out, done = t["out"], 0
    slot = torch.tensor([2], dtype=torch.int32, device=DEV)
    none = torch.tensor([-1], dtype=torch.int32, device=DEV)
    for n in (100, 1, 1, 64, 17, 3, 114):
        part = {x: t[x][done:done + n] for x in "qkv"}
        g = t["g"][done:done + n].contiguous()
        qsl = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        pk.pa_linear_attention(part["q"], part["k"], part["v"], qsl, g, t["state"],
                               none if done == 0 else slot, slot, s.scale, out[done:done + n])
        done += n
    s.state_out[0] = 2
    s.check(t)
    assert_status_clean()


def test_contiguous_and_padded_strides():
    run([40, 1, 130], 6, 3, 64, fused=False, seed=1)
    s = Step([40, 1, 130], 6, 3, 64, seed=2)
    t = s.to_dev()
    for x in "qkv":  # token rows 8 elements further apart than their heads need
        wide = torch.full((171, t[x].shape[1] * 64 + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, :-8] = t[x].reshape(171, -1)
        t[x] = wide[:, :-8].view(171, -1, 64)
    s.call(t)
    s.check(t)
    assert_status_clean()


def test_bad_slots_and_starts_are_flagged():
    s = Step([3, 100, 2], 4, 2, 64, seed=3)
    t = s.to_dev()
    t["state_in"][0] = len(s.state)
    t["state_out"][1] = len(s.state) + 5
    s.call(t)
    s.state_in[0] = s.state_out[1] = -1
    s.check(t)
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_SLOT
    for starts in ([0, 3, 2, 105], [0, 3, 103, 106], [-1, 3, 103, 105], [0, 3, 2**31 - 1, 105]):
        t = s.to_dev()
        t["qsl"].copy_(torch.tensor(starts))
        before = t["state"].clone()
        s.call(t)
        torch.cuda.synchronize()
        assert pk.read_device_status(clear=True) & pk.PA_DEV_BAD_METADATA
        bad = [b for b in range(3) if not 0 <= starts[b] <= starts[b + 1] <= s.total]
        for b in bad:
            if s.state_out[b] >= 0:
                assert torch.equal(t["state"][s.state_out[b]], before[s.state_out[b]])


def test_padded_graphs_share_a_workspace():
    graphs = []
    ws = pk.alloc_workspace(max(pk.linear_workspace_size(12, 400, 8, 2, 128),
                                pk.linear_workspace_size(5, 300, 8, 2, 128)), DEV)
    for size, tokens in ((12, 400), (5, 300)):
        s = Step([tokens] + [0] * (size - 1), 8, 2, 128)
        t = s.to_dev()
        s.call(t, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.call(t, workspace=ws)
        graphs.append((size, tokens, t, graph))
    rng = np.random.default_rng(1)
    for turn in range(6):
        size, tokens, t, graph = graphs[turn % 2]
        n = size - turn // 2
        lens = [int(x) for x in rng.choice([1, 1, 5, 30, 70, 90], n)]
        while sum(lens) > tokens:
            lens[lens.index(max(lens))] = 1
        s = Step(lens + [0] * (size - n), 8, 2, 128, seed=turn, pad=tokens - sum(lens),
                 fresh=range(n, size), drop=range(n, size))
        u = s.to_dev()
        for x in ("q", "k", "v", "qsl", "g", "state", "state_in", "state_out", "out"):
            t[x].copy_(u[x])
        graph.replay()
        s.check(t)
    assert_status_clean()


def test_other_stream_and_repeat():
    s = Step([300, 1, 5, 100], 8, 2, 128, seed=6)
    t = s.to_dev()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = s.call(t, stream=side)
    side.synchronize()
    s.check(t)
    first, state = t["out"].clone(), t["state"].clone()
    for _ in range(5):
        s.call(t, workspace=ws)
        assert torch.equal(first, t["out"]) and torch.equal(state, t["state"])
    assert_status_clean()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [2, 6])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_rows_stay_other_rows(bad, hq, d):
    """What stands in the next request's rows, or behind the last, reaches no sum."""
    lens = [70, 33, 1, 100, 5, 64, 9, 200]
    s = Step(lens, hq, 2, d, seed=8, pad=150)
    t, u = s.to_dev(), s.to_dev()
    s.call(t)
    starts = s.qsl.tolist()
    spoilt = (1, 4)
    for x in "qkv":
        for b in spoilt:
            u[x][starts[b]:starts[b + 1]] = bad
        u[x][s.total:] = bad
    u["g"][s.total:] = bad
    s.call(u)
    torch.cuda.synchronize()
    for b in set(range(len(lens))) - set(spoilt):
        rows = slice(starts[b], starts[b + 1])
        assert torch.equal(t["out"][rows], u["out"][rows]), b
        slot = s.state_out[b]
        assert torch.equal(t["state"][slot], u["state"][slot]), b
    assert torch.all(u["out"][s.total:] == 7)
    assert_status_clean()


def test_steps_behind_each_other_and_beside():
    """Steps of prompts and short rows in place, one behind the other without a wait, and the
    same on two streams at once, give what they give one by one."""
    lens = [300, 1, 1, 5, 90, 1, 8, 9] + [1] * 40
    s = Step(lens, 4, 2, 128, seed=9, in_place=True)
    one = s.to_dev()
    for _ in range(4):
        s.call(one)
        torch.cuda.synchronize()
    s.g = s.g.clone()
    steps = [s.to_dev() for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for t, side in zip(steps, streams):
            s.call(t, stream=side)
    torch.cuda.synchronize()
    for t in steps:
        assert torch.equal(t["out"], one["out"]) and torch.equal(t["state"], one["state"])
    assert_status_clean()


@pytest.mark.parametrize("n", [5, 70])
def test_offsets_past_32_bits(n):
    """A pool of more than 2^32 bytes of states, and token rows 2^29 elements apart."""
    s = Step([n, 1], 4, 2, 64, seed=n)
    t = s.to_dev()
    pool = torch.empty((264000, 2, 64, 64), device=DEV)   # 8192 elements a slot, 8.6 GB
    slots = [263999, 262145, 131073, 5]
    t["state_in"].copy_(torch.tensor(slots[:2]))
    t["state_out"].copy_(torch.tensor(slots[2:]))
    pool[slots[:2]] = t["state"][s.state_in.long().to(DEV)]
    rows = torch.empty(((s.total - 1) << 29) + 1024, dtype=torch.bfloat16, device=DEV) \
        if n == 5 else None
    if rows is not None:
        far = rows.as_strided((s.total, 4, 64), (1 << 29, 64, 1))
        far.copy_(t["q"])
        t["q"] = far
    small = t["state"]
    t["state"] = pool
    s.call(t)
    small[s.state_out.long().to(DEV)] = pool[slots[2:]]
    t["state"] = small
    s.check(t)
    assert_status_clean()


def test_refusals():
    s = Step([3, 2], 4, 2, 64)
    t = s.to_dev()
    ws = s.call(t)
    for kw in ({}, {"workspace": ws}):
        for name in ("qsl", "g", "state", "state_in", "state_out", "q", "k", "v", "out"):
            with pytest.raises(TypeError):
                s.call({**t, name: t[name].double()}, **kw)
            with pytest.raises(ValueError):
                s.call({**t, name: t[name].cpu()}, **kw)
        for name in ("qsl", "g", "state_out", "k", "v", "out"):
            with pytest.raises(ValueError):
                s.call({**t, name: t[name][:-1]}, **kw)
        with pytest.raises(ValueError):
            s.call({**t, "state": t["state"][:, :1].contiguous()}, **kw)
        with pytest.raises(pk.PaError):
            s.scale = float("inf")
            s.call(t, **kw)
        s.scale = 0.125
    assert_status_clean()


def test_a_wait_that_runs_out():
    """CTA 0 loads one chunk: its waits give up after 2 s, the status says so, and the next call
    is right again.  One CTA to a request, and a cluster (whose barriers are met all the same)."""
    for lens in ([200] * 90, [900]):
        s = Step(lens, 4, 2, 128, seed=1)
        t = s.to_dev()
        pk.set_test_stall(pk.PA_TEST_STALL_LINEAR)
        try:
            s.call(t)
        finally:
            pk.set_test_stall(pk.PA_TEST_STALL_NONE)
        torch.cuda.synchronize()
        assert pk.read_device_status(clear=True) == pk.PA_DEV_WAIT_TIMEOUT
        assert pk.read_device_status() == 0
        t = s.to_dev()
        s.call(t)
        s.check(t)
        assert_status_clean()
