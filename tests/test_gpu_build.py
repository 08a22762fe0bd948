"""pa_build_step on the GPU against the row-by-row definition: every output equal, every
table entry and list word that the call has no business with untouched."""
import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean
from oracle import ops

pytestmark = pytest.mark.gpu


class Batch:
    """A persistent batch: rows' lengths, tables and a free list whose ring starts anywhere."""

    def __init__(self, rows, bs, width, spare=8, pad=0, head=None, holes=False, seed=0):
        rng = np.random.default_rng(seed)
        self.bs, self.width, self.q = bs, width, np.array([n for n, _ in rows], np.int32)
        self.cached = np.array([c for _, c in rows], np.int32)
        up = lambda x: -(-x // bs)  # noqa: E731
        have = [up(c) for _, c in rows]
        need = sum(up(c + n) - up(c) for n, c in rows if n > 0)
        free = max(0, need + spare)
        self.num_blocks = sum(have) + free + 1
        perm = rng.permutation(self.num_blocks).astype(np.int32)
        self.table = rng.integers(-9, -1, (len(rows), width)).astype(np.int32)  # never to be read
        at = 0
        for b, n in enumerate(have):
            self.table[b, :n] = perm[at:at + n]
            if holes and n > 3:  # blocks given back behind a window
                self.table[b, 1:n - 1][rng.random(n - 2) < 0.5] = -1
            at += n
        cap = self.num_blocks
        self.head = int(rng.integers(cap)) if head is None else head % cap
        self.count = free
        self.ring = np.full(cap, -7, np.int32)
        self.ring[(self.head + np.arange(free)) % cap] = perm[at:at + free]
        self.tokens = int(np.maximum(self.q, 0).sum()) + pad

    def expected(self):
        return ops.build_step(self.q, self.cached, self.table, self.ring, self.head, self.count,
                              self.tokens, self.bs)

    def on_gpu(self):
        t = lambda x: torch.from_numpy(np.array(x)).to(DEV)  # noqa: E731
        B, i32 = len(self.q), dict(dtype=torch.int32, device=DEV)
        return {"q": t(self.q), "cached": t(self.cached), "table": t(self.table),
                "ring": t(self.ring), "state_in": torch.tensor([self.head, self.count, 5, 6], **i32),
                "state": torch.full((4,), -3, **i32), "qsl": torch.full((B + 1,), -3, **i32),
                "ctx": torch.full((B,), -3, **i32), "seq": torch.full((B,), -3, **i32),
                "slots": torch.full((self.tokens,), -3, dtype=torch.int64, device=DEV),
                "positions": torch.full((self.tokens,), -3, **i32)}

    def call(self, t, stream=None):
        pk.pa_build_step(t["q"], t["cached"], t["table"], t["ring"], t["state_in"],
                         self.num_blocks, self.bs, t["qsl"], t["ctx"], t["seq"], t["slots"],
                         t["positions"], free_state_out=t["state"], stream=stream)


def same(t, want):
    torch.cuda.synchronize()
    for name in ("qsl", "ctx", "seq", "slots", "positions", "table", "ring", "state"):
        got = t[name].cpu().numpy()
        assert np.array_equal(got, want[name]), (name, got, want[name])


def check(batch, status=0):
    t, want = batch.on_gpu(), batch.expected()
    batch.call(t)
    same(t, want)
    assert pk.read_device_status(clear=True) == status
    assert torch.equal(t["cached"].cpu(), torch.from_numpy(batch.cached))
    return want


def random_rows(n, seed, longest=100, ctx=300):
    rng = np.random.default_rng(seed)
    kind = rng.choice([-1, 0, 1, 5, 2], n, p=[0.15, 0.2, 0.4, 0.1, 0.15])
    return [(int(rng.integers(1, longest)) if k == 2 else int(k), int(rng.integers(0, ctx)))
            for k in kind]


@pytest.mark.parametrize("rows", [[(1, 0)], [(1, 15)], [(1, 16)], [(1, 17)], [(16, 0)], [(17, 0)],
                                  [(0, 5)], [(-1, 33)], [(-1, 0)], [(0, 0), (3, 13), (0, 7)],
                                  [(-4, 40), (40, 0), (-1, 16)], [(33, 31)] * 3])
def test_small(rows):
    check(Batch(rows, 16, 8))
    assert check(Batch(rows, 16, 8, spare=0, pad=3))["state"][2] == 0


@pytest.mark.parametrize("bs", [16, 48, 256])
@pytest.mark.parametrize("n", [2, 31, 33, 300, 1023, 1024, 1025, 2500])
def test_batches(n, bs):
    check(Batch(random_rows(n, n + bs), bs, 26, pad=n % 70, holes=n % 2 == 1, seed=n))


@pytest.mark.parametrize("head", [0, 1, -1, -5])
def test_the_list_goes_round(head):
    check(Batch([(70, 3), (-1, 90), (1, 16), (-1, 200)], 16, 20, head=head, spare=1))


def test_most_rows_and_many_tokens():
    check(Batch([(1, i % 37) for i in range(8192)], 16, 4))
    check(Batch([(5000, 123), (-1, 4000), (0, 9), (61000, 0), (1, 64)], 32, 2000, pad=777))


def test_all_rows_done_or_idle():
    check(Batch([(-1, 37), (0, 12), (-1, 0)], 16, 5, pad=4))
    check(Batch([(0, 0)] * 3, 16, 5, pad=0))
    check(Batch([], 16, 5, pad=4))


@pytest.mark.parametrize("holes", [False, True])
def test_long_rows_given_back(holes):
    check(Batch([(-1, 20000), (1, 5), (-1, 31999), (-1, 16)], 16, 2000, holes=holes))


def test_list_too_short():
    b = Batch([(40, 10), (-1, 50), (1, 16)], 16, 8, spare=-1, pad=2)
    want = check(b, pk.PA_DEV_NO_BLOCKS)
    assert want["state"].tolist() == [b.head, b.count, 1, 0] and want["qsl"][-1] == 0
    assert np.array_equal(want["table"], b.table) and np.array_equal(want["ring"], b.ring)
    # blocks given back by this very step do not count
    check(Batch([(40, 0), (-1, 160)], 16, 10, spare=-1), pk.PA_DEV_NO_BLOCKS)


@pytest.mark.parametrize("what", ["tokens", "table", "negative", "head", "count", "huge"])
def test_refused_steps(what):
    b = Batch([(3, 10), (-1, 50), (30, 97), (0, 3)], 16, 8, pad=5)
    if what == "tokens":
        b.tokens -= 6
    elif what == "table":
        b.q[2] = 32
    elif what == "negative":
        b.cached[3] = -1
    elif what == "head":
        b.head = len(b.ring)
    elif what == "count":
        b.count = len(b.ring) + 1
    else:
        b.q[:] = 2**31 - 1
    assert check(b, pk.PA_DEV_BAD_METADATA)["bad"]


def test_ids_outside_the_pool():
    b = Batch([(1, 16), (1, 20)], 16, 4)
    b.ring[b.head] = b.num_blocks + 3      # row 0's new block
    b.table[1, 1] = -2                     # row 1's open block
    t = b.on_gpu()
    b.call(t)
    torch.cuda.synchronize()
    assert t["slots"].tolist() == [-1, -1]
    assert t["table"][0, 1].item() == b.num_blocks - 1 and t["table"][1, 1].item() == -2
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_BLOCK


def test_a_list_that_would_overflow():
    """Ids that stand twice (a row and the list) can give back more than the ring holds."""
    b = Batch([(-1, 64)], 16, 4)
    t = b.on_gpu()
    cap = len(b.ring)
    t["state_in"][1] = cap - 1
    before = t["ring"].clone()
    b.call(t)
    torch.cuda.synchronize()
    assert t["state"].tolist() == [b.head, cap, 0, 0]
    last = (b.head + cap - 1) % cap
    before[last] = t["table"][0, 0]
    assert torch.equal(t["ring"], before)
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_METADATA


@pytest.mark.parametrize("what", ["tokens", "table", "negative", "head", "count", "huge", "short"])
def test_refused_large_steps(what):
    rows = [(700, 10), (-1, 50), (1500, 97), (0, 3), (-1, 2000), (9, 40)]
    b = Batch(rows, 16, 130, pad=5, spare=-1 if what == "short" else 8)
    if what == "tokens":
        b.tokens -= 6
    elif what == "table":
        b.q[2] = 130 * 16 - 96
    elif what == "negative":
        b.cached[3] = -1
    elif what == "head":
        b.head = -1
    elif what == "count":
        b.count = -1
    elif what == "huge":
        b.q[:] = 2**31 - 1
    want = check(b, pk.PA_DEV_NO_BLOCKS if what == "short" else pk.PA_DEV_BAD_METADATA)
    assert want["qsl"][-1] == 0 and np.array_equal(want["table"], b.table)


def test_ids_outside_the_pool_in_a_large_step():
    b = Batch([(1, 16), (1500, 20), (-1, 70)], 16, 100)
    b.ring[b.head] = -5                    # row 0's new block
    b.table[1, 1] = b.num_blocks           # row 1's open block
    b.table[2, 3] = b.num_blocks + 9       # a block to be given back
    want, t = b.expected(), b.on_gpu()
    b.call(t)
    torch.cuda.synchronize()
    slots = t["slots"].cpu().numpy()
    assert np.all(slots[:1 + 12] == -1) and np.array_equal(slots[13:], want["slots"][13:])
    assert t["table"][0, 1].item() == 0 and t["table"][1, 1].item() == b.num_blocks
    back = b.table[2, [0, 1, 2, 4]]
    at = (b.head + b.count + np.arange(4)) % len(b.ring)
    assert np.array_equal(t["ring"].cpu().numpy()[at], back)
    assert t["state"][1].item() == b.count - 94 + 4
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_BLOCK


def test_a_list_that_would_overflow_in_a_large_step():
    """As above, by the cluster: given back by many rows, no further than the ring goes."""
    b = Batch([(-1, 64)] * 40 + [(1100, 0)], 16, 80, spare=0)
    t = b.on_gpu()
    cap, taken = len(b.ring), 69
    t["state_in"][1] = cap - 100
    b.call(t)
    torch.cuda.synchronize()
    assert t["state"].tolist() == [(b.head + taken) % cap, cap - 100 - taken + 100, 0, 0]
    at = (b.head + cap - 100 + np.arange(100)) % cap
    assert np.array_equal(t["ring"].cpu().numpy()[at], b.table[:25, :4].reshape(-1))
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_METADATA


@pytest.mark.parametrize("rows", [5, 3000])
def test_in_place(rows):
    """seq_lens over cached_lens and the list's state over itself."""
    b = Batch(random_rows(rows, 4), 16, 30)
    t, want = b.on_gpu(), b.expected()
    pk.pa_build_step(t["q"], t["cached"], t["table"], t["ring"], t["state_in"], b.num_blocks, b.bs,
                     t["qsl"], t["ctx"], t["cached"], t["slots"], t["positions"])
    t["seq"], t["state"] = t["cached"], t["state_in"]
    same(t, want)
    assert_status_clean()


def test_captured_loop_runs_by_itself():
    """Twenty steps of one graph: rows grow, finish and start over, with the list and the
    lengths carried from replay to replay."""
    rng = np.random.default_rng(3)
    b = Batch([(9, 0), (1, 30), (0, 0), (1, 15), (4, 100)], 16, 40, spare=60, pad=80)
    t = b.on_gpu()
    plan = np.where(rng.random((20, 5)) < 0.2, -1, rng.integers(0, 18, (20, 5))).astype(np.int32)
    args = (t["q"], t["cached"], t["table"], t["ring"], t["state_in"], b.num_blocks, b.bs,
            t["qsl"], t["ctx"], t["cached"], t["slots"], t["positions"])
    saved = {x: t[x].clone() for x in ("cached", "table", "ring", "state_in")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.pa_build_step(*args)
    for x in saved:
        t[x].copy_(saved[x])
    t["seq"], t["state"] = t["cached"], t["state_in"]
    for step in plan:
        t["q"].copy_(torch.from_numpy(step))
        b.q = step
        want = b.expected()
        graph.replay()
        same(t, want)
        b.cached, b.table, b.ring = want["seq"], want["table"], want["ring"]
        b.head, b.count = int(want["state"][0]), int(want["state"][1])
        live = [x for i, c in enumerate(b.cached) for x in b.table[i, :-(-c // 16)]]
        live += [b.ring[(b.head + i) % len(b.ring)] for i in range(b.count)]
        assert len(set(live)) == len(live) == b.num_blocks - 1   # every block once
    assert_status_clean()


def test_captured_loop_of_large_steps():
    """As above with prompts of thousands of tokens: in place, one replay behind the other."""
    rng = np.random.default_rng(5)
    b = Batch([(900, 0), (1, 30), (0, 0), (1, 15), (700, 100)], 32, 200, spare=600, pad=1500)
    t = b.on_gpu()
    plan = np.where(rng.random((12, 5)) < 0.25, -1, rng.choice([0, 1, 5, 333, 600], (12, 5)))
    plan = torch.from_numpy(plan.astype(np.int32)).to(DEV)
    graph = torch.cuda.CUDAGraph()
    saved = {x: t[x].clone() for x in ("cached", "table", "ring", "state_in")}
    with torch.cuda.graph(graph):
        pk.pa_build_step(t["q"], t["cached"], t["table"], t["ring"], t["state_in"], b.num_blocks,
                         b.bs, t["qsl"], t["ctx"], t["cached"], t["slots"], t["positions"])
    for x in saved:
        t[x].copy_(saved[x])
    for step in plan:   # (nothing waits for the one before)
        t["q"].copy_(step)
        graph.replay()
    for step in plan.cpu().numpy():
        b.q = step
        want = b.expected()
        assert not want["bad"] and want["state"][2] == 0
        b.cached, b.table, b.ring = want["seq"], want["table"], want["ring"]
        b.head, b.count = int(want["state"][0]), int(want["state"][1])
    t["seq"], t["state"] = t["cached"], t["state_in"]
    same(t, want)
    assert_status_clean()


def test_more_tokens_than_one_round():
    check(Batch([(7, 100), (170000, 3), (1, 8), (-1, 5000)], 256, 700, pad=41))


def test_other_stream_and_slices():
    b = Batch(random_rows(40, 8), 16, 30)
    t, want = b.on_gpu(), b.expected()
    for name in ("qsl", "ctx", "seq", "positions", "slots"):   # only element-aligned
        t[name] = torch.cat([t[name][:1], t[name]])[1:]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.call(t, stream=side)
    side.synchronize()
    same(t, want)
    assert_status_clean()


def test_refusals_of_the_binding():
    b = Batch([(1, 3), (2, 20)], 16, 4)
    t = b.on_gpu()
    names = ("q", "cached", "table", "ring", "state_in", "qsl", "ctx", "seq", "slots", "positions")
    for name in names:
        bad = dict(t)
        bad[name] = t[name].to(torch.int16)
        with pytest.raises(TypeError):
            b.call(bad)
        bad[name] = t[name].cpu()
        with pytest.raises(ValueError):
            b.call(bad)
    for name in ("cached", "table", "qsl", "ctx", "seq", "positions", "state"):
        with pytest.raises(ValueError):
            b.call({**t, name: t[name][:-1]})
    b.bs = 24
    with pytest.raises(pk.PaError):
        b.call(t)
