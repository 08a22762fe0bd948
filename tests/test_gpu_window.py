"""pa_window_attention on the GPU against the float64 definition: every table
entry and every key that no row sees is poisoned (-1 entries, NaN keys), so a
read of anything hidden shows.

Tolerances.  out is rounded to bf16 (at most 2^-8 of its value), and the
probabilities are rounded once before P V (bf16 2^-8, f16 less), which moves
out by at most 2^-8 sum_j p_j |v_j|; scores and sums in fp32 add less than
2^-12 of that sum (a score of 128 products has an error below
128 * 2^-24 * scale * sum |q k| < 2^-13 for the inputs here; the normaliser as
much).  lse inherits the scores' error, 2^-13, and fp32's own 2^-22 of it."""
import time

import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean, plan_header
from oracle import ops

pytestmark = pytest.mark.gpu

E4M3_NAN = 0x7F


class Step:
    """One windowed step: bf16 or e4m3 pool whose visible keys are normal values
    and whose every other element is NaN; hidden blocks' table entries are -1."""

    def __init__(self, requests, hq, hkv, d, bs, window, sinks, kv="bf16", seed=0, pad=0,
                 keep_tables=False):
        g = torch.Generator().manual_seed(seed)
        self.window, self.sinks, self.bs, self.kv, self.hkv = window, sinks, bs, kv, hkv
        self.requests = requests
        width = max(1, max(-(-(c + n) // bs) for c, n in requests))
        seen = [set(int(j) for p in range(c, c + n) for j in ops.visible_keys(p, window, sinks))
                for c, n in requests]
        need = [sorted({j // bs for j in s}) for s in seen]
        used = sum(len(x) for x in need)
        self.num_blocks = used + 3
        perm = torch.randperm(self.num_blocks, generator=g).tolist()
        table = torch.full((len(requests), width), -1, dtype=torch.int32)
        live = torch.zeros(self.num_blocks, bs, dtype=torch.bool)
        at = 0
        for b, cols in enumerate(need):
            for col in cols:
                table[b, col] = perm[at]
                for off in range(bs):
                    live[perm[at], off] = col * bs + off in seen[b]
                at += 1
        shape = (self.num_blocks, hkv, bs, d)
        k, v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        hidden = ~live[:, None, :, None]
        if kv == "bf16":
            self.k = k.masked_fill(hidden, float("nan")).to(torch.bfloat16)
            self.v = v.masked_fill(hidden, float("nan")).to(torch.bfloat16)
            self.ks = self.vs = None
            self.k64, self.v64 = self.k.double().numpy(), self.v.double().numpy()
        else:
            self.k, self.v = ((x * 16).to(torch.float8_e4m3fn).view(torch.uint8)
                              .masked_fill(hidden, E4M3_NAN) for x in (k, v))
            self.ks, self.vs = (0.04 + 0.05 * torch.rand(hkv, generator=g) for _ in "kv")
            self.k64, self.v64 = (x.view(torch.float8_e4m3fn).double().numpy() *
                                  s.double().numpy()[:, None, None]
                                  for x, s in ((self.k, self.ks), (self.v, self.vs)))
        i32 = dict(dtype=torch.int32)
        self.table = table
        self.qsl = torch.tensor(np.concatenate([[0], np.cumsum([n for _, n in requests])]), **i32)
        self.ctx = torch.tensor([c for c, _ in requests], **i32)
        self.seq = torch.tensor([c + n for c, n in requests], **i32)
        self.total = int(self.qsl[-1])
        self.q = torch.randn((self.total + pad, hq, d), generator=g).to(torch.bfloat16)
        self.scale = d ** -0.5
        self.staging = sum(len(x) for x, (_, n) in zip(need, requests) if n * hq // hkv > 64)

    def to_dev(self):
        t = {x: getattr(self, x).to(DEV) for x in ("q", "k", "v", "table", "qsl", "ctx", "seq")}
        t["ks"], t["vs"] = ((None, None) if self.ks is None
                            else (self.ks.to(DEV), self.vs.to(DEV)))
        t["out"] = torch.full_like(t["q"], 7.0)
        t["lse"] = torch.full(t["q"].shape[:2], 7.0, device=DEV)
        return t

    def call(self, t, **kw):
        kw.setdefault("staging_blocks", self.staging if self.kv == "e4m3" else 0)
        return pk.pa_window_attention(t["q"], t["k"], t["v"], t["table"], t["qsl"], t["ctx"],
                                      t["seq"], self.scale, self.window, self.sinks, t["out"],
                                      t["lse"], k_scale=t["ks"], v_scale=t["vs"], **kw)

    def check(self, t, what=""):
        n = self.total
        ref_o, ref_l, mag = ops.window_attention(
            self.q.double().numpy()[:n], self.k64, self.v64, self.table.numpy(), self.qsl.numpy(),
            self.ctx.numpy(), self.scale, self.window, self.sinks, self.bs)
        out, lse = t["out"].double().cpu().numpy(), t["lse"].double().cpu().numpy()
        assert np.all(out[n:] == 7.0) and np.all(lse[n:] == 7.0), "rows of no request written"
        err, lerr = np.abs(out[:n] - ref_o), np.abs(lse[:n] - ref_l)
        tol = 2.0 ** -8 * np.abs(ref_o) + (2.0 ** -8 + 2.0 ** -12) * mag
        ltol = 2.0 ** -13 + 2.0 ** -22 * np.abs(ref_l)
        assert np.all(np.isfinite(out[:n])) and np.all(np.isfinite(lse[:n])), what
        assert np.all(err <= tol), f"{what}: {np.max(err / tol)} of the tolerance"
        assert np.all(lerr <= ltol), f"{what}: lse {np.max(lerr / ltol)} of the tolerance"

    def run_and_check(self, **kw):
        t = self.to_dev()
        self.call(t, **kw)
        torch.cuda.synchronize()
        self.check(t, f"{self.requests[:4]} W={self.window} S={self.sinks} bs={self.bs}")
        assert_status_clean()
        return t


DECODE = [(0, 1), (1, 1), (15, 1), (16, 1), (63, 1), (64, 1), (100, 1), (333, 1), (700, 1)]
VERIFY = [(0, 5), (3, 2), (60, 5), (130, 3), (411, 5), (15, 7)]
CHUNKS = [(0, 150), (37, 70), (260, 129)]
MIXED = [(0, 90), (500, 1), (77, 5), (211, 64), (1, 1), (300, 140), (0, 0), (40, 0)]
WINDOWS = [(1, 0), (1, 3), (7, 0), (16, 4), (33, 17), (64, 1), (100, 130), (128, 0), (5000, 0),
           (31, 5000)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("requests", [DECODE, VERIFY, CHUNKS, MIXED],
                         ids=["decode", "verify", "chunks", "mixed"])
def test_bf16_128(requests, window, sinks):
    Step(requests, 8, 2, 128, 16, window, sinks, seed=window).run_and_check()


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("requests", [DECODE, MIXED], ids=["decode", "mixed"])
def test_e4m3(requests, window, sinks):
    Step(requests, 8, 2, 128, 16, window, sinks, kv="e4m3", seed=window).run_and_check()


@pytest.mark.parametrize("staged", [0, 1, 12])
def test_e4m3_long_requests_without_enough_staging_room(staged):
    st = Step(MIXED, 16, 2, 128, 32, 90, 9, kv="e4m3", seed=5)
    st.run_and_check(staging_blocks=staged)


@pytest.mark.parametrize("hq,hkv,d,bs,kv", [
    (4, 4, 64, 16, "bf16"), (14, 2, 64, 32, "bf16"), (16, 1, 128, 64, "bf16"),
    (5, 1, 128, 256, "bf16"), (6, 3, 64, 48, "bf16"), (128, 1, 64, 16, "bf16"),
    (14, 2, 128, 48, "e4m3"), (3, 3, 128, 16, "e4m3"), (32, 1, 128, 256, "e4m3")])
@pytest.mark.parametrize("window,sinks", [(20, 3), (200, 40)])
def test_heads_and_block_sizes(hq, hkv, d, bs, kv, window, sinks):
    Step([(0, 1), (250, 1), (90, 4), (130, 35), (0, 0), (600, 1)], hq, hkv, d, bs, window, sinks,
         kv=kv, seed=hq).run_and_check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_long_contexts_split_over_the_window(kv):
    """Few rows over long windows (the split and its fold), far into a context
    whose other blocks are gone."""
    Step([(20000, 1), (9000, 2)], 8, 2, 128, 16, 6000, 37, kv=kv, seed=3).run_and_check()


def test_far_positions_have_a_table_of_gone_blocks():
    """A position past 2^20 keys: table columns far out, all but the window's and
    the sinks' blocks given back."""
    Step([(1 << 20, 1), ((1 << 20) + 5, 3)], 4, 2, 64, 256, 300, 4, seed=4).run_and_check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_more_requests_than_a_plan_keeps_in_shared_memory(kv):
    """Over a thousand requests, decode rows and chunks among them."""
    rng = np.random.default_rng(5)
    reqs = [(int(c), 1) for c in rng.integers(0, 90, 1100)]
    reqs[7] = reqs[600] = (33, 40)
    reqs[1099] = (5, 70)
    Step(reqs, 4, 2, 128, 16, 30, 2, kv=kv, seed=6).run_and_check()


def test_many_pieces_of_an_unstaged_prompt():
    """An e4m3 prompt without staging room: one piece per 4 tokens, split-KV."""
    Step([(100, 700), (20, 3)], 16, 1, 128, 16, 64, 5, kv="e4m3",
         seed=7).run_and_check(staging_blocks=0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_padding_rows_are_left_alone(kv):
    Step([(30, 3), (0, 0), (200, 70)], 8, 2, 128, 16, 40, 4, kv=kv, pad=9).run_and_check()


def test_no_lse_and_a_kept_workspace():
    st = Step(MIXED, 8, 2, 128, 16, 50, 4)
    t = st.to_dev()
    ws = st.call(t)
    first = t["out"].clone()
    t["out"].fill_(3.0)
    assert st.call(t, workspace=ws) is ws
    torch.cuda.synchronize()
    assert torch.equal(t["out"], first)
    small = pk.alloc_workspace(4096, DEV)          # too small: a fresh one is used
    assert st.call(t, workspace=small) is not small
    torch.cuda.synchronize()
    assert torch.equal(t["out"], first)
    t["lse"], lse = None, t["lse"]
    st.call(t, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(t["out"], first)
    t["lse"] = lse
    st.check(t)
    assert_status_clean()


def test_a_window_past_every_context_equals_pa_attention():
    """The same keys as plain causal attention: both within the definition's
    tolerance, and the plain call's own result unchanged by a windowed one."""
    st = Step([(100, 1), (0, 90), (33, 5)], 8, 2, 128, 16, 10 ** 6, 0)
    t = st.to_dev()
    args = (t["q"], t["k"], t["v"], t["table"], t["qsl"], t["ctx"], t["seq"], st.scale)
    pk.pa_attention(*args, t["out"], t["lse"])
    torch.cuda.synchronize()
    plain = t["out"].clone()
    st.check(t, "pa_attention")
    st.call(t)
    torch.cuda.synchronize()
    st.check(t, "pa_window_attention")
    pk.pa_attention(*args, t["out"], t["lse"])
    torch.cuda.synchronize()
    assert torch.equal(t["out"], plain)
    assert_status_clean()


def test_other_stream_and_interleaved_calls():
    a = Step(DECODE, 8, 2, 128, 16, 50, 4, seed=1)
    b = Step(MIXED, 8, 2, 128, 16, 9, 0, kv="e4m3", seed=2)
    ta, tb = a.to_dev(), b.to_dev()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    wa = a.call(ta, stream=s1)
    wb = b.call(tb, stream=s2)
    for _ in range(4):
        a.call(ta, workspace=wa, stream=s1)
        b.call(tb, workspace=wb, stream=s2)
    torch.cuda.synchronize()
    a.check(ta)
    b.check(tb)
    assert_status_clean()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_graph_captured_once_serves_other_metadata(kv):
    """Captured on one batch, replayed on another of the same sizes (other
    contexts, another split of the tokens, one request empty)."""
    first = Step([(40, 1), (300, 5), (7, 70), (90, 1)], 8, 2, 128, 16, 60, 4, kv=kv, seed=1)
    other = Step([(511, 1), (0, 70), (13, 5), (480, 0)], 8, 2, 128, 16, 60, 4, kv=kv, seed=2, pad=1)
    assert other.q.shape == first.q.shape
    t, o = first.to_dev(), other.to_dev()
    width = max(t["table"].shape[1], o["table"].shape[1])
    n = max(t["k"].shape[0], o["k"].shape[0])

    def grown(x, size, dim, value):
        shape = list(x.shape)
        shape[dim] = size - shape[dim]
        return torch.cat([x, torch.full(shape, value, dtype=x.dtype, device=x.device)], dim)
    for x in (t, o):
        x["table"] = grown(x["table"], width, 1, -1).contiguous()
        for c in "kv":
            x[c] = grown(x[c], n, 0, E4M3_NAN if kv == "e4m3" else float("nan")).contiguous()
    room = max(first.staging, other.staging) if kv == "e4m3" else 0
    ws = first.call(t, staging_blocks=room)
    torch.cuda.synchronize()
    eager = t["out"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        first.call(t, workspace=ws, staging_blocks=room)
    t["out"].fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(t["out"], eager)
    first.check(t)
    for name in t:
        if t[name] is not None:
            t[name].copy_(o[name])
    g.replay()
    torch.cuda.synchronize()
    other.check(t)
    assert_status_clean()


def test_bad_block_and_bad_metadata_are_flagged():
    """A visible entry outside the pool is clamped and flagged; a request whose
    lengths disagree is skipped and flagged; the others are right."""
    st = Step([(40, 1), (50, 2), (60, 1)], 4, 2, 64, 16, 20, 2)
    t = st.to_dev()
    t["table"][0, 2] = st.num_blocks
    t["seq"][1] += 1
    st.call(t)
    torch.cuda.synchronize()
    assert pk.read_device_status() == pk.PA_DEV_BAD_BLOCK | pk.PA_DEV_BAD_METADATA
    assert torch.all(t["out"][1:3] == 7.0)
    ref, _, _ = ops.window_attention(st.q.double().numpy(), st.k64, st.v64, st.table.numpy(),
                                     st.qsl.numpy(), st.ctx.numpy(), st.scale, 20, 2, 16)
    assert np.abs(t["out"][3].double().cpu().numpy() - ref[3]).max() < 0.05


# Batches of at most 16 rows a request on average run as one kernel: clusters of
# CTAs for each (piece of 16 rows, kv head), in several rounds when there are many.
def many(n, spread, rng, new=(1, 2)):
    return [(int(c), int(m)) for c, m in zip(rng.integers(0, spread, n), rng.integers(*new, n))]


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (33, 17), (100, 130), (700, 5)])
def test_large_batches(kv, d, window, sinks):
    rng = np.random.default_rng(window)
    reqs = many(45, 900, rng, (1, 6)) + [(0, 1), (15, 1), (16, 1), (0, 0), (63, 4), (5, 0)]
    Step(reqs, 28, 7, d, 16, window, sinks, kv=kv, seed=window, pad=3).run_and_check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("group,bs,new", [(1, 64, 17), (5, 16, 5), (8, 48, 3), (16, 32, 3),
                                          (17, 16, 2)])
def test_large_batches_of_other_groups(kv, group, bs, new):
    """Pieces of 16 / group tokens; a group of 17 stays with the planned kernels."""
    rng = np.random.default_rng(group)
    reqs = many(80, 400, rng, (1, new)) + [(0, 0)] * 60
    assert group == 17 or sum(n for _, n in reqs) * group <= 16 * len(reqs)
    Step(reqs, 4 * group, 4, 128, bs, 130, 7, kv=kv, seed=group).run_and_check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_large_batches_of_many_jobs(kv):
    """Over 2000 jobs, a few of them long."""
    rng = np.random.default_rng(8)
    Step(many(260, 120, rng) + [(3000, 1), (2500, 2)], 16, 8, 128, 16, 2000, 20, kv=kv,
         seed=8).run_and_check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_large_batches_split_over_the_window(kv):
    Step([(5000 - 37 * i, 1) for i in range(40)], 16, 8, 128, 16, 1500, 37, kv=kv,
         seed=9).run_and_check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_large_batch_beside_prompt_chunks(kv):
    rng = np.random.default_rng(10)
    reqs = many(330, 400, rng, (1, 3)) + [(100, 300), (0, 140), (411, 70)]
    assert 512 <= sum(n for _, n in reqs) <= 4 * len(reqs)
    st = Step(reqs, 8, 2, 128, 16, 150, 9, kv=kv, seed=10)
    t = st.run_and_check()
    first = t["out"].clone()
    for _ in range(3):
        st.call(t)
    torch.cuda.synchronize()
    assert torch.equal(t["out"], first)


def test_a_large_batch_flags_a_bad_block_and_reads_inside_the_pool():
    rng = np.random.default_rng(11)
    st = Step(many(60, 300, rng), 16, 8, 128, 16, 100, 4, seed=11)
    t = st.to_dev()
    last = (int(st.ctx[5])) // 16
    t["table"][5, last] = st.num_blocks + 7
    st.call(t)
    torch.cuda.synchronize()
    assert pk.read_device_status(clear=True) & pk.PA_DEV_BAD_BLOCK
    t["table"][5, last] = st.table[5, last].item()
    st.call(t)
    torch.cuda.synchronize()
    st.check(t)
    assert_status_clean()


def test_a_large_batch_times_out_when_chunks_never_come():
    rng = np.random.default_rng(12)
    st = Step(many(60, 300, rng), 16, 8, 128, 16, 100, 4, seed=12)
    t = st.to_dev()
    pk.set_test_stall(pk.PA_TEST_STALL_SPLIT_KV)
    try:
        st.call(t)
        torch.cuda.synchronize()
    finally:
        pk.set_test_stall(pk.PA_TEST_STALL_NONE)
    assert pk.read_device_status(clear=True) & pk.PA_DEV_WAIT_TIMEOUT
    st.call(t)
    torch.cuda.synchronize()
    st.check(t)
    assert_status_clean()


# The same for steps whose pieces, kv heads and windows bound little work, whatever
# their requests are.
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("requests,window,sinks", [
    ([(0, 1)], 1, 0), ([(700, 1)], 128, 4), ([(5000, 1)], 4000, 9), ([(300, 3)], 40, 0),
    ([(31, 5), (0, 0), (64, 1), (15, 9)], 33, 17), ([(9, 40)], 7, 100),
    ([(100 * i, 1 + i % 3) for i in range(30)], 90, 3),
    ([(3 * i, i % 2) for i in range(128)], 20, 2)])
def test_small_steps(kv, d, requests, window, sinks):
    Step(requests, 8, 2, d, 16, window, sinks, kv=kv, seed=len(requests), pad=2).run_and_check()


@pytest.mark.parametrize("hq,hkv,bs", [(1, 1, 32), (16, 1, 64), (15, 3, 256), (17, 1, 16)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_small_steps_of_other_groups(hq, hkv, bs, kv):
    Step([(250, 1), (90, 4), (130, 18), (0, 2)], hq, hkv, 128, bs, 150, 20, kv=kv,
         seed=hq).run_and_check()


def test_small_step_in_a_graph_beside_another_on_its_own_stream():
    a = Step([(500, 1), (60, 2)], 8, 2, 128, 16, 300, 4, seed=1)
    b = Step([(80, 1)], 4, 4, 64, 16, 50, 0, seed=2)
    ta, tb = a.to_dev(), b.to_dev()
    wa, wb = a.call(ta), b.call(tb)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            a.call(ta, workspace=wa)
    s = torch.cuda.Stream()
    for _ in range(5):
        g.replay()
        b.call(tb, workspace=wb, stream=s)
    torch.cuda.synchronize()
    a.check(ta)
    b.check(tb)
    assert_status_clean()


def test_small_step_flags_bad_blocks_bad_metadata_and_a_wait_that_runs_out():
    st = Step([(40, 1), (50, 2), (900, 1)], 4, 2, 64, 16, 600, 2)
    t = st.to_dev()
    t["table"][0, 2] = st.num_blocks
    t["seq"][1] += 1
    st.call(t)
    torch.cuda.synchronize()
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_BLOCK | pk.PA_DEV_BAD_METADATA
    assert torch.all(t["out"][1:3] == 7.0)
    # overlapping requests want more pieces than the step's tokens allow
    over = Step([(5, 9), (5, 9), (5, 9)], 4, 1, 64, 16, 600, 0)
    t = over.to_dev()
    t["qsl"] = torch.tensor([0, 27, 0, 27], dtype=torch.int32, device=DEV)
    t["ctx"][0] = t["ctx"][2] = 0
    t["seq"][0] = t["seq"][2] = 27
    t["table"].clamp_(min=0)
    t["table"] = t["table"].repeat(1, 4).contiguous()
    over.call(t)
    torch.cuda.synchronize()
    status = pk.read_device_status(clear=True)
    assert status & pk.PA_DEV_PLAN_OVERFLOW and torch.all(t["out"] == 7.0)
    # request 0's first worker has two chunks, asks for one
    late = Step([(1000, 1)], 32, 8, 128, 16, 900, 0)
    t = late.to_dev()
    pk.set_test_stall(pk.PA_TEST_STALL_SPLIT_KV)
    try:
        late.call(t)
        torch.cuda.synchronize()
    finally:
        pk.set_test_stall(pk.PA_TEST_STALL_NONE)
    assert pk.read_device_status(clear=True) & pk.PA_DEV_WAIT_TIMEOUT
    late.run_and_check()


# The planned kernels: steps with more work and more rows a request, in which they
# run one after the other (under 512 tokens) or side by side.
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("kv,d,staged", [("bf16", 128, 0), ("bf16", 64, 0), ("e4m3", 128, 0),
                                         ("e4m3", 128, 1), ("e4m3", 128, 12),
                                         ("e4m3", 128, None)])
def test_planned_steps(kv, d, staged, window, sinks):
    kw = {} if staged is None else {"staging_blocks": staged}
    Step(MIXED, 64, 8, d, 16, window, sinks, kv=kv, seed=window).run_and_check(**kw)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_planned_steps_split_over_the_window(kv):
    Step([(16000 - 300 * i, 8) for i in range(8)], 8, 1, 128, 16, 14000, 37, kv=kv,
         seed=3).run_and_check()


def test_planned_step_at_far_positions():
    Step(MIXED + [((1 << 20) + 5, 70)], 64, 8, 64, 256, 300, 4, seed=4).run_and_check()


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128)])
def test_large_planned_steps(kv, d, window, sinks):
    Step(MIXED * 2 + CHUNKS + VERIFY * 4 + DECODE * 4, 16, 4, d, 16, window, sinks, kv=kv,
         seed=window).run_and_check()


def test_binding_takes_plain_calls_and_leaves_the_others():
    """The direct binding launches a documented call and hands every other back
    (-1) without a launch."""
    st = Step([(40, 1), (50, 2)], 4, 2, 64, 16, 20, 2)
    t = st.to_dev()
    ws = st.call(t)
    torch.cuda.synchronize()
    call = pk._load_direct().window_attention
    good = [t["q"], t["k"], t["v"], t["table"], t["qsl"], t["ctx"], t["seq"], st.scale, 20, 2,
            t["out"], t["lse"], ws, None, None, None]
    t["out"].fill_(7.0)
    assert call(*good) == 0 and call(*good[:13], torch.cuda.Stream(), None, None) == 0
    torch.cuda.synchronize()
    st.check(t)
    before = pk.lib().pa_kernel_launches()
    wrong = {0: [t["q"].float(), t["q"].cpu(), t["q"].transpose(0, 1), None, 3],
             1: [t["k"].view(torch.uint8), t["k"][0], t["k"][:, :, ::2]],
             2: [t["v"][1:]], 3: [t["table"].long(), t["table"][0], t["table"].t()],
             4: [t["qsl"][1:]], 5: [t["ctx"].cpu()], 6: [t["seq"].float()],
             7: ["1", t["ctx"]], 8: [20.5, 1 << 40, None], 9: ["2"],
             10: [t["out"][:, :1], t["out"].half()], 11: [t["lse"][1:], t["lse"].double()],
             12: [None, ws.cpu(), 5], 13: [7, "stream"], 14: [t["lse"]]}
    for i, values in wrong.items():
        for v in values:
            assert call(*good[:i], v, *good[i + 1:]) == -1, (i, v)
    assert call(*good[:15]) == -1 and call() == -1
    assert call(*good[:12], ws[:256], *good[13:]) == pk.PA_ERR_WORKSPACE
    assert call(*good[:8], 0, *good[9:]) == pk.PA_ERR_INVALID_ARG
    assert pk.lib().pa_kernel_launches() == before


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (33, 17), (90, 0)])
def test_many_short_jobs_of_a_warp_each(kv, d, window, sinks):
    rng = np.random.default_rng(window)
    reqs = many(150, 500, rng, (1, 4)) + [(0, 0)] * 40 + many(3, 40, rng, (9, 10))
    Step(reqs, 32, 8, d, 16, window, sinks, kv=kv, seed=window, pad=2).run_and_check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,window", [(129, 200), (300, 40), (1024, 20)])
def test_more_requests_than_threads_of_a_cta(kv, n, window):
    """Each thread scans several requests; few jobs, so clusters share them."""
    rng = np.random.default_rng(n)
    reqs = many(n, 300, rng)
    for i in range(0, n, 7):
        reqs[i] = (0, 0)
    reqs[n // 2] = (77, 9)
    Step(reqs, 4, 1, 128, 32, window, 5, kv=kv, seed=n).run_and_check()


@pytest.mark.parametrize("kv,d,n", [("bf16", 64, 300), ("bf16", 128, 300), ("e4m3", 128, 200)])
def test_many_requests_over_one_long_prefix(kv, d, n):
    """Every request has the same blocks, position and query, so each warp walks
    dozens of chunks (several batches of block ids) and all rows are equal."""
    one = Step([(4400, 1)], 4, 1, d, 16, 4300, 20, kv=kv, seed=n)
    t = one.to_dev()
    one.call(t)
    torch.cuda.synchronize()
    one.check(t)
    t["q"] = t["q"].repeat(n, 1, 1).contiguous()
    t["table"] = t["table"].repeat(n, 1).contiguous()
    t["qsl"] = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    t["ctx"], t["seq"] = t["ctx"].repeat(n), t["seq"].repeat(n)
    t["out"] = torch.full_like(t["q"], 7.0)
    t["lse"] = torch.full((n, 4), 7.0, device=DEV)
    one.call(t)
    torch.cuda.synchronize()
    assert torch.equal(t["out"], t["out"][:1].expand_as(t["out"]))
    assert torch.equal(t["lse"], t["lse"][:1].expand_as(t["lse"]))
    one.check({"out": t["out"][:1], "lse": t["lse"][:1]})
    assert_status_clean()


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 128), (32, 8, 64), (16, 1, 128)])
def test_prompts_and_short_rows_without_a_plan(hq, hkv, d, window, sinks):
    """bf16 steps of at most 8 requests: short rows in the one-kernel form, long
    requests' tiles found by the tensor-core kernel itself."""
    reqs = CHUNKS + [(0, 0), (100, 1), (40, 16), (64, 17), (300, 300)]
    Step(reqs, hq, hkv, d, 16, window, sinks, seed=window, pad=3).run_and_check()


def test_a_step_without_a_plan_skips_bad_and_overlapping_requests():
    st = Step([(40, 200), (50, 300), (60, 1), (700, 150)], 32, 8, 128, 16, 600, 2)
    t = st.to_dev()
    t["seq"][1] += 1
    st.call(t)
    torch.cuda.synchronize()
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_METADATA
    assert torch.all(t["out"][200:500] == 7.0)
    ref, _, mag = ops.window_attention(st.q.double().numpy(), st.k64, st.v64, st.table.numpy(),
                                       st.qsl.numpy(), st.ctx.numpy(), st.scale, 600, 2, 16)
    err = np.abs(t["out"].double().cpu().numpy() - ref)
    ok = err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mag
    assert ok[:200].all() and ok[500:].all()
    t = st.to_dev()
    t["qsl"][:] = torch.tensor([0, 200, 0, 651, 651], dtype=torch.int32, device=DEV)
    t["qsl"][1:4] = torch.tensor([651, 0, 651], dtype=torch.int32, device=DEV)
    t["ctx"][:] = 0
    t["seq"][:] = torch.tensor([651, 1, 651, 0], dtype=torch.int32, device=DEV)
    t["table"] = t["table"].clamp_(min=0).repeat(1, 4).contiguous()
    st.call(t)
    torch.cuda.synchronize()
    assert pk.read_device_status(clear=True) & pk.PA_DEV_PLAN_OVERFLOW
    assert torch.all(t["out"] == 7.0)


@pytest.mark.parametrize("window,sinks", [(2**32 + 3, 0), (2**70, 2**32), (1, 2**32 + 1),
                                          (2**31 - 1, 2**31 - 1)])
def test_windows_and_sinks_past_int32_see_every_key(window, sinks):
    st = Step(DECODE + [(33, 5)], 8, 2, 128, 16, 10 ** 6, 0)
    t = st.to_dev()
    st.window, st.sinks = window, sinks
    st.call(t)
    st.call(t, workspace=pk.alloc_workspace(1 << 26, DEV))   # (a kept one)
    torch.cuda.synchronize()
    st.window, st.sinks = 10 ** 6, 0
    st.check(t)
    assert_status_clean()


@pytest.mark.parametrize("group,n", [(1, 1), (1, 3), (3, 1), (5, 3), (7, 1), (15, 1)])
@pytest.mark.parametrize("window,sinks", [(40, 1), (700, 5), (3000, 0)])
def test_clusters_fold_an_odd_number_of_rows(group, n, window, sinks):
    """At head_dim 64 an odd number of rows leaves a warp of the fold half idle; few jobs,
    so that clusters of 2, 4 and 8 CTAs share them."""
    assert group * n % 2 == 1
    st = Step([(3500, n), (90, n), (2100, n)], group, 1, 64, 16, window, sinks, seed=group)
    t = st.run_and_check()
    first = t["out"].clone()
    for _ in range(5):
        st.call(t)
    torch.cuda.synchronize()
    assert torch.equal(t["out"], first)
    assert_status_clean()


def stalled(st):
    """The step with keys that never come: its tensors, seconds and status."""
    t = st.to_dev()
    torch.cuda.synchronize()
    pk.set_test_stall(pk.PA_TEST_STALL_TENSOR_CORE)
    try:
        t0 = time.perf_counter()
        st.call(t)
        torch.cuda.synchronize()
        seconds = time.perf_counter() - t0
    finally:
        pk.set_test_stall(pk.PA_TEST_STALL_NONE)
    return t, seconds, pk.read_device_status(clear=True)


STALLED = [("bf16", 128, [(300, 400), (5, 1), (700, 200)]),              # no plan
           ("bf16", 64, [(300, 400), (5, 1), (700, 200)]),
           ("bf16", 128, [(300, 400), (700, 60)] + [(50, 9)] * 8),       # planned
           ("bf16", 64, [(900, 1000), (700, 60)] + [(2900, 9)] * 10),    # side by side
           ("e4m3", 128, [(300, 400), (700, 60), (5, 1)])]               # staged


@pytest.mark.parametrize("kv,d,requests", STALLED)
def test_a_prompt_kernel_whose_keys_never_come_returns(kv, d, requests):
    """The wait for CTA 0's second tile of keys runs out (2 s a grid): every role gives
    up, and the next call is right."""
    st = Step(requests, 32, 8, d, 16, 2500, 4, kv=kv, seed=d)
    t, seconds, _ = stalled(st)
    assert 1.5 < seconds < 60.0, seconds
    t["out"].fill_(7.0)
    t["lse"].fill_(7.0)
    st.call(t)
    torch.cuda.synchronize()
    st.check(t)
    assert_status_clean()


@pytest.mark.parametrize("kv,d,requests", STALLED)
def test_a_prompt_kernel_whose_keys_never_come_flags_it(kv, d, requests):
    """The warp that loads keys has left when the others' waits run out: the status says
    so all the same."""
    _, _, status = stalled(Step(requests, 32, 8, d, 16, 2500, 4, kv=kv, seed=d))
    assert status == pk.PA_DEV_WAIT_TIMEOUT


@pytest.mark.parametrize("call", ["pa_window_attention", "pa_attention"])
def test_a_workspace_made_for_another_stream_is_not_handed_out_while_in_use(call):
    """A call on a busy stream makes its workspace, and the caller drops it: the
    allocator keeps it until that stream is done."""
    st = Step(MIXED, 16, 4, 128, 16, 10 ** 6, 0)
    t = st.to_dev()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    args = (t["q"], t["k"], t["v"], t["table"], t["qsl"], t["ctx"], t["seq"], st.scale)
    if call == "pa_window_attention":
        args += (st.window, st.sinks)
    getattr(pk, call)(*args, t["out"], t["lse"])    # (loading a kernel waits for the device)
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(1e9))     # about half a second
    ws = getattr(pk, call)(*args, t["out"], t["lse"], stream=side)
    at, size = ws.data_ptr(), ws.numel()
    del ws
    other = torch.empty(size, dtype=torch.uint8, device=DEV)
    busy, other_at = not side.query(), other.data_ptr()
    torch.cuda.synchronize()
    assert busy and other_at != at
    st.check(t)
    assert_status_clean()


def launches(st, t, **kw):
    """Kernels that the step launches (one: the one-kernel form)."""
    ws = st.call(t, **kw)
    torch.cuda.synchronize()
    before = pk.lib().pa_kernel_launches()
    st.call(t, workspace=ws, **kw)
    torch.cuda.synchronize()
    return pk.lib().pa_kernel_launches() - before


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("requests,hq,hkv,kernels", [
    ([(17000, 1)], 4, 1, 2), ([(16000, 1)], 4, 1, 1),      # 4 rows: from 1024 chunks on
    ([(17000, 1), (300, 1)], 8, 2, 2), ([(17000, 2)], 4, 1, 1),
    ([(33500, 2), (20000, 2)], 4, 1, 2)])
def test_a_few_long_jobs_are_split_over_the_whole_device(kv, d, requests, hq, hkv, kernels):
    """Decode and verify rows that see all of a long context: plan and split-KV kernel."""
    st = Step(requests, hq, hkv, d, 16, 10 ** 6, 0, kv=kv, seed=hkv)
    t = st.to_dev()
    assert launches(st, t) == kernels
    st.check(t)
    assert_status_clean()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_few_long_jobs_behind_a_gap(kv):
    """The same with blocks between the sinks and the window given back."""
    st = Step([(26000, 1), (25000, 1)], 4, 1, 128, 16, 18000, 37, kv=kv, seed=5)
    t = st.to_dev()
    assert launches(st, t) == 2
    st.check(t)
    assert_status_clean()


# Steps whose path is asserted by what they launch: the planned kernels one after the
# other (plan, [staging,] split-KV, tensor core) and side by side (one more tensor-core
# grid), with blocks given back between sinks and windows.
PROMPTS = [(2000, 150), (3100, 200), (0, 130), (1500, 90)]


def beside(n, seed):
    """n decode and verify rows of contexts past the windows."""
    rng = np.random.default_rng(seed)
    return [(int(c), int(m)) for c, m in zip(rng.integers(1300, 4000, n), rng.integers(1, 6, n))]


@pytest.mark.parametrize("window,sinks", [(1, 0), (33, 17), (100, 130), (700, 5), (31, 5000)])
@pytest.mark.parametrize("kv,d,staged", [("bf16", 128, 0), ("bf16", 64, 0), ("e4m3", 128, None)])
def test_planned_steps_of_many_requests(kv, d, staged, window, sinks):
    st = Step(MIXED + CHUNKS[1:] + [(900, 3), (1400, 5)], 64, 8, d, 16, window, sinks, kv=kv,
              seed=window, pad=2)
    assert len(st.requests) > 8 and st.total < 512
    t = st.to_dev()
    kw = {} if staged is None else {"staging_blocks": staged}
    assert launches(st, t, **kw) == (3 if kv == "bf16" else 4)
    st.check(t)
    assert_status_clean()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(14000, 37), (9000, 0)])
def test_planned_steps_of_many_requests_split_over_the_window(kv, window, sinks):
    """Split-KV items cut over the packed chunks, and their fold: 64 rows at 12 requests."""
    st = Step([(16000 - 300 * i, 8) for i in range(12)], 8, 1, 128, 16, window, sinks, kv=kv, seed=3)
    t = st.to_dev()
    ws = st.call(t)
    torch.cuda.synchronize()
    header = plan_header(ws)
    assert header["short_items"] > 12 and header["long_items"] == 0
    st.check(t)
    first = t["out"].clone()
    for _ in range(3):
        st.call(t, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(t["out"], first)
    assert_status_clean()


@pytest.mark.parametrize("window,sinks", [(1024, 5), (1200, 300), (1100, 0)])
@pytest.mark.parametrize("kv,d,staged", [("bf16", 128, 0), ("bf16", 64, 0), ("e4m3", 128, None),
                                         ("e4m3", 128, 90)])
def test_side_by_side_behind_a_gap(kv, d, staged, window, sinks):
    st = Step(PROMPTS + beside(22, window), 16, 4, d, 16, window, sinks, kv=kv, seed=window, pad=1)
    assert st.total >= 512
    t = st.to_dev()
    kw = {} if staged is None else {"staging_blocks": staged}
    assert launches(st, t, **kw) == (4 if kv == "bf16" else 5)
    st.check(t)
    first = t["out"].clone()
    for _ in range(3):
        st.call(t, **kw)
    torch.cuda.synchronize()
    assert torch.equal(t["out"], first)
    assert_status_clean()


def test_side_by_side_in_a_graph():
    """Captured on one batch, replayed on it while its outputs are cleared, with the
    workspace's counters as the replay before left them."""
    st = Step(PROMPTS + beside(22, 7), 16, 4, 128, 16, 1024, 5, seed=7)
    t = st.to_dev()
    ws = st.call(t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.call(t, workspace=ws)
    for _ in range(3):
        t["out"].fill_(7.0)
        g.replay()
    torch.cuda.synchronize()
    st.check(t)
    assert_status_clean()


def test_the_last_grid_of_a_windowed_step_times_out_waiting_for_a_missing_cta():
    st = Step(PROMPTS + beside(22, 8), 16, 4, 64, 16, 1024, 5, seed=8)
    t = st.to_dev()
    assert launches(st, t) == 4
    t["out"].fill_(7.0)
    pk.set_test_stall(pk.PA_TEST_STALL_LAST_GRID)
    try:
        st.call(t)
        torch.cuda.synchronize()
    finally:
        pk.set_test_stall(pk.PA_TEST_STALL_NONE)
    assert pk.read_device_status(clear=True) == pk.PA_DEV_WAIT_TIMEOUT
    st.check(t)     # every item ran before the wait
    assert_status_clean()


@pytest.mark.parametrize("requests,hq,hkv,kernels", [
    ([(500, 1)] * 3, 8, 2, 1),                                    # one kernel
    (CHUNKS + [(300, 300)], 32, 8, 2),                            # no plan
    ([(500, 1)] * 1025, 4, 1, 4),                                 # over 1024 requests
    ([(500, 1)] * 3, 34, 2, 2),                                   # a group of 17
    ([(500, 1)] * 20, 34, 2, 3)])
def test_what_a_step_launches(requests, hq, hkv, kernels):
    st = Step(requests, hq, hkv, 128, 16, 90, 3, seed=len(requests))
    t = st.to_dev()
    assert launches(st, t) == kernels
    st.check(t)
    assert_status_clean()
