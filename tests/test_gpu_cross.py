"""pa_cross_attention on the GPU against the float64 definition.  Table entries that no
key needs are -1, slots behind the last key hold NaN.

Tolerances.  out is rounded to bf16 (at most 2^-8 of its value) and the probabilities are
rounded once before P V (bf16 2^-8, f16 less), which moves out by at most 2^-8 sum_j p_j
|v_j|; scores and sums in fp32 add less than 2^-12 of that sum (a score of 128 products has
an error below 128 * 2^-24 * scale * sum |q k| < 2^-13 for the inputs here; the normaliser as
much).  lse inherits the scores' error, 2^-13, and fp32's own 2^-22 of it."""
import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean
from oracle import ops

pytestmark = pytest.mark.gpu


class Step:
    """requests: (keys, query tokens) pairs."""

    def __init__(self, requests, hq, hkv, d, bs, kv="bf16", seed=0, pad=0, width=0):
        g = torch.Generator().manual_seed(seed)
        self.bs, self.kv, self.requests = bs, kv, requests
        blocks = [-(-n // bs) for n, _ in requests]
        self.num_blocks = sum(blocks) + 3
        perm = torch.randperm(self.num_blocks, generator=g).to(torch.int32)
        self.table = torch.full((len(requests), max([width, 1] + blocks)), -1, dtype=torch.int32)
        live = torch.zeros(self.num_blocks, bs, dtype=torch.bool)
        at = 0
        for b, (n, _) in enumerate(requests):
            ids = perm[at:at + blocks[b]]
            self.table[b, :blocks[b]] = ids
            at += blocks[b]
            for i, x in enumerate(ids.tolist()):
                live[x, :min(bs, n - i * bs)] = True
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
                              .masked_fill(hidden, 0x7F) for x in (k, v))
            self.ks, self.vs = (0.04 + 0.05 * torch.rand(hkv, generator=g) for _ in "kv")
            self.k64, self.v64 = (x.view(torch.float8_e4m3fn).double().numpy() *
                                  s.double().numpy()[:, None, None]
                                  for x, s in ((self.k, self.ks), (self.v, self.vs)))
        i32 = dict(dtype=torch.int32)
        self.qsl = torch.tensor(np.concatenate([[0], np.cumsum([n for _, n in requests])]), **i32)
        self.lens = torch.tensor([n for n, _ in requests], **i32)
        self.total = int(self.qsl[-1])
        self.q = torch.randn((self.total + pad, hq, d), generator=g).to(torch.bfloat16)
        self.scale = d ** -0.5
        self.staging = sum(x for x, (_, n) in zip(blocks, requests) if n * hq // hkv > 64)

    def to_dev(self):
        t = {x: getattr(self, x).to(DEV) for x in ("q", "k", "v", "table", "qsl", "lens")}
        t["ks"], t["vs"] = ((None, None) if self.ks is None
                            else (self.ks.to(DEV), self.vs.to(DEV)))
        t["out"] = torch.full_like(t["q"], 7.0)
        t["lse"] = torch.full(t["q"].shape[:2], 7.0, device=DEV)
        return t

    def call(self, t, **kw):
        kw.setdefault("staging_blocks", self.staging)
        return pk.pa_cross_attention(t["q"], t["k"], t["v"], t["table"], t["qsl"], t["lens"],
                                     self.scale, t["out"], t["lse"], k_scale=t["ks"],
                                     v_scale=t["vs"], **kw)

    def check(self, t):
        torch.cuda.synchronize()
        out, lse, mag = ops.cross_attention(self.q[:self.total].double().numpy(), self.k64,
                                            self.v64, self.table.numpy(), self.qsl.numpy(),
                                            self.lens.numpy(), self.scale, self.bs)
        got, got_lse = t["out"].double().cpu().numpy(), t["lse"].double().cpu().numpy()
        assert np.all(got[self.total:] == 7) and np.all(got_lse[self.total:] == 7)
        got, got_lse = got[:self.total], got_lse[:self.total]
        bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -12) * mag + 1e-30
        assert np.all(np.abs(got - out) <= bound), np.max(np.abs(got - out) / bound)
        none = np.isneginf(lse)
        assert np.array_equal(none, np.isneginf(got_lse))
        err = np.abs(got_lse[~none] - lse[~none])
        assert np.all(err <= 2.0 ** -13 + 2.0 ** -22 * np.abs(lse[~none])), err.max()


def run(requests, hq, hkv, d, bs, kv="bf16", status=0, call=None, **kw):
    s = Step(requests, hq, hkv, d, bs, kv, **kw)
    t = s.to_dev()
    s.call(t, **(call or {}))
    s.check(t)
    assert pk.read_device_status(clear=True) == status
    return s, t


SMALL = [(1, 1), (15, 1), (16, 1), (17, 1), (64, 1), (0, 1), (129, 1), (700, 1), (33, 3), (0, 4),
         (257, 16), (500, 21)]


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("bf16", 128), ("e4m3", 128)])
@pytest.mark.parametrize("request_", SMALL)
def test_one_request(request_, kv, d):
    run([request_], 4, 2, d, 16, kv, seed=request_[0])


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("bf16", 128), ("e4m3", 128)])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 6), (14, 2), (16, 1), (17, 1), (32, 8), (64, 1)])
def test_heads(hq, hkv, kv, d):
    run([(77, 1), (0, 2), (130, 5), (16, 0), (200, 1)], hq, hkv, d, 32, kv, seed=hq, pad=2)


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("bf16", 128), ("e4m3", 128)])
@pytest.mark.parametrize("n", [65, 128, 200])
def test_prompts(n, kv, d):
    """Tensor-core tiles, alone (without a plan) and among many requests (planned), with
    requests that have no keys between them."""
    run([(300, n), (0, 90), (128, 129)], 8, 2, d, 16, kv, seed=n, pad=1)
    run([(40 * i, [n, 1, 3, 0, 70][i % 5]) for i in range(12)], 8, 2, d, 16, kv, seed=n, pad=3)


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("bf16", 128), ("e4m3", 128)])
def test_step_of_everything_side_by_side(kv, d):
    """At least 512 tokens and 6144 chunks: both tensor-core grids beside the split-KV one."""
    reqs = [(0, 1)] + [(900 + 13 * i, 1) for i in range(70)] + [(0, 70), (1500, 300), (700, 260)]
    run(reqs, 8, 2, d, 16, kv, seed=9, width=700)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_keys_few_rows(kv):
    """Planned splits and their fold: one row over many keys (a wide table leaves the
    one-kernel form), with requests that have none."""
    run([(9000, 1), (0, 1), (4100, 2)], 4, 1, 128, 64, kv, seed=3, width=300)
    run([(40000, 1), (0, 1)], 4, 1, 128, 256, kv, seed=3, width=160)


def test_beams_of_one_request_are_rows():
    """Rows of one request and requests that share a table give the same rows."""
    s = Step([(333, 5)], 8, 2, 64, 16, seed=2)
    t = s.to_dev()
    s.call(t)
    u = dict(t, table=t["table"].expand(5, -1).contiguous(), lens=t["lens"].expand(5).contiguous(),
             qsl=torch.arange(6, dtype=torch.int32, device=DEV), out=torch.zeros_like(t["out"]),
             lse=torch.zeros_like(t["lse"]))
    s.call(u)
    s.check(t)
    s.check(u)
    assert_status_clean()


def test_padded_graph_replays():
    """One graph for every batch up to its size: empty requests and padding rows; two graphs
    of different sizes share a workspace, replayed in turn."""
    graphs = []
    big = Step([(200, 1)] * 24, 8, 2, 128, 16)
    ws = pk.alloc_workspace(pk.workspace_size(24, 24, 8, 2, 128), DEV)
    for size in (24, 9):
        t = Step([(200, 1)] * size, 8, 2, 128, 16).to_dev()
        t["k"], t["v"] = big.k.to(DEV), big.v.to(DEV)
        t["table"] = torch.zeros((size, 40), dtype=torch.int32, device=DEV)
        big.call(t, workspace=ws, staging_blocks=0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            big.call(t, workspace=ws, staging_blocks=0)
        graphs.append((size, t, graph))
    for turn in range(4):
        size, t, graph = graphs[turn % 2]
        n = size - 2 * turn
        s = Step([(17 * i, 1) for i in range(n)], 8, 2, 128, 16, seed=turn, pad=size - n)
        for x in ("k", "v"):
            t[x].zero_()
            t[x][:min(len(t[x]), s.num_blocks)] = getattr(s, x)[:len(t[x])].to(DEV)
        assert s.num_blocks <= len(t["k"])
        t["table"].fill_(-1)
        t["table"][:n, :s.table.shape[1]] = s.table.to(DEV)
        t["q"].copy_(s.q)
        t["lens"].zero_()
        t["lens"][:n] = s.lens.to(DEV)
        t["qsl"].fill_(n)
        t["qsl"][:n + 1] = s.qsl.to(DEV)
        t["out"].fill_(7)
        t["lse"].fill_(7)
        graph.replay()
        s.check(t)
    assert_status_clean()


def test_bad_metadata_is_flagged():
    s = Step([(50, 1), (60, 1), (70, 1)], 4, 2, 64, 16)
    t = s.to_dev()
    t["lens"][1] = s.table.shape[1] * 16 + 1
    t["lens"][2] = -1
    s.call(t)
    torch.cuda.synchronize()
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_METADATA
    assert torch.all(t["out"][1:] == 7)
    t = s.to_dev()
    t["table"][0, 0] = s.num_blocks
    s.call(t)
    torch.cuda.synchronize()
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_BLOCK


def test_other_stream_and_repeat():
    s = Step([(300, 1), (4, 2), (600, 40), (90, 90)], 8, 2, 128, 16, seed=6)
    t = s.to_dev()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = s.call(t, stream=side)
    side.synchronize()
    s.check(t)
    first = t["out"].clone()
    for _ in range(5):
        s.call(t, workspace=ws)
        assert torch.equal(first, t["out"])
    assert_status_clean()


@pytest.mark.parametrize("requests", [[(300, 1), (17, 2)], [(300, 70), (40, 1)]])
def test_pool_past_32_bits(requests):
    """Blocks more than 2^31 elements into the pool."""
    s = Step(requests, 16, 8, 128, 16, seed=4)
    t = s.to_dev()
    at = 131100   # 16384 elements a block
    for x in "kv":
        pool = torch.empty((at + s.num_blocks, 8, 16, 128), dtype=torch.bfloat16, device=DEV)
        pool[at:] = t[x]
        t[x] = pool
    t["table"][t["table"] >= 0] += at
    s.call(t)
    s.check(t)
    assert_status_clean()


def test_refusals():
    s = Step([(50, 1), (60, 2)], 4, 2, 64, 16)
    t = s.to_dev()
    ws = s.call(t)
    for kw in ({}, {"workspace": ws}):
        with pytest.raises(pk.PaError):
            s.scale = 0.0
            s.call(t, **kw)
        s.scale = 0.125
        for name in ("table", "qsl", "lens"):
            with pytest.raises(TypeError):
                s.call({**t, name: t[name].long()}, **kw)
            with pytest.raises(ValueError):
                s.call({**t, name: t[name].cpu()}, **kw)
            with pytest.raises(ValueError):
                s.call({**t, name: t[name][:-1]}, **kw)
        with pytest.raises(ValueError):
            s.call({**t, "out": t["out"][:-1]}, **kw)
        with pytest.raises(TypeError):
            s.call({**t, "q": t["q"].float()}, **kw)
    assert_status_clean()
