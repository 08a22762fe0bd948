"""The step builder, the rotated cache write, attention over the own cache, cross attention and
linear attention one after the other in one captured graph, as a decoder's loop runs them:
prompts, decode and verify rows, rows that finish and start over, with lengths, tables and the
free list carried on the GPU.  Each operator against its definition on the inputs that the one
before it left, with its own test's tolerance."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, OUT_MAX_ABS, assert_status_clean, bits
from oracle import ops

pytestmark = pytest.mark.gpu

BS, WIDTH, TOKENS = 16, 24, 240
STEPS = [[70, 5, 0, 90, 1], [1, 5, 33, 1, 1], [1, -1, 1, 5, 1], [0, 20, 1, 5, -1], [-1, 1, 100, 1, 2],
         [65, 1, 1, 1, 64], [1, 1, 1, 1, 1], [1, 5, 5, -1, 1]]


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (4, 4, 128), (8, 2, 128)])
def test_one_graph_for_every_step(hq, hkv, d):
    g = torch.Generator().manual_seed(d + hq)
    rows, scale, blocks = 5, d ** -0.5, 90
    randn = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)  # noqa: E731
    q_lens, seq, table = i32([0] * rows), i32([0] * rows), i32(np.zeros((rows, WIDTH)))
    ring, state = i32(np.random.default_rng(1).permutation(blocks)), i32([40, blocks, 0, 0])
    qsl, ctx, positions = i32([0] * (rows + 1)), i32([0] * rows), i32([0] * TOKENS)
    slots = torch.zeros(TOKENS, dtype=torch.int64, device=DEV)
    cache = [torch.zeros((blocks, hkv, BS, d), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    q, k, v = (torch.zeros((TOKENS, h, d), dtype=torch.bfloat16, device=DEV) for h in (hq, hkv, hkv))
    rotated, own, cross, out = (torch.zeros_like(q) for _ in range(4))
    inv_freq = torch.tensor(10000.0 ** -(np.arange(d // 2) / (d // 2)), device=DEV)
    enc_lens = [37, 0, 200, 16, 1]
    enc_table = np.random.default_rng(2).permutation(5 * 13).reshape(5, 13)
    enc = [randn(5 * 13, hkv, BS, d).to(DEV) for _ in "kv"]
    e_table, e_lens = i32(enc_table), i32(enc_lens)
    decay = -torch.rand((TOKENS, hkv), generator=g).to(DEV)
    states = torch.zeros((rows, hkv, d, d), device=DEV)
    row_slots = i32(range(rows))
    size = (rows, TOKENS, hq, hkv, d)
    ws = pk.alloc_workspace(max(pk.workspace_size(*size), pk.linear_workspace_size(*size)), DEV)

    def step():
        pk.pa_build_step(q_lens, seq, table, ring, state, blocks, BS, qsl, ctx, seq, slots, positions)
        pk.pa_rope_write_kv(q, k, v, positions, inv_freq, None, slots, *cache, rotated)
        pk.pa_attention(rotated, *cache, table, qsl, ctx, seq, scale, own, workspace=ws)
        pk.pa_cross_attention(own, *enc, e_table, qsl, e_lens, scale, cross, workspace=ws)
        state_in = torch.where(ctx == 0, -1, row_slots)
        pk.pa_linear_attention(cross, k, v, qsl, decay, states, state_in, row_slots, scale, out,
                               workspace=ws)

    step()   # (all rows idle)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    host = dict(cached=np.zeros(rows, np.int32), table=table.cpu().numpy(), ring=ring.cpu().numpy(),
                head=40, count=blocks)
    enc64 = [x.double().cpu().numpy() for x in enc]
    how = (np.arange(d // 2) * 0, d, False)
    for n, lens in enumerate(STEPS):
        new = [randn(TOKENS, h, d) for h in (hq, hkv, hkv)]
        for dst, src in zip((q, k, v), new):
            dst.copy_(src)
        q_lens.copy_(i32(lens))
        before = states.double().cpu().numpy()
        graph.replay()
        torch.cuda.synchronize()
        assert_status_clean()

        want = ops.build_step(lens, host["cached"], host["table"], host["ring"], host["head"],
                              host["count"], TOKENS, BS)
        for name, got in (("qsl", qsl), ("ctx", ctx), ("seq", seq), ("slots", slots),
                          ("positions", positions), ("table", table), ("ring", ring),
                          ("state", state)):
            assert np.array_equal(got.cpu().numpy(), want[name]), (n, name)
        host = dict(cached=want["seq"], table=want["table"], ring=want["ring"],
                    head=int(want["state"][0]), count=int(want["state"][1]))
        total = int(want["qsl"][-1])
        q64, k64, v64 = (x[:total].double().numpy() for x in new)
        at = (want["slots"][:total] // BS, slice(None), want["slots"][:total] % BS)
        pos = want["positions"][None, :total]
        for x, got in ((q64, rotated[:total].cpu()), (k64, cache[0].cpu()[at])):
            ref = ops.rope(x, pos, inv_freq.cpu().numpy(), *how)
            half = np.abs(x[..., :d // 2]) + np.abs(x[..., d // 2:])
            tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * np.concatenate([half, half], -1)
            assert np.all(np.abs(got.double().numpy() - ref) <= tol), n
        assert np.array_equal(cache[1].cpu()[at].double().numpy(), v64)

        ref, _ = oracle.attention(rotated[:total].cpu(), bits(cache[0]), bits(cache[1]),
                                  want["table"], want["qsl"], want["ctx"], want["seq"], scale)
        own64 = own[:total].double().cpu().numpy()
        assert np.max(np.abs(own64 - ref)) <= OUT_MAX_ABS, n

        ref, _, mag = ops.cross_attention(own64, *enc64, enc_table, want["qsl"], enc_lens, scale, BS)
        cross64 = cross[:total].double().cpu().numpy()
        assert np.all(np.abs(cross64 - ref) <= 2.0 ** -8 * np.abs(ref) +
                      (2.0 ** -8 + 2.0 ** -12) * mag), n

        start = np.where(want["ctx"] == 0, -1, np.arange(rows))
        ref, new_states, mag, smag = ops.linear_attention(
            cross64, k64, v64, want["qsl"], decay[:total].double().cpu().numpy(), before, start,
            np.arange(rows), scale)
        err = np.abs(out[:total].double().cpu().numpy() - ref)
        assert np.all(err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mag + 1e-30), n
        tol = (2.0 ** -16 + (2 * max(lens) + 2 * d) * 2.0 ** -23) * smag + 1e-30
        assert np.all(np.abs(states.double().cpu().numpy() - new_states) <= tol), n
