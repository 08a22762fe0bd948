"""A serving loop of long-lived streams: the block manager's copy-on-write
copies, the rotary cache write, windowed attention over the paged pool, the
blocks behind the window given back, and now and then a compaction -- two
layers deep, forks among the requests.  Every step's output is compared with
attention over dense per-request arrays that know nothing of pages."""
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean
from oracle import ops
from paged_kv_cache_284_gb300.blocks import BlockManager

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, ROT, NB, LAYERS = 8, 2, 128, 16, 64, 40, 2


def rows_of(seq, layer):
    """The projected q, k, v rows of the last token of a sequence."""
    g = torch.Generator().manual_seed((hash(tuple(seq)) * 2 + layer) & 0x7FFFFFFF)
    return torch.randn((HQ + 2 * HKV) * D, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("kv,window,sinks", [("bf16", 37, 4), ("e4m3", 37, 4), ("bf16", 16, 0),
                                             ("bf16", 200, 20)])
def test_loop(kv, window, sinks):
    rng = random.Random(window)
    bm = BlockManager(NB, BS)
    shape = (NB, HKV, BS, D)
    if kv == "bf16":
        kc, vc = ([torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)
                   for _ in range(LAYERS)] for _ in "kv")
        ks = vs = None
    else:
        kc, vc = ([torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV)
                   for _ in range(LAYERS)] for _ in "kv")
        ks, vs = (torch.tensor([0.02, 0.05], device=DEV) for _ in "kv")
    layers = pk.kv_layers(kc, vc)
    inv = 1e4 ** (-torch.arange(ROT // 2, dtype=torch.float64) / (ROT // 2))
    axis = (torch.arange(ROT // 2) % 3).to(torch.int32)
    inv_d, axis_d = inv.to(DEV), axis.to(DEV)
    scale = D ** -0.5
    seqs, pos_of = {}, lambda p: (p, p // 7, p % 7)   # three axes
    released = moved = copied = 0

    def admit(rid, n):
        seqs[rid] = [rng.randrange(50) for _ in range(n)]
        bm.add_request(rid, seqs[rid])

    admit(9, 5)    # computes its prompt, idles, and leaves a hole at the low end
    admit(0, 70)
    admit(1, 3)
    for step in range(26):
        for at, src, dst in ((6, 0, 2), (9, 1, 4)):
            if step == at:
                bm.fork(src, dst)
                seqs[dst] = list(seqs[src])
        if step in (14, 21):
            for rid in ((1, 4, 9) if step == 14 else (0,)):
                bm.free_request(rid)
                del seqs[rid]
        if step == 16:
            admit(3, 41)
        if step in (14, 21):
            moves = bm.compact()
            pk.pa_validate_copies(moves, NB)
            pk.pa_copy_blocks(layers, torch.from_numpy(moves).to(DEV))
            moved += len(moves)
        rids, new = sorted((r for r in seqs if r != 9 or step == 0), key=lambda r: (r != 9, r)), []
        for rid in rids:
            done = bm.num_computed(rid)
            if done == len(seqs[rid]):
                t = [rng.randrange(50) for _ in range(rng.choice([1, 1, 1, 4]))]
                seqs[rid] += t
                bm.append_tokens(rid, t)
            new.append(min(len(seqs[rid]) - done, 48))
        meta = bm.schedule(rids, new, 32)
        if len(meta["copies"]):
            pk.pa_validate_copies(meta["copies"], NB)
            pk.pa_copy_blocks(layers, torch.from_numpy(meta["copies"]).to(DEV))
            copied += len(meta["copies"])
        dev = {k: torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for k, v in meta.items()}
        pk.pa_validate_metadata(*(torch.from_numpy(meta[x]) for x in
                                  ("block_tables", "query_start_loc", "context_lens", "seq_lens")),
                                num_blocks=NB, block_size=BS, window=window, num_sinks=sinks,
                                slot_mapping=torch.from_numpy(meta["slot_mapping"]))
        place = [(rid, p) for i, rid in enumerate(rids)
                 for p in range(meta["context_lens"][i], meta["seq_lens"][i])]
        T = len(place)
        positions = torch.tensor([pos_of(p) for _, p in place], dtype=torch.int32).T.contiguous()
        for layer in range(LAYERS):
            qkv = torch.stack([rows_of(seqs[r][:p + 1], layer) for r, p in place]).to(DEV)
            q, k, v = (x.view(T, -1, D) for x in qkv.split([HQ * D, HKV * D, HKV * D], dim=1))
            q_rot = torch.empty((T, HQ, D), dtype=torch.bfloat16, device=DEV)
            out, lse = torch.empty_like(q_rot), torch.empty((T, HQ), device=DEV)
            pk.pa_rope_write_kv(q, k, v, positions.to(DEV), inv_d, axis_d, dev["slot_mapping"],
                                kc[layer], vc[layer], q_rot, k_scale=ks, v_scale=vs)
            pk.pa_window_attention(q_rot, kc[layer], vc[layer], dev["block_tables"],
                                   dev["query_start_loc"], dev["context_lens"], dev["seq_lens"],
                                   scale, window, sinks, out, lse, k_scale=ks, v_scale=vs,
                                   staging_blocks=20)
            got = out.double().cpu().numpy()
            for i, rid in enumerate(rids):
                L = int(meta["seq_lens"][i])
                x = torch.stack([rows_of(seqs[rid][:p + 1], layer) for p in range(L)])
                qd, kd, vd = (y.double().numpy().reshape(L, -1, D)
                              for y in x.split([HQ * D, HKV * D, HKV * D], dim=1))
                how = (np.array([pos_of(p) for p in range(L)]).T, inv.numpy(), axis.numpy(), ROT,
                       False)
                qd = torch.from_numpy(ops.rope(qd, *how)).to(torch.bfloat16).double().numpy()
                kd = ops.rope(kd, *how)
                if kv == "bf16":
                    kd = torch.from_numpy(kd).to(torch.bfloat16).double().numpy()
                else:
                    s = np.array([0.02, 0.05], np.float32).astype(np.float64)[:, None]
                    kd, vd = (torch.from_numpy(np.clip(y / s, -448, 448)).to(torch.float8_e4m3fn)
                              .double().numpy() * s for y in (kd, vd))
                n = new[i]
                pad = -L % BS
                kd, vd = (np.concatenate([y, np.zeros((pad, HKV, D))]).reshape(-1, BS, HKV, D)
                          .transpose(0, 2, 1, 3) for y in (kd, vd))
                ref, _, mag = ops.window_attention(qd[L - n:], kd, vd,
                                                   np.arange(kd.shape[0])[None], [0, n], [L - n],
                                                   scale, window, sinks, BS)
                at = int(meta["query_start_loc"][i])
                err = np.abs(got[at:at + n] - ref)
                # the bf16 output and the probabilities' rounding (see the
                # windowed attention's own test), and q and k that may be
                # rounded the other way at a tie of the fp32 rotation: one
                # step of a single element of a 128-term score
                tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mag
                step_k = 2.0 ** -7 if kv == "bf16" else 2.0 ** -3
                tol += 2 * scale * step_k * 16 * mag
                assert np.all(err <= tol), (step, layer, rid, np.max(err / tol))
        for rid in rids:
            released += bm.release_window(rid, window, sinks)
    assert copied >= 1 and moved >= 1
    assert released >= 1 or window == 200
    assert_status_clean()


@pytest.mark.parametrize("kv,window,sinks", [("bf16", 37, 4), ("e4m3", 37, 4), ("bf16", 16, 0),
                                             ("e4m3", 200, 20), ("e4m3", 3, 1)])
def test_loop_against_the_rows_written(kv, window, sinks):
    """The same run of calls, with the rounding of q, k and v taken out of the comparison:
    every new row is read back from its slot and checked against the rotation, and kept
    with its request; attention over the kept rows, with the rotated q that the call itself
    used, has the windowed attention's own tolerance.  A lost sink, a window off by one, a
    block copied too late or to the wrong place changes far more than that."""
    rng = random.Random(window + 1)
    bm = BlockManager(NB, BS)
    shape = (NB, HKV, BS, D)
    fp8 = kv == "e4m3"
    kc, vc = ([torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV) if fp8 else
               torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)
               for _ in range(LAYERS)] for _ in "kv")
    ks = vs = None
    step_of = np.ones((HKV, 1))
    if fp8:
        ks, vs = (torch.tensor([0.02, 0.05], device=DEV) for _ in "kv")
        step_of = ks.cpu().double().numpy()[:, None]
    layers = pk.kv_layers(kc, vc)
    inv = 1e4 ** (-torch.arange(ROT // 2, dtype=torch.float64) / (ROT // 2))
    axis = (torch.arange(ROT // 2) % 3).to(torch.int32)
    inv_d, axis_d = inv.to(DEV), axis.to(DEV)
    scale = D ** -0.5
    seqs, kept, pos_of = {}, {}, lambda p: (p, p // 7, p % 7)
    copied = moved = released = 0

    def values(pool, slots):
        rows = pool.cpu()[slots // BS, :, slots % BS]
        return (rows.view(torch.float8_e4m3fn) if fp8 else rows).double().numpy() * step_of

    def admit(rid, n):
        seqs[rid] = [rng.randrange(50) for _ in range(n)]
        hits = bm.add_request(rid, seqs[rid])
        assert hits == 0
        kept[rid] = [([], []) for _ in range(LAYERS)]

    admit(0, 75)
    admit(1, 6)
    admit(8, 20)
    for step in range(24):
        for at, src, dst in ((4, 0, 2), (4, 1, 3), (11, 2, 5)):
            if step == at:
                bm.fork(src, dst)
                seqs[dst] = list(seqs[src])
                kept[dst] = [(list(k), list(v)) for k, v in kept[src]]
        if step in (9, 17):
            for rid in ((8, 1) if step == 9 else (0,)):
                bm.free_request(rid)
                del seqs[rid], kept[rid]
        if step == 13:
            admit(6, 52)
        if step in (9, 17):
            moves = bm.compact(5)
            pk.pa_validate_copies(moves, NB)
            pk.pa_copy_blocks(layers, torch.from_numpy(moves).to(DEV))
            moved += len(moves)
        rids, new = sorted(seqs), []
        for rid in rids:
            done = bm.num_computed(rid)
            if done == len(seqs[rid]):
                t = [rng.randrange(50) for _ in range(rng.choice([1, 1, 3]))]
                seqs[rid] += t
                bm.append_tokens(rid, t)
            new.append(min(len(seqs[rid]) - done, 40))
        meta = bm.schedule(rids, new, 32)
        if len(meta["copies"]):
            pk.pa_copy_blocks(layers, torch.from_numpy(meta["copies"]).to(DEV))
            copied += len(meta["copies"])
        dev = {k: torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for k, v in meta.items()}
        place = [(rid, p) for i, rid in enumerate(rids)
                 for p in range(meta["context_lens"][i], meta["seq_lens"][i])]
        T = len(place)
        positions = torch.tensor([pos_of(p) for _, p in place], dtype=torch.int32).T.contiguous()
        how = (positions.numpy(), inv.numpy(), axis.numpy(), ROT, False)
        slots = torch.from_numpy(meta["slot_mapping"])
        for layer in range(LAYERS):
            qkv = torch.stack([rows_of(seqs[r][:p + 1], layer) for r, p in place]).to(DEV)
            q, k, v = (x.view(T, -1, D) for x in qkv.split([HQ * D, HKV * D, HKV * D], dim=1))
            q_rot = torch.empty((T, HQ, D), dtype=torch.bfloat16, device=DEV)
            out, lse = torch.empty_like(q_rot), torch.empty((T, HQ), device=DEV)
            pk.pa_rope_write_kv(q, k, v, positions.to(DEV), inv_d, axis_d, dev["slot_mapping"],
                                kc[layer], vc[layer], q_rot, k_scale=ks, v_scale=vs)
            pk.pa_window_attention(q_rot, kc[layer], vc[layer], dev["block_tables"],
                                   dev["query_start_loc"], dev["context_lens"], dev["seq_lens"],
                                   scale, window, sinks, out, lse, k_scale=ks, v_scale=vs,
                                   staging_blocks=20)
            q64, k64, v64 = (x.double().cpu().numpy() for x in (q, k, v))
            # one rounding to bf16, or to e4m3 of value / scale (half a step: 2^-4 of the
            # value, 2^-10 below the normal range), and the fp32 rotation's (|a| + |b|) 2^-21
            for name, got, want, rounds in (
                    ("q", q_rot.double().cpu().numpy(), ops.rope(q64, *how), False),
                    ("k", values(kc[layer], slots), ops.rope(k64, *how), fp8),
                    ("v", values(vc[layer], slots), v64, fp8)):
                pair = np.zeros_like(want)
                src = {"q": q64, "k": k64}.get(name)
                if src is not None:
                    a, b = np.abs(src[..., :ROT // 2]), np.abs(src[..., ROT // 2:ROT])
                    pair[..., :ROT // 2] = pair[..., ROT // 2:ROT] = (a + b) * 2.0 ** -21
                tol = 2.0 ** -8 * np.abs(want) + pair
                if rounds:
                    want = np.clip(want, -448 * step_of, 448 * step_of)
                    tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * step_of + pair
                assert np.all(np.abs(got - want) <= tol), (step, layer, name)
            k_new, v_new = values(kc[layer], slots), values(vc[layer], slots)
            for t, (rid, p) in enumerate(place):
                rows_k, rows_v = kept[rid][layer]
                assert len(rows_k) == p
                rows_k.append(k_new[t])
                rows_v.append(v_new[t])
            got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
            q64 = q_rot.double().cpu().numpy()
            for i, rid in enumerate(rids):
                L, n, at = int(meta["seq_lens"][i]), new[i], int(meta["query_start_loc"][i])
                kd, vd = (np.concatenate([np.stack(y), np.zeros((-L % BS, HKV, D))])
                          .reshape(-1, BS, HKV, D).transpose(0, 2, 1, 3) for y in kept[rid][layer])
                ref, ref_l, mag = ops.window_attention(q64[at:at + n], kd, vd,
                                                       np.arange(kd.shape[0])[None], [0, n],
                                                       [L - n], scale, window, sinks, BS)
                err = np.abs(got[at:at + n] - ref)
                tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mag
                assert np.all(err <= tol), (step, layer, rid, np.max(err / tol))
                lerr = np.abs(got_lse[at:at + n] - ref_l)
                assert np.all(lerr <= 2.0 ** -13 + 2.0 ** -22 * np.abs(ref_l)), (step, layer, rid)
        for rid in rids:
            released += bm.release_window(rid, window, sinks)
    assert copied >= 1 and moved >= 1
    assert released >= 1 or window == 200
    assert_status_clean()
