"""Host side of windowed attention, the rotary cache write and block copies:
the block manager's release and compaction against the plain model, the host
validators, and every refusal of the new entry points -- all before any CUDA
call."""
import ctypes
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from oracle.blocks import BlockManagerModel, INVALID, OK
from paged_kv_cache_284_gb300.blocks import BlockManager


# ---- block manager ----------------------------------------------------------------

def advance(m, bm, rid, n):
    tokens = [(rid * 31 + i) % 7 for i in range(n)]
    m.append_tokens(rid, tokens)
    bm.append_tokens(rid, tokens)
    code, meta = m.schedule([rid], [n], 64, 8)
    assert code == OK
    got = bm.schedule([rid], [n], 64, max_copies=8)
    assert got["block_tables"].tolist() == meta["block_tables"]
    assert got["slot_mapping"].tolist() == meta["slot_mapping"]
    return meta


def same(m, bm):
    assert bm.num_free_blocks == m.available()
    assert bm.num_cached_blocks == len(m.cache)
    assert [bm.ref_count(b) for b in range(m.n)] == m.ref
    for rid, r in m.reqs.items():
        assert bm.blocks_of(rid) == r.table and bm.num_computed(rid) == r.computed


@pytest.mark.parametrize("window,sinks,gone", [
    (1, 0, 9), (1, 4, 8), (3, 0, 9), (4, 0, 8), (5, 0, 8), (6, 1, 7), (40, 0, 0), (13, 9, 3), (1, 1000, 0),
    (2**31 - 1, 0, 0), (1, 2**31 - 1, 0)])
def test_release_window_gives_back_what_no_later_row_sees(window, sinks, gone):
    """38 computed tokens in blocks of 4: the next row (position 38) sees keys
    from 39 - window on and the sinks."""
    m, bm = BlockManagerModel(16, 4), BlockManager(16, 4)
    for x in (m, bm):
        x.add_request(1, [5])
    advance(m, bm, 1, 38)
    code, n = m.release_window(1, window, sinks)
    assert code == OK
    assert bm.release_window(1, window, sinks) == n
    same(m, bm)
    table = bm.blocks_of(1)
    for j, b in enumerate(table):
        hidden = all(p < 38 - window + 1 and p >= sinks for p in range(4 * j, 4 * j + 4))
        assert (b == -1) == hidden
    assert bm.release_window(1, window, sinks) == 0       # nothing twice
    assert n == gone
    advance(m, bm, 1, 3)
    same(m, bm)


def test_release_window_keeps_shared_and_cached_blocks():
    m, bm = BlockManagerModel(16, 4), BlockManager(16, 4)
    for x in (m, bm):
        x.add_request(1, list(range(17)))
    for x, kw in ((m, {}), (bm, {})):
        x.schedule([1], [17], 16, 4)
        x.fork(1, 2)
    for rid in (2, 1):
        m.release_window(rid, 2, 0)
        bm.release_window(rid, 2, 0)
        same(m, bm)
    # the cached prefix is still matched by a third request
    assert bm.add_request(3, list(range(17))) == m.add_request(3, list(range(17)))[1] == 16
    same(m, bm)
    for rid in (1, 2, 3):
        bm.free_request(rid)
        m.free_request(rid)
        same(m, bm)


def test_release_window_refusals():
    bm = BlockManager(4, 4)
    bm.add_request(1, [1, 2])
    for args in ((9, 4, 0), (1, 0, 0), (1, 4, -1)):
        with pytest.raises(pk.PaError) as e:
            bm.release_window(*args)
        assert e.value.code == pk.PA_ERR_INVALID_ARG
    assert BlockManagerModel(4, 4).release_window(9, 4, 0)[0] == INVALID
    assert pk.lib().pa_bm_release_window(None, 1, 1, 0, None) == pk.PA_ERR_INVALID_ARG
    assert pk.lib().pa_bm_compact(None, 1, None, None) == pk.PA_ERR_INVALID_ARG
    with pytest.raises(pk.PaError):
        bm.compact(-1)


@pytest.mark.parametrize("seed", range(10))
def test_manager_matches_the_model_with_releases_and_compaction(seed):
    rng = random.Random(seed)
    m, bm = BlockManagerModel(40, 4), BlockManager(40, 4)
    next_id = 0
    for step in range(300):
        live = sorted(m.reqs)
        r = rng.random()
        if not live or r < 0.15:
            t = [rng.randrange(2) for _ in range(rng.randint(1, 20))]
            assert bm.add_request(next_id, t) == m.add_request(next_id, t)[1]
            next_id += 1
        elif r < 0.25:
            src = rng.choice(live)
            m.fork(src, next_id)
            bm.fork(src, next_id)
            next_id += 1
        elif r < 0.35:
            rid = rng.choice(live)
            m.free_request(rid)
            bm.free_request(rid)
        elif r < 0.50:
            rid, w, s = rng.choice(live), rng.randint(1, 12), rng.randint(0, 6)
            assert bm.release_window(rid, w, s) == m.release_window(rid, w, s)[1]
        elif r < 0.60:
            limit = rng.choice([0, 1, 3, 40])
            before = [list(x.table) for x in m.reqs.values()]
            want = m.compact(limit)
            got = bm.compact(limit)
            assert [tuple(x) for x in got.tolist()] == want
            pk.pa_validate_copies(got, 40)
            if limit == 40:
                used = [b for b in range(40) if b not in m.free_blocks()]
                assert used == list(range(len(used)))
            # a table names the same contents as before
            moved = dict(want)
            after = [list(x.table) for x in m.reqs.values()]
            assert after == [[moved.get(b, b) for b in t] for t in before]
        else:
            rid = rng.choice(live)
            q = m.reqs[rid]
            if len(q.tokens) == q.computed:
                t = [rng.randrange(2) for _ in range(rng.randint(1, 6))]
                m.append_tokens(rid, t)
                bm.append_tokens(rid, t)
            n = rng.randint(1, len(q.tokens) - q.computed)
            code, meta = m.schedule([rid], [n], 64, 4)
            got = bm.try_schedule([rid], [n], 64, max_copies=4)
            if code != OK:
                assert got == code
            else:
                assert got["block_tables"].tolist() == meta["block_tables"]
                assert [tuple(c) for c in got["copies"].tolist()] == meta["copies"]
                pk.pa_validate_copies(got["copies"], 40)
        same(m, bm)
    bm.close()


# ---- validators --------------------------------------------------------------------

@pytest.mark.parametrize("pairs,ok", [
    ([], True), ([(0, 1)], True), ([(0, 1), (0, 2)], True), ([(-1, 1), (0, 1)], True),
    ([(3, 3), (0, 3)], True), ([(0, 1), (2, 1)], False), ([(0, 1), (1, 2)], False),
    ([(1, 2), (0, 1)], False), ([(0, 9)], False), ([(9, 0)], False), ([(9, -1)], True)])
def test_validate_copies(pairs, ok):
    p = np.array(pairs, np.int32).reshape(-1, 2)
    if ok:
        pk.pa_validate_copies(p, 9)
        return
    with pytest.raises(pk.PaError) as e:
        pk.pa_validate_copies(p, 9)
    assert e.value.code == pk.PA_ERR_BAD_METADATA


def test_validate_window_metadata_looks_at_visible_blocks_only():
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    # position 96..97 of a 98-token request, blocks of 16: window 20 sees keys
    # 77.. (block 4 on), 3 sinks see block 0
    good = torch.tensor([[2, -1, -1, -7, 3, 0, 1]], dtype=torch.int32)
    meta = (i32(0, 2), i32(96), i32(98))
    kw = dict(num_blocks=4, block_size=16)
    pk.pa_validate_metadata(good, *meta, window=20, num_sinks=3, **kw)
    with pytest.raises(pk.PaError):
        pk.pa_validate_metadata(good, *meta, **kw)
    for window, sinks in ((34, 3), (20, 17), (2**31 - 1, 0), (20, 2**31 - 1)):
        with pytest.raises(pk.PaError):
            pk.pa_validate_metadata(good, *meta, window=window, num_sinks=sinks, **kw)
    for j in (0, 4, 6):
        bad = good.clone()
        bad[0, j] = 4
        with pytest.raises(pk.PaError):
            pk.pa_validate_metadata(bad, *meta, window=20, num_sinks=3, **kw)
    with pytest.raises(pk.PaError) as e:
        pk.pa_validate_metadata(good, *meta, window=0, num_sinks=3, **kw)
    assert e.value.code == pk.PA_ERR_INVALID_ARG
    # an empty request reads nothing
    pk.pa_validate_metadata(torch.full((1, 7), -1, dtype=torch.int32), i32(0, 0), i32(96), i32(96),
                            window=20, num_sinks=3, **kw)


# ---- refusals of the entry points (pointers that are never followed) -----------------

F = ctypes.c_void_p(1 << 20)
WS = ctypes.c_void_p(1 << 22)


def desc(num_blocks=100, block_size=16, hkv=8, d=128, dtype=0, scales=None, k=1 << 20):
    return pk.KVDesc(k, 1 << 21, num_blocks, block_size, hkv, d, dtype, 0, scales, scales)


def call_window(kv=None, q=F, table=F, width=4, hq=32, scale=0.1, window=8, sinks=2, ws=WS,
                ws_bytes=1 << 30, seqs=2, tokens=3):
    kv = kv or desc()
    return pk.lib().pa_window_attention(q, ctypes.byref(kv), table, width, F, F, F, seqs, tokens, hq,
                                        scale, window, sinks, F, None, ws, ws_bytes, None)


@pytest.mark.parametrize("want,kw", [
    ("INVALID_ARG", dict(window=0)), ("INVALID_ARG", dict(window=-5)),
    ("INVALID_ARG", dict(sinks=-1)), ("INVALID_ARG", dict(scale=0.0)),
    ("INVALID_ARG", dict(scale=-0.1)), ("INVALID_ARG", dict(scale=float("nan"))),
    ("INVALID_ARG", dict(scale=float("inf"))), ("INVALID_ARG", dict(scale=3e38)),
    ("INVALID_ARG", dict(q=None)), ("INVALID_ARG", dict(q=ctypes.c_void_p((1 << 20) + 8))),
    ("INVALID_ARG", dict(table=None)), ("INVALID_ARG", dict(width=0)),
    ("INVALID_ARG", dict(hq=30)), ("INVALID_ARG", dict(seqs=-1)), ("INVALID_ARG", dict(tokens=-1)),
    ("UNSUPPORTED", dict(width=(1 << 26) + 1)), ("UNSUPPORTED", dict(kv=desc(d=96))),
    ("UNSUPPORTED", dict(kv=desc(block_size=24))), ("INVALID_ARG", dict(kv=desc(dtype=1))),
    ("WORKSPACE", dict(ws=None)), ("WORKSPACE", dict(ws_bytes=1024)),
    ("WORKSPACE", dict(ws=ctypes.c_void_p((1 << 22) + 16)))])
def test_window_attention_refusals(want, kw):
    assert call_window(**kw) == getattr(pk, "PA_ERR_" + want)


def test_window_attention_of_nothing_is_ok():
    assert call_window(seqs=0) == pk.PA_OK
    assert call_window(tokens=0, q=None) == pk.PA_OK


def call_rope(kv=None, q=F, qs=4096, k=F, ks=1024, vs=1024, pos=F, inv=1 << 20, axis=None, rot=128,
              axes=1, adjacent=0, factor=1.0, slots=F, tokens=4, hq=32, q_out=WS):
    kv = kv or desc()
    r = pk.RopeDesc(inv, axis, rot, axes, adjacent, factor)
    return pk.lib().pa_rope_write_kv(q, qs, k, ks, F, vs, pos, ctypes.byref(r), slots, tokens, hq,
                                     ctypes.byref(kv), q_out, None)


@pytest.mark.parametrize("want,kw", [
    ("INVALID_ARG", dict(q=None)), ("INVALID_ARG", dict(k=None)), ("INVALID_ARG", dict(pos=None)),
    ("INVALID_ARG", dict(inv=None)), ("INVALID_ARG", dict(slots=None)),
    ("INVALID_ARG", dict(q_out=None)), ("INVALID_ARG", dict(q=ctypes.c_void_p((1 << 20) + 2))),
    ("INVALID_ARG", dict(qs=4092)), ("INVALID_ARG", dict(qs=2048)), ("INVALID_ARG", dict(ks=1023)),
    ("INVALID_ARG", dict(vs=512)), ("INVALID_ARG", dict(ks=-1024)),
    ("INVALID_ARG", dict(tokens=-1)), ("INVALID_ARG", dict(hq=-1)),
    ("INVALID_ARG", dict(adjacent=2)), ("INVALID_ARG", dict(factor=float("nan"))),
    ("INVALID_ARG", dict(q_out=F, qs=8192)),                       # in place, not contiguous
    ("INVALID_ARG", dict(pos=ctypes.c_void_p((1 << 20) + 2))),
    ("INVALID_ARG", dict(slots=ctypes.c_void_p((1 << 20) + 4))),
    ("INVALID_ARG", dict(inv=(1 << 20) + 4)), ("INVALID_ARG", dict(axis=(1 << 20) + 1)),
    ("UNSUPPORTED", dict(rot=136)), ("UNSUPPORTED", dict(rot=144)), ("UNSUPPORTED", dict(rot=0)),
    ("UNSUPPORTED", dict(rot=24)), ("UNSUPPORTED", dict(axes=0)), ("UNSUPPORTED", dict(axes=9)),
    ("UNSUPPORTED", dict(kv=desc(d=80))), ("INVALID_ARG", dict(kv=desc(dtype=1)))])
def test_rope_write_refusals(want, kw):
    assert call_rope(**kw) == getattr(pk, "PA_ERR_" + want)


def test_rope_write_of_nothing_is_ok():
    assert call_rope(tokens=0) == pk.PA_OK
    assert pk.lib().pa_rope_write_kv(F, 0, F, 0, F, 0, F, None, F, 4, 32, ctypes.byref(desc()), F,
                                     None) == pk.PA_ERR_INVALID_ARG


def call_copy(kvs, pairs=F, n=2, layers=None):
    arr = (pk.KVDesc * max(len(kvs), 1))(*kvs)
    return pk.lib().pa_copy_blocks(arr, len(kvs) if layers is None else layers, pairs, n, None)


def test_copy_blocks_refusals():
    assert call_copy([desc(), desc(block_size=32)]) == pk.PA_ERR_INVALID_ARG
    assert call_copy([desc(), desc(num_blocks=99)]) == pk.PA_ERR_INVALID_ARG
    assert call_copy([desc(), desc(dtype=1)]) == pk.PA_ERR_INVALID_ARG
    assert call_copy([desc(k=(1 << 20) + 8)]) == pk.PA_ERR_INVALID_ARG
    assert call_copy([desc(d=96)]) == pk.PA_ERR_UNSUPPORTED
    assert call_copy([desc()], pairs=None) == pk.PA_ERR_INVALID_ARG
    assert call_copy([desc()], pairs=ctypes.c_void_p((1 << 20) + 4)) == pk.PA_ERR_INVALID_ARG
    assert call_copy([desc()], n=-1) == pk.PA_ERR_INVALID_ARG
    assert call_copy([desc()], layers=-1) == pk.PA_ERR_INVALID_ARG
    assert pk.lib().pa_copy_blocks(None, 1, F, 1, None) == pk.PA_ERR_INVALID_ARG
    # nothing to do; codes move without their scales
    assert call_copy([]) == pk.PA_OK and call_copy([desc()], n=0) == pk.PA_OK
    assert call_copy([desc(dtype=1)], n=0) == pk.PA_OK


def test_rope_descriptor_layout():
    assert ctypes.sizeof(pk.RopeDesc) == 32 and pk.RopeDesc.attn_factor.offset == 28


def test_binding_refuses_host_tensors_and_wrong_types():
    z = torch.zeros(2, 4, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pk.pa_window_attention(q, z, z, i[None], i, i[:1], i[:1], 0.1, 4, 0, q)
    with pytest.raises(TypeError):
        pk.pa_window_attention(q.float(), z, z, i[None], i, i[:1], i[:1], 0.1, 4, 0, q)
    with pytest.raises(ValueError):
        pk.pa_rope_write_kv(q, q, q, i, i.double(), None, i.long(), z, z, q)
    with pytest.raises(TypeError):
        pk.pa_rope_write_kv(q, q.half(), q, i, i.double(), None, i.long(), z, z, q)
    with pytest.raises(ValueError):
        pk.kv_layers([z], [z])
    with pytest.raises(ValueError):
        pk.kv_layers([z], [])
    with pytest.raises(TypeError):
        pk.kv_layers([z.float()], [z])
    with pytest.raises(TypeError):
        pk.pa_copy_blocks(pk.kv_layers([], []), i.long())
    with pytest.raises(ValueError):
        pk.pa_copy_blocks(pk.kv_layers([], []), i)


# ---- numbers past int32 ------------------------------------------------------------

@pytest.mark.parametrize("window,sinks,gone", [
    (2**32 + 1, 0, 0), (2**40, 0, 0), (2**63, 0, 0), (1, 2**32, 0), (1, 2**70, 0), (1, 0, 9)])
def test_release_window_with_numbers_past_int32(window, sinks, gone):
    """A window or sinks past any request's keys hide nothing, whatever their low 32
    bits are."""
    bm = BlockManager(16, 4)
    bm.add_request(1, [5])
    bm.append_tokens(1, [1] * 37)
    bm.schedule([1], [38], 64)
    assert bm.release_window(1, window, sinks) == gone
    assert bm.blocks_of(1).count(-1) == gone


@pytest.mark.parametrize("window,sinks", [(-2**32 + 5, 0), (5, -2**32 + 5), (-2**70, 0), (2**32, -1)])
def test_negative_numbers_past_int32_are_refused(window, sinks):
    bm = BlockManager(16, 4)
    bm.add_request(1, [5])
    with pytest.raises(pk.PaError) as e:
        bm.release_window(1, window, sinks)
    assert e.value.code == pk.PA_ERR_INVALID_ARG
    t = [torch.tensor(x, dtype=torch.int32) for x in ([[0]], [0, 1], [0], [1])]
    with pytest.raises(pk.PaError) as e:
        pk.pa_validate_metadata(*t, num_blocks=4, block_size=16, window=window, num_sinks=sinks)
    assert e.value.code == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("window,sinks", [(2**32 + 1, 0), (2**40, 0), (1, 2**32 + 16), (1, 2**70)])
def test_window_metadata_with_numbers_past_int32(window, sinks):
    """Every block of a request of 51 tokens is visible then, -1 entries are not."""
    kw = dict(num_blocks=4, block_size=16, window=window, num_sinks=sinks)
    rest = [torch.tensor(x, dtype=torch.int32) for x in ([0, 1], [50], [51])]
    pk.pa_validate_metadata(torch.tensor([[0, 1, 2, 3]], dtype=torch.int32), *rest, **kw)
    with pytest.raises(pk.PaError) as e:
        pk.pa_validate_metadata(torch.tensor([[0, -1, 2, 3]], dtype=torch.int32), *rest, **kw)
    assert e.value.code == pk.PA_ERR_BAD_METADATA


def test_compact_with_numbers_past_int32():
    def pool():
        bm = BlockManager(8, 4)
        for rid in (1, 2):
            bm.add_request(rid, [rid] * 4)
            bm.schedule([rid], [4], 8)
        bm.append_tokens(2, [7] * 4)
        bm.schedule([2], [4], 8)
        bm.free_request(1)
        bm.add_request(3, [9] * 4)
        return bm
    for most in (2**32 + 3, 2**70):
        assert pool().compact(most).tolist() == pool().compact().tolist()
    for most in (-2**32 + 3, -2**70, -1):
        with pytest.raises(pk.PaError) as e:
            pool().compact(most)
        assert e.value.code == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("pairs", [torch.tensor([1, 2, 3, 4]), torch.tensor([[1], [2], [3]]),
                                   torch.tensor([[1, 2, 0], [3, 4, 0]]), torch.zeros(1, 2, 2),
                                   torch.tensor(3), [5, 6]])
def test_validate_copies_refuses_what_is_no_list_of_pairs(pairs):
    """(A flat list or one column holds fewer than two numbers a row.)"""
    with pytest.raises(ValueError, match="pairs"):
        pk.pa_validate_copies(pairs, 10)


@pytest.mark.parametrize("pairs", [[], torch.empty(0, 2, dtype=torch.int32), [[1, 2], [3, 4]],
                                   np.array([[0, 9]], np.int64)])
def test_validate_copies_takes_pairs(pairs):
    pk.pa_validate_copies(pairs, 10)


def test_blocks_of_a_stream_longer_than_the_pool():
    """200 tokens through a pool of 6 blocks of 4: the whole table, given back
    entries and the last blocks alike."""
    m, bm = BlockManagerModel(6, 4), BlockManager(6, 4)
    for x in (m, bm):
        x.add_request(1, [5])
    for i in range(50):
        advance(m, bm, 1, 4 if i else 3)
        assert bm.release_window(1, 7, 2) == m.release_window(1, 7, 2)[1]
        same(m, bm)
    table = bm.blocks_of(1)
    assert len(table) == 50 and table[0] >= 0 and table[-1] >= 0 and table.count(-1) == 47
    assert bm.blocks_of(2) is None
    bm.add_request(2, [1])
    assert bm.blocks_of(2) == []


# ---- the direct binding's answers ---------------------------------------------------

class Answers:
    """Stands in for the direct binding: every call gives `code`."""

    def __init__(self, code):
        self.code, self.calls = code, 0

    def window_attention(self, *args):
        self.calls += 1
        return self.code
    rope_write_kv = copy_blocks = window_attention


def direct_calls():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    n = torch.zeros(3, dtype=torch.int32)
    layers = pk.KVLayers((pk.KVDesc * 1)(), [x])
    return {
        "pa_window_attention": lambda: pk.pa_window_attention(
            x, x, x, n, n, n, n, 1.0, 4, 0, x, workspace=torch.zeros(8, dtype=torch.uint8)),
        "pa_rope_write_kv": lambda: pk.pa_rope_write_kv(x, x, x, n, n, None, n, x, x, x),
        "pa_copy_blocks": lambda: pk.pa_copy_blocks(layers, torch.zeros(1, 2, dtype=torch.int64))}


@pytest.mark.parametrize("name", ["pa_window_attention", "pa_rope_write_kv", "pa_copy_blocks"])
@pytest.mark.parametrize("code", [pk.PA_ERR_INVALID_ARG, pk.PA_ERR_UNSUPPORTED, pk.PA_ERR_CUDA])
def test_a_failed_call_is_not_made_again(monkeypatch, name, code):
    """What the library refuses, or what fails on the device, is raised as it came."""
    answers = Answers(code)
    monkeypatch.setattr(pk, "_direct", answers)
    with pytest.raises(pk.PaError) as e:
        direct_calls()[name]()
    assert e.value.code == code and answers.calls == 1 and name in str(e.value)


@pytest.mark.parametrize("name", ["pa_window_attention", "pa_rope_write_kv", "pa_copy_blocks"])
def test_calls_that_are_not_plain_reach_the_checks(monkeypatch, name):
    monkeypatch.setattr(pk, "_direct", Answers(-1))
    with pytest.raises((TypeError, ValueError)):     # (CPU tensors, int64 pairs)
        direct_calls()[name]()
