"""pa_rope_write_kv on the GPU against the float64 definition.

Tolerances: one rounding to bf16 (2^-8 of the value), or to e4m3 (2^-4 of the
code's value, half the subnormal step 2^-10 below that); the fp32 rotation
adds at most |f| (|a| + |b|) 2^-21 (cos and sin good to 2^-22, three fp32
roundings of 2^-24 each).  v and the unrotated elements are exact in bf16."""
import time

import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean
from oracle import ops

pytestmark = pytest.mark.gpu


def make(T, hq, hkv, d, rot, bs, axes=1, kv="bf16", fused=True, max_pos=5000, seed=0, pad=0,
         far=False):
    g = torch.Generator().manual_seed(seed)
    nb = -(-T // bs) + 2
    x = torch.randn((T, (hq + 2 * hkv) * d), generator=g).to(torch.bfloat16)
    s = dict(T=T, hq=hq, hkv=hkv, d=d, rot=rot, bs=bs, kv=kv)
    s["qkv"] = x
    lo, hi = (-2**31, 2**31) if far else (0, max_pos)
    s["positions"] = torch.randint(lo, hi, (axes, T), generator=g).to(torch.int32)
    s["inv_freq"] = 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    s["axis"] = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32) if axes > 1 else None
    slots = torch.randperm(nb * bs, generator=g)[:T]
    if pad:
        slots[torch.randperm(T, generator=g)[:pad]] = -1
    s["slots"] = slots
    shape = (nb, hkv, bs, d)
    if kv == "bf16":
        s["kc"], s["vc"] = (torch.randn(shape, generator=g).to(torch.bfloat16) for _ in "kv")
        s["ks"] = s["vs"] = None
    else:
        s["kc"], s["vc"] = ((torch.randn(shape, generator=g) * 16).to(torch.float8_e4m3fn)
                            .view(torch.uint8) for _ in "kv")
        s["ks"], s["vs"] = (0.004 + 0.05 * torch.rand(hkv, generator=g) for _ in "kv")
    return s


def split(s, qkv):
    T, hq, hkv, d = s["T"], s["hq"], s["hkv"], s["d"]
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
    return q.view(T, hq, d), k.view(T, hkv, d), v.view(T, hkv, d)


def to_dev(s):
    return {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in s.items()}


def call(s, t, fused=True, adjacent=False, factor=1.0, q_out=None, stream=None):
    q, k, v = split(s, t["qkv"])
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if q_out is None:
        q_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    pk.pa_rope_write_kv(q, k, v, t["positions"], t["inv_freq"], t["axis"], t["slots"], t["kc"],
                        t["vc"], q_out, adjacent=adjacent, attn_factor=factor, k_scale=t["ks"],
                        v_scale=t["vs"], stream=stream)
    return q_out


def check(s, t, q_out, adjacent=False, factor=1.0):
    torch.cuda.synchronize()
    axis = None if s["axis"] is None else s["axis"].numpy()
    how = (s["positions"].numpy(), s["inv_freq"].numpy(), axis, s["rot"], adjacent, factor)
    q, k, v = (x.double().numpy() for x in split(s, s["qkv"]))

    def spread(x):  # |a| + |b| of each rotated element's pair, 0 for the others
        z = np.zeros_like(x)
        i, r = np.arange(s["rot"] // 2), s["rot"]
        ia, ib = (2 * i, 2 * i + 1) if adjacent else (i, i + r // 2)
        z[..., ia] = z[..., ib] = (np.abs(x[..., ia]) + np.abs(x[..., ib])) * abs(factor) * 2.0 ** -21
        return z
    ref = ops.rope(q, *how)
    got = q_out.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + spread(q))
    assert np.array_equal(got[..., s["rot"]:], q[..., s["rot"]:])
    live = s["slots"].numpy() >= 0
    slots = s["slots"].numpy()[live]
    for name, rows, new, slack in (("kc", ops.rope(k, *how), t["kc"], spread(k)),
                                   ("vc", v, t["vc"], np.zeros_like(v))):
        old, got = s[name].clone(), new.cpu()
        at = (slots // s["bs"], slice(None), slots % s["bs"])
        if s["kv"] == "bf16":
            y = got[at].double().numpy()
            assert np.all(np.abs(y - rows[live]) <= 2.0 ** -8 * np.abs(rows[live]) + slack[live])
            exact = slice(s["rot"] if name == "kc" else 0, None)
            assert np.array_equal(y[..., exact], rows[live][..., exact])
        else:
            scale = s["ks" if name == "kc" else "vs"].double().numpy()[:, None]
            y = got[at].view(torch.float8_e4m3fn).double().numpy()
            want = np.clip(rows[live] / scale, -448, 448)
            tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + slack[live] / scale
            assert np.all(np.abs(y - want) <= tol)
        old[at] = got[at]
        assert torch.equal(old, got), f"{name}: a slot of no token changed"
    assert_status_clean()


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 96),
                                   (128, 112)])
def test_rotated_widths(d, rot, adjacent):
    for kv in ("bf16", "e4m3")[:1 + (d == 128)]:
        s = make(37, 8, 2, d, rot, 16, axes=3, kv=kv, seed=rot)
        t = to_dev(s)
        check(s, t, call(s, t, adjacent=adjacent), adjacent)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 33, 257])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (32, 8), (14, 2), (1, 1), (16, 1), (3, 3)])
def test_tokens_and_heads(T, hq, hkv):
    s = make(T, hq, hkv, 128, 128, 32, seed=T)
    t = to_dev(s)
    check(s, t, call(s, t))
    s = make(T, hq, hkv, 128, 64, 16, axes=3, kv="e4m3", seed=T, pad=T // 3)
    t = to_dev(s)
    check(s, t, call(s, t, fused=False, adjacent=True), True)


def test_many_tokens():
    s = make(5003, 32, 8, 128, 128, 16, axes=3, seed=1, pad=100)
    t = to_dev(s)
    check(s, t, call(s, t))


@pytest.mark.parametrize("adjacent", [False, True])
def test_far_and_negative_positions(adjacent):
    """Any int32 position: the angle is reduced without loss."""
    s = make(200, 2, 1, 64, 64, 16, axes=2, far=True, seed=9)
    s["positions"][:, :4] = torch.tensor([[2**31 - 1, -2**31, 0, -1], [1, 2, 3, 4]])
    t = to_dev(s)
    check(s, t, call(s, t, adjacent=adjacent), adjacent)


def test_frequencies_of_whole_turns_and_negative_ones():
    s = make(20, 2, 1, 64, 64, 16, seed=2, max_pos=1000)
    s["inv_freq"][:4] = torch.tensor([2 * np.pi, 0.0, -0.7, 40.0], dtype=torch.float64)
    t = to_dev(s)
    check(s, t, call(s, t))


def test_factor_scales_the_rotated_part_alone():
    s = make(21, 4, 2, 128, 64, 16, axes=3, seed=3)
    t = to_dev(s)
    check(s, t, call(s, t, factor=1.37), factor=1.37)


def test_q_in_place():
    s = make(50, 8, 2, 128, 96, 16, seed=4)
    t = to_dev(s)
    q, k, v = split(s, t["qkv"])
    q = q.contiguous()
    pk.pa_rope_write_kv(q, k, v, t["positions"], t["inv_freq"], None, t["slots"], t["kc"], t["vc"], q)
    check(s, t, q)


def test_keys_and_values_without_queries():
    s = make(9, 2, 2, 64, 64, 16, seed=5)
    t = to_dev(s)
    q, k, v = split(s, t["qkv"])
    pk.pa_rope_write_kv(None, k, v, t["positions"], t["inv_freq"], None, t["slots"], t["kc"],
                        t["vc"], None)
    whole = call(s, to_dev(s))
    check(s, t, whole)


def test_position_zero_writes_what_pa_write_kv_writes():
    for kv in ("bf16", "e4m3"):
        s = make(40, 4, 2, 128, 128, 16, kv=kv, seed=6, pad=5)
        s["positions"].zero_()
        t, u = to_dev(s), to_dev(s)
        q_out = call(s, t)
        q, k, v = split(s, u["qkv"])
        pk.pa_write_kv(k.contiguous(), v.contiguous(), u["slots"], u["kc"], u["vc"], k_scale=u["ks"],
                       v_scale=u["vs"])
        torch.cuda.synchronize()
        assert torch.equal(t["kc"], u["kc"]) and torch.equal(t["vc"], u["vc"])
        assert torch.equal(q_out, q)


def test_bad_slots_and_axes_are_flagged():
    s = make(12, 2, 1, 64, 64, 16, axes=3, seed=7)
    t = to_dev(s)
    t["slots"][3] = t["kc"].shape[0] * 16
    call(s, t)
    torch.cuda.synchronize()
    assert pk.read_device_status() == pk.PA_DEV_BAD_SLOT
    old = s["kc"].clone()
    live = [i for i in range(12) if i != 3]
    at = (s["slots"][live] // 16, slice(None), s["slots"][live] % 16)
    old[at] = t["kc"].cpu()[at]
    assert torch.equal(old, t["kc"].cpu())
    t = to_dev(s)
    t["axis"][5], t["axis"][6] = 3, -1
    q_out = call(s, t)
    torch.cuda.synchronize()
    assert pk.read_device_status() == pk.PA_DEV_BAD_METADATA
    s["axis"][5], s["axis"][6] = 2, 0   # what the clamp makes of them
    check(s, t, q_out)


def test_graph_and_stream():
    s = make(30, 8, 2, 128, 128, 16, axes=3, seed=8)
    t = to_dev(s)
    q_out = torch.empty((30, 8, 128), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(s, t, q_out=q_out, stream=side)
    torch.cuda.synchronize()
    check(s, t, q_out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(s, t, q_out=q_out)
    other = make(30, 8, 2, 128, 128, 16, axes=3, seed=88)
    o = to_dev(other)
    for name in ("qkv", "positions", "axis", "slots", "kc", "vc"):
        t[name].copy_(o[name])
    g.replay()
    check(other, t, q_out)


def test_binding_takes_plain_calls_and_leaves_the_others():
    """The direct binding launches a documented call and hands every other back
    (-1) without a launch."""
    dev, T, d = torch.device("cuda:0"), 5, 64
    q = torch.randn(T, 4, d, device=dev).to(torch.bfloat16)
    k, v = (torch.randn(T, 2, d, device=dev).to(torch.bfloat16) for _ in "kv")
    kc, vc = (torch.zeros(3, 2, 16, d, device=dev, dtype=torch.bfloat16) for _ in "kv")
    pos = torch.arange(T, device=dev, dtype=torch.int32)
    freq = torch.ones(d // 2, device=dev, dtype=torch.float64)
    axis = torch.zeros(d // 2, device=dev, dtype=torch.int32)
    slots = torch.arange(T, device=dev, dtype=torch.int64)
    out = torch.empty_like(q)
    call = pk._load_direct().rope_write_kv
    good = [q, k, v, pos, freq, axis, slots, kc, vc, out, False, 1.0, None, None, None]
    assert call(*good) == 0
    assert call(None, *good[1:9], None, *good[10:]) == 0
    assert call(*good[:5], None, *good[6:]) == 0
    torch.cuda.synchronize()
    before = pk.lib().pa_kernel_launches()
    wrong = {0: [q.float(), q[:3], None, q[..., ::2]], 1: [k.cpu(), k[:, :1], k[0]],
             2: [v[1:], v.half()], 3: [pos.long(), pos[1:], pos.view(1, 1, T)],
             4: [freq.float(), freq[1:]], 5: [axis[1:], axis.long()], 6: [slots.int(), slots[1:]],
             7: [kc[0], kc.float(), vc.view(torch.uint8)], 8: [vc[1:]], 9: [None, out[1:]],
             10: [0, None], 11: ["1", None], 12: [5], 13: [freq]}
    for i, values in wrong.items():
        for x in values:
            assert call(*good[:i], x, *good[i + 1:]) == -1, (i, x)
    assert call() == -1
    assert pk.lib().pa_kernel_launches() == before
    with pytest.raises((TypeError, ValueError)):
        pk.pa_rope_write_kv(*good[:3], pos.long(), *good[4:10])


# Scales: ordinary, both sides of 2^-60 and 2^60, where the quotient is taken another
# way, and the ends of fp32.
@pytest.mark.parametrize("scales", [(1.0, 0.0371), (2.0 ** -59, 1.7 * 2.0 ** 59),
                                    (2.0 ** -61, 1.3 * 2.0 ** 61), (0.3, 7.0 / 3.0),
                                    (2.0 ** -126, 3.0e38), (1.1e-5, 450.7)])
@pytest.mark.parametrize("adjacent", [False, True])
def test_every_bf16_value_gets_the_code_of_pa_write_kv(scales, adjacent):
    """All 65536 bit patterns (zeros of both signs, subnormals, infinities, NaN) as
    values and as unrotated key elements, at two scales: the same codes, bit for bit."""
    T, hkv, d, bs, rot = 592, 2, 128, 16, 16
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    # 112 unrotated elements a head: 592 tokens hold every pattern
    rows = torch.zeros(T * (d - rot), dtype=torch.bfloat16)
    rows[:65536] = every
    x = torch.zeros(T, hkv, d, dtype=torch.bfloat16)
    x[:, :, rot:] = rows.view(T, 1, d - rot)
    x[:, :, :rot] = x[:, :, rot:2 * rot]
    k, v = x.clone(), x
    k[:, :, :rot] = 0.5
    slots = torch.randperm(T, generator=torch.Generator().manual_seed(1))
    k, v, slots = k.to(DEV), v.to(DEV), slots.to(DEV)
    ks = torch.tensor(scales, dtype=torch.float32, device=DEV)
    vs = ks.flip(0).contiguous()
    new, want = ([torch.full((T // bs, hkv, bs, d), 0x11, dtype=torch.uint8, device=DEV)
                  for _ in "kv"] for _ in range(2))
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    freq = torch.ones(rot // 2, dtype=torch.float64, device=DEV)
    pk.pa_rope_write_kv(None, k, v, pos, freq, None, slots, *new, None, adjacent=adjacent,
                        k_scale=ks, v_scale=vs)
    pk.pa_write_kv(k, v, slots, *want, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    for name, a, b in (("k", new[0], want[0]), ("v", new[1], want[1])):
        wrong = (a != b).nonzero()
        assert len(wrong) == 0, (name, len(wrong), wrong[:4].tolist(), a[a != b][:4].tolist(),
                                 b[a != b][:4].tolist())
    # (an e4m3 zero keeps its sign: both codes appear)
    assert (want[1] == 0x80).any() and (want[1] == 0x00).any()
    assert_status_clean()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_rows_that_never_come_time_out(kv):
    """The first warp's second item is not fetched: its wait runs out (2 s), the status
    says so, the rows before it are written, and the next call is right."""
    s = make(2500, 32, 8, 128, 128, 16, axes=3, kv=kv, seed=10)
    t = to_dev(s)
    torch.cuda.synchronize()
    pk.set_test_stall(pk.PA_TEST_STALL_ROPE)
    try:
        t0 = time.perf_counter()
        q_out = call(s, t)
        torch.cuda.synchronize()
        seconds = time.perf_counter() - t0
    finally:
        pk.set_test_stall(pk.PA_TEST_STALL_NONE)
    assert 1.5 < seconds < 60.0, seconds
    assert pk.read_device_status(clear=True) == pk.PA_DEV_WAIT_TIMEOUT
    whole = call(s, to_dev(s))
    lost = (q_out != whole).flatten(1).any(1).nonzero().flatten().tolist()
    assert lost and max(lost) < 20, lost
    assert torch.equal(q_out[0, 0], whole[0, 0]) and torch.all(q_out[0, -1] == 7.0)
    check(s, t, call(s, t))
