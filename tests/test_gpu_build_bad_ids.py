"""An id outside the pool in pa_build_step's free list: what the step after it does."""
import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV
from test_gpu_build import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, -5, 2**31 - 1, None])
@pytest.mark.parametrize("rows", [[(1, 16), (1, 20), (2, 7)], [(1, 16), (1500, 20), (-1, 70), (3, 45)]])
def test_no_later_step_writes_where_the_id_was_clamped_to(rows, bad):
    """The list holds a bad id where row 0 takes its block, or (large steps) where a later row
    does: that row's tokens get no slot, and no later step is made, in place or with the lengths
    and the list's state carried over by the caller."""
    for row in (0, 1) if rows[1][0] > 1 else (0,):
        b = Batch(rows, 16, 100)
        at = b.head + (0 if row == 0 else 1 + 40)
        b.ring[at % len(b.ring)] = b.num_blocks if bad is None else bad
        t = b.on_gpu()
        b.call(t)
        torch.cuda.synchronize()
        assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_BLOCK
        good = b.expected()
        head, count = int(good["state"][0]), int(good["state"][1])
        assert t["state"].tolist() == [-1 - head, count, 0, 0]
        assert torch.equal(t["seq"].cpu(), torch.from_numpy(good["seq"]))
        kept = {x: t[x].clone() for x in ("table", "ring", "seq", "state")}
        # the next step: all rows one token on
        t["q"].fill_(1)
        t["cached"], t["state_in"] = t["seq"], t["state"]
        t["seq"], t["state"] = torch.zeros_like(t["seq"]), torch.zeros_like(t["state"])
        for _ in range(3):
            b.call(t)
            torch.cuda.synchronize()
            assert torch.all(t["slots"] == -1) and torch.all(t["qsl"] == 0)
            assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_METADATA
            assert torch.equal(t["table"], kept["table"]) and torch.equal(t["ring"], kept["ring"])
            assert torch.equal(t["seq"], kept["seq"])
            assert t["state"].tolist() == kept["state"].tolist()
            t["cached"], t["seq"] = t["seq"], t["cached"]
            t["state_in"], t["state"] = t["state"], t["state_in"]


@pytest.mark.parametrize("more", [0, 1500])
def test_after_the_caller_has_mended_table_and_list(more):
    """The head that was left names the place: with the list's head and the row's entry put right
    the batch goes on."""
    b = Batch([(1, 16), (1 + more, 20)], 16, 100)
    good = b.expected()
    at = b.head % len(b.ring)
    right = int(b.ring[at])
    b.ring[at] = -2
    t = b.on_gpu()
    b.call(t)
    torch.cuda.synchronize()
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_BLOCK
    t["table"][0, 1] = right
    t["state"][0] = -1 - t["state"][0]
    assert np.array_equal(t["table"].cpu().numpy(), good["table"])
    assert np.array_equal(t["state"].cpu().numpy(), good["state"])
    b.q[:] = 1
    b.cached, b.table = good["seq"], good["table"]
    b.ring = t["ring"].cpu().numpy()
    b.head, b.count = int(good["state"][0]), int(good["state"][1])
    t["q"].fill_(1)
    t["cached"], t["state_in"] = t["seq"].clone(), t["state"].clone()
    b.call(t)
    torch.cuda.synchronize()
    want = b.expected()
    for name in ("qsl", "ctx", "seq", "slots", "positions", "table", "state"):
        assert np.array_equal(t[name].cpu().numpy(), want[name]), name
    assert pk.read_device_status(clear=True) == 0
