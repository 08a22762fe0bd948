"""Lengths far beyond the block tables in an e4m3 step with a staging area: flagged, left out, and
counted so that no sum of their blocks wraps."""
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV
from test_gpu_window import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("count,length", [(40, 2**31 - 1), (17, 2**31 - 1), (1100, 2**31 - 1), (33, 2**31 - 300)])
def test_huge_lengths(count, length, first):
    """`count` requests of 17 tokens with the length, no context and so a length that is none of
    theirs, behind or before three good ones, two of which are staged."""
    n = 17
    s = Step([(300, 70), (40, 1), (100, 90)], 8, 2, 128, 16, 100000, 0, kv="e4m3", seed=1, pad=count * n)
    t = s.to_dev()
    i32 = dict(dtype=torch.int32, device=DEV)
    bad = torch.arange(1, count + 1, **i32) * n
    good = t["qsl"][1:]
    if first:   # the good rows move to the end
        q = torch.cat([t["q"][s.total:], t["q"][:s.total]])
        qsl = torch.cat([torch.zeros(1, **i32), bad, good + count * n])
    else:
        q, qsl = t["q"], torch.cat([torch.zeros(1, **i32), good, bad + s.total])
    order = (lambda a, b: torch.cat([b, a])) if first else (lambda a, b: torch.cat([a, b]))
    table = order(t["table"], torch.zeros((count, t["table"].shape[1]), **i32))
    ctx = order(t["ctx"], torch.zeros(count, **i32))
    seq = order(t["seq"], torch.full((count,), length, **i32))
    out = torch.full_like(q, 7)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    pk.pa_attention(q, t["k"], t["v"], table, qsl, ctx, seq, s.scale, out, lse, k_scale=t["ks"],
                    v_scale=t["vs"], staging_blocks=s.staging + 5)
    torch.cuda.synchronize()
    assert pk.read_device_status(clear=True) == pk.PA_DEV_BAD_METADATA
    if first:
        out, lse = (torch.cat([x[count * n:], x[:count * n]]) for x in (out, lse))
    s.check({"out": out, "lse": lse})
