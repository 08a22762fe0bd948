"""Groups of more than 64 query heads: one token's rows are more than a split-KV piece holds, so
they run on the tensor-core kernels alone; an e4m3 pool, which may need pieces, refuses them."""
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
import test_gpu_cross
import test_gpu_window
from gpu_helpers import DEV, assert_status_clean

pytestmark = pytest.mark.gpu

GROUPS = [(65, 1), (100, 1), (128, 1), (200, 2)]
KEYS = [(0, 1), (300, 1), (17, 2), (1, 1), (0, 3), (700, 1), (129, 0), (64, 5)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", GROUPS)
def test_cross(hq, hkv, d):
    s = test_gpu_cross.Step(KEYS, hq, hkv, d, 16, seed=hq, pad=2)
    t = s.to_dev()
    s.call(t)
    s.check(t)
    assert_status_clean()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", GROUPS)
@pytest.mark.parametrize("window", [40, 100000])
def test_windowed_and_plain(window, hq, hkv, d):
    s = test_gpu_window.Step(KEYS, hq, hkv, d, 16, window, 0, seed=hq, pad=2)
    t = s.run_and_check()
    if window == 100000:   # (sees all keys)
        t["out"].fill_(7)
        t["lse"].fill_(7)
        pk.pa_attention(t["q"], t["k"], t["v"], t["table"], t["qsl"], t["ctx"], t["seq"], s.scale,
                        t["out"], t["lse"])
        torch.cuda.synchronize()
        s.check(t)
        assert_status_clean()


@pytest.mark.parametrize("hq", [65, 128])
def test_an_e4m3_pool_of_such_groups_is_refused(hq):
    for step in (test_gpu_window.Step(KEYS, hq, 1, 128, 16, 100000, 0, kv="e4m3", seed=1),
                 test_gpu_cross.Step(KEYS, hq, 1, 128, 16, "e4m3", seed=1)):
        t = step.to_dev()
        for staging in (0, step.staging):
            with pytest.raises(pk.PaError, match="group size"):
                step.call(t, staging_blocks=staging)
        torch.cuda.synchronize()
        assert torch.all(t["out"] == 7) and torch.all(t["lse"] == 7)
    assert_status_clean()
