"""Prompts whose tensor-core kernels' waits end at other times in each run: beside copies on
another stream, the same calls give the same bits as alone, and no wait runs out.  (What an
issuing thread reads between a barrier and its MMAs must not depend on when the barrier was
ready.)"""
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
import test_gpu_cross
import test_gpu_linear
import test_gpu_window
from gpu_helpers import DEV, assert_status_clean

pytestmark = pytest.mark.gpu

RAGGED = [(0, 300), (700, 129), (33, 128), (1500, 65), (4, 1), (900, 513)]


def repeat(call, outputs, times=12):
    """`call` alone, then `times` times beside copies; its outputs each time."""
    call()
    torch.cuda.synchronize()
    first = [x.clone() for x in outputs]
    side, a = torch.cuda.Stream(), torch.ones(64 << 20, device=DEV)
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    for turn in range(times):
        with torch.cuda.stream(side):
            for _ in range(1 + turn % 4):
                b.copy_(a)
        for x in outputs:
            x.zero_()
        call()
        torch.cuda.synchronize()
        for x, want in zip(outputs, first):
            assert torch.equal(x, want), turn
    assert_status_clean()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(200, 4), (100000, 0)])
def test_windowed(window, sinks, d):
    s = test_gpu_window.Step(RAGGED * 3, 8, 2, d, 16, window, sinks, seed=1)
    t = s.to_dev()
    repeat(lambda: s.call(t), [t["out"], t["lse"]])


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("bf16", 128), ("e4m3", 128)])
def test_cross(kv, d):
    s = test_gpu_cross.Step([(n + 1, m) for n, m in RAGGED * 3], 8, 2, d, 16, kv, seed=2)
    t = s.to_dev()
    repeat(lambda: s.call(t), [t["out"], t["lse"]])


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (6, 6, 64)])
def test_linear(hq, hkv, d):
    s = test_gpu_linear.Step([m for _, m in RAGGED * 3], hq, hkv, d, seed=3)
    t = s.to_dev()
    repeat(lambda: s.call(t), [t["out"]])
