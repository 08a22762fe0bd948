"""pa_copy_blocks on the GPU: bit-exact, every other block untouched."""
import numpy as np
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean
from oracle import ops

pytestmark = pytest.mark.gpu


def pools(layers, nb, hkv, bs, d, kv="bf16", seed=0):
    """Arbitrary bit patterns, NaNs among them."""
    g = torch.Generator().manual_seed(seed)
    if kv == "bf16":
        make = lambda: torch.randint(-2**15, 2**15, (nb, hkv, bs, d), generator=g,  # noqa: E731
                                     dtype=torch.int16).view(torch.bfloat16)
    else:
        make = lambda: torch.randint(0, 256, (nb, hkv, bs, d), generator=g, dtype=torch.uint8)  # noqa: E731
    return [make() for _ in range(layers)], [make() for _ in range(layers)]


def raw(t):
    return t.cpu().view(torch.uint8).numpy()


def run(layers, nb, hkv, bs, d, pairs, kv="bf16", seed=0, stream=None):
    ks, vs = pools(layers, nb, hkv, bs, d, kv, seed)
    kd, vd = [x.to(DEV) for x in ks], [x.to(DEV) for x in vs]
    torch.cuda.synchronize()
    p = torch.tensor(np.array(pairs, np.int32).reshape(-1, 2), device=DEV)
    torch.cuda.synchronize()
    pk.pa_copy_blocks(pk.kv_layers(kd, vd), p, stream=stream)
    torch.cuda.synchronize()
    return ks, vs, kd, vd


def check(ks, vs, kd, vd, pairs):
    for old, new in zip(ks + vs, kd + vd):
        assert np.array_equal(ops.copy_blocks(raw(old), pairs), raw(new))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("layers,hkv,bs,d", [(1, 1, 16, 128), (3, 8, 16, 128), (2, 5, 48, 128),
                                             (1, 3, 256, 128), (5, 2, 32, 128)])
@pytest.mark.parametrize("n", [1, 2, 7, 40])
def test_copies(layers, hkv, bs, d, kv, n):
    nb = 2 * n + 3
    perm = np.random.default_rng(n).permutation(nb)
    pairs = np.stack([perm[:n], perm[n:2 * n]], 1)
    check(*run(layers, nb, hkv, bs, d, pairs, kv, seed=n), pairs)
    assert_status_clean()


def test_head_dim_64_and_the_smallest_block():
    pairs = [(0, 2), (3, 1)]
    check(*run(2, 4, 1, 16, 64, pairs), pairs)
    assert_status_clean()


def test_one_block_to_many_and_padding():
    pairs = [(5, 0), (5, 1), (-1, 3), (5, 2), (4, -7), (6, 6), (-1, -1), (7, 9)]
    check(*run(2, 10, 2, 16, 128, pairs), pairs)
    assert_status_clean()


@pytest.mark.parametrize("layers", [63, 64, 65, 130])
def test_more_layers_than_one_launch_takes(layers):
    pairs = [(0, 4), (1, 3)]
    check(*run(layers, 5, 1, 16, 64, pairs), pairs)
    assert_status_clean()


def test_ids_past_the_pool_are_skipped_and_flagged():
    pairs = [(0, 4), (5, 1), (1, 5), (2**31 - 1, 3), (2, 3)]
    got = run(2, 5, 2, 16, 128, pairs)
    assert pk.read_device_status() == pk.PA_DEV_BAD_BLOCK
    check(*got, [(0, 4), (2, 3)])


def test_stream_and_graph_with_other_pairs():
    pairs = [(0, 4), (1, 5), (-1, -1)]
    side = torch.cuda.Stream()
    check(*run(2, 6, 2, 16, 128, pairs, stream=side), pairs)
    ks, vs = pools(2, 6, 2, 16, 128)
    kd, vd = [x.to(DEV) for x in ks], [x.to(DEV) for x in vs]
    p = torch.tensor(pairs, dtype=torch.int32, device=DEV)
    layers = pk.kv_layers(kd, vd)
    pk.pa_copy_blocks(layers, p)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.pa_copy_blocks(layers, p)
    for new, old in zip(kd + vd, ks + vs):
        new.copy_(old)
    other = [(3, 0), (-1, -1), (3, 1)]
    p.copy_(torch.tensor(other, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    check(ks, vs, kd, vd, other)


def test_offsets_past_32_bits():
    """Blocks beyond the first 4 GiB of a cache array."""
    nb = (1 << 32) // (8 * 256 * 128 * 2) + 9   # 8193 + 8 blocks of 512 KiB
    k = torch.zeros((nb, 8, 256, 128), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    k[3], v[3] = 3.0, -3.0
    k[nb - 2], v[nb - 2] = 5.0, -5.0
    p = torch.tensor([(3, nb - 1), (nb - 2, 0)], dtype=torch.int32, device=DEV)
    pk.pa_copy_blocks(pk.kv_layers([k], [v]), p)
    torch.cuda.synchronize()
    want = {0: 5.0, 3: 3.0, nb - 2: 5.0, nb - 1: 3.0}
    for b in (0, 1, 2, 3, 4, nb - 3, nb - 2, nb - 1):
        assert torch.all(k[b] == want.get(b, 0.0)) and torch.all(v[b] == -want.get(b, 0.0))
    assert_status_clean()


def test_binding_takes_plain_calls_and_leaves_the_others():
    dev = torch.device("cuda:0")
    k, v = (torch.randn(6, 2, 16, 64, device=dev).to(torch.bfloat16) for _ in "kv")
    layers = pk.kv_layers([k], [v])
    pairs = torch.tensor([[0, 3], [1, 4], [-1, -1]], dtype=torch.int32, device=dev)
    call = pk._load_direct().copy_blocks
    good = [layers.address, 1, layers.device, pairs, None]
    assert call(*good) == 0
    torch.cuda.synchronize()
    assert torch.equal(k[3], k[0]) and torch.equal(v[4], v[1])
    before = pk.lib().pa_kernel_launches()
    wrong = {0: [None, 1.5], 1: [0, None], 2: [-1, 99], 4: [3],
             3: [pairs.long(), pairs.cpu(), pairs[0], pairs.t(), pairs[:, :1], None]}
    for i, values in wrong.items():
        for x in values:
            assert call(*good[:i], x, *good[i + 1:]) == -1, (i, x)
    assert call() == -1
    assert pk.lib().pa_kernel_launches() == before
    pk.pa_copy_blocks(layers, pairs[:0])  # nothing to copy
    torch.cuda.synchronize()
