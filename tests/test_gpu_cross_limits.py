"""pa_cross_attention at the longest encoder lengths that its tables can hold.

One block of ordinary keys stands in every table entry but the first, whose first key has a score
of 60 beside 2^30 scores of 0: e^60 > 2^86, so it takes all of the softmax (the others together
less than 2^-56) and the output is its value, exactly.  A row that does not see it gets 0."""
import pytest
import torch

import paged_kv_cache_284_gb300 as pk
from gpu_helpers import DEV, assert_status_clean

pytestmark = pytest.mark.gpu

LONGEST = 1 << 30


@pytest.mark.parametrize("d,kv,hq", [(64, "bf16", 1), (128, "e4m3", 4)])
@pytest.mark.parametrize("behind,tokens", [(0, 1), (0, 7), (3, 16), (LONGEST - 40000, 16)])
def test_first_key_at_the_longest_lengths(behind, tokens, d, kv, hq):
    """L = 2^30 - behind, for the last rows of a piece too."""
    bs, n = 256, LONGEST - behind
    width = -(-n // bs)
    table = torch.ones((1, width), dtype=torch.int32, device=DEV)
    table[0, 0] = 0
    k = torch.zeros((2, 1, bs, d), device=DEV)
    v = torch.zeros((2, 1, bs, d), device=DEV)
    k[0, 0, 0, 0], v[0, 0, 0] = 60, 3
    scales = {}
    if kv == "e4m3":   # (60 and 3 are codes)
        k, v = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        scales = {x: torch.ones(1, device=DEV) for x in ("k_scale", "v_scale")}
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    q = torch.zeros((tokens, hq, d), dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 8
    out = torch.full_like(q, 7)
    lse = torch.full((tokens, hq), 7.0, device=DEV)
    pk.pa_cross_attention(q, k, v, table, torch.tensor([0, tokens], dtype=torch.int32, device=DEV),
                          torch.tensor([n], dtype=torch.int32, device=DEV), 0.125, out, lse, **scales)
    torch.cuda.synchronize()
    assert torch.all(out == 3), out[:, 0, 0]
    assert torch.all((lse - 60).abs() <= 2.0 ** -13 + 60 * 2.0 ** -22), lse[:, 0]
    assert_status_clean()


def test_later_pieces_of_a_prompt_at_the_longest_lengths():
    """An e4m3 prompt without staging room runs in pieces of 64 rows: every piece's rows stand
    right behind the keys, however many pieces are before it."""
    d, bs, n, tokens = 128, 256, LONGEST - 150, 200
    table = torch.ones((1, LONGEST // bs), dtype=torch.int32, device=DEV)
    table[0, 0] = 0
    k, v = torch.zeros((2, 1, bs, d), device=DEV), torch.zeros((2, 1, bs, d), device=DEV)
    k[0, 0, 0, 0], v[0, 0, 0] = 60, 3
    k, v = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    q = torch.zeros((tokens, 1, d), dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 8
    out, one = torch.full_like(q, 7), torch.ones(1, device=DEV)
    pk.pa_cross_attention(q, k, v, table, torch.tensor([0, tokens], dtype=torch.int32, device=DEV),
                          torch.tensor([n], dtype=torch.int32, device=DEV), 0.125, out,
                          k_scale=one, v_scale=one)
    torch.cuda.synchronize()
    assert torch.all(out == 3), out[:, 0, 0]
    assert_status_clean()
