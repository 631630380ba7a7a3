"""The attention sublayer's operators at the edges of what they take."""
import math

import pytest
import torch

from test_attention_ops import BF, F32, paged_inputs
from transformer_depth_wise_gb300 import api

gpu_only = pytest.mark.gpu


# --------------------------------------------------------------------------
# paged attention
# --------------------------------------------------------------------------
# one tile of 64 tokens (written by the CTA that has it), pairs cut into a tile per CTA, pairs of many tiles per CTA
PAGED_NAN = [(5, 64), (0, 5, 777), (40000,), (300, 20000, 1)]


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lengths", PAGED_NAN)
def test_paged_nan_query(gpu, dtype, lengths):
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, len(lengths), 8, 2, 128, 16, list(lengths), sum(lengths))
    want, wlse = api.paged_attention(q, kc, vc, table, n, scale)
    q[:, 3, 17] = math.nan
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    some = n > 0
    assert bool(out[some, 3].isnan().all()) and bool(lse[some, 3].isnan().all())
    assert bool((out[~some] == 0).all()) and bool((lse[~some] == -math.inf).all())
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(out[:, keep], want[:, keep]) and torch.equal(lse[:, keep], wlse[:, keep])


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("length,first,last", [(777, 64, 128), (777, 0, 64), (40000, 12800, 13312), (40000, 39999, 40000)])
def test_paged_nan_keys(gpu, dtype, length, first, last):
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, 1, 8, 2, 128, 16, [length], length)
    want, wlse = api.paged_attention(q, kc, vc, table, n, scale)
    for j in range(first, last):
        kc[int(table[0, j // 16]), 1, j % 16] = math.nan
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    assert bool(out[0, 4:].isnan().all()) and bool(lse[0, 4:].isnan().all())
    assert torch.equal(out[0, :4], want[0, :4]) and torch.equal(lse[0, :4], wlse[0, :4])


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("length,at", [(5, 4), (777, 300), (40000, 12803)])
def test_paged_nan_values(gpu, dtype, length, at):
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, 1, 8, 2, 128, 16, [length], length)
    want, wlse = api.paged_attention(q, kc, vc, table, n, scale)
    vc[int(table[0, at // 16]), 0, at % 16, 9] = math.nan
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    hit = torch.zeros(8, 128, dtype=torch.bool, device=gpu)
    hit[:4, 9] = True
    assert torch.equal(lse, wlse) and bool(out[0][hit].isnan().all()) and torch.equal(out[0][~hit], want[0][~hit])
