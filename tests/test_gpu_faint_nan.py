"""A NaN among V rows whose weight is far below the others': the steps over the 4-bit
and the 8-bit cache, in one shard and in several."""
import math

import pytest
import torch

from tests.chunk_reference import chunk_attention, ragged
from tests.test_gpu_fp4 import F16, cache, pkg, reference  # noqa: F401
from tests.test_gpu_fp4 import run as run_fp4
from tests.test_gpu_quant import run
from tests.test_gpu_quant_range import pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["block", "row"])
@pytest.mark.parametrize("kw", [dict(split_min=10000), dict(force_chunk=64, schedule=1),
                                dict(force_chunk=64, schedule=2)], ids=["one", "grid", "cluster"])
@pytest.mark.parametrize("Hq,D", [(4, 64), (8, 128), (16, 128), (4, 256)])
def test_fp4_a_nan_far_below_the_others(pkg, Hq, D, kw, what):  # noqa: F811
    """A unit of positions 200 nats below the others with a NaN among its V rows: a
    weight is above zero, however small, so the rows that attend it are NaN there."""
    L = 256
    for t in (5, 40, 70, 127, 130, 255):
        d = cache(901, [L], 1, Hq=Hq, Hkv=1, D=D, PS=32, dtype=F16, loud=False)
        pos = torch.arange(L)
        page, slot = d["table"][0, pos // 32].long(), pos % 32
        # keys of ones: the scores are the row scales
        d["cache"][0].fill_(0x22)
        d["cache"][4].view(torch.uint8).fill_(0x38)
        d["cache"][2].zero_()
        unit = pos // 32 == t // 32
        d["cache"][2][page, :, slot] = torch.where(unit, -200.0, 0.0)[:, None]
        d["q"].fill_(1.0)
        clean, _ = reference(d, scale=1.0 / D)
        if what == "block":
            d["cache"][5].view(torch.uint8)[page[t], 0, slot[t], 2] = 0x7f
        else:
            d["cache"][3][page[t], 0, slot[t]] = math.nan
        got, err = run_fp4(pkg, d, 1, scale=1.0 / D, **kw)
        assert err == 0
        hit = torch.zeros(got.shape, dtype=torch.bool)
        hit[..., 32:48] = True
        if what == "row":
            hit[:] = True
        got = got.double().cpu()
        assert torch.equal(torch.isnan(got), hit), t
        near = (got - clean).abs()[~hit] <= 2.0 ** -10 * clean.abs().max()
        assert bool(near.all()), t


@pytest.mark.parametrize("kw", [dict(split_min=10000), dict(force_chunk=64, schedule=1),
                                dict(force_chunk=64, schedule=2)], ids=["one", "grid", "cluster"])
@pytest.mark.parametrize("Hq,D", [(4, 64), (8, 128), (16, 128), (4, 256)])
def test_a_nan_far_below_the_others(pkg, Hq, D, kw):  # noqa: F811
    """A block of positions 200 nats below the others with a NaN code in one of its V
    rows: a weight is above zero, however small, so that dim of the output is NaN."""
    L = 256
    g = torch.Generator().manual_seed(561)
    w, q, off = ragged(560, [L], [1], Hq=Hq, Hkv=1, D=D, PS=32, dtype=F16)
    q.fill_(1.0)
    v = torch.randn((L, 1, D), generator=g)
    for t in (5, 40, 70, 127, 130, 255):
        unit = torch.arange(L) // 32 == t // 32
        k = torch.where(unit, -200.0, 0.0)[:, None, None].expand(L, 1, D)
        d = pool(w, k, v, q, off)
        clean, _ = chunk_attention(q, d["k_pages"], d["v_pages"], d["table"], off, d["lens"],
                                   1.0 / D, 0, d["k_scales"], d["v_scales"])
        page, slot = int(w.page_table[0, t // 32]), t % 32
        d["v_pages"].view(torch.uint8)[page, slot, 0, 33] = 0x7f
        got, err = run(pkg, d, 1, scale=1.0 / D, **kw)
        assert err == 0
        got = got.double().cpu()
        hit = torch.zeros(got.shape, dtype=torch.bool)
        hit[..., 33] = True
        assert torch.equal(torch.isnan(got), hit), t
        near = (got - clean).abs()[~hit] <= 2.0 ** -10 * clean.abs().max()
        assert bool(near.all()), t
