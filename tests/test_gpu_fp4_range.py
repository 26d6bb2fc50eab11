"""decode_attn_fp4 where row scales lie further apart than a 32-bit exponent
reaches.  Against the exact softmax in 64 bits over the same cells."""
import pytest
import torch

from tests.chunk_reference import assert_rows
from tests.fp4_reference import pools4
from tests.test_gpu_fp4 import (BF16, cache, least_weights, pkg, reference, run,  # noqa: F401
                                weight)

pytestmark = pytest.mark.gpu


def at(d, L):
    """(page, slot) of the first sequence's positions."""
    PS = d["cache"][0].shape[1]
    pos = torch.arange(L)
    return d["table"][0, pos // PS].long(), pos % PS


SPLITS = [dict(split_min=10000), dict(force_chunk=128, schedule=1),
          dict(force_chunk=128, schedule=2)]
# positions whose V rows are the large ones: of 700, in shards of 128 and units of 32
LARGE = {"last half": lambda t: t >= 350, "first half": lambda t: t < 350,
         "odd units": lambda t: t // 32 % 2 == 1, "two warps": lambda t: t // 32 % 4 >= 2,
         "last unit of a warp": lambda t: t // 32 >= 20, "odd positions": lambda t: t % 2 == 1,
         "first shard": lambda t: t < 128}


@pytest.mark.parametrize("kw", SPLITS, ids=["one", "grid", "cluster"])
@pytest.mark.parametrize("large", list(LARGE))
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (8, 1, 64), (16, 1, 128), (8, 2, 256)])
def test_fp4_v_scales_far_apart(pkg, Hq, Hkv, D, large, kw):  # noqa: F811
    """Zero V rows, or rows of 2^-110, beside rows of 2^40 to 2^110: every row has its
    share of the sum, in whichever order they come."""
    L = 700
    for exponent, small in ((50, 0.0), (90, 0.0), (120, 0.0), (120, 2.0 ** -100)):
        d = cache(900, [L], 1, Hq=Hq, Hkv=Hkv, D=D, PS=16, dtype=BF16, loud=False)
        page, slot = at(d, L)
        factor = torch.where(LARGE[large](torch.arange(L)), 2.0 ** exponent, small)
        d["cache"][3][page, :, slot] *= factor[:, None]
        assert torch.isfinite(pools4(d["cache"])[1]).all()
        got, err = run(pkg, d, 1, **kw)
        assert err == 0
        ref, mass = reference(d)
        # scores and references below 256 in magnitude: their difference is off by half
        # a step of that, 2^-17, where a weight is taken and where it is carried on
        w = weight(d) + 2.0 ** -16
        assert_rows(got, ref, mass + least_weights(d) / (2 * w), BF16, w, exponent)


@pytest.mark.parametrize("T,Hq,Hkv,D,window", [(1, 8, 2, 128, 0), (2, 8, 2, 64, 0),
                                               (3, 4, 2, 128, 0), (3, 5, 1, 128, 300)])
def test_fp4_v_scales_far_apart_in_large_steps(pkg, T, Hq, Hkv, D, window):  # noqa: F811
    """The same with two KV heads per CTA and with several tokens: zero rows and rows of
    2^60 to 2^110 mixed over positions and heads."""
    cap = 131072 // 16 * 8
    d = cache(901, [900, 1, 0, 77, 2300, 64], T, Hq=Hq, Hkv=Hkv, D=D, PS=16, dtype=BF16,
              max_pages=cap, loud=False)
    if Hkv == 2:
        p = pkg.DecodeAttnParams(6, Hq, Hkv, D, 16, cap, d["cache"][0].shape[0], 0, 1.0, window,
                                 0, 0, 0, T, 1, 0)
        plan = pkg.decode_attn_fp4_make_plan(p, 152)
        assert (plan.grid_x if plan.head_fastest else plan.grid_y) == 1
    g = torch.Generator().manual_seed(902)
    shape = d["cache"][3].shape
    kinds = torch.tensor([0.0, 0.0, 2.0 ** 70, 2.0 ** 120])
    for per_page in (False, True):  # rows of one page alike, or each its own
        n = shape[:2] + (1,) if per_page else shape
        e = dict(d, cache=list(d["cache"]))
        e["cache"][3] = d["cache"][3] * kinds[torch.randint(0, 4, n, generator=g)]
        ref, mass = reference(e, window)
        w = weight(e) + 2.0 ** -16
        for kw in ({}, dict(force_chunk=256, schedule=1)):
            got, err = run(pkg, e, T, window, **kw)
            assert err == 0
            assert_rows(got, ref, mass + least_weights(e, window) / (2 * w), BF16, w)
