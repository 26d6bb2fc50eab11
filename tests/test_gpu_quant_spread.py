"""decode_attn_quant where row scales lie further apart than a 32-bit exponent
reaches.  Against the exact softmax in 64 bits over the same codes and scales."""
import pytest
import torch

from tests.chunk_reference import chunk_attention, ragged, weight_error
from tests.test_gpu_quant import BF16, cache, pkg, run, weight  # noqa: F401
from tests.test_gpu_quant_range import assert_close, exact, pool

pytestmark = pytest.mark.gpu

SPLITS = [dict(split_min=10000), dict(force_chunk=128, schedule=1),
          dict(force_chunk=128, schedule=2)]
LARGE = {"last half": lambda t: t >= 350, "first half": lambda t: t < 350,
         "odd halves of a stage": lambda t: t // 32 % 2 == 1,
         "some warps": lambda t: t // 32 % 6 >= 3, "odd positions": lambda t: t % 2 == 1,
         "first shard": lambda t: t < 128}


@pytest.mark.parametrize("kw", SPLITS, ids=["one", "grid", "cluster"])
@pytest.mark.parametrize("large", list(LARGE))
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (8, 1, 64), (16, 1, 128), (8, 2, 256)])
def test_v_scales_far_apart(pkg, Hq, Hkv, D, large, kw):  # noqa: F811
    """Zero V rows, or rows of 2^-110, beside rows of 2^40 to 2^110: every row has its
    share of the sum, in whichever order they come."""
    L = 700
    g = torch.Generator().manual_seed(551)
    k, v = (torch.randn((L, Hkv, D), generator=g) for _ in range(2))
    w, q, off = ragged(550, [L], [1], Hq=Hq, Hkv=Hkv, D=D, PS=16, dtype=BF16)
    for exponent, small in ((50, 0.0), (90, 0.0), (118, 0.0), (118, 2.0 ** -100)):
        factor = torch.where(LARGE[large](torch.arange(L)), 2.0 ** exponent, small)
        d = pool(w, k, v, q, off)
        page, slot = w.page_table[0, torch.arange(L) // 16].long(), torch.arange(L) % 16
        d["v_scales"][page, :, slot] *= factor[:, None]
        got, err = run(pkg, d, 1, scale=0.05, **kw)
        assert err == 0
        ref, mass = exact(d, 0.05)
        size = 0.05 * float(q.double().norm(dim=-1).max()) * \
            float(k.double().norm(dim=-1).max() * 1.07)  # codes within 2^-4 of the value
        # scores and references below 256 in magnitude: their difference is off by half
        # a step of that, 2^-17, where a weight is taken and where it is carried on
        assert_close(got, ref, mass, BF16, weight_error(D, size) + 2.0 ** -21 + 2.0 ** -16, 0.0)


@pytest.mark.parametrize("T,Hq,Hkv,D,window", [(1, 8, 2, 128, 0), (2, 8, 2, 64, 0),
                                               (3, 5, 1, 128, 300)])
def test_v_scales_far_apart_in_large_steps(pkg, T, Hq, Hkv, D, window):  # noqa: F811
    """The same over a table long enough for two KV heads per CTA, and with several
    tokens: zero rows and rows of 2^60 to 2^110 mixed over positions and heads."""
    d = cache(552, [900, 1, 0, 77, 2300, 64], T, Hq=Hq, Hkv=Hkv, D=D, PS=16, dtype=BF16,
              max_pages=16384, loud=False)
    g = torch.Generator().manual_seed(553)
    kinds = torch.tensor([0.0, 0.0, 2.0 ** 70, 2.0 ** 118])
    for per_page in (False, True):  # rows of one page alike, or each its own
        n = d["v_scales"].shape[:2] + (1,) if per_page else d["v_scales"].shape
        e = dict(d, v_scales=d["v_scales"] * kinds[torch.randint(0, 4, n, generator=g)])
        ref, mass = chunk_attention(e["q"], e["k_pages"], e["v_pages"], e["table"], e["off"],
                                    e["lens"], e["scale"], window, e["k_scales"], e["v_scales"])
        for kw in ({}, dict(force_chunk=256, schedule=1)):
            got, err = run(pkg, e, T, window, **kw)
            assert err == 0
            assert_close(got, ref, mass, BF16, weight(e) + 2.0 ** -16, 0.0)
