"""decode_attn_fp4 with two KV heads per CTA and a window, which a large step takes:
against the exact softmax, and a NaN among several tokens."""
import pytest
import torch

from tests.chunk_reference import assert_rows
from tests.test_gpu_fp4 import (BF16, F16, cache, least_weights, pkg, reference,  # noqa: F401
                                run, weight)

pytestmark = pytest.mark.gpu

LENS = [2600, 1, 0, 900, 2461, 64]
TIMES = 8


def many(d, T):
    """The sequences TIMES times over."""
    return dict(d, q=d["q"].repeat(TIMES, 1, 1), table=d["table"].repeat(TIMES, 1),
                lens=d["lens"].repeat(TIMES))


def heads_of(pkg, d, T, window):
    B, Hq, D = len(d["lens"]), d["q"].shape[1], d["q"].shape[2]
    P, PS, Hkv, _ = d["cache"][0].shape
    p = pkg.DecodeAttnParams(B, Hq, Hkv, D, PS, d["table"].shape[1], P, max(LENS), 1.0, window, 0,
                             0, 0, T, 1 if d["q"].dtype is BF16 else 0, 0)
    plan = pkg.decode_attn_fp4_make_plan(p, 152)
    return plan.grid_x if plan.head_fastest else plan.grid_y


@pytest.mark.parametrize("T,Hq,Hkv,D,PS,window,dtype", [
    (1, 8, 4, 64, 16, 2200, F16), (1, 16, 4, 128, 32, 2200, BF16), (3, 4, 2, 128, 16, 2300, F16),
    (2, 16, 4, 64, 8, 2301, BF16), (1, 12, 6, 128, 256, 2000, F16),
])
def test_fp4_two_heads_per_cta_with_a_window(pkg, T, Hq, Hkv, D, PS, window, dtype):  # noqa: F811
    d = cache(910, LENS, T, Hq=Hq, Hkv=Hkv, D=D, PS=PS, dtype=dtype)
    ref, mass = reference(d, window)
    w, n = weight(d), len(LENS) * T
    mass = mass + least_weights(d, window) / (2 * w)
    d = many(d, T)
    assert heads_of(pkg, d, T, window) == Hkv // 2
    for kw in ({}, dict(force_chunk=256, schedule=1)):
        got, err = run(pkg, d, T, window, max_seq_len=max(LENS), **kw)
        assert err == 0
        for k in range(TIMES):
            assert torch.equal(got[k * n:(k + 1) * n], got[:n])
        assert_rows(got[:n], ref, mass, dtype, w)


@pytest.mark.parametrize("T,Hq,Hkv,D,window", [(3, 4, 2, 128, 2300), (3, 8, 4, 64, 0),
                                               (2, 8, 4, 128, 2300)])
def test_fp4_a_nan_with_two_heads_per_cta(pkg, T, Hq, Hkv, D, window):  # noqa: F811
    """A NaN among the V blocks of the second head of a CTA, at the window's edge and at
    the last positions: the rows of that head that attend it, in its 16 dims."""
    PS, G, L = 16, Hq // Hkv, LENS[0]
    n = len(LENS) * T
    first = L - T - window if window else 0  # before every row's window, then inside
    spots = [first, first + 1, first + 2, first + T, 1300, L - 3, L - 2, L - 1]
    for t in spots:
        d = cache(911, LENS, T, Hq=Hq, Hkv=Hkv, D=D, PS=PS, dtype=F16)
        clean, _ = reference(d, window)
        page, slot = int(d["table"][0, t // PS]), t % PS
        h, blk = 1, D // 16 - 2
        d["cache"][5].view(torch.uint8)[page, h, slot, blk] = 0xff
        d = many(d, T)
        assert heads_of(pkg, d, T, window) == Hkv // 2
        got, err = run(pkg, d, T, window, max_seq_len=max(LENS))
        assert err == 0
        got = got[(TIMES - 1) * n:].double().cpu()
        hit = torch.zeros(got.shape, dtype=torch.bool)
        for i in range(T):
            p = L - T + i
            if t <= p and (window == 0 or t > p - window):
                hit[i, h * G:(h + 1) * G, 16 * blk:16 * blk + 16] = True
        assert torch.equal(torch.isnan(got), hit), t
        near = (got - clean).abs()[~hit] <= 0.02 * clean.abs().max()
        assert bool(near.all()), t
