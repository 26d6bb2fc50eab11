"""decode_attn_quant with several new tokens per sequence: what a token does not
attend never reaches its rows, though another token of the step attends it."""
import pytest
import torch

from tests.test_gpu_quant import BF16, DEV, F16, cache, check, pkg, run  # noqa: F401

pytestmark = pytest.mark.gpu

KW = [{}, dict(force_chunk=128, schedule=1), dict(force_chunk=128, schedule=2)]


@pytest.mark.parametrize("kw", KW, ids=["auto", "grid", "cluster"])
@pytest.mark.parametrize("T,Hq,Hkv,D,PS,window", [
    (2, 8, 2, 128, 16, 0), (3, 8, 2, 64, 32, 0), (4, 8, 2, 128, 16, 0), (5, 3, 1, 256, 8, 0),
    (3, 8, 2, 128, 16, 100), (2, 4, 1, 64, 64, 70),
])
def test_a_nan_reaches_the_tokens_that_attend_it(pkg, T, Hq, Hkv, D, PS, window, kw):  # noqa: F811
    """NaN codes in V of the last tokens, and of the first positions that only
    the first tokens' windows hold; a NaN in K too."""
    lens = [333, 290, T]
    d = cache(480 + T + D, lens, T, Hq=Hq, Hkv=Hkv, D=D, PS=PS, dtype=F16)
    clean, err = run(pkg, d, T, window, **kw)
    assert err == 0
    bad = {0: [332, 331] if T > 2 else [332], 1: [290 - T + 1], 2: [T - 1]}
    if window:
        bad[0].append(333 - T + 1 - window)  # the first token's first position
    for b, ts in bad.items():
        for n, t in enumerate(ts):
            page, slot = int(d["table"][b, t // PS]), t % PS
            d["v_pages"].view(torch.uint8)[page, slot, 0, 5 + n] = 0x7f
            d["v_pages"].view(torch.uint8)[page, slot, Hkv - 1, D - 1 - n] = 0xff
    got, err = run(pkg, d, T, window, **kw)
    assert err == 0
    G = Hq // Hkv
    want = clean.clone()
    for b, ts in bad.items():
        for i in range(T):
            p = lens[b] - T + i
            for n, t in enumerate(ts):
                if t <= p and (not window or t > p - window):
                    want[b * T + i, :G, 5 + n] = float("nan")
                    want[b * T + i, (Hkv - 1) * G:, D - 1 - n] = float("nan")
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0))
    # K of a token: the rows that attend it, whole
    page, slot = int(d["table"][0, 332 // PS]), 332 % PS
    d["k_pages"].view(torch.uint8)[page, slot, 0, 0] = 0x7f
    again, err = run(pkg, d, T, window, **kw)
    assert err == 0 and torch.isnan(again[T - 1, :G]).all()
    keep = torch.ones(got.shape[0], dtype=torch.bool)
    keep[T - 1] = False
    assert torch.equal(torch.nan_to_num(again[keep], nan=9.0), torch.nan_to_num(got[keep], nan=9.0))


@pytest.mark.parametrize("T", [2, 3])
def test_an_inf_reaches_the_tokens_that_attend_it(pkg, T):  # noqa: F811
    """A scale of 2^120 (an Inf was appended) on the last token's V row."""
    d = cache(490 + T, [333], T, Hq=8, Hkv=2, D=128, PS=16, dtype=BF16)
    clean, err = run(pkg, d, T)
    page, slot = int(d["table"][0, 332 // 16]), 332 % 16
    d["v_scales"][page, 1, slot] = 2.0 ** 120
    codes = torch.zeros(128, dtype=torch.uint8)
    codes[9] = 0x7e  # 448
    d["v_pages"].view(torch.uint8)[page, slot, 1] = codes
    got, err = run(pkg, d, T)
    assert err == 0 and torch.equal(got[:T - 1], clean[:T - 1])
    assert torch.equal(got[T - 1, :4], clean[T - 1, :4])
    assert torch.isinf(got[T - 1, 4:, 9]).all()
    rest = [x for x in range(128) if x != 9]
    assert torch.isfinite(got[T - 1, 4:][:, rest]).all()


@pytest.mark.parametrize("T,Hq,Hkv,D,PS,window", [
    (1, 8, 2, 64, 16, 40000), (3, 4, 2, 128, 16, 20000), (1, 6, 2, 256, 8, 10000),
    (2, 8, 2, 64, 8, 33333),
])
def test_two_heads_per_cta_with_a_window(pkg, T, Hq, Hkv, D, PS, window):  # noqa: F811
    """Windows long enough that the plan takes two KV heads per CTA, over short
    sequences (inside the window) and one that it cuts inside a tile."""
    cap = 65536 // PS
    lens = [900, 1, 0, 77, window + 555, 64, 301, 12]
    d = cache(500 + D, lens, T, Hq=Hq, Hkv=Hkv, D=D, PS=PS, dtype=F16, max_pages=cap)
    for kw in ({}, dict(force_chunk=4096)):
        p = pkg.DecodeAttnParams(len(lens), Hq, Hkv, D, PS, cap, d["k_pages"].shape[0], 0, 1.0,
                                 window, 0, 0, kw.get("force_chunk", 0), T, 0, 0)
        plan = pkg.decode_attn_quant_make_plan(p, 152)
        assert (plan.grid_x if plan.head_fastest else plan.grid_y) == Hkv // 2
        check(pkg, d, T, window, **kw)
    bad = dict(d, table=d["table"].clone())
    bad["table"][4, 500 // PS] = -3  # before the window: nobody looks
    assert run(pkg, bad, T, window)[1] == 0
    bad["table"][4, (window + 500) // PS] = -3
    got, err = run(pkg, bad, T, window)
    assert err == pkg.DEV_BAD_PAGE and torch.all(got[4 * T:5 * T] == 0)
