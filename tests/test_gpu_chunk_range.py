"""decode_attn_chunk where numbers of very different sizes meet: values near
the top of bf16 under rising scores, rows whose scores rise apart.  Against the exact softmax in 64 bits."""
import pytest
import torch

from tests.chunk_reference import chunk_attention, half_step, ragged, weight_error
from tests.test_gpu_chunk import BF16, DEV, F16, pkg, run  # noqa: F401

pytestmark = pytest.mark.gpu


def put(w, k, v):
    """K and V rows [L, Hkv, D] into the pages of the one sequence."""
    PS = w.k_pages.shape[1]
    pos = torch.arange(k.shape[0])
    page, slot = w.page_table[0, pos // PS].long(), pos % PS
    w.k_pages[page, slot], w.v_pages[page, slot] = k.to(w.k_pages.dtype), v.to(w.v_pages.dtype)


def assert_close(got, ref, mass, dtype, weight, floor=0.0):
    """chunk_reference.assert_rows with an absolute error of the sums beside."""
    g, u = got.double().cpu(), half_step(dtype)
    tol = 2 * weight * mass + floor + (u + 2.0 ** -22) * ref.abs() + \
        torch.finfo(dtype).smallest_normal * u
    assert torch.isfinite(g).all()
    over = (g - ref).abs() - tol
    assert float(over.max()) <= 0, (float(over.max()), float((g - ref).abs().max()))


@pytest.mark.parametrize("force", [0, 384])
@pytest.mark.parametrize("rise", [5.0, 27.0, 40.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_values_under_rising_scores(pkg, D, rise, force):  # noqa: F811
    """bf16 values of 2^110 and scores that rise by `rise` nats after the first
    tiles: the weights must not grow with them."""
    L, n = 900, 40
    w, _, off = ragged(610, [L], [n], Hq=8, Hkv=2, D=D, PS=16, dtype=BF16)
    g = torch.Generator().manual_seed(611)
    k = torch.randn((L, 2, D), generator=g) * 0.02
    v = torch.randn((L, 2, D), generator=g) * 2.0 ** 110
    steps = torch.clamp((torch.arange(L) - 200) / 500.0, 0.0, 1.0)
    k += steps[:, None, None]
    put(w, k, v)
    q, scale = torch.ones((n, 8, D), dtype=BF16), rise / D
    got, err = run(pkg, w, q, off, scale=scale, force_chunk=force)
    assert err == 0
    ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, [L], scale)
    assert_close(got, ref, mass, BF16, half_step(BF16) + weight_error(D, rise * 1.1))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("D", [128, 256])
def test_scores_that_rise_row_by_row(pkg, D, dtype):  # noqa: F811
    """Rows of one warp whose scores rise at different tiles and by different
    amounts, some by less than the reference allows, and fall again."""
    L, n = 1500, 64
    w, q, off = ragged(620, [L], [n], Hq=8, Hkv=2, D=D, PS=32, dtype=dtype)
    g = torch.Generator().manual_seed(621)
    k = torch.randn((L, 2, D), generator=g) * 0.3
    v = torch.randn((L, 2, D), generator=g)
    hot = torch.randint(0, L - n, (30,), generator=g)
    who = torch.randint(0, n, (30,), generator=g)
    for t, i in zip(hot.tolist(), who.tolist()):
        amount = float(torch.rand((), generator=g)) * 2.0
        k[t, 0] = q[i, 1].float() * amount
        k[t, 1] = q[i, 6].float() * amount
    put(w, k, v)
    for force in (0, 512):
        got, err = run(pkg, w, q, off, scale=0.1, force_chunk=force)
        assert err == 0
        ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, [L], 0.1)
        size = 0.1 * float(q.double().norm(dim=-1).max() * w.k_pages.double().norm(dim=-1).max())
        assert_close(got, ref, mass, dtype, half_step(dtype) + weight_error(D, size))
