"""decode_attn_chunk where numbers of very different sizes meet: weights far
below the first tile's largest, values near the top of bf16 under rising
scores.  Against the exact softmax in 64 bits."""
import math

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


@pytest.mark.parametrize("force", [1 << 20, 0, 16384], ids=["one", "auto", "eight"])
@pytest.mark.parametrize("D,nats,dtype", [(64, 17.5, F16), (128, 17.0, F16), (128, 17.5, F16),
                                          (256, 17.5, F16), (128, 17.5, BF16)])
def test_a_context_far_below_its_first_token(pkg, D, nats, dtype, force):  # noqa: F811
    """A first token that draws the attention (e^nats over the others) and has no
    value of its own: the output is the small weights' alone."""
    L, n = 131072, 3
    w, _, off = ragged(600, [L], [n], Hq=4, Hkv=1, D=D, PS=64, dtype=dtype)
    g = torch.Generator().manual_seed(601)
    k = torch.randn((L, 1, D), generator=g) * 0.02
    v = torch.randn((L, 1, D), generator=g).abs() + 0.25
    k[0], v[0] = 1.5, 0.0
    put(w, k, v)
    q, scale = torch.ones((n, 4, D), dtype=dtype), nats / (1.5 * D)
    got, err = run(pkg, w, q, off, scale=scale, max_seq_len=L, force_chunk=force)
    assert err == 0
    ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, [L], scale)
    # weights rounded to the type while they are normal numbers: e^-17.5 is
    # 2^-25.25 (2^-25.6 with the others' spread), 2^-13.6 in the first tile,
    # where the largest is 2^12, and near the largest in the others; sum |q k|
    # is the first token's score, all of one sign
    assert_close(got, ref, mass, dtype, half_step(dtype) + weight_error(D, nats))


@pytest.mark.parametrize("force", [1 << 20, 1024], ids=["one", "shards"])
@pytest.mark.parametrize("nats", [21.0, 26.0, 31.0])
@pytest.mark.parametrize("D", [128, 256])
def test_a_context_below_every_fp16_number(pkg, D, nats, force):  # noqa: F811
    """Weights that fp16 could not hold beside the first token's: those of the
    other tiles count in full, those of the first token's own tile are lost
    below 2^-25 where its weight is 2^12.  Values that keep the result in fp16."""
    L = 8192
    w, _, off = ragged(602, [L], [1], Hq=4, Hkv=1, D=D, PS=64)
    g = torch.Generator().manual_seed(603)
    k = torch.randn((L, 1, D), generator=g) * 0.02
    v = ((torch.randn((L, 1, D), generator=g).abs() + 0.25) * 15000.0).clamp(max=60000.0)
    k[0], v[0] = 1.5, 0.0
    put(w, k, v)
    q, scale = torch.ones((1, 4, D)).half(), nats / (1.5 * D)
    got, err = run(pkg, w, q, off, scale=scale, max_seq_len=L, force_chunk=force)
    assert err == 0
    ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, [L], scale)
    tile = v.double()[1:128 if D == 128 else 64].sum(0)[0]
    own = tile * min(2.0 ** -37, 1.2 * math.exp(-nats))
    assert_close(got, ref, mass, F16, half_step(F16) + weight_error(D, nats), own)


@pytest.mark.parametrize("place", [0, 700, 4095])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_large_weight_between_small_ones(pkg, D, place):  # noqa: F811
    """A token that draws the attention at the start, inside or at the end of
    the context, 25 nats over the rest and without a value of its own; the
    values are large enough for fp16 to hold the result."""
    L, nats = 4096, 25.0
    w, _, off = ragged(604, [L], [1], Hq=4, Hkv=1, D=D, PS=32)
    g = torch.Generator().manual_seed(605)
    k = torch.randn((L, 1, D), generator=g) * 0.02
    v = (torch.randn((L, 1, D), generator=g).abs() + 0.25) * 8192.0
    v = v.clamp(max=60000.0)
    k[place], v[place] = 1.5, 0.0
    put(w, k, v)
    q, scale = torch.ones((1, 4, D)).half(), nats / (1.5 * D)
    got, err = run(pkg, w, q, off, scale=scale, max_seq_len=L, force_chunk=1 << 20)
    assert err == 0
    ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, [L], scale)
    # e^-25 is 2^-36.07: the tile of the large weight loses what is below 2^-25
    # where that weight is 2^12 (the first tile) or 2^2
    tile = 64 if D == 256 else 128
    first = place // tile * tile
    own = v.double()[first:first + tile].sum(0)[0]
    lost = own * min(2.0 ** -37 if first == 0 else 2.0 ** -27, 1.2 * math.exp(-nats))
    assert_close(got, ref, mass, F16, half_step(F16) + weight_error(D, nats), lost)


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


@pytest.mark.parametrize("exponent", [-60, -100, -112])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_bf16_values(pkg, D, exponent):  # noqa: F811
    """bf16 values far below fp16's: the first weights of 2^-16 must not take
    them out of the 32-bit accumulators."""
    L, n = 700, 30
    w, q, off = ragged(630, [L], [n], Hq=8, Hkv=2, D=D, PS=16, dtype=BF16)
    g = torch.Generator().manual_seed(631)
    k = torch.randn((L, 2, D), generator=g)
    v = (torch.randn((L, 2, D), generator=g).abs() + 0.5) * 2.0 ** exponent
    put(w, k, v)
    got, err = run(pkg, w, q, off)
    assert err == 0
    ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, [L], w.scale)
    size = w.scale * float(q.double().norm(dim=-1).max() * w.k_pages.double().norm(dim=-1).max())
    # (a 32-bit sum near 2^-128 has steps of 2^-149: 2^-21 of it)
    assert_close(got, ref, mass, BF16, half_step(BF16) + weight_error(D, size) + 2.0 ** -20)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gap", [40.0, 60.0, 120.0, 400.0])
def test_towering_keys_at_any_distance(pkg, D, gap, dtype):  # noqa: F811
    """Keys whose scores stand `gap` powers of two above all others, at two
    places: sums and accumulators stay finite however far the reference could
    follow the tiles between them."""
    L, n = 1400, 20
    w, _, off = ragged(640, [L], [n], Hq=4, Hkv=1, D=D, PS=16, dtype=dtype)
    g = torch.Generator().manual_seed(641)
    k = torch.randn((L, 1, D), generator=g) * 0.02
    v = torch.randn((L, 1, D), generator=g)
    k[5], k[700] = 1.0, 1.5
    put(w, k, v)
    q, scale = torch.ones((n, 4, D), dtype=dtype), gap * 0.6931 / D
    for force in (0, 1 << 20):
        got, err = run(pkg, w, q, off, scale=scale, force_chunk=force)
        assert err == 0
        ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, [L], scale)
        assert_close(got, ref, mass, dtype, half_step(dtype) + weight_error(D, gap * 1.1))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_bf16_values_behind_a_masked_tile(pkg, D):  # noqa: F811
    """Windows that leave a CTA's first tile to some of its rows only: the others
    take their reference in a later one."""
    L, n, window = 900, 130, 100
    w, q, off = ragged(650, [L], [n], Hq=2, Hkv=2, D=D, PS=16, dtype=BF16)
    g = torch.Generator().manual_seed(651)
    k = torch.randn((L, 2, D), generator=g)
    v = (torch.randn((L, 2, D), generator=g).abs() + 0.5) * 2.0 ** -112
    put(w, k, v)
    got, err = run(pkg, w, q, off, window)
    assert err == 0
    ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, [L], w.scale, window)
    size = w.scale * float(q.double().norm(dim=-1).max() * w.k_pages.double().norm(dim=-1).max())
    assert_close(got, ref, mass, BF16, half_step(BF16) + weight_error(D, size) + 2.0 ** -20)
