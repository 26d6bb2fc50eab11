"""decode_attn_quant where numbers of very different sizes meet: weights far
below the largest, the largest V scales, q rows with an outlier.  Against the
exact softmax in 64 bits over the same codes and scales."""
import pytest
import torch

from tests.chunk_reference import chunk_attention, half_step, quantise, ragged, weight_error
from tests.test_gpu_quant import BF16, DEV, F16, pkg, run  # noqa: F401

pytestmark = pytest.mark.gpu


def pool(w, k, v, q, off):
    """The tests' dictionary from K and V rows [L, Hkv, D] of one sequence, in
    its pages (quantised; any 32-bit scale)."""
    d = dict(q=q, off=off, table=w.page_table, lens=w.seq_lens, scale=w.scale)
    P, PS = w.k_pages.shape[:2]
    pos = torch.arange(k.shape[0])
    page, slot = w.page_table[0, pos // PS].long(), pos % PS
    for n, x in (("k", k), ("v", v)):
        code, s = quantise(x)
        full = torch.zeros((P, PS, *x.shape[1:]), dtype=torch.uint8)
        full[page, slot] = code.view(torch.uint8)
        scales = torch.zeros((P, PS, x.shape[1]))
        scales[page, slot] = s
        d[n + "_pages"] = full.view(torch.float8_e4m3fn)
        d[n + "_scales"] = scales.transpose(1, 2).contiguous()
    return d


def exact(d, scale, window=0):
    return chunk_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["off"], d["lens"],
                           scale, window, d["k_scales"], d["v_scales"])


def assert_close(got, ref, mass, dtype, weight, floor):
    """chunk_reference.assert_rows with an absolute error of the sums beside."""
    g, u = got.double().cpu(), half_step(dtype)
    tol = 2 * weight * mass + floor + (u + 2.0 ** -22) * ref.abs() + \
        torch.finfo(dtype).smallest_normal * u
    assert torch.isfinite(g).all()
    over = (g - ref).abs() - tol
    assert float(over.max()) <= 0, (float(over.max()), float((g - ref).abs().max()))


SPLITS = [dict(force_chunk=65536), dict(schedule=1), dict(force_chunk=8192, schedule=2)]


@pytest.mark.parametrize("kw", SPLITS, ids=["one", "grid", "cluster"])
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, F16), (128, BF16), (256, F16)])
def test_small_weights_beside_a_large_one(pkg, D, dtype, kw):  # noqa: F811
    """A first token that draws the attention (17.5 nats over the others) and
    whose value lies in one dim: the other dims are the small weights' alone."""
    L, nats = 65536, 17.5
    w, _, off = ragged(500, [L], [1], Hq=4, Hkv=1, D=D, PS=64, dtype=dtype)
    g = torch.Generator().manual_seed(501)
    k = torch.randn((L, 1, D), generator=g) * 0.05
    v = torch.randn((L, 1, D), generator=g).abs()
    k[0], v[0] = 1.5, 0.0
    v[0, 0, 0] = 3.0
    d = pool(w, k, v, torch.ones((1, 4, D), dtype=dtype), off)
    scale = nats / (1.5 * D)
    got, err = run(pkg, d, 1, scale=scale, max_seq_len=L, **kw)
    assert err == 0
    ref, mass = exact(d, scale)
    # sum |q k| of a row is the first one's score, all of one sign; of a weight's
    # fp16 head and remainder 2^-25 may be lost where the largest is 2^14
    weight = weight_error(D, nats) + 2.0 ** -21
    floor = L * 2.0 ** -39 * 448 * float(d["v_scales"].max())
    assert_close(got, ref, mass, dtype, weight, floor)
    assert float(got.double()[:, :, 1:].min()) > 0.5 * float(ref[:, :, 1:].min())


@pytest.mark.parametrize("kw", [{}, dict(force_chunk=128, schedule=1),
                                dict(force_chunk=128, schedule=2)], ids=["auto", "grid", "cluster"])
@pytest.mark.parametrize("exponent", [99, 106, 112, 118])
def test_the_largest_v_scales(pkg, exponent, kw):  # noqa: F811
    """V rows near the top of bf16, all of them or one that few tokens attend:
    scales of 2^exponent, up to what the append writes for finite rows."""
    L, D = 600, 128
    w, q, off = ragged(510, [L], [1], Hq=8, Hkv=2, D=D, PS=16, dtype=BF16)
    g = torch.Generator().manual_seed(511)
    k, v = (torch.randn((L, 2, D), generator=g) for _ in range(2))
    for rows in (slice(None), slice(77, 78)):
        big = v.double().clone()
        top = big[rows].abs().amax(-1, keepdim=True)
        big[rows] = big[rows] / top * 440.0 * 2.0 ** exponent
        d = pool(w, k, big, q, off)
        assert float(d["v_scales"].max()) == 2.0 ** exponent
        got, err = run(pkg, d, 1, scale=0.05, **kw)
        assert err == 0
        ref, mass = exact(d, 0.05)
        size = 0.05 * float((q.double().abs().norm(dim=-1)).max()) * \
            float(k.double().norm(dim=-1).max() * 1.07)  # codes within 2^-4 of the value
        # every weight within 2^-20 of the largest is in the sum (2^-22 at 2^118)
        raw = 0.05 * 1.4427 * torch.einsum("hd,td->ht", q[0].double(), k.double()[:, 0])
        assert float(raw.max() - raw.min()) < 18
        # an exponent s + log2(vs) - m of numbers below 128 is off by half a
        # step of those, 2^-18, where it is taken and where m was
        assert_close(got, ref, mass, BF16, weight_error(D, size) + 2.0 ** -21 + 2.0 ** -17, 0.0)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("kw", [{}, dict(force_chunk=128, schedule=1),
                                dict(force_chunk=128, schedule=2)], ids=["auto", "grid", "cluster"])
def test_a_row_with_an_inf_stays_its_own(pkg, kw, D):  # noqa: F811
    """A V row with an Inf, appended (scale 2^120, code 448) and attended: that
    dim is Inf in the rows of its head; the other dims and the rows of other
    heads are the other tokens' values, to the tolerance of any other cache."""
    L, Hkv = 600, 2
    w, q, off = ragged(520, [L], [1], Hq=4, Hkv=Hkv, D=D, PS=16, dtype=BF16)
    g = torch.Generator().manual_seed(521)
    k, v = (torch.randn((L, Hkv, D), generator=g).bfloat16() for _ in range(2))
    v[50, 1, 7], v[599, 1, 7] = float("inf"), float("inf")
    v[300, 1, 30] = float("-inf")
    v[301, 0, 11], v[302, 0, 11] = float("inf"), float("-inf")
    P = w.k_pages.shape[0]
    codes = [torch.zeros((P, 16, Hkv, D), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    scales = [torch.zeros((P, Hkv, 16), device=DEV) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkg.decode_kv_append_chunk(k.to(DEV), v.to(DEV),
                               torch.tensor([0, L], dtype=torch.int32, device=DEV),
                               w.seq_lens.to(DEV), *codes, w.page_table.to(DEV), *scales,
                               err_flag=err)
    d = dict(q=q, off=off, table=w.page_table, lens=w.seq_lens, scale=w.scale,
             k_pages=codes[0].cpu(), v_pages=codes[1].cpu(), k_scales=scales[0].cpu(),
             v_scales=scales[1].cpu())
    assert float(d["v_scales"].max()) == 2.0 ** 120
    got, bits = run(pkg, d, 1, **kw)
    assert int(err.item()) == bits == 0
    ref, mass = exact(d, w.scale)
    assert (got[0, 2:, 7] == float("inf")).all() and (got[0, 2:, 30] == float("-inf")).all()
    assert torch.isnan(got[0, :2, 11]).all()
    for x in (got, ref, mass):
        x[0, 2:, 7] = x[0, 2:, 30] = x[0, :2, 11] = 0.0
    size = w.scale * float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()) * 1.07
    assert_close(got, ref, mass, BF16, weight_error(D, size) + 2.0 ** -21, 0.0)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_bf16_query_with_an_outlier(pkg, D):  # noqa: F811
    """One dim of q far above the others (2^22), where K is zero: the scores are
    the other dims' alone, which keep bf16's precision."""
    L = 700
    w, q, off = ragged(530, [L], [1], Hq=8, Hkv=2, D=D, PS=16, dtype=BF16)
    g = torch.Generator().manual_seed(531)
    k, v = (torch.randn((L, 2, D), generator=g) for _ in range(2))
    q[:, :, 3], k[:, :, 3] = 2.0 ** 22, 0.0
    d = pool(w, k, v, q, off)
    got, err = run(pkg, d, 1, scale=0.2)
    assert err == 0
    ref, mass = exact(d, 0.2)
    # sum |q_d k_d| of the dims that count; q in fp16 with its largest at 2^14:
    # below 2^-9 = 2^(22 - 31) it loses bits, by at most 2^-25 of 2^14 each
    rest = q.double().clone()
    rest[:, :, 3] = 0.0
    kn = float(k.double().norm(dim=-1).max()) * 1.07
    size = 0.2 * float(rest.norm(dim=-1).max()) * kn
    lost = 0.2 * kn * D ** 0.5 * 2.0 ** (22 - 39)
    assert_close(got, ref, mass, BF16, weight_error(D, size) + 2.0 ** -21 + 2 * lost, 0.0)


def test_an_inf_and_a_nan_with_two_heads_per_cta(pkg):  # noqa: F811
    """A table long enough that the plan takes two KV heads per CTA: what is
    beside the products stays with its own head."""
    L, Hkv, D, cap = 600, 2, 64, 16384
    w, q, off = ragged(540, [L], [1], Hq=4, Hkv=Hkv, D=D, PS=16, dtype=BF16, max_pages=cap)
    g = torch.Generator().manual_seed(541)
    k, v = (torch.randn((L, Hkv, D), generator=g) for _ in range(2))
    d = pool(w, k, v, q, off)
    p = pkg.DecodeAttnParams(1, 4, Hkv, D, 16, cap, d["k_pages"].shape[0], 0, 1.0, 0, 0, 0, 0, 1, 1,
                             0)
    plan = pkg.decode_attn_quant_make_plan(p, 152)
    assert (plan.grid_x if plan.head_fastest else plan.grid_y) == 1
    page, slot = int(d["table"][0, 500 // 16]), 500 % 16
    d["v_scales"][page, 1, slot] = 2.0 ** 120
    codes = torch.zeros(D, dtype=torch.uint8)
    codes[20], codes[21], codes[22] = 0x7e, 0xfe, 0x7f  # 448, -448, NaN
    d["v_pages"].view(torch.uint8)[page, slot, 1] = codes
    got, err = run(pkg, d, 1)
    assert err == 0
    assert (got[0, 2:, 20] == float("inf")).all() and (got[0, 2:, 21] == float("-inf")).all()
    assert torch.isnan(got[0, 2:, 22]).all()
    ref, mass = exact(d, w.scale)
    for x in (got, ref, mass):
        x[0, 2:, 20:23] = 0.0
    size = w.scale * float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()) * 1.07
    assert_close(got, ref, mass, BF16, weight_error(D, size) + 2.0 ** -21, 0.0)
