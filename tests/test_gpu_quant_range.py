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
