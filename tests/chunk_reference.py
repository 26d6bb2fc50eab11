"""Plain implementations in 64 bits (numpy / torch on the CPU) of the ragged
operators, written from their definitions, and the inputs their tests share."""
import math

import torch

from paged_gqa_decode_06_gb300 import workloads


def ragged(seed, lens, news, *, Hq, Hkv, D, PS, dtype=torch.float16, decoys=3, max_pages=None):
    """A pool holding `lens` positions per sequence and `news` query tokens
    each (at the last positions), ragged: (workload, q, offsets)."""
    w = workloads.make_custom("ragged", batch=len(lens), num_q_heads=Hq, num_kv_heads=Hkv,
                              head_dim=D, page_size=PS, seq_lens=lens, seed=seed,
                              decoy_pages=decoys, max_pages=max_pages, dtype=dtype)
    g = torch.Generator().manual_seed(seed + 1)
    off = [0]
    for n in news:
        off.append(off[-1] + n)
    q = torch.randn((off[-1], Hq, D), generator=g).to(dtype)
    return w, q, torch.tensor(off, dtype=torch.int32)


def cache_rows(pages, table_row, lo, hi, scales=None):
    """Positions [lo, hi) of one sequence, [n, Hkv, D] in 64 bits."""
    PS = pages.shape[1]
    pos = torch.arange(lo, hi)
    page, slot = table_row[pos // PS].long(), pos % PS
    if scales is None:
        return pages[page, slot].double()
    codes = pages.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).double()
    return codes * scales[page, :, slot].double()[..., None]


def chunk_attention(q, k_pages, v_pages, table, off, lens, scale, window=0, k_scales=None,
                    v_scales=None):
    """One exact softmax per row, in 64 bits; a row without a key is zero.
    Returns (out, weighted): out [total, Hq, D], and the sum of p |v| beside
    it, which bounds what an error of the weights does to an element."""
    Hq = q.shape[1]
    G = Hq // k_pages.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64)
    mass = torch.zeros(q.shape, dtype=torch.float64)
    for b, L in enumerate(lens):
        L, a, z = int(L), int(off[b]), int(off[b + 1])
        n = z - a
        if n == 0 or L <= 0:
            continue
        first = max(0, L - n + 1 - window) if window > 0 else 0
        K = cache_rows(k_pages, table[b], first, L, k_scales).repeat_interleave(G, 1)
        V = cache_rows(v_pages, table[b], first, L, v_scales).repeat_interleave(G, 1)
        s = torch.einsum("nhd,thd->hnt", q[a:z].double(), K) * scale
        p = torch.arange(L - n, L)[:, None]
        t = torch.arange(first, L)[None]
        hide = t > p
        if window > 0:
            hide = hide | (t <= p - window)
        s = s.masked_fill(hide, -math.inf)
        top = s.amax(-1, keepdim=True)
        w = torch.where(hide, torch.zeros_like(s),
                        torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top)))
        tot = w.sum(-1, keepdim=True)
        w = torch.where(tot == 0, torch.zeros_like(w), w / tot)
        out[a:z] = torch.einsum("hnt,thd->nhd", w, V)
        mass[a:z] = torch.einsum("hnt,thd->nhd", w, V.abs())
    return out, mass


def score_size(q, k_pages, scale, k_scales=None):
    """An upper bound of scale * sum_d |q_d k_d| over all rows (norms)."""
    k = k_pages.view(torch.uint8).view(torch.float8_e4m3fn).double() if k_scales is not None \
        else k_pages.double()
    if k_scales is not None:
        k = k * k_scales.transpose(1, 2).double()[..., None]
    k = torch.nan_to_num(k, nan=0.0, posinf=0.0, neginf=0.0)
    return float(abs(scale) * q.double().norm(dim=-1).max() * k.norm(dim=-1).max())


def half_step(dtype):
    """Largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def weight_error(D, size):
    """Relative error of a softmax weight whose scores are summed in 32 bits:
    D products in any order, each addition off by at most one step (the
    tensor cores may cut where they add), twice over for the maximum and the
    score, and the exponential (2^-22) with its argument's rounding."""
    return 2 * D * 2.0 ** -23 * size + 2.0 ** -21 + 2 * size * 2.0 ** -23


def assert_rows(got, out, mass, dtype, weight, tag=""):
    """|got - out| at most: the weights' error on p |v|, once for the products
    and once for their sum; two roundings of the result (the value itself, and
    its division by the sum in 32 bits, 2^-23); the type's smallest step."""
    g = got.double().cpu()
    u = half_step(dtype)
    tol = 2 * weight * mass + (u + 2.0 ** -22) * out.abs() + torch.finfo(dtype).smallest_normal * u
    over = ((g - out).abs() - tol)
    assert torch.isfinite(g).all(), tag
    assert float(over.max()) <= 0, (tag, float(over.max()), float((g - out).abs().max()))


def quantise(x):
    """Rows [..., D] -> (e4m3 codes, scales [...]) from the definition: the
    least power of two with max |x| <= 448 * scale (0 below 2^-100), the
    nearest code, ties to even."""
    x = x.double()
    top = x.abs().amax(-1)
    scale = torch.zeros_like(top)
    flat, out = top.reshape(-1), scale.view(-1)
    for i, t in enumerate(flat.tolist()):
        if t >= 2.0 ** -100:
            e = math.frexp(t)[1] - 9  # 2^(e + 8) <= t < 2^(e + 9)
            if t > 448.0 * 2.0 ** e:
                e += 1
            out[i] = 2.0 ** e
    y = torch.where(scale[..., None] > 0, x / scale.clamp(min=1e-300)[..., None],
                    torch.zeros_like(x))
    return y.float().to(torch.float8_e4m3fn), scale.float()
