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
    """[total, Hq, D] in 64 bits: one exact softmax per row; a row without a
    key is zero."""
    Hq = q.shape[1]
    G = Hq // k_pages.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64)
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
        w = torch.where(hide, torch.zeros_like(s),
                        torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300)))
        tot = w.sum(-1, keepdim=True)
        w = torch.where(tot > 0, w / tot.clamp(min=1e-300), torch.zeros_like(w))
        # (a row outside the mask contributes nothing, whatever it holds)
        o = torch.einsum("hnt,thd->nhd", w, torch.nan_to_num(V, nan=0.0, posinf=0.0, neginf=0.0))
        out[a:z] = o
    return out


def half_step(dtype):
    """Largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2
