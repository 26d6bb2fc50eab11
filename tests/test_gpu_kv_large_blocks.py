"""Appends and reads of as many rows as fill the row kernels' largest blocks."""
import pytest
import torch

from tests.chunk_reference import quantise
from tests.fp4_reference import quantise4, rope_table, rotate, values4
from tests.test_gpu_kv_rope import (BF16, DEV, E4M3, F16, bits, new_rows, offsets,  # noqa: F401
                                    pkg, pools, run_append, same)

pytestmark = pytest.mark.gpu


def layout(lens, PS):
    """A table of random pages for sequences of `lens`, and every position's cell."""
    g = torch.Generator().manual_seed(32)
    need = [-(-L // PS) for L in lens]
    P = sum(need) + 3
    ids = torch.randperm(P, generator=g).int()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at, page, slot = 0, [], []
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
        p = torch.arange(lens[b])
        page.append(table[b, p // PS].long())
        slot.append(p % PS)
    return P, table, page, slot


# rows of a block (8 blocks an SM, up to 64 rows each), and rows over
@pytest.mark.parametrize("per,over", [(5, 3), (32, -1), (33, 0), (64, -65), (64, 700)])
@pytest.mark.parametrize("fmt", ["16", "fp8", "fp4"])
def test_append_in_large_blocks(pkg, fmt, per, over):
    """Whole sequences of thousands of rows, empty and short ones between them, an odd
    number of query heads: cells, queries and all other cells to the bit."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    total = per * 8 * sms + over
    Hq, Hkv, D, PS, dtype, before = 3, 1, 64, 64, BF16, 11
    cut = [total // 3, 1, 0, 77, total // 5, 2]
    news = cut + [total - sum(cut)]
    lens = [n + before for n in news]
    P, table, page, slot = layout(lens, PS)
    d, _ = pools(33, [1], Hkv, D, PS, fmt, dtype)
    d = {n: torch.zeros((P, *t.shape[1:]), dtype=torch.uint8).to(t.dtype)
         if t.element_size() > 1 else torch.zeros((P, *t.shape[1:]), dtype=torch.uint8)
         .view(t.dtype) for n, t in d.items()}
    off = offsets(news)
    k, v, q = (new_rows(34 + i, total, h, D, dtype) for i, h in enumerate((Hkv, Hkv, Hq)))
    rope = rope_table(48, max(lens))
    pos = torch.cat([torch.arange(before, L) for L in lens])
    turned = [torch.cat([rotate(x[i:i + 8192].float(), pos[i:i + 8192], rope).to(dtype)
                         for i in range(0, total, 8192)]) for x in (k, q)]
    got, q_out, err = run_append(pkg, d, table, k, v, off, lens, rope, q)
    assert err == 0
    assert torch.equal(bits(q_out), bits(turned[1]))
    pg, sl = (torch.cat([x[before:] for x in y]) for y in (page, slot))
    want = {n: t.clone() for n, t in d.items()}
    for n, new in (("k", turned[0]), ("v", v)):
        if fmt == "fp4":
            code, row, block = quantise4(new)
            want[n + "_pages"][pg, sl] = code
            want[n + "_scales"][pg, :, sl] = row
            bits(want[n + "_blocks"])[pg, :, sl] = bits(block)
        elif fmt == "fp8":
            code, scale = quantise(new)
            bits(want[n + "_pages"])[pg, sl] = bits(code)
            want[n + "_scales"][pg, :, sl] = scale
        else:
            want[n + "_pages"][pg, sl] = new
    same(got, want)


@pytest.mark.parametrize("per,over", [(5, 3), (32, -1), (33, 0), (64, -65), (64, 700)])
def test_read_in_large_blocks(pkg, per, over):
    """As many rows read back, from a position of their own in each sequence."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    total = per * 8 * sms + over
    Hkv, D, PS = 1, 64, 64
    cut = [total // 3, 1, 0, 77, total // 5, 2]
    rows, first = cut + [total - sum(cut)], 7
    P, table, page, slot = layout([n + first + 3 for n in rows], PS)
    g = torch.Generator().manual_seed(36)
    levels = torch.randint(0, 127, (2, P, Hkv, PS, D // 16), dtype=torch.uint8, generator=g)
    cache = [torch.randint(0, 256, (P, PS, Hkv, D // 2), dtype=torch.uint8, generator=g)
             for _ in range(2)]
    cache += [torch.randn((P, Hkv, PS), generator=g) for _ in range(2)]
    cache += [x.contiguous().view(E4M3) for x in levels]
    off = offsets(rows)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = [torch.full((total + 5, Hkv, D), 9.0, dtype=F16, device=DEV) for _ in range(2)]
    pkg.decode_kv_read_fp4(*[t.to(DEV) for t in cache], table.to(DEV), off.to(DEV), total + 5,
                           starts=torch.full((len(rows),), first, dtype=torch.int32, device=DEV),
                           k_out=out[0], v_out=out[1], err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pg, sl = (torch.cat([x[first:len(x) - 3] for x in y]) for y in (page, slot))
    for i in range(2):
        part = values4(cache[i][pg, sl], torch.ones((total, Hkv)),
                       cache[4 + i].view(torch.uint8)[pg, :, sl].view(E4M3))
        want = (part.float() * cache[2 + i][pg, :, sl][..., None]).half()
        got = out[i].cpu()
        assert torch.equal(got[:total], want) and bool((got[total:] == 9).all())
