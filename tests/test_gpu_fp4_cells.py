"""Rows of 4 bits at the end of their type's range, appended and read back."""
import math

import pytest
import torch

from tests.fp4_reference import values4
from tests.test_gpu_kv_rope import (BF16, DEV, E4M3, F16, NAMES, bits, offsets,  # noqa: F401
                                    pkg, pools, run_append)

pytestmark = pytest.mark.gpu


def read(pkg, got, table, n, dtype):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pkg.decode_kv_read_fp4(*[got[x].to(DEV) for x in NAMES], table.to(DEV),
                                 offsets([n]).to(DEV), n, dtype=dtype, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return [x.cpu() for x in out]


def cells(got, i, table, n):
    """What the first sequence's cells stand for, in 64 bits."""
    PS = got["k_pages"].shape[1]
    p = torch.arange(n)
    page, slot = table[0, p // PS].long(), p % PS
    return values4(got[NAMES[i]][page, slot], got[NAMES[2 + i]][page, :, slot],
                   got[NAMES[4 + i]].view(torch.uint8)[page, :, slot].view(E4M3))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
def test_finite_rows_read_back_finite(pkg, dtype):
    """A block whose maximum is near the type's largest number can get a scale whose code
    6 stands for a larger one (fp16: from 64512 on, 67584): it reads back as the type's
    largest, not as an Inf."""
    top = torch.finfo(dtype).max
    i = torch.arange(256, dtype=torch.int16)
    large = (torch.tensor([top], dtype=dtype).view(torch.int16) - i).view(dtype)
    D, n = 64, 256
    x = torch.zeros((n, 1, D), dtype=dtype)
    x[:, 0, 0], x[:, 0, 17], x[:, 0, 40] = large, -large, large / 8
    x[:, 0, 41] = large / 4
    d, table = pools(30, [n], 1, D, 16, "fp4", dtype)
    got, _, err = run_append(pkg, d, table, x, -x, offsets([n]), [n])
    assert err == 0
    for i, y in enumerate(read(pkg, got, table, n, dtype)):
        assert torch.isfinite(y).all()
        want = cells(got, i, table, n)
        assert float(want.abs().max()) > top
        assert torch.equal(bits(y), bits(want.clamp(-top, top).float().to(dtype)))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
def test_cells_beyond_the_type(pkg, dtype):
    """Cells with finite scales beyond the type's range, whichever scale takes them there,
    read back as its largest number; those with an Inf or a NaN as that."""
    D, n, PS = 64, 48, 16
    d, table = pools(31, [n], 1, D, PS, "fp4", dtype)
    page, slot = table[0, torch.arange(n) // PS].long(), torch.arange(n) % PS
    scales = torch.tensor([2.0 ** 14, -2.0 ** 14, 2.0 ** 127, -3e38, 2.0 ** 120, 30.0, math.inf,
                           -math.inf, math.nan, 1e-3, 0.0, 2.0 ** -140])
    for i in range(2):
        d[NAMES[2 + i]][page, :, slot] = scales.repeat(4)[:, None]
        b = torch.randint(0, 0x7f, d[NAMES[4 + i]].shape, dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(i))
        d[NAMES[4 + i]] = b.view(E4M3)
    top = torch.finfo(dtype).max
    for i, y in enumerate(read(pkg, d, table, n, dtype)):
        code = cells(dict(d, **{NAMES[2 + i]: torch.ones_like(d[NAMES[2 + i]])}), i, table, n)
        s = d[NAMES[2 + i]][page, :, slot][..., None]
        want = torch.where(torch.isfinite(s), (code.double() * s.double()).clamp(-top, top),
                           code.double() * s.double())
        want = want.float().to(dtype)
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        keep = ~torch.isnan(want)
        assert torch.equal(y[keep], want[keep])
