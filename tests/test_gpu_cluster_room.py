"""Clusters of 15 CTAs with 16 query rows, whose receive buffer is the largest
there is: the 8-bit step against the exact softmax, the 16-bit step bit for bit
against its merge through the workspace."""
import pytest
import torch

from tests.chunk_reference import ragged
from tests.test_gpu_quant import BF16, DEV, F16, cache, check, pkg  # noqa: F401

pytestmark = pytest.mark.gpu

# (head_dim, query heads, KV heads, T, length, keywords): 15 shards each; the
# first is what the planner takes by itself
CASES = [
    (256, 16, 1, 1, 2800, {}),
    (256, 16, 2, 2, 2800, {}),
    (256, 16, 1, 1, 1900, dict(force_chunk=128, schedule=2)),
    (128, 16, 1, 1, 1900, dict(force_chunk=128, schedule=2)),
    (64, 16, 1, 1, 1900, dict(force_chunk=128, schedule=2)),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_cluster_of_15_over_the_8_bit_cache(pkg, case, dtype):  # noqa: F811
    D, Hq, Hkv, T, L, kw = CASES[case]
    d = cache(460 + case, [L], T, Hq=Hq, Hkv=Hkv, D=D, PS=16, dtype=dtype)
    p = pkg.DecodeAttnParams(1, Hq, Hkv, D, 16, d["table"].shape[1], d["k_pages"].shape[0], L, 1.0,
                             0, 0, 0, kw.get("force_chunk", 0), T, 0, kw.get("schedule", 0))
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    if sms == 152 and not (case == 1):
        assert pkg.decode_attn_quant_make_plan(p, sms).cluster == 15
    check(pkg, d, T, max_seq_len=L, **kw)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_cluster_of_15_over_the_16_bit_cache(pkg, case):  # noqa: F811
    D, Hq, Hkv, T, L, kw = CASES[case]
    w, q, _ = ragged(470 + case, [L], [T], Hq=Hq, Hkv=Hkv, D=D, PS=16)
    q = q.view(1, T, Hq, D) if T > 1 else q
    args = [q.to(DEV), w.k_pages.to(DEV), w.v_pages.to(DEV), w.page_table.to(DEV),
            w.seq_lens.to(DEV), w.scale]
    kw = dict(kw, max_seq_len=L)
    got = pkg.decode_attn(*args, **kw)
    grid = pkg.decode_attn(*args, **dict(kw, schedule=1))
    torch.cuda.synchronize()
    assert torch.equal(got, grid)
