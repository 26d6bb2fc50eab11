"""No sequences: every call of the ragged and 8-bit set returns before it looks
at a pointer (an empty tensor has none)."""
import pytest
import torch

from tests.test_ragged_host import calls, params, pkg  # noqa: F401


def test_no_sequences_need_no_pointers(pkg):  # noqa: F811
    assert set(calls(pkg, params(pkg, batch=0)).values()) == {0}
    # what is wrong with the other arguments is still said
    assert calls(pkg, params(pkg, batch=0), fmt=7)["quant"] == -2
    assert calls(pkg, params(pkg, batch=0, head_dim=96))["quant"] == -3


@pytest.mark.gpu
def test_no_sequences_from_python(pkg):  # noqa: F811
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")

    def z(*shape, dtype=torch.float16):
        return torch.zeros(shape, dtype=dtype, device="cuda:0")

    codes, s = z(4, 16, 2, 64, dtype=torch.float8_e4m3fn), z(4, 2, 16, dtype=torch.float32)
    t, n, off = z(0, 2, dtype=torch.int32), z(0, dtype=torch.int32), z(1, dtype=torch.int32)
    for shape in ((0, 8, 64), (0, 2, 8, 64)):
        q = z(*shape)
        assert pkg.decode_attn_quant(q, codes, codes, s, s, t, n, 0.1).shape == q.shape
    pool = z(4, 16, 2, 64)
    assert pkg.decode_attn_chunk(z(0, 8, 64), pool, pool, t, off, n, 0.1).shape == (0, 8, 64)
    pkg.decode_kv_append_chunk(z(0, 2, 64), z(0, 2, 64), off, n, codes, codes, t, s, s)
    k, v = pkg.decode_kv_read(codes, codes, t, off, 0, k_scales=s, v_scales=s)
    assert k.shape == v.shape == (0, 2, 64)
