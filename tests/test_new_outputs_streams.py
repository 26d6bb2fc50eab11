"""Outputs that a call creates itself for work on another stream than the
current one lie in that stream's memory: what the current stream's allocator
hands out may still be waiting for earlier work of that stream."""
import contextlib

import pytest
import torch

from tests.chunk_reference import quantise, ragged

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pkg():
    from paged_gqa_decode_06_gb300 import build
    build.build()
    import paged_gqa_decode_06_gb300 as p
    p.load_library()
    return p


def test_outputs_are_allocated_on_the_stream_that_fills_them(pkg, monkeypatch):
    log, inside = [], []

    @contextlib.contextmanager
    def stream(s):
        inside.append(s)
        yield
        inside.pop()

    empty = torch.empty_like
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty_like", lambda t: log.append(list(inside)) or empty(t))
    t = torch.zeros(3)
    pkg._new_like(t, "side")
    pkg._new_like(t)
    pkg._new_like(t, None)
    assert log == [["side"], [], []] and not inside


def calls(pkg):
    """{entry point: (the call with keywords, its expected outputs)}"""
    w, q, off = ragged(700, [3000, 77], [1, 1], Hq=64, Hkv=8, D=128, PS=16)
    a = [q.to(DEV), w.k_pages.to(DEV), w.v_pages.to(DEV), w.page_table.to(DEV)]
    L, off = w.seq_lens.to(DEV), off.to(DEV)
    pools = [quantise(x) for x in (w.k_pages, w.v_pages)]
    codes = [c.to(DEV) for c, _ in pools]
    scales = [s.transpose(1, 2).contiguous().to(DEV) for _, s in pools]
    rows = torch.tensor([0, 3000, 3077], dtype=torch.int32, device=DEV)
    new = [torch.randn(2, 8, 128, device=DEV).half() for _ in range(2)]
    return {
        "decode_attn": lambda **kw: pkg.decode_attn(*a, L, w.scale, **kw),
        "decode_attn_append": lambda **kw: pkg.decode_attn_append(a[0], *new, *a[1:], L, w.scale,
                                                                  **kw),
        "decode_attn_static_scratch": lambda **kw: pkg.decode_attn_static_scratch(*a, L, w.scale,
                                                                                  **kw),
        "decode_attn_chunk": lambda **kw: pkg.decode_attn_chunk(*a, off, L, w.scale, **kw),
        "decode_attn_quant": lambda **kw: pkg.decode_attn_quant(a[0], *codes, *scales, a[3], L,
                                                                w.scale, **kw),
        "decode_kv_read": lambda **kw: pkg.decode_kv_read(*codes, a[3], rows, 3077,
                                                          k_scales=scales[0], v_scales=scales[1],
                                                          **kw),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["decode_attn", "decode_attn_append",
                                  "decode_attn_static_scratch", "decode_attn_chunk",
                                  "decode_attn_quant", "decode_kv_read"])
def test_pending_work_of_the_current_stream_does_not_reach_new_outputs(pkg, name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    call = calls(pkg)[name]
    want = call()
    want = want if isinstance(want, tuple) else (want,)
    side = torch.cuda.Stream(DEV)
    call(stream=side)  # its workspace is there already
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)  # the current stream is busy for some 30 ms
    pending = [torch.empty_like(t).fill_(7.0) for t in want for _ in range(3)]
    del pending
    got = call(stream=side)
    torch.cuda.synchronize()
    got = got if isinstance(got, tuple) else (got,)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
