"""One zeroed workspace for calls of very different sizes: a step with more
than 16384 (sequence, KV head) groups, whose last tickets lie where smaller
calls keep their partials, before and after such a call, by each entry point."""
import pytest
import torch

from tests.chunk_reference import quantise, ragged
from tests.test_gpu_quant import DEV, F16, pkg  # noqa: F401

pytestmark = pytest.mark.gpu

B, HKV, D, PS, BOUND = 2100, 8, 128, 64, 4096
LAST = 40  # sequences at the end that are cut into shards


@pytest.fixture(scope="module")
def large():
    """Many sequences of one position, and long ones among the last groups,
    all over one small pool."""
    g = torch.Generator().manual_seed(480)
    P = 100
    lens = torch.ones(B, dtype=torch.int32)
    lens[-LAST:] = torch.randint(2100, BOUND + 1, (LAST,), generator=g).to(torch.int32)
    d = dict(q=torch.randn((B, HKV, D), generator=g).half(),
             table=torch.randint(0, P, (B, BOUND // PS), generator=g).to(torch.int32), lens=lens)
    for n in ("k", "v"):
        x = torch.randn((P, PS, HKV, D), generator=g).half()
        code, s = quantise(x)
        d[n], d[n + "_codes"], d[n + "_scales"] = x, code, s.transpose(1, 2).contiguous()
    return {n: t.to(DEV) for n, t in d.items()}


def step(pkg, d, name, ws, err):  # noqa: F811
    kw = dict(max_seq_len=BOUND, workspace=ws, err_flag=err, schedule=1)
    if name == "quant":
        return pkg.decode_attn_quant(d["q"], d["k_codes"], d["v_codes"], d["k_scales"],
                                     d["v_scales"], d["table"], d["lens"], D ** -0.5, **kw)
    return pkg.decode_attn(d["q"], d["k"], d["v"], d["table"], d["lens"], D ** -0.5, **kw)


def small(pkg, name, ws, err):  # noqa: F811
    w, q, off = ragged(481, [3000], [1], Hq=64, Hkv=8, D=64, PS=16)
    a = [q.to(DEV), w.k_pages.to(DEV), w.v_pages.to(DEV), w.page_table.to(DEV)]
    L = w.seq_lens.to(DEV)
    kw = dict(max_seq_len=3000, workspace=ws, err_flag=err, force_chunk=128)
    if name == "chunk":
        return pkg.decode_attn_chunk(*a, off.to(DEV), L, w.scale, **kw)
    if name == "quant":
        pools = [quantise(x) for x in (w.k_pages, w.v_pages)]
        return pkg.decode_attn_quant(a[0], *[c.to(DEV) for c, _ in pools],
                                     *[s.transpose(1, 2).contiguous().to(DEV) for _, s in pools],
                                     a[3], L, w.scale, schedule=1, **kw)
    return pkg.decode_attn(*a, L, w.scale, schedule=1, **kw)


def shape(pkg):  # noqa: F811
    return pkg.DecodeAttnParams(B, HKV, HKV, D, PS, BOUND // PS, 100, BOUND, 1.0, 0, 0, 0, 0, 1, 0,
                                1)


def test_the_large_step_has_tickets_behind_64_kib(pkg):  # noqa: F811
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    for plan in (pkg.decode_attn_make_plan(shape(pkg), sms),
                 pkg.decode_attn_quant_make_plan(shape(pkg), sms)):
        assert plan.max_shards > 1 and not plan.cluster
        heads = plan.grid_x if plan.head_fastest else plan.grid_y
        assert (B - LAST) * heads > 16384


@pytest.mark.parametrize("between", ["decode", "quant", "chunk"])
@pytest.mark.parametrize("name", ["decode", "quant"])
def test_large_small_large_on_one_buffer(pkg, large, name, between):  # noqa: F811
    ws = torch.zeros(96 << 20, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    first = step(pkg, large, name, ws, err)
    alone = small(pkg, between, torch.zeros_like(ws), err)
    for _ in range(2):
        got = small(pkg, between, ws, err)
        again = torch.full_like(first, float("nan"))
        again.copy_(step(pkg, large, name, ws, err))
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert torch.equal(first, again) and torch.equal(got, alone)
    # the sequences of one position: their value row itself
    page = large["table"][:B - LAST, 0].long()
    if name == "decode":
        assert torch.equal(first[:B - LAST], large["v"][page, 0])


@pytest.mark.parametrize("name", ["decode", "quant"])
def test_large_small_large_on_the_cached_buffer(pkg, large, name):  # noqa: F811
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    first = step(pkg, large, name, None, err)
    small(pkg, name, None, err)
    again = step(pkg, large, name, None, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(first, again)


@pytest.mark.parametrize("name", ["decode", "quant"])
def test_large_step_in_a_graph_between_small_ones(pkg, large, name):  # noqa: F811
    """The clearing is captured with the launch."""
    ws = torch.zeros(96 << 20, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = step(pkg, large, name, ws, err)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(pkg, large, name, ws, err)
    for _ in range(3):
        small(pkg, name, ws, err)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and torch.equal(out, want)
