"""decode_attn_quant (the decode step over an e4m3 cache) against an exact
softmax in 64 bits over the same codes and scales, element by element, and
the operators together as a server runs them.

Nothing but the result is rounded to 16 bits (weights are kept as an fp16 head
and remainder, 2^-22), so the tolerance is one rounding of the result and the
32-bit sums (chunk_reference)."""
import os

import pytest
import torch

from tests.chunk_reference import (assert_rows, chunk_attention, half_step, quantise, ragged,
                                   score_size, weight_error)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_gqa_decode_06_gb300 import build
    build.build()
    import paged_gqa_decode_06_gb300 as p
    p.load_library()
    return p


def cache(seed, lens, T, *, Hq, Hkv, D, PS, dtype, loud=True, max_pages=None):
    """q [B, T, Hq, D], codes, scales (not powers of two, magnitudes spread
    over 2^-12..2^8 when loud), table and lengths."""
    w, q, off = ragged(seed, lens, [T] * len(lens), Hq=Hq, Hkv=Hkv, D=D, PS=PS, dtype=dtype,
                       max_pages=max_pages)
    g = torch.Generator().manual_seed(seed + 2)
    d = dict(q=q, off=off, table=w.page_table, lens=w.seq_lens, scale=w.scale)
    for n in ("k", "v"):
        x = getattr(w, n + "_pages").float()
        if loud and n == "v":
            x = x * torch.exp2(torch.randint(-12, 9, (*x.shape[:-1], 1), generator=g).float())
        code, s = quantise(x.half())
        s = s * (0.6 + torch.rand(s.shape, generator=g))
        d[n + "_pages"], d[n + "_scales"] = code, s.transpose(1, 2).contiguous()
    return d


def run(pkg, d, T, window=0, scale=None, **kw):
    B, Hq, D = len(d["lens"]), d["q"].shape[1], d["q"].shape[2]
    q = d["q"].view(B, T, Hq, D) if T > 1 else d["q"]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pkg.decode_attn_quant(
        q.to(DEV), d["k_pages"].to(DEV), d["v_pages"].to(DEV), d["k_scales"].to(DEV),
        d["v_scales"].to(DEV), d["table"].to(DEV), d["lens"].to(DEV),
        d["scale"] if scale is None else scale, window=window, err_flag=err, **kw)
    torch.cuda.synchronize()
    return got.view(B * T, Hq, D), int(err.item())


def weight(d, scale=None):
    """The weights' error: the 32-bit sums, 2^-22 of the split, and a bf16 q's
    values below 2^-14 of its row's largest, off by 2^-25 of it in fp16."""
    size = score_size(d["q"], d["k_pages"], d["scale"] if scale is None else scale, d["k_scales"])
    D = d["q"].shape[-1]
    return weight_error(D, size) + 2.0 ** -21 + 2 * size * D ** 0.5 * 2.0 ** -24


def check(pkg, d, T, window=0, scale=None, lens=None, **kw):
    got, err = run(pkg, d, T, window, scale, **kw)
    assert err == 0
    ref, mass = chunk_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["off"],
                                d["lens"], d["scale"] if scale is None else scale, window,
                                d["k_scales"], d["v_scales"])
    assert_rows(got, ref, mass, d["q"].dtype, weight(d, scale))
    return got


# (lengths, T, Hq, Hkv, D, page, window, keywords)
CASES = [
    ([1], 1, 4, 1, 64, 8, 0, {}),
    ([1, 2, 63, 64, 65], 1, 8, 2, 128, 16, 0, {}),
    ([0, 255, 256, 0], 1, 32, 8, 128, 16, 0, {}),
    ([257, 3060, 700], 1, 32, 8, 128, 16, 0, {}),
    ([3060], 1, 16, 4, 256, 16, 0, {}),
    ([3060], 1, 32, 8, 64, 16, 0, {}),
    ([2000, 77], 1, 16, 1, 128, 64, 0, {}),                      # 16 query rows
    ([900, 1500], 2, 8, 1, 128, 32, 0, {}),
    ([900, 3], 5, 3, 1, 64, 128, 0, {}),                         # more queries than positions
    ([5000, 4097, 30], 1, 14, 2, 128, 256, 300, {}),
    ([5000, 4097, 30], 3, 4, 1, 256, 8, 1, {}),
    ([1100, 900], 1, 8, 2, 128, 16, 0, dict(force_chunk=128)),
    ([1100, 900], 1, 8, 2, 256, 16, 0, dict(force_chunk=256, schedule=2)),
    ([1100, 900], 1, 8, 2, 64, 16, 0, dict(force_chunk=192, schedule=1)),
    ([700, 120], 1, 8, 2, 128, 16, 0, dict(split_min=10000)),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_quant_matches_exact_softmax(pkg, case, dtype):
    lens, T, Hq, Hkv, D, PS, window, kw = CASES[case]
    d = cache(400 + case, lens, T, Hq=Hq, Hkv=Hkv, D=D, PS=PS, dtype=dtype)
    check(pkg, d, T, window, **kw)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_quant_every_page_size(pkg, D, page):
    d = cache(430, [417, 260, 33], 1, Hq=6, Hkv=2, D=D, PS=page, dtype=F16)
    check(pkg, d, 1)
    check(pkg, d, 1, window=100)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_quant_scales(pkg, scale):
    d = cache(431, [500, 40], 1, Hq=8, Hkv=2, D=128, PS=16, dtype=BF16)
    check(pkg, d, 1, scale=scale)


def test_quant_bf16_rows_beyond_fp16(pkg):
    """Rows of q whose magnitudes no fp16 holds."""
    d = cache(432, [300], 1, Hq=8, Hkv=2, D=128, PS=16, dtype=BF16)
    factor = torch.exp2(torch.tensor([20.0, -30, 60, -60, 90, -90, 0, 1]))[None, :, None]
    d["q"] = (d["q"].float() * factor).bfloat16()
    # each head with a scale that brings its scores back
    for h in range(8):
        s = d["scale"] / float(factor[0, h, 0])
        got, err = run(pkg, d, 1, scale=s)
        assert err == 0
        one = dict(d, q=d["q"][:, h:h + 1].repeat(1, 8, 1))
        ref, mass = chunk_attention(one["q"], d["k_pages"], d["v_pages"], d["table"], d["off"],
                                    d["lens"], s, 0, d["k_scales"], d["v_scales"])
        assert_rows(got[:, h], ref[:, h], mass[:, h], BF16, weight(one, s))


def test_quant_zero_and_uneven_values(pkg):
    """Zero V rows (scale 0) beside tiny and large ones."""
    d = cache(433, [600, 64], 1, Hq=8, Hkv=2, D=128, PS=16, dtype=F16, loud=False)
    d["v_scales"][:, :, ::3] = 0.0
    d["v_scales"][:, :, 1::3] *= 2.0 ** -20
    check(pkg, d, 1)
    d["v_scales"][:] = 0.0
    got, err = run(pkg, d, 1)
    assert err == 0 and torch.all(got == 0)
    # a cache whose every value is far below 16-bit magnitudes.  The exponents
    # s + log2(vs) - m are differences of numbers near 70, so each carries
    # half a step of those, 2^-24 * 128, twice (s + log2(vs), and minus m), and
    # the weight that relative error times ln 2 < 1: 2^-16 in all.
    d = cache(434, [600], 1, Hq=8, Hkv=2, D=128, PS=16, dtype=BF16, loud=False)
    d["v_scales"] *= 2.0 ** -60
    got, err = run(pkg, d, 1)
    ref, mass = chunk_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["off"],
                                d["lens"], d["scale"], 0, d["k_scales"], d["v_scales"])
    assert err == 0
    assert_rows(got, ref, mass, BF16, weight(d) + 2.0 ** -16)


@pytest.mark.parametrize("kw", [{}, dict(force_chunk=128, schedule=1),
                                dict(force_chunk=128, schedule=2)], ids=["auto", "grid", "cluster"])
def test_quant_unattended_codes_never_matter(pkg, kw):
    d = cache(435, [333, 200], 1, Hq=8, Hkv=2, D=128, PS=32, dtype=F16)
    clean, err = run(pkg, d, 1, window=170, **kw)
    used = torch.zeros(d["k_pages"].shape[:2], dtype=torch.bool)
    for b, L in enumerate((333, 200)):
        for t in range(max(0, L - 170), L):
            used[d["table"][b, t // 32], t % 32] = True
    for n in ("k", "v"):
        d[n + "_pages"].view(torch.uint8)[~used] = 0x7f  # NaN
        s = d[n + "_scales"].transpose(1, 2).contiguous()
        s[~used] = float("nan")
        d[n + "_scales"] = s.transpose(1, 2).contiguous()
    again, err2 = run(pkg, d, 1, window=170, **kw)
    assert err == err2 == 0 and torch.equal(clean, again)


@pytest.mark.parametrize("kw", [{}, dict(force_chunk=128, schedule=1),
                                dict(force_chunk=128, schedule=2)], ids=["auto", "grid", "cluster"])
def test_quant_bad_lengths_and_pages(pkg, kw):
    d = cache(436, [300, 50, 50, 300], 1, Hq=8, Hkv=2, D=128, PS=16, dtype=F16)
    want, _ = run(pkg, d, 1, **kw)
    d["lens"] = torch.tensor([300, -1, 100000, 300], dtype=torch.int32)
    d["table"] = d["table"].clone()
    d["table"][3, 9] = d["k_pages"].shape[0]
    got, err = run(pkg, d, 1, **kw)
    assert err == pkg.DEV_BAD_LEN | pkg.DEV_BAD_PAGE
    assert torch.equal(got[0], want[0]) and torch.all(got[1:] == 0)


def test_quant_same_bits_every_run_and_beside_decode(pkg):
    """The same bits run after run, also with 16-bit decode steps sharing the
    workspace between them."""
    d = cache(437, [3000, 777], 1, Hq=32, Hkv=8, D=128, PS=16, dtype=BF16)
    w, _, _ = ragged(438, [900], [1], Hq=32, Hkv=8, D=128, PS=16)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    a, err = run(pkg, d, 1, workspace=ws)
    assert err == 0
    for _ in range(3):
        pkg.decode_attn(w.q.to(DEV), w.k_pages.to(DEV), w.v_pages.to(DEV), w.page_table.to(DEV),
                        w.seq_lens.to(DEV), w.scale, workspace=ws, schedule=1)
        b, err = run(pkg, d, 1, workspace=ws)
        assert err == 0 and torch.equal(a, b)


@pytest.mark.parametrize("T,Hq,Hkv,D,PS,window", [
    (1, 8, 2, 64, 8, 0), (1, 8, 2, 64, 16, 100), (1, 32, 4, 128, 16, 0), (1, 8, 2, 128, 8, 0),
    (2, 8, 2, 64, 32, 0), (3, 4, 2, 128, 16, 70), (1, 6, 2, 256, 8, 0), (1, 4, 4, 64, 64, 0),
])
def test_quant_two_heads_per_cta(pkg, T, Hq, Hkv, D, PS, window):
    """Small boxes and a step that the bound on the lengths calls large: the
    plan takes two KV heads per CTA.  Short and empty sequences among them."""
    cap = 65536 // PS * 8
    d = cache(450, [900, 1, 0, 77, 2300, 64], T, Hq=Hq, Hkv=Hkv, D=D, PS=PS, dtype=BF16,
              max_pages=cap)
    p = pkg.DecodeAttnParams(6, Hq, Hkv, D, PS, cap, d["k_pages"].shape[0], 0, 1.0, window, 0, 0,
                             0, T, 1, 0)
    plan = pkg.decode_attn_quant_make_plan(p, 152)
    heads = plan.grid_x if plan.head_fastest else plan.grid_y
    assert heads == Hkv // 2 or window
    check(pkg, d, T, window)
    check(pkg, d, T, window, force_chunk=256)  # shards and their merge
    d["table"] = d["table"].clone()
    d["table"][4, 20] = -3
    got, err = run(pkg, d, T, window)
    bad = 20 * PS + PS > (max(0, 2300 - T + 1 - window) if window else 0)
    assert err == (pkg.DEV_BAD_PAGE if bad else 0)
    assert torch.all(got[4 * T:5 * T] == 0) == bad


def test_quant_long_context(pkg):
    d = cache(439, [40000], 1, Hq=8, Hkv=1, D=128, PS=64, dtype=F16)
    check(pkg, d, 1, max_seq_len=40000)


def test_quant_large_batch(pkg):
    """More (sequence, head) units than CTA slots: several waves."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 300, (260,), generator=g).tolist()
    d = cache(440, lens, 1, Hq=8, Hkv=2, D=64, PS=16, dtype=F16)
    check(pkg, d, 1)
    check(pkg, d, 1, force_chunk=64)


def test_quant_graphs_do_not_share_a_workspace(pkg):
    sets, graphs = [], []
    for seed in (441, 442):
        d = cache(seed, [3000], 1, Hq=32, Hkv=8, D=128, PS=16, dtype=F16)
        g = [d[n].to(DEV) for n in ("q", "k_pages", "v_pages", "k_scales", "v_scales", "table",
                                    "lens")]
        sets.append((g, pkg.decode_attn_quant(*g, d["scale"], schedule=1)))
        torch.cuda.synchronize()
        graph, out = torch.cuda.CUDAGraph(), torch.empty_like(g[0])
        with torch.cuda.graph(graph):
            pkg.decode_attn_quant(*g, d["scale"], schedule=1, out=out)
        graphs.append((graph, out))
    streams = [torch.cuda.Stream(DEV) for _ in sets]
    for _ in range(20):
        for st, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out), (_, ref) in zip(graphs, sets):
        assert torch.equal(out, ref)


def test_quant_stalled_wait_reports_and_recovers(pkg):
    d = cache(443, [500], 1, Hq=8, Hkv=2, D=128, PS=16, dtype=F16)
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device=DEV)
    want, _ = run(pkg, d, 1, workspace=ws)
    os.environ["DECODE_ATTN_TEST_STALL_TX"] = "64"
    try:
        got, err = run(pkg, d, 1, workspace=ws)
    finally:
        del os.environ["DECODE_ATTN_TEST_STALL_TX"]
    assert err & pkg.DEV_TIMEOUT and torch.all(got == 0)
    ws.zero_()
    got, err = run(pkg, d, 1, workspace=ws)
    assert err == 0 and torch.equal(got, want)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
def test_serving_over_an_8_bit_cache(pkg, dtype):
    """Two prompts by the chunk, then decode steps, as a server with an 8-bit
    cache runs them: each chunk's rows are quantised into their pages, the
    cache is read back into 16-bit pages that the chunk attends, and the
    decode steps run on the codes.  Every output against the exact softmax
    over the codes written so far."""
    Hq, Hkv, D, PS = 16, 4, 128, 16
    chunks = [[40, 16], [33, 70], [1, 1], [1, 1]]
    B, cap = 2, 10
    g = torch.Generator().manual_seed(7)
    P = B * cap + 2
    table = torch.randperm(P, generator=g)[:B * cap].view(B, cap).to(torch.int32)
    kp, vp = (torch.zeros((P, PS, Hkv, D), dtype=torch.float8_e4m3fn, device=DEV)
              for _ in range(2))
    ks, vs = (torch.zeros((P, Hkv, PS), device=DEV) for _ in range(2))
    tb = table.to(DEV)
    lens = [0, 0]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for news in chunks:
        lens = [a + b for a, b in zip(lens, news)]
        off = torch.tensor([0, news[0], sum(news)], dtype=torch.int32)
        q, k, v = (torch.randn((sum(news), h, D), generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
        L = torch.tensor(lens, dtype=torch.int32, device=DEV)
        pkg.decode_kv_append_chunk(k.to(DEV), v.to(DEV), off.to(DEV), L, kp, vp, tb, ks, vs,
                                   err_flag=err)
        if max(news) > 1:
            pages = [-(-x // PS) for x in lens]
            whole = torch.tensor([0, pages[0] * PS, sum(pages) * PS], dtype=torch.int32)
            k16, v16 = pkg.decode_kv_read(kp, vp, tb, whole.to(DEV), sum(pages) * PS,
                                          k_scales=ks, v_scales=vs, dtype=dtype, err_flag=err)
            ids = torch.full((B, cap), -1, dtype=torch.int32)
            for b in range(B):
                ids[b, :pages[b]] = torch.arange(pages[b]) + (pages[0] if b else 0)
            got = pkg.decode_attn_chunk(q.to(DEV), k16.view(-1, PS, Hkv, D),
                                        v16.view(-1, PS, Hkv, D), ids.to(DEV), off.to(DEV), L,
                                        D ** -0.5, max_seq_len=max(lens), err_flag=err)
            step = half_step(dtype)  # the weights' rounding
        else:
            got = pkg.decode_attn_quant(q.to(DEV), kp, vp, ks, vs, tb, L, D ** -0.5,
                                        max_seq_len=max(lens), err_flag=err)
            step = 0.0
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        c = [t.cpu() for t in (kp, vp, ks, vs)]
        ref, mass = chunk_attention(q, c[0], c[1], table, off, lens, D ** -0.5, 0, c[2], c[3])
        d = dict(q=q, k_pages=c[0], k_scales=c[2], scale=D ** -0.5)
        # read back in fp16, a value below 2^-14 may round (bf16 holds them all)
        assert_rows(got, ref, mass + 2.0 ** -25, dtype, weight(d) + step)
