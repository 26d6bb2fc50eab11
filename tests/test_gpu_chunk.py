"""decode_attn_chunk against an exact softmax in 64 bits, element by element.

The tolerance counts the roundings (chunk_reference): the weights are rounded
once to the element type for the second product, half a step each, beside the
32-bit sums of the scores; the result is rounded once."""
import os

import pytest
import torch

from tests.chunk_reference import (assert_rows, chunk_attention, half_step, ragged, score_size,
                                   weight_error)

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


def run(pkg, w, q, off, window=0, scale=None, lens=None, table=None, out=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pkg.decode_attn_chunk(
        q.to(DEV), w.k_pages.to(DEV), w.v_pages.to(DEV),
        (w.page_table if table is None else table).to(DEV), off.to(DEV),
        (w.seq_lens if lens is None else lens).to(DEV), w.scale if scale is None else scale,
        window=window, err_flag=err, out=out, **kw)
    torch.cuda.synchronize()
    return got, int(err.item())


def check(pkg, w, q, off, window=0, scale=None, **kw):
    scale = w.scale if scale is None else scale
    got, err = run(pkg, w, q, off, window, scale, **kw)
    assert err == 0
    ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, w.seq_lens, scale,
                                window)
    weight = half_step(q.dtype) + weight_error(q.shape[-1], score_size(q, w.k_pages, scale))
    assert_rows(got, ref, mass, q.dtype, weight)
    return got


# (lengths, new tokens, Hq, Hkv, D, page, window, force_chunk)
CASES = [
    ([1], [1], 4, 1, 64, 16, 0, 0),
    ([1, 2, 3], [1, 2, 3], 8, 2, 128, 8, 0, 0),
    ([64, 64], [16, 1], 8, 2, 128, 16, 0, 0),
    ([128, 129, 127], [128, 129, 127], 8, 2, 128, 64, 0, 0),
    ([300, 77, 5], [300, 20, 5], 8, 2, 128, 16, 0, 0),
    ([300, 77, 5], [300, 20, 5], 8, 2, 64, 16, 0, 0),
    ([300, 77, 5], [300, 20, 5], 8, 2, 256, 32, 0, 0),
    ([500, 0, 700, 33], [3, 0, 0, 33], 32, 8, 128, 16, 0, 0),
    ([1300, 77, 5], [30, 20, 5], 12, 4, 128, 8, 0, 128),     # G = 3: two rows of a tile unused
    ([900, 700], [90, 70], 14, 2, 64, 256, 100, 0),          # G = 7, window inside a tile
    ([900, 700], [90, 70], 10, 2, 256, 128, 1, 0),           # only the token itself
    ([1100, 640], [1100, 7], 16, 1, 128, 128, 257, 0),       # G = 16
    ([600, 401], [600, 100], 3, 3, 128, 32, 0, 0),           # G = 1
    ([2300, 700, 5], [600, 20, 5], 14, 2, 256, 16, 1000, 256),
    ([2000], [5], 40, 8, 128, 16, 0, 300),                   # shards and their merge
    ([2000, 90], [5, 3], 8, 8, 64, 8, 0, 128),
    ([2000, 1500], [200, 130], 16, 4, 256, 64, 0, 512),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_chunk_matches_exact_softmax(pkg, case, dtype):
    lens, news, Hq, Hkv, D, PS, window, force = CASES[case]
    w, q, off = ragged(100 + case, lens, news, Hq=Hq, Hkv=Hkv, D=D, PS=PS, dtype=dtype)
    check(pkg, w, q, off, window, force_chunk=force)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_every_page_size(pkg, D, page):
    w, q, off = ragged(200, [417, 260], [66, 260], Hq=6, Hkv=2, D=D, PS=page)
    check(pkg, w, q, off)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("D", [128, 256])
def test_chunk_scales(pkg, scale, D):
    """A scale of 0 is the mean of the attended values; a negative one turns
    the order of the scores around; a large one leaves one key per row."""
    w, q, off = ragged(210, [500, 40], [200, 40], Hq=8, Hkv=2, D=D, PS=16)
    check(pkg, w, q, off, window=150, scale=scale)


def test_chunk_growing_scores(pkg):
    """Keys whose scores rise along the sequence make the running maximum
    follow tile after tile."""
    w, q, off = ragged(211, [1500], [40], Hq=8, Hkv=2, D=128, PS=16)
    q = q.abs()
    flat = w.k_pages[w.page_table[0].long()].reshape(-1, 2, 128)
    ramp = torch.linspace(0.01, 1.5, flat.shape[0])[:, None, None]
    w.k_pages[w.page_table[0].long()] = (flat.float().abs() * ramp).half().view(
        -1, 16, 2, 128)
    check(pkg, w, q, off)
    check(pkg, w, q, off, force_chunk=384)


def test_chunk_equals_decode_steps(pkg):
    """The last token of each sequence gets what the decode step gives it."""
    w, q, off = ragged(212, [700, 130, 64], [9, 1, 30], Hq=16, Hkv=4, D=128, PS=16)
    got, err = run(pkg, w, q, off)
    last = (off[1:] - 1).long()
    one = pkg.decode_attn(q[last].to(DEV), w.k_pages.to(DEV), w.v_pages.to(DEV),
                          w.page_table.to(DEV), w.seq_lens.to(DEV), w.scale)
    torch.cuda.synchronize()
    assert err == 0
    a, b = got[last.to(DEV)].double(), one.double()
    assert float((a - b).norm() / b.norm()) <= 2 * half_step(F16)


@pytest.mark.parametrize("D,force", [(64, 0), (128, 0), (256, 0), (128, 256)])
def test_chunk_unattended_values_never_matter(pkg, D, force):
    """NaN and Inf everywhere a token must not look: pages of no sequence,
    positions past the length, before the window, and later tokens' rows."""
    lens, news, window = [333, 290], [40, 290], 70
    w, q, off = ragged(220, lens, news, Hq=8, Hkv=2, D=D, PS=32, dtype=BF16)
    clean, err = run(pkg, w, q, off, window, force_chunk=force)
    assert err == 0
    used = torch.zeros(w.k_pages.shape[:2], dtype=torch.bool)
    for b, (L, n) in enumerate(zip(lens, news)):
        for t in range(max(0, L - n + 1 - window), L):
            used[w.page_table[b, t // 32], t % 32] = True
    w.k_pages[~used] = float("nan")
    w.v_pages[~used] = float("inf")
    again, err = run(pkg, w, q, off, window, force_chunk=force)
    assert err == 0 and torch.equal(clean, again)
    # a later token's rows: what comes before it does not change
    for b, t in ((0, 310), (0, 332), (1, 150)):
        page, slot = int(w.page_table[b, t // 32]), t % 32
        w.k_pages[page, slot, 0] = float("nan")
        w.v_pages[page, slot, 1, 3] = float("inf")
        w.v_pages[page, slot, 1, 5] = float("nan")
    spoilt, err = run(pkg, w, q, off, window, force_chunk=force)
    assert err == 0
    G = 4
    for b, bad in ((0, [310, 332]), (1, [150])):
        for i in range(news[b]):
            p = lens[b] - news[b] + i
            hit = any(t <= p and t > p - window for t in bad)
            row, was = spoilt[int(off[b]) + i], clean[int(off[b]) + i]
            if not hit:
                assert torch.equal(row, was), (b, i)
            else:
                assert torch.isnan(row[:G]).all(), (b, i)  # K of head 0
                assert torch.isinf(row[G:, 3]).all() and torch.isnan(row[G:, 5]).all(), (b, i)
                keep = [d for d in range(D) if d not in (3, 5)]
                assert torch.equal(row[G:, keep], was[G:, keep]), (b, i)


def test_chunk_rows_of_no_sequence_stay(pkg):
    w, q, off = ragged(230, [100, 60], [7, 60], Hq=8, Hkv=2, D=128, PS=16)
    total = int(off[-1])
    q = torch.cat([q, torch.full((5, 8, 128), float("nan"), dtype=q.dtype)])
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    got, err = run(pkg, w, q, off, out=out)
    ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, w.seq_lens, w.scale)
    assert err == 0 and torch.all(got[total:] == 7.0)
    assert_rows(got[:total], ref[:total], mass[:total], F16,
                half_step(F16) + weight_error(128, score_size(q[:total], w.k_pages, w.scale)))


def test_chunk_tokens_before_position_zero(pkg):
    """More new tokens than positions: the first ones get zero rows."""
    w, q, off = ragged(231, [5, 40], [9, 40], Hq=8, Hkv=2, D=128, PS=16)
    got = check(pkg, w, q, off)
    assert torch.all(got[:4] == 0) and bool((got[4:] != 0).any())


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 48, 47, 39])
def test_chunk_windows_beyond_every_position(pkg, window):
    """Windows as long as the table (48 positions here) and longer attend
    everything, also where tokens before position 0 come with them."""
    w, q, off = ragged(233, [5, 40], [9, 40], Hq=8, Hkv=2, D=128, PS=16, max_pages=3)
    got = check(pkg, w, q, off, window)
    assert torch.all(got[:4] == 0) and bool((got[4:] != 0).any())


@pytest.mark.parametrize("force", [0, 128])
def test_chunk_bad_lengths_and_pages(pkg, force):
    lens = torch.tensor([300, -1, 5000, 300], dtype=torch.int32)
    w, q, off = ragged(232, [300, 50, 50, 300], [20, 10, 10, 100], Hq=8, Hkv=2, D=128, PS=16)
    table = w.page_table.clone()
    table[3, 15] = w.k_pages.shape[0]  # positions 240..255 of the last sequence
    got, err = run(pkg, w, q, off, lens=lens, table=table, force_chunk=force)
    assert err == pkg.DEV_BAD_LEN | pkg.DEV_BAD_PAGE
    assert torch.all(got[20:40] == 0)
    ref, mass = chunk_attention(q, w.k_pages, w.v_pages, w.page_table, off, [300, 0, 0, 300],
                                w.scale)
    weight = half_step(F16) + weight_error(128, score_size(q, w.k_pages, w.scale))
    assert_rows(got[:20], ref[:20], mass[:20], F16, weight)
    # the tokens at 200..239 do not attend the bad page, those from 240 on do
    assert_rows(got[40:80], ref[40:80], mass[40:80], F16, weight)
    assert torch.all(got[80:] == 0)


@pytest.mark.parametrize("offsets", [[0, 20, 10, 30], [0, 10, 20, 31], [-5, 10, 20, 30]])
def test_chunk_bad_offsets_are_reported(pkg, offsets):
    w, q, _ = ragged(233, [300, 50, 50], [10, 10, 10], Hq=8, Hkv=2, D=128, PS=16)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    _, err = run(pkg, w, q, torch.tensor(offsets, dtype=torch.int32), out=out)
    assert err & pkg.DEV_BAD_LEN


@pytest.mark.parametrize("force", [0, 256])
def test_chunk_same_bits_every_run(pkg, force):
    w, q, off = ragged(234, [3000, 777], [130, 64], Hq=32, Hkv=8, D=128, PS=16, dtype=BF16)
    a, _ = run(pkg, w, q, off, force_chunk=force)
    for _ in range(3):
        b, _ = run(pkg, w, q, off, force_chunk=force)
        assert torch.equal(a, b)


def test_chunk_max_seq_len_only_steers(pkg):
    w, q, off = ragged(235, [1500, 20], [10, 10], Hq=8, Hkv=2, D=128, PS=16)
    for bound in (1, 64, 700, 1500, 100000):
        check(pkg, w, q, off, max_seq_len=bound)


def test_chunk_long_context_rows(pkg):
    """131072 positions, the first and last rows of a chunk of 40."""
    L, n = 131072, 40
    w, q, off = ragged(236, [L], [n], Hq=8, Hkv=1, D=128, PS=64, dtype=BF16)
    got, err = run(pkg, w, q, off, max_seq_len=L)
    assert err == 0
    for i in (0, n - 1):
        end = L - n + 1 + i
        ref, mass = chunk_attention(q[i:i + 1], w.k_pages, w.v_pages, w.page_table,
                                    torch.tensor([0, 1]), [end], w.scale)
        assert_rows(got[i:i + 1], ref, mass, BF16,
                    half_step(BF16) + weight_error(128, score_size(q, w.k_pages, w.scale)))


def test_chunk_many_sequences(pkg):
    """Over a thousand sequences, some without a token: three search steps."""
    g = torch.Generator().manual_seed(1)
    news = torch.randint(0, 4, (1100,), generator=g).tolist()
    lens = [max(n, int(x)) for n, x in zip(news, torch.randint(0, 40, (1100,), generator=g))]
    w, q, off = ragged(237, lens, news, Hq=2, Hkv=1, D=64, PS=8)
    check(pkg, w, q, off)


def test_chunk_empty_calls(pkg):
    w, q, off = ragged(238, [30], [4], Hq=8, Hkv=2, D=128, PS=16)
    got, err = run(pkg, w, q[:0], torch.zeros(2, dtype=torch.int32))
    assert err == 0 and got.shape[0] == 0
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    got, err = run(pkg, w, q, torch.zeros(2, dtype=torch.int32), out=out)
    assert err == 0 and torch.all(got == 7.0)


def test_chunk_two_streams_and_graphs(pkg):
    """Calls on two streams at once, and two captured graphs replayed side by
    side: neither shares a workspace with the other."""
    sets = []
    for seed in (240, 241):
        w, q, off = ragged(seed, [4000, 900], [6, 3], Hq=32, Hkv=8, D=128, PS=16)
        d = [q.to(DEV), w.k_pages.to(DEV), w.v_pages.to(DEV), w.page_table.to(DEV), off.to(DEV),
             w.seq_lens.to(DEV)]
        sets.append((d, w.scale, pkg.decode_attn_chunk(*d, w.scale, max_seq_len=4000)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in sets]
    outs = []
    for _ in range(20):
        for st, (d, scale, _) in zip(streams, sets):
            outs.append(pkg.decode_attn_chunk(*d, scale, max_seq_len=4000, stream=st))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, sets[i % 2][2])
    graphs = []
    for d, scale, _ in sets:
        out = torch.empty_like(d[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkg.decode_attn_chunk(*d, scale, max_seq_len=4000, out=out)
        graphs.append((g, out))
    for _ in range(20):
        for st, (g, out) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_, out), (_, _, ref) in zip(graphs, sets):
        assert torch.equal(out, ref)


def test_chunk_stalled_wait_reports_and_recovers(pkg):
    """A load whose bytes never all arrive (the library's test hook): the
    bounded waits give up, the rows are zero, and the next call is right."""
    w, q, off = ragged(242, [300], [20], Hq=8, Hkv=2, D=128, PS=16)
    want, _ = run(pkg, w, q, off)
    os.environ["DECODE_ATTN_TEST_STALL_TX"] = "64"
    try:
        got, err = run(pkg, w, q, off)
    finally:
        del os.environ["DECODE_ATTN_TEST_STALL_TX"]
    assert err & pkg.DEV_TIMEOUT and torch.all(got == 0)
    got, err = run(pkg, w, q, off)
    assert err == 0 and torch.equal(got, want)
