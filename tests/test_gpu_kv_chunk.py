"""decode_kv_append_chunk and decode_kv_read: rows into the paged cache and
back, 16-bit and e4m3.  Both are defined to the bit (a copy; a power-of-two
scale and the nearest code; code * scale rounded once), so every comparison
is of bits."""
import pytest
import torch

from paged_gqa_decode_06_gb300 import workloads
from tests.chunk_reference import quantise

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_gqa_decode_06_gb300 import build
    build.build()
    import paged_gqa_decode_06_gb300 as p
    p.load_library()
    return p


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def pools(seed, lens, Hkv, D, PS, dtype, decoys=3):
    """(pools and scales, table): random content, 16-bit or e4m3."""
    w = workloads.make_custom("kv", batch=len(lens), num_q_heads=Hkv, num_kv_heads=Hkv,
                              head_dim=D, page_size=PS, seq_lens=lens, seed=seed,
                              decoy_pages=decoys, dtype=F16 if dtype == E4M3 else dtype)
    if dtype != E4M3:
        return {"k_pages": w.k_pages, "v_pages": w.v_pages}, w.page_table
    d = {}
    for n in ("k", "v"):
        code, scale = quantise(getattr(w, n + "_pages"))
        d[n + "_pages"], d[n + "_scales"] = code, scale.transpose(1, 2).contiguous()
    return d, w.page_table


def new_rows(seed, total, Hkv, D, dtype):
    """Rows of very different magnitudes, some of them zero."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        x = torch.randn((total, Hkv, D), generator=g)
        x = x * torch.exp2(torch.randint(-14, 12, (total, Hkv, 1), generator=g).float())
        if total:
            x[torch.randint(0, total, (1 + total // 9,), generator=g), 0] = 0.0
        out.append(x.to(dtype))
    return out


def offsets(news):
    return torch.tensor([0] + list(torch.tensor(news).cumsum(0)), dtype=torch.int32)


def expect_append(d, table, k_new, v_new, off, lens, PS):
    want = {n: t.clone() for n, t in d.items()}
    capacity = table.shape[1] * PS
    for b, L in enumerate(lens):
        a, z = int(off[b]), int(off[b + 1])
        for r in range(a, z):
            pos = int(L) - (z - a) + (r - a)
            if pos < 0 or pos >= capacity or L > capacity:
                continue
            page, slot = int(table[b, pos // PS]), pos % PS
            if not 0 <= page < d["k_pages"].shape[0]:
                continue
            for n, new in (("k", k_new), ("v", v_new)):
                if n + "_scales" in want:
                    code, scale = quantise(new[r])
                    bits(want[n + "_pages"])[page, slot] = bits(code)
                    want[n + "_scales"][page, :, slot] = scale
                else:
                    want[n + "_pages"][page, slot] = new[r]
    return want


def run_append(pkg, d, table, k_new, v_new, off, lens, **kw):
    g = {n: t.to(DEV) for n, t in d.items()}
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkg.decode_kv_append_chunk(k_new.to(DEV), v_new.to(DEV), off.to(DEV),
                               torch.as_tensor(lens, dtype=torch.int32).to(DEV), g["k_pages"],
                               g["v_pages"], table.to(DEV), k_scales=g.get("k_scales"),
                               v_scales=g.get("v_scales"), err_flag=err, **kw)
    torch.cuda.synchronize()
    return {n: t.cpu() for n, t in g.items()}, int(err.item())


APPEND = [
    ([1], [1], 1, 64, 8),
    ([16, 5, 33], [1, 1, 1], 2, 128, 16),
    ([100, 0, 64, 31], [100, 0, 3, 31], 4, 128, 16),
    ([700, 650, 3], [513, 1, 3], 8, 128, 64),
    ([90, 300], [90, 299], 3, 64, 32),
    ([90, 300], [17, 255], 5, 256, 256),
    ([2000, 1900], [1700, 1900], 1, 64, 128),
]


@pytest.mark.parametrize("new_dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("quant", [False, True], ids=["copy", "e4m3"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_chunk_to_the_bit(pkg, case, quant, new_dtype):
    lens, news, Hkv, D, PS = APPEND[case]
    d, table = pools(300 + case, lens, Hkv, D, PS, E4M3 if quant else new_dtype)
    off = offsets(news)
    k, v = new_rows(301 + case, int(off[-1]), Hkv, D, new_dtype)
    want = expect_append(d, table, k, v, off, lens, PS)
    got, err = run_append(pkg, d, table, k, v, off, lens)
    assert err == 0
    for n in want:
        assert torch.equal(bits(got[n]), bits(want[n])), n


@pytest.mark.parametrize("quant", [False, True], ids=["copy", "e4m3"])
def test_append_chunk_refused_rows_write_nothing(pkg, quant):
    """Rows before position 0, past the table, in a page outside the pool, of
    a sequence with a negative length, and rows that no sequence owns."""
    lens, news = [4, 200, 60, -3, 40], [6, 3, 20, 2, 10]
    d, table = pools(320, [4, 80, 60, 8, 40], 2, 128, 16, E4M3 if quant else F16)
    table = table.clone()
    table[2, 3] = -7
    off = offsets(news)
    k, v = new_rows(321, int(off[-1]) + 4, 2, 128, F16)
    want = expect_append(d, table, k, v, off, [4, 200, 60, -3, 40], 16)
    got, err = run_append(pkg, d, table, k, v, off, lens)
    assert err == pkg.DEV_BAD_LEN | pkg.DEV_BAD_PAGE
    for n in want:
        assert torch.equal(bits(got[n]), bits(want[n])), n


@pytest.mark.parametrize("off", [[0, 8, 9, 10, 2, 20], [0, 8, 9, 2, 3, 20], [3, 9, 9, 12, 1, 20],
                                 [0, 30, 5, 6, 7, 20], [-4, 4, 8, 12, 16, 20]])
def test_append_with_offsets_that_do_not_ascend(pkg, off):
    """Reported, and nothing is written but the rows of the sequences whose own
    offsets ascend, at their own positions."""
    lens, PS = [40, 50, 60, 70, 40], 16
    d, table = pools(325, lens, 2, 64, PS, E4M3)
    k, v = new_rows(326, 20, 2, 64, F16)
    mine = torch.zeros(d["k_pages"].shape[:2], dtype=torch.bool)
    for b, L in enumerate(lens):
        if 0 <= off[b] <= off[b + 1] <= 20:
            for pos in range(max(0, L - (off[b + 1] - off[b])), L):
                mine[table[b, pos // PS], pos % PS] = True
    got, err = run_append(pkg, d, table, k, v, torch.tensor(off, dtype=torch.int32), lens)
    assert err == pkg.DEV_BAD_LEN
    for n in d:
        x, y = bits(got[n]), bits(d[n])
        if n.endswith("_scales"):
            x, y = x.transpose(1, 2), y.transpose(1, 2)
        assert torch.equal(x[~mine], y[~mine]), n


def test_append_quantises_the_edges(pkg):
    """Rows at the scale's border (448 times a power of two and its
    neighbours), the smallest and largest magnitudes, ties, NaN and Inf."""
    D = 64
    x = torch.zeros((12, 1, D))
    x[0, 0, 0] = 448.0
    x[1, 0, 0] = 448.25
    x[2, 0, 0] = 447.75
    x[3, 0, :] = torch.linspace(-1, 1, D)
    x[4, 0, 0] = 65504.0
    x[5, 0, 0] = 2.0 ** -24
    x[6, 0, :4] = torch.tensor([448.0, 17.0, 19.0, -21.0])  # ties between codes of step 2
    x[7, 0, :3] = torch.tensor([448.0, 2.0 ** -10, 3 * 2.0 ** -10])  # below the smallest code
    x[8, 0, :2] = torch.tensor([1.0, float("nan")])
    x[9, 0, :2] = torch.tensor([float("inf"), 1.0])
    x[10, 0, 0] = 0.875
    x[11, 0, 0] = 0.8755
    k = x.half()
    lens, off = [12], offsets([12])
    d, table = pools(330, lens, 1, D, 16, E4M3)
    got, err = run_append(pkg, d, table, k, k, off, lens)
    assert err == 0
    page = int(table[0, 0])
    code, scale = got["k_pages"][page, :12, 0].float(), got["k_scales"][page, 0, :12]
    # (an Inf takes the scale of the largest 32-bit number, 2^128 (1 - 2^-24) <=
    # 448 * 2^120, so that it reads back as Inf)
    want_scale = [1, 2, 1, 2.0 ** -8, 256, 2.0 ** -32, 1, 1, 2.0 ** -8, 2.0 ** 120, 2.0 ** -9,
                  2.0 ** -8]
    assert scale.tolist() == want_scale
    assert code[6, :4].tolist() == [448.0, 16.0, 20.0, -20.0]
    assert code[7, :3].tolist() == [448.0, 0.0, 2.0 ** -8]  # 2^-10 is a tie with 0, 3 with 2^-8
    assert code[8, 0] == 256.0 and torch.isnan(code[8, 1])
    assert code[9, 0] == 448.0
    for i in (0, 1, 2, 3, 4, 5, 10, 11):
        ref, s = quantise(k[i])
        assert torch.equal(bits(got["k_pages"][page, i]), bits(ref)) and float(s) == float(scale[i])
    # bf16 reaches beyond: tiny rows are zeros with scale 0, huge ones finite codes
    b = torch.zeros((3, 1, D), dtype=BF16)
    b[0, 0, 0], b[1, 0, 0], b[2, 0, 0] = 2.0 ** -101, 2.0 ** -100, 2.0 ** 127
    got, err = run_append(pkg, d, table, b, b, offsets([3]), [3])
    assert err == 0
    assert got["k_scales"][page, 0, :3].tolist() == [0.0, 2.0 ** -108, 2.0 ** 119]
    assert got["k_pages"][page, :3, 0, 0].float().tolist() == [0.0, 256.0, 256.0]


def expect_read(d, table, off, starts, total, dtype, PS, fill):
    outs = []
    P, capacity = d["k_pages"].shape[0], table.shape[1] * PS
    for n in ("k", "v"):
        out = torch.full((total, *d["k_pages"].shape[2:]), fill, dtype=dtype)
        for b in range(table.shape[0]):
            a, z = int(off[b]), int(off[b + 1])
            for r in range(a, z):
                pos = int(starts[b]) + r - a
                page = int(table[b, pos // PS]) if 0 <= pos < capacity else -1
                if not 0 <= page < P:
                    out[r] = 0
                    continue
                x = d[n + "_pages"][page, pos % PS]
                if n + "_scales" in d:
                    x = x.float() * d[n + "_scales"][page, :, pos % PS][:, None]
                out[r] = x.to(dtype)
        outs.append(out)
    return outs


READ = [
    ([1], [0], [1], 1, 64, 8),
    ([100, 64, 31], [0, 60, 30], [100, 4, 1], 4, 128, 16),
    ([700, 650, 3], [1, 640, 0], [699, 10, 0], 8, 128, 64),
    ([90, 300], [0, 7], [90, 290], 3, 64, 32),
    ([600], [11], [500], 5, 256, 256),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("quant", [False, True], ids=["copy", "e4m3"])
@pytest.mark.parametrize("case", range(len(READ)))
def test_read_to_the_bit(pkg, case, quant, dtype):
    lens, starts, news, Hkv, D, PS = READ[case]
    d, table = pools(340 + case, lens, Hkv, D, PS, E4M3 if quant else dtype)
    if quant:  # any scale, not only the quantiser's powers of two
        g = torch.Generator().manual_seed(case)
        for n in ("k_scales", "v_scales"):
            d[n] = d[n] * (0.5 + torch.rand(d[n].shape, generator=g))
    off = offsets(news)
    total = int(off[-1]) + 3  # three rows that no sequence owns
    want = expect_read(d, table, off, starts, total, dtype, PS, 7.0)
    g = {n: t.to(DEV) for n, t in d.items()}
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = [torch.full(w.shape, 7.0, dtype=dtype, device=DEV) for w in want]
    got = pkg.decode_kv_read(g["k_pages"], g["v_pages"], table.to(DEV), off.to(DEV), total,
                             starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                             k_scales=g.get("k_scales"), v_scales=g.get("v_scales"), dtype=dtype,
                             k_out=outs[0], v_out=outs[1], err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for x, y in zip(got, want):
        assert torch.equal(bits(x.cpu()), bits(y))


def test_read_refused_rows_are_zero(pkg):
    lens = [80, 60, 40]
    d, table = pools(360, lens, 2, 128, 16, E4M3)
    table = table.clone()
    table[1, 1] = d["k_pages"].shape[0] + 5
    starts, off = [76, 10, -2], offsets([8, 20, 6])  # past the table, a bad page, before 0
    want = expect_read(d, table, off, starts, int(off[-1]), F16, 16, 0.0)
    g = {n: t.to(DEV) for n, t in d.items()}
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pkg.decode_kv_read(g["k_pages"], g["v_pages"], table.to(DEV), off.to(DEV), 34,
                             starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                             k_scales=g["k_scales"], v_scales=g["v_scales"], err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pkg.DEV_BAD_LEN | pkg.DEV_BAD_PAGE
    for x, y in zip(got, want):
        assert torch.equal(bits(x.cpu()), bits(y))


def test_rows_many_sequences(pkg):
    """Over a thousand sequences, many without a row."""
    g = torch.Generator().manual_seed(5)
    news = torch.randint(0, 3, (1300,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(news, torch.randint(0, 20, (1300,), generator=g))]
    d, table = pools(370, lens, 1, 64, 8, E4M3)
    off = offsets(news)
    k, v = new_rows(371, int(off[-1]), 1, 64, F16)
    want = expect_append(d, table, k, v, off, lens, 8)
    got, err = run_append(pkg, d, table, k, v, off, lens)
    assert err == 0
    for n in want:
        assert torch.equal(bits(got[n]), bits(want[n])), n


def test_append_in_a_captured_graph_and_on_another_stream(pkg):
    lens, news = [300, 90], [40, 90]
    d, table = pools(380, lens, 4, 128, 16, E4M3)
    off = offsets(news)
    k, v = new_rows(381, 130, 4, 128, BF16)
    want = expect_append(d, table, k, v, off, lens, 16)
    args = [k.to(DEV), v.to(DEV), off.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)]
    for captured in (False, True):
        g = {n: t.to(DEV) for n, t in d.items()}
        tail = (g["k_pages"], g["v_pages"], table.to(DEV), g["k_scales"], g["v_scales"])
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                pkg.decode_kv_append_chunk(*args, *tail)
            graph.replay()
        else:
            st = torch.cuda.Stream(DEV)
            st.wait_stream(torch.cuda.current_stream())
            pkg.decode_kv_append_chunk(*args, *tail, stream=st)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(bits(g[n].cpu()), bits(want[n])), (captured, n)
