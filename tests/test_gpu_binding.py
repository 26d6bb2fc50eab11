"""The two ways of the rotary and 4-bit calls (C++ and Python) on unusual arguments:
the same values, or the same refusal in the same words."""
import pytest
import torch

from tests.fp4_reference import rope_table
from tests.test_gpu_kv_rope import BF16, DEV, F16, NAMES, bits, new_rows, offsets, pkg, pools  # noqa: F401

pytestmark = pytest.mark.gpu


def outcome(f):
    try:
        r = f()
    except Exception as e:  # noqa: BLE001
        return type(e).__name__, str(e)
    torch.cuda.synchronize()
    r = r if isinstance(r, tuple) else (r,)
    return [None if t is None else (tuple(t.shape), t.stride(), t.dtype, bits(t.contiguous()).cpu())
            for t in r]


def agree(pkg, monkeypatch, calls):
    monkeypatch.setattr(pkg, "_quick_module", pkg._UNSET)
    assert pkg._quick() is not None
    quick = pkg._quick()
    for i, make in enumerate(calls):
        got = []
        for module in (quick, None):
            monkeypatch.setattr(pkg, "_quick_module", module)
            got.append(outcome(make()))
        a, b = got
        assert type(a) is type(b) and len(a) == len(b), (i, a, b)
        if isinstance(a, tuple):
            assert a == b, (i, a, b)
            continue
        for x, y in zip(a, b):
            assert (x is None) == (y is None), i
            if x is not None:
                assert x[:3] == y[:3] and torch.equal(x[3], y[3]), i


def test_rotations(pkg, monkeypatch):  # noqa: F811
    D, table = 64, rope_table(32, 50).to(DEV)
    wide = new_rows(1, 9, 12, D, F16).to(DEV)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)

    def call(x, out=None, p=pos, t=table, **kw):
        return lambda: lambda: pkg.decode_rope(x, p[:x.shape[0]] if p is pos else p, t,
                                               out=None if out is None else out(), **kw)

    flat = wide.flatten()
    calls = [call(x) for x in (
        wide, wide[:, 2:5], wide[:1], wide[:1, 2:5], wide[:0], wide[:0, 3:], wide[:, :0],
        wide[:, 5:6], wide[:, ::2], wide[..., :32], wide[..., ::2], wide[::2], wide[:1].expand(9, 12, D),
        wide.transpose(0, 1), wide[:, :, None].squeeze(2), flat[8:8 + 6 * 2 * D].view(6, 2, D),
        flat[4:4 + 6 * 2 * D].view(6, 2, D), flat.as_strided((6, 3, D), (196, D, 1)),
        flat.as_strided((6, 3, D), (200, D, 1)), flat.as_strided((1, 3, D), (7, D, 1)),
        flat.as_strided((6, 1, D), (72, 3, 1)), flat.as_strided((6, 3, D), (128, D, 1)),
        wide[0], wide.float(), wide.cpu(), wide.bfloat16(), wide[..., :48].contiguous(),
        wide[..., :24].contiguous(), torch.nn.Parameter(wide, requires_grad=False))]
    calls += [call(wide, lambda o=o: o()) for o in (
        lambda: torch.zeros_like(wide), lambda: torch.zeros(9, 20, D, device=DEV).half()[:, 4:16],
        lambda: torch.zeros(9, 12, 2 * D, device=DEV).half()[..., :D],
        lambda: torch.zeros(8, 12, D, device=DEV).half(), lambda: torch.zeros_like(wide).bfloat16(),
        lambda: torch.zeros(9, 12, D).half(), lambda: wide[:1].expand(9, 12, D),
        lambda: wide.clone())]
    calls += [call(wide, p=p) for p in (
        pos.long(), pos[:4], pos[:, None], pos.cpu(), torch.zeros(18, device=DEV).int()[::2],
        pos + 45, None)]
    calls += [call(wide, t=t) for t in (
        table[:0], table[0], table.double(), table.t(), table.cpu(), rope_table(80, 50).to(DEV),
        table[:, :16], table[:, :24].contiguous(), None)]
    calls += [call(wide, **kw) for kw in (
        dict(interleaved=1), dict(interleaved=True, backward=True), dict(backward=None),
        dict(err_flag=torch.zeros(1, device=DEV)), dict(err_flag=torch.zeros(1).int()))]
    agree(pkg, monkeypatch, calls)


@pytest.mark.parametrize("fmt", ["16", "fp8", "fp4"])
def test_appends(pkg, monkeypatch, fmt):  # noqa: F811
    Hkv, D, PS = 2, 64, 16
    d, table = pools(2, [40, 33], Hkv, D, PS, fmt, F16)
    wide = new_rows(3, 10, 12, D, F16).to(DEV)
    off, L = offsets([9, 1]).to(DEV), torch.tensor([40, 33], dtype=torch.int32, device=DEV)
    base = dict(k_new=wide[:, 8:10], v_new=wide[:, 10:], row_offsets=off, seq_lens=L,
                page_table=table.to(DEV), table=rope_table(48, 50).to(DEV), q=wide[:, :8])

    def call(**kw):
        def fresh():
            c = {n: t.to(DEV) for n, t in d.items()}
            args = {**base, **c, **{k: v(c) if callable(v) else v for k, v in kw.items()}}

            def run():
                out = pkg.decode_kv_append_rope(**args)
                return (out, *[args[n] for n in c])
            return run
        return fresh

    calls = [call(), call(q=None), call(q=None, q_out=lambda c: wide[:, :8].clone()),
             call(q=wide[:, :7].contiguous()), call(q=wide[:, :0]), call(q=wide[:9, :8]),
             call(q=wide[:, :8].bfloat16()), call(q_out=lambda c: torch.zeros_like(wide)),
             call(q_out=lambda c: torch.zeros_like(wide)[:, 2:10]),
             call(q_out=lambda c: torch.zeros(10, 8, D, device=DEV)),
             call(k_new=wide[:, 8:11]), call(v_new=wide[:9, 10:]), call(k_new=wide[:, 8::2]),
             call(k_new=wide[:, 8:10].cpu()), call(k_new=wide[:, 8:10].bfloat16()),
             call(k_new=wide[:, 8:10].bfloat16(), v_new=wide[:, 10:].bfloat16(), q=None),
             call(k_new=wide[:0, 8:10], v_new=wide[:0, 10:], q=None, row_offsets=off * 0),
             call(k_new=wide[:0, 8:10], v_new=wide[:0, 10:], q=wide[:0, :8], row_offsets=off * 0),
             call(seq_lens=L[:1]), call(seq_lens=L.long()), call(seq_lens=None),
             call(row_offsets=off[:2]), call(row_offsets=off.cpu()), call(row_offsets=off * 3),
             call(page_table=table.to(DEV)[0]), call(page_table=table.to(DEV).t()),
             call(page_table=table.to(DEV)[:1]), call(table=rope_table(80, 50).to(DEV)),
             call(table=rope_table(48, 20).to(DEV)), call(interleaved=True), call(interleaved=1),
             call(err_flag=torch.zeros(1, device=DEV)), call(v_pages=lambda c: c["v_pages"][:-1]),
             call(k_pages=lambda c: c["k_pages"].transpose(0, 1)),
             call(k_pages=lambda c: c["k_pages"].cpu())]
    for n in NAMES[2:]:
        calls += [call(**{n: None}), call(**{n: torch.zeros(3, device=DEV)})]
    agree(pkg, monkeypatch, calls)


def test_4_bit_reads_and_steps(pkg, monkeypatch):  # noqa: F811
    Hkv, D, PS = 2, 64, 16
    d, table = pools(4, [40, 33], Hkv, D, PS, "fp4", F16)
    c, tb = [d[n].to(DEV) for n in NAMES], table.to(DEV)
    off, L = offsets([40, 33]).to(DEV), torch.tensor([40, 33], dtype=torch.int32, device=DEV)
    q = new_rows(5, 2, 8, D, F16).to(DEV)
    packed = [c[0].view(torch.float4_e2m1fn_x2), c[1].view(torch.float4_e2m1fn_x2), *c[2:]]

    def read(cache=c, t=tb, o=off, n=73, **kw):
        return lambda: lambda: pkg.decode_kv_read_fp4(*cache, t, o, n, **kw)

    new = torch.zeros(73, Hkv, D, device=DEV)
    agree(pkg, monkeypatch, [
        read(), read(packed), read(n=0, o=off * 0), read(dtype=BF16), read(dtype=torch.float32),
        read(k_out=new.half()), read(v_out=new.bfloat16()), read(k_out=new),
        read(k_out=new.half(), v_out=new.bfloat16()), read(k_out=new.half(), dtype=BF16),
        read(k_out=new.half()[:5]), read(starts=L * 0 + 1), read(starts=L.long()),
        read(starts=L[:1]), read(o=off[:2]), read(t=tb[0]), read([c[0], packed[1], *c[2:]]),
        read([*c[:5], c[5][..., :2]]), read([*c[:4], c[4].view(torch.uint8), c[5]]),
        read([c[0].cpu(), *c[1:]]), read([None, *c[1:]])])

    def step(x=q, cache=c, t=tb, lens=L, scale=0.1, **kw):
        return lambda: lambda: pkg.decode_attn_fp4(x, *cache, t, lens, scale, **kw)

    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    agree(pkg, monkeypatch, [
        step(), step(cache=packed), step(scale=1), step(q[:, None]), step(q[:0], t=tb[:0], lens=L[:0]),
        step(q.bfloat16()), step(q.float()), step(q[0]), step(q[..., ::2]), step(q[:, :7]),
        step(q[:, :7].contiguous()), step(lens=L[:1]), step(lens=None), step(t=tb[:1]),
        step(scale=float("nan")), step(window=20), step(window=-3), step(max_seq_len=40),
        step(max_seq_len=20), step(out=torch.empty_like(q)), step(out=torch.empty_like(q)[:1]),
        step(out=torch.empty_like(q).bfloat16()), step(workspace=ws, force_chunk=64),
        step(workspace=ws[:64], force_chunk=64, schedule=1), step(workspace=ws.cpu(), force_chunk=64),
        step(workspace=ws[::2], force_chunk=64), step(force_chunk=1 << 20), step(schedule=7),
        step(q.repeat(1, 17, 1)), step(cache=[*c[:3], c[3].half(), *c[4:]])])
