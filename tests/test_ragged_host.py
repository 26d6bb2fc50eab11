"""Host-side checks of the ragged and 8-bit entry points (no GPU needed):
arguments refused before any CUDA call, the planners' contracts, the binding's
refusals and struct mirror."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 152


@pytest.fixture(scope="module")
def pkg():
    from paged_gqa_decode_06_gb300 import build
    build.build()
    import paged_gqa_decode_06_gb300 as p
    p.load_library()
    return p


def params(pkg, **kw):
    base = dict(batch=4, num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16,
                max_pages_per_seq=192, num_pages=256, max_seq_len=3060, scale=0.088,
                num_queries=1)
    base.update(kw)
    return pkg.DecodeAttnParams(**base)


def calls(pkg, p, ptr=None, total=8, fmt=1, ws=None, ws_bytes=0):
    """Each entry point with every pointer `ptr`: {name: status}."""
    lib, r = pkg.load_library(), ctypes.byref(p) if p is not None else None
    return {
        "chunk": lib.decode_attn_chunk(r, total, *[ptr] * 7, ws, ws_bytes, None, None),
        "append": lib.decode_kv_append_chunk(r, fmt, total, *[ptr] * 9, None, None),
        "read": lib.decode_kv_read(r, fmt, total, *[ptr] * 9, None, None),
        "quant": lib.decode_attn_quant(r, fmt, *[ptr] * 8, ws, ws_bytes, None, None),
    }


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 96, -3), ("page_size", 24, -4), ("num_q_heads", 30, -2), ("num_kv_heads", 0, -2),
    ("batch", -1, -2), ("batch", 65536, -2), ("max_pages_per_seq", 0, -2), ("num_pages", 0, -2),
    ("scale", float("nan"), -2), ("num_q_heads", 8 * 32, -5), ("dtype", 2, -2),
    ("num_pages", 1 << 28, -2),
])
def test_bad_params(pkg, field, value, code):
    for name, st in calls(pkg, params(pkg, **{field: value})).items():
        assert st == code, name


def test_null_and_misaligned_pointers(pkg):
    for name, st in calls(pkg, None).items():
        assert st == -1, name
    for name, st in calls(pkg, params(pkg)).items():
        assert st == -1, name
    for name, st in calls(pkg, params(pkg), ptr=4096 + 8).items():
        assert st == -7, name


def test_negative_totals_and_formats(pkg):
    got = calls(pkg, params(pkg), total=-1)
    assert got["chunk"] == got["append"] == got["read"] == -2
    got = calls(pkg, params(pkg), fmt=7)
    assert got["append"] == got["read"] == got["quant"] == -2
    assert calls(pkg, params(pkg), fmt=0)["quant"] == -2  # a 16-bit pool: decode_attn's


def test_empty_calls_need_no_device(pkg):
    got = calls(pkg, params(pkg), total=0)
    assert got["chunk"] == got["append"] == got["read"] == 0
    got = calls(pkg, params(pkg, batch=0))
    assert got["chunk"] == got["append"] == got["read"] == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (8, 8), (12, 4), (14, 2), (16, 1), (40, 8)])
@pytest.mark.parametrize("total", [1, 4, 100, 8192, 200000])
def test_chunk_plan(pkg, D, Hq, Hkv, total):
    G = Hq // Hkv
    for B, max_len, window in ((1, 3060, 0), (4, 130000, 0), (64, 8192, 0), (3, 4099, 1024),
                               (4, 0, 0)):
        p = params(pkg, batch=B, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, window=window,
                   max_pages_per_seq=16384, num_pages=40000, max_seq_len=max_len)
        plan = pkg.decode_attn_chunk_make_plan(p, total, SMS)
        assert plan.tile_tokens == 128 // G and plan.tile_tokens * G <= 128
        assert plan.item_tokens == plan.tile_tokens * (1 if D == 256 else 2)
        # slots cover any way of cutting `total` into B sequences
        assert plan.slots >= total // plan.item_tokens + min(B, total)
        assert 1 <= plan.max_shards <= 128
        assert plan.shard_keys % (64 if D == 256 else 128) == 0
        span = min(max_len or 262144, 262144)
        if window:
            span = min(span, window + plan.item_tokens)
        assert plan.shard_keys * plan.max_shards >= span
        assert plan.grid == plan.slots * plan.max_shards * Hkv
        if plan.max_shards == 1:
            assert plan.workspace_bytes == 0
        else:
            rows = total * Hq * plan.max_shards
            assert plan.workspace_bytes >= 65536 + rows * 8 + rows * D * 4
            assert rows * D * 4 <= 1 << 29


def test_chunk_plan_splits_when_sms_are_idle(pkg):
    one = params(pkg, batch=1, max_seq_len=3060)
    assert pkg.decode_attn_chunk_make_plan(one, 16, SMS).max_shards > 4
    # a long prompt fills the SMs with its own tiles
    prompt = params(pkg, batch=1, max_pages_per_seq=512, num_pages=512, max_seq_len=8192)
    assert pkg.decode_attn_chunk_make_plan(prompt, 8192, SMS).max_shards == 1
    forced = params(pkg, batch=1, max_seq_len=3060, force_chunk=1000)
    plan = pkg.decode_attn_chunk_make_plan(forced, 16, SMS)
    assert plan.max_shards == 3 and plan.shard_keys == 1024


def test_chunk_plan_refusals(pkg):
    lib, plan = pkg.load_library(), pkg.DecodeAttnChunkPlan()
    r = ctypes.byref(params(pkg))
    assert lib.decode_attn_chunk_make_plan(r, 8, SMS, None) == -1
    assert lib.decode_attn_chunk_make_plan(r, 8, 0, ctypes.byref(plan)) == -2
    assert lib.decode_attn_chunk_make_plan(r, -8, SMS, ctypes.byref(plan)) == -2
    with pytest.raises(pkg.DecodeAttnError):
        pkg.decode_attn_chunk_make_plan(params(pkg, head_dim=32), 8, SMS)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_quant_plan(pkg, D):
    for B, L, window in ((1, 3060, 0), (64, 8192, 0), (4, 131072, 0), (1000, 512, 0), (1, 200, 0),
                         (4, 131072, 4096), (1, 131072, 0)):
        p = params(pkg, batch=B, head_dim=D, max_pages_per_seq=8192, num_pages=40000,
                   max_seq_len=L, window=window)
        plan = pkg.decode_attn_quant_make_plan(p, SMS)
        span = L if not window else min(L, window) + 63
        assert plan.variant == pkg.VARIANT_MMA and plan.chunk_tokens % 64 == 0
        assert plan.chunk_tokens * plan.max_shards >= span
        assert plan.split == (1 if plan.max_shards > 1 else 0)
        assert plan.cluster in (0, plan.max_shards) and plan.cluster <= 16
        # one or two KV heads per CTA, and the ring of its CTAs fits an SM
        assert plan.grid_x * plan.grid_y in (plan.max_shards * 8, plan.max_shards * 4)
        assert plan.grid_z == B and plan.ring_stages * 128 * D * plan.ctas_per_sm <= 192 * 1024
        assert (plan.workspace_bytes > 0) == bool(plan.split)
    short = pkg.decode_attn_quant_make_plan(params(pkg, max_seq_len=256, head_dim=D), SMS)
    assert short.split == 0 and short.workspace_bytes == 0


@pytest.mark.parametrize("kw,code", [
    (dict(num_queries=5), -10), (dict(variant=1), -10), (dict(schedule=2, max_seq_len=100), -10),
    (dict(schedule=3), -2), (dict(force_chunk=1 << 20), -2),
])
def test_quant_plan_refusals(pkg, kw, code):
    lib, plan = pkg.load_library(), pkg.DecodeAttnPlan()
    p = params(pkg, **kw)
    assert lib.decode_attn_quant_make_plan(ctypes.byref(p), 1, SMS, ctypes.byref(plan)) == code


def test_chunk_plan_struct_matches_the_header(pkg, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    cls = pkg.DecodeAttnChunkPlan
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "decode_attn.h"',
           'int main(void) {', '  printf("%zu\\n", sizeof(decode_attn_chunk_plan));']
    src += [f'  printf("%zu\\n", offsetof(decode_attn_chunk_plan, {n}));' for n, _ in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(src + ["  return 0;", "}"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"),
                    str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout
    assert [int(x) for x in got.split()] == [ctypes.sizeof(cls)] + [
        getattr(cls, n).offset for n, _ in cls._fields_]


def tensors():
    z = torch.zeros
    return dict(q=z(5, 8, 64).half(), k=z(4, 16, 2, 64).half(), t=z(2, 2, dtype=torch.int32),
                off=z(3, dtype=torch.int32), lens=z(2, dtype=torch.int32),
                codes=z(4, 16, 2, 64).to(torch.float8_e4m3fn), s=z(4, 2, 16),
                rows=z(5, 2, 64).half())


def test_binding_refuses_host_tensors(pkg):
    x = tensors()
    with pytest.raises(ValueError, match="CUDA"):
        pkg.decode_attn_chunk(x["q"], x["k"], x["k"], x["t"], x["off"], x["lens"], 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.decode_kv_append_chunk(x["rows"], x["rows"], x["off"], x["lens"], x["k"], x["k"],
                                   x["t"])
    with pytest.raises(ValueError, match="CUDA"):
        pkg.decode_kv_read(x["k"], x["k"], x["t"], x["off"], 5)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.decode_attn_quant(x["q"][:2], x["codes"], x["codes"], x["s"], x["s"], x["t"],
                              x["lens"], 1.0)


def test_binding_checks_pools_and_scales(pkg):
    x, dev = tensors(), -1  # the index of a CPU tensor
    assert pkg._kv_pools(x["k"], x["k"], None, None, dev) == pkg.KV_16BIT
    assert pkg._kv_pools(x["codes"], x["codes"], x["s"], x["s"], dev) == pkg.KV_E4M3
    for bad, exc in (((x["k"], x["k"], x["s"], None), ValueError),
                     ((x["codes"], x["codes"], None, x["s"]), ValueError),
                     ((x["codes"], x["codes"], x["s"], x["s"].double()), TypeError),
                     ((x["codes"], x["codes"], x["s"].transpose(1, 2).contiguous(), x["s"]),
                      ValueError),
                     ((x["codes"], x["k"], x["s"], x["s"]), TypeError),
                     ((x["k"], x["k"].bfloat16(), None, None), TypeError),
                     ((x["k"].float(), x["k"].float(), None, None), TypeError),
                     ((x["k"].transpose(0, 1), x["k"], None, None), ValueError),
                     ((x["k"][:, :, :, None], x["k"], None, None), ValueError),
                     ((None, x["k"], None, None), TypeError)):
        with pytest.raises(exc):
            pkg._kv_pools(*bad, dev)


def test_binding_checks_offsets_and_tables(pkg):
    x, dev = tensors(), -1  # the index of a CPU tensor
    pkg._check_offsets(x["off"], 2, "off", dev)
    for bad, exc in ((x["off"][:2], ValueError), (x["off"].long(), TypeError),
                     (x["off"].view(3, 1), ValueError), ([0, 1, 2], TypeError)):
        with pytest.raises(exc):
            pkg._check_offsets(bad, 2, "off", dev)
    pkg._check_table(x["t"], x["lens"], dev)
    for t, lens, exc in ((x["t"].long(), x["lens"], TypeError), (x["t"][0], x["lens"], ValueError),
                         (x["t"], x["lens"][:1], ValueError), (x["t"].t(), x["lens"], ValueError),
                         (x["t"], x["lens"].long(), TypeError)):
        with pytest.raises(exc):
            pkg._check_table(t, lens, dev)


@pytest.mark.parametrize("heads,T,page,D,cluster", [
    ((64, 8), 1, 64, 128, True),     # 8 rows of one head
    ((64, 8), 1, 16, 128, False),    # 16 rows of two heads
    ((64, 8), 2, 64, 128, False),    # 16 rows of one head
    ((64, 8), 2, 64, 64, True),      # 16 rows of 64: 4.6 KB, 5.0 KB of room
    ((64, 8), 1, 16, 64, False),     # 5.1 KB
    ((64, 8), 1, 16, 256, False),    # one CTA per SM: no clusters of 8 on a full grid
])
def test_cluster_plans_leave_room_for_both_ctas(pkg, heads, T, page, D, cluster):
    """An automatic plan merges through a cluster only where its receive buffer
    (rows x D fp32) fits beside the rings of the CTAs of an SM."""
    p = params(pkg, batch=8, num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=D,
               page_size=page, max_pages_per_seq=8192 // page, num_pages=8 * 8192 // page,
               max_seq_len=8192, num_queries=T)
    plan = pkg.decode_attn_quant_make_plan(p, SMS)
    assert plan.split == 1 and plan.max_shards > 1
    if cluster:
        assert plan.cluster == plan.max_shards
    else:
        assert plan.cluster == 0


def test_long_steps_of_several_sequences_are_cut_into_pieces(pkg):
    """One wave of equal shards for a few sequences, pieces in the order the
    SMs take them where more may differ in length."""
    def ctas(batch, ctx):
        p = params(pkg, batch=batch, num_q_heads=16, num_kv_heads=4, head_dim=64, page_size=32,
                   max_pages_per_seq=ctx // 32, num_pages=batch * ctx // 32, max_seq_len=ctx)
        plan = pkg.decode_attn_quant_make_plan(p, SMS)
        return plan.grid_x * plan.grid_y * plan.grid_z, 2 * SMS

    for batch, ctx in ((4, 131072), (2, 65536), (16, 8192)):
        n, slots = ctas(batch, ctx)
        assert n <= slots
    for batch, ctx in ((16, 32768), (8, 131072)):
        n, slots = ctas(batch, ctx)
        assert n > 1.5 * slots
