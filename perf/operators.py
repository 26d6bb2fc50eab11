"""Cases of the paged-cache operators beyond the decode step, for measurement.

Four operators, each as one call a serving program makes:
  chunk   decode_attn_chunk: attention of a ragged batch of new tokens over a
          paged 16-bit cache (prompt chunks, verification of drafted tokens)
  append  decode_kv_append_chunk: the chunk's K/V rows written into their
          pages, as they are or quantised to 8 bits with a scale per row
  read    decode_kv_read: rows of a paged cache read back as contiguous
          16-bit rows
  quant   decode_attn_quant: the decode step over an 8-bit cache

``own`` False computes the plain form (elementary torch operations in 32
bits), True calls the library.
"""
import math

import torch

own = False

MAX_SCORES = 4 << 30   # bytes of the plain form's scores of one KV head
MAX_FLOPS = 4.4e12     # of the plain form, padding included
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    llama = dict(hq=32, hkv=8, d=128, page=16)
    return [
        # 16 drafted tokens verified at once on the Llama shape: latency
        dict(name="chunk 16 of 3060", op="chunk", dtype="fp16", batch=1, new=16, ctx=3060,
             spread=False, window=0, **llama),
        # one whole prompt, nothing cached before it
        dict(name="chunk prompt 8192", op="chunk", dtype="bf16", batch=1, new=8192, ctx=8192,
             spread=False, window=0, **llama),
        # a serving mix: each sequence brings its own number of new tokens
        dict(name="chunk mix of 64", op="chunk", dtype="bf16", batch=64, new=512, ctx=8192,
             spread=True, window=0, **llama),
        # the next chunk of a long document
        dict(name="chunk 1024 of 131072", op="chunk", dtype="fp16", batch=1, new=1024,
             ctx=131072, spread=False, window=0, hq=64, hkv=8, d=128, page=64),
        # sliding window, head_dim 256, odd lengths
        dict(name="chunk window d256", op="chunk", dtype="fp16", batch=3, new=1001, ctx=4099,
             spread=False, window=1024, hq=16, hkv=4, d=256, page=32),
        # the step's own row of every sequence, quantised: latency
        dict(name="append one each to fp8", op="append", dtype="bf16", fmt="fp8", batch=64,
             new=1, ctx=2048, spread=True, **llama),
        # the rows of a serving mix's chunks, quantised
        dict(name="append mix to fp8", op="append", dtype="fp16", fmt="fp8", batch=64, new=1024,
             ctx=2048, spread=True, **llama),
        # one sequence's cache taken back to 16 bits before its next chunk
        dict(name="read 3060 of fp8", op="read", dtype="fp16", fmt="fp8", batch=1, new=3060,
             ctx=3060, spread=False, **llama),
        # the same for long sequences
        dict(name="read 4 x 32768 of fp8", op="read", dtype="bf16", fmt="fp8", batch=4,
             new=32768, ctx=32768, spread=False, hq=64, hkv=8, d=128, page=64),
        # decode on the Llama shape over an 8-bit cache: latency
        dict(name="decode fp8 3060", op="quant", dtype="fp16", fmt="fp8", batch=1, new=1,
             ctx=3060, spread=False, window=0, **llama),
        # decode of a serving mix
        dict(name="decode fp8 mix of 64", op="quant", dtype="bf16", fmt="fp8", batch=64, new=1,
             ctx=8192, spread=True, window=0, **llama),
        # decode at long context, the whole cache streamed
        dict(name="decode fp8 4 x 131072", op="quant", dtype="fp16", fmt="fp8", batch=4, new=1,
             ctx=131072, spread=False, window=0, hq=64, hkv=8, d=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "append", "read", "quant"])
    hq, hkv = rng.choice([(32, 8), (64, 8), (16, 4), (4, 1), (8, 8), (12, 4), (14, 2), (40, 8),
                          (16, 1)])
    c = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), hq=hq, hkv=hkv,
             d=rng.choice([64, 128, 256]), page=rng.choice([8, 16, 32, 64, 128, 256]),
             batch=_log_int(rng, 1, 128), ctx=_log_int(rng, 1, 131072), spread=rng.random() < 0.7)
    if op in ("chunk", "quant"):
        c["window"] = rng.choice([0, 0, _log_int(rng, 1, 4096)])
    if op == "chunk":
        c["new"] = _log_int(rng, 1, min(8192, c["ctx"]))
    elif op == "quant":
        c["fmt"] = "fp8"
        c["new"] = rng.choice([1, 1, 1, max(1, min(16 // (hq // hkv), 2, c["ctx"]))])
        c["spread"] = c["spread"] and c["new"] == 1
    elif op == "append":
        c["fmt"] = rng.choice(["fp8", "fp8", "16"])
        c["new"] = _log_int(rng, 1, min(1024, c["ctx"]))
    else:
        c["fmt"] = rng.choice(["fp8", "fp8", "16"])
        c["new"] = _log_int(rng, 1, c["ctx"])
    while True:  # at most the largest listed case's memory and work
        pool = c["batch"] * c["ctx"] * hkv * c["d"]
        scores = c["batch"] * c["new"] * (c["ctx"] + c["new"]) * 4 * (hq // hkv)
        flops = c["batch"] * c["new"] * (c["ctx"] + c["new"]) * 4 * hq * c["d"]
        attends = op in ("chunk", "quant")
        if pool <= (1 << 28) and (not attends or (scores <= MAX_SCORES // 2 and
                                                  flops <= MAX_FLOPS / 2)):
            return c
        if c["batch"] > 1:
            c["batch"] = (c["batch"] + 1) // 2
        else:
            c["ctx"] = (c["ctx"] + 1) // 2
            c["new"] = max(1, min(c["new"], c["ctx"]) // (2 if op == "chunk" else 1))


def _lengths(c):
    """(cached positions with the new rows, new rows) of each sequence: the
    same numbers for every seed, prepare() only shuffles them."""
    out = []
    for b in range(c["batch"]):
        if c["spread"]:
            u, v = ((b + 1) * 0.6180339887498949) % 1.0, ((b + 1) * 0.41421356237309515) % 1.0
            n = 1 + int(v * (c["new"] - 1) + 0.5)
            out.append((max(n, 1 + int(u * (c["ctx"] - 1) + 0.5)), n))
        else:
            out.append((c["ctx"], c["new"]))
    return out


def _attended(c, L, n):
    """(query, key) pairs of one sequence, and the distinct keys among them."""
    w = c.get("window", 0)
    if w <= 0 or w >= L:
        return n * (L - n) + n * (n + 1) // 2, L
    first = L - n + 1  # keys the first query sees without a window
    full = max(0, min(n, L - max(first, w) + 1)) if L >= w else 0
    part = n - full
    return full * w + part * first + part * (part - 1) // 2, min(L, w + n - 1)


def work(case):
    c = case
    rows = sum(n for _, n in _lengths(c))
    row = c["hkv"] * c["d"] * 2  # values of one position's K and V
    cell = 1 if c.get("fmt") == "fp8" else 2
    scales = c["hkv"] * 2 * 4 if c.get("fmt") == "fp8" else 0
    if c["op"] == "append":
        return {"bytes": rows * (row * 2 + row * cell + scales), "flops": 2 * rows * row}
    if c["op"] == "read":
        return {"bytes": rows * (row * 2 + row * cell + scales), "flops": rows * row}
    pairs = [_attended(c, L, n) for L, n in _lengths(c)]
    keys = sum(k for _, k in pairs)
    return {"bytes": keys * (row * cell + scales) + rows * c["hq"] * c["d"] * 4,
            "flops": sum(p for p, _ in pairs) * 4 * c["hq"] * c["d"]}


# -------------------------------------------------------------- the inputs

def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    order = torch.Generator()
    order.manual_seed(int(seed))
    lens = _lengths(c)
    lens = [lens[i] for i in torch.randperm(len(lens), generator=order).tolist()]
    B, Hq, Hkv, D, PS = c["batch"], c["hq"], c["hkv"], c["d"], c["page"]
    dt = DTYPES[c["dtype"]]
    need = [-(-L // PS) for L, _ in lens]
    P = sum(need) + max(1, sum(need) // 16)
    perm = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    off = [0]
    for _, n in lens:
        off.append(off[-1] + n)
    total = off[-1]

    def rows(*shape):
        x = torch.randn(shape, generator=g, device=dev)
        return x if len(shape) < 3 else x * torch.exp2(
            torch.randn((*shape[:-1], 1), generator=g, device=dev) * 0.5)

    s = dict(case=dict(c), table=table, total=total, max_new=max(n for _, n in lens),
             max_len=max(L for L, _ in lens),
             lens=torch.tensor([L for L, _ in lens], dtype=torch.int32, device=dev),
             off=torch.tensor(off, dtype=torch.int32, device=dev), scale=1.0 / math.sqrt(D))
    if c.get("fmt") == "fp8":
        for n in ("k", "v"):
            code, sc = _quantise(rows(P, PS, Hkv, D))
            s[n + "_pages"], s[n + "_scales"] = code, sc.transpose(1, 2).contiguous()
    else:
        for n in ("k", "v"):
            s[n + "_pages"] = rows(P, PS, Hkv, D).to(dt)
    if c["op"] in ("chunk", "quant"):
        s["q"] = torch.randn((total, Hq, D), generator=g, device=dev).to(dt)
        if c["op"] == "quant":
            s["q"] = s["q"].view(B, c["new"], Hq, D) if c["new"] > 1 else s["q"]
    elif c["op"] == "append":
        s["k_new"], s["v_new"] = rows(total, Hkv, D).to(dt), rows(total, Hkv, D).to(dt)
    else:  # the positions read are the last rows of each sequence
        s["starts"] = torch.tensor([L - n for L, n in lens], dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------ the operators

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import paged_gqa_decode_06_gb300 as pgd
    c = s["case"]
    if c["op"] == "chunk":
        return pgd.decode_attn_chunk(s["q"], s["k_pages"], s["v_pages"], s["table"], s["off"],
                                     s["lens"], s["scale"], window=c["window"],
                                     max_seq_len=s["max_len"])
    if c["op"] == "quant":
        return pgd.decode_attn_quant(s["q"], s["k_pages"], s["v_pages"], s["k_scales"],
                                     s["v_scales"], s["table"], s["lens"], s["scale"],
                                     window=c["window"], max_seq_len=s["max_len"])
    if c["op"] == "append":
        pgd.decode_kv_append_chunk(s["k_new"], s["v_new"], s["off"], s["lens"], s["k_pages"],
                                   s["v_pages"], s["table"], k_scales=s.get("k_scales"),
                                   v_scales=s.get("v_scales"))
        return _pools(s)
    return pgd.decode_kv_read(s["k_pages"], s["v_pages"], s["table"], s["off"], s["total"],
                              starts=s["starts"], k_scales=s.get("k_scales"),
                              v_scales=s.get("v_scales"), dtype=DTYPES[c["dtype"]])


def _pools(s):
    return [s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales") if n in s]


def _quantise(x):
    """fp32 rows [..., D] -> (e4m3 values, scale [...]): the scale is the
    least power of two with max |x| <= 448 * scale, and 0 for a row below
    2^-100, whose values are 0."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    live = amax >= 2.0 ** -100
    zero = torch.zeros_like(amax)  # 2^e and 2^-e put together from their bits
    scale = torch.where(live, ((e + 127) << 23).view(torch.float32), zero)
    inv = torch.where(live, ((127 - e) << 23).view(torch.float32), zero)
    return (x * inv.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _row_sequences(s):
    """Sequence of each of the ragged rows, and its place in the sequence."""
    r = torch.arange(s["total"], device=s["off"].device)
    b = torch.searchsorted(s["off"][1:].long(), r, right=True)
    return b, r - s["off"].long()[b]


def _plain(s):
    c = s["case"]
    if c["op"] in ("chunk", "quant"):
        return _plain_attention(s)
    b, i = _row_sequences(s)
    PS = c["page"]
    if c["op"] == "append":
        pos = s["lens"].long()[b] - (s["off"][1:] - s["off"][:-1]).long()[b] + i
        page, slot = s["table"][b, pos // PS].long(), pos % PS
        for n in ("k", "v"):
            new, pool = s[n + "_new"], s[n + "_pages"]
            if c["fmt"] == "fp8":
                code, sc = _quantise(new.float())
                pool.view(torch.uint8)[page, slot] = code.view(torch.uint8)
                s[n + "_scales"][page, :, slot] = sc
            else:
                pool[page, slot] = new
        return _pools(s)
    pos = s["starts"].long()[b] + i
    page, slot = s["table"][b, pos // PS].long(), pos % PS
    out = []
    for n in ("k", "v"):
        if c["fmt"] == "fp8":
            x = s[n + "_pages"].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float()
            x = x * s[n + "_scales"][page, :, slot].unsqueeze(-1)
        else:
            x = s[n + "_pages"][page, slot]
        out.append(x.to(DTYPES[c["dtype"]]))
    return tuple(out)


def _plain_attention(s):
    """Softmax attention of the padded batch, one KV head at a time."""
    c = s["case"]
    B, Hq, Hkv, D, PS = c["batch"], c["hq"], c["hkv"], c["d"], c["page"]
    G, dev = Hq // Hkv, s["q"].device
    n, L = s["max_new"], s["max_len"]
    off, lens = s["off"].long(), s["lens"].long()
    count = off[1:] - off[:-1]
    i, t = torch.arange(n, device=dev), torch.arange(L, device=dev)
    q = s["q"].reshape(-1, Hq, D)
    q = q[(off[:-1, None] + i).clamp(max=q.shape[0] - 1)].float()      # [B, n, Hq, D]
    at = (lens - count)[:, None] + i                                    # position of each query
    last = torch.where(i < count[:, None], at, torch.full_like(at, -1))
    seen = t <= last[:, :, None]                                        # [B, n, L]
    if c["window"] > 0:
        seen &= t > last[:, :, None] - c["window"]
    page, slot = s["table"][:, t // PS].long().clamp(min=0), (t % PS).expand(B, L)
    out = torch.zeros((B, n, Hq, D), device=dev)
    for h in range(Hkv):
        kv = []
        for x in ("k", "v"):
            pool = s[x + "_pages"]
            if "fmt" in c:
                r = pool.view(torch.uint8)[page, slot, h].view(torch.float8_e4m3fn).float()
                r = r * s[x + "_scales"][page, h, slot].unsqueeze(-1)
            else:
                r = pool[page, slot, h].float()
            kv.append(r)                                                # [B, L, D]
        k, v = kv
        qh = q[:, :, h * G:(h + 1) * G].transpose(1, 2).reshape(B, G * n, D)
        w = torch.matmul(qh, k.transpose(1, 2)).mul_(s["scale"]).view(B, G, n, L)
        w.masked_fill_(~seen[:, None], float("-inf"))
        top = w.amax(-1, keepdim=True)
        w.sub_(torch.where(top == float("-inf"), torch.zeros_like(top), top)).exp_()
        total = w.sum(-1, keepdim=True)
        o = torch.matmul(w.view(B, G * n, L), v).view(B, G, n, D)
        o = torch.where(total > 0, o / total, torch.zeros_like(o))
        out[:, :, h * G:(h + 1) * G] = o.transpose(1, 2)
        del w, o, k, v, kv
    return out[i < count[:, None]].view(s["q"].shape).to(s["q"].dtype)


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    lens, off, table = s["lens"].tolist(), s["off"].tolist(), s["table"].long()
    if c["op"] in ("chunk", "quant"):
        return _exact_attention(s, lens, off, table)
    if c["op"] == "read":
        out = []
        for n in ("k", "v"):
            got = torch.empty((s["total"], c["hkv"], c["d"]), dtype=torch.float64, device="cuda")
            for b, start in enumerate(s["starts"].tolist()):
                rows = _rows64(s, n, table[b], start, start + off[b + 1] - off[b], None)
                got[off[b]:off[b + 1]] = rows
            out.append(got)
        return tuple(out)
    # append: the scale from the definition's inequality, the value to the
    # nearest number of four significant bits (three below 2^-6)
    pools = [p.double() if c["fmt"] == "fp8" and p.dtype == torch.float8_e4m3fn else p.clone()
             for p in _pools(s)]
    if c["fmt"] != "fp8":
        pools = [p.double() for p in pools]
    for b in range(c["batch"]):
        n = off[b + 1] - off[b]
        pos = torch.arange(lens[b] - n, lens[b], device="cuda")
        page, slot = table[b, pos // c["page"]], pos % c["page"]
        for k, name in enumerate(("k_new", "v_new")):
            x = s[name][off[b]:off[b + 1]].double()
            if c["fmt"] == "fp8":
                top = x.abs().amax(-1)
                e = torch.ceil(torch.log2(top.clamp(min=1e-30) / 448.0)).long()
                e = torch.where(448.0 * _pow2(e - 1) >= top, e - 1, e)
                e = torch.where(448.0 * _pow2(e) < top, e + 1, e)
                sc = torch.where(top >= _pow2(torch.full_like(e, -100)), _pow2(e),
                                 torch.zeros_like(top))
                y = torch.where(sc[..., None] > 0, x / sc[..., None], torch.zeros_like(x))
                step = _pow2(torch.frexp(y.abs().clamp(min=0.015625))[1].long() - 4)
                x = torch.round(y / step) * step
                pools[2 + k][page, :, slot] = sc.float()
            pools[k][page, slot] = x
    return pools


def _pow2(e):
    """2^e in 64 bits, exactly."""
    return ((e + 1023) << 52).view(torch.float64)


def _rows64(s, n, pages, lo, hi, h):
    """K or V of positions [lo, hi) of one sequence in 64 bits (head h or all)."""
    c = s["case"]
    pos = torch.arange(lo, hi, device="cuda")
    page, slot = pages[pos // c["page"]], pos % c["page"]
    heads = slice(None) if h is None else slice(h, h + 1)
    pool = s[n + "_pages"][:, :, heads]
    if c.get("fmt") == "fp8":
        x = pool.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).double()
        return x * s[n + "_scales"][:, heads][page, :, slot].double().unsqueeze(-1)
    return pool[page, slot].double()


def _exact_attention(s, lens, off, table):
    c = s["case"]
    Hq, Hkv, D, w = c["hq"], c["hkv"], c["d"], c["window"]
    if work(c)["flops"] > 6e12:
        return None
    G = Hq // Hkv
    q = s["q"].reshape(-1, Hq, D)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(lens):
        n = off[b + 1] - off[b]
        for h in range(Hkv):
            first = max(0, L - n + 1 - w) if w > 0 else 0
            k, v = (_rows64(s, x, table[b], first, L, h)[:, 0] for x in ("k", "v"))
            step = max(1, (1 << 28) // (G * (L - first)))
            for a in range(0, n, step):
                z = min(n, a + step)
                p = torch.arange(L - n + a, L - n + z, device="cuda")[:, None]
                top = L - n + z  # one past the last key these queries see
                t = torch.arange(first, top, device="cuda")
                hide = t > p
                if w > 0:
                    hide |= t <= p - w
                for g in range(G):
                    x = q[off[b] + a:off[b] + z, h * G + g].double() @ k[:top - first].T
                    x = (x * s["scale"]).masked_fill(hide, -math.inf)
                    out[off[b] + a:off[b] + z, h * G + g] = \
                        torch.softmax(x, -1) @ v[:top - first]
    return out.view(s["q"].shape)
