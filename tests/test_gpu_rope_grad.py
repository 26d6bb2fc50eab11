"""decode_rope under autograd: its gradient is the rotation by the negative angle,
against the formula's in 64 bits and against differences."""
import pytest
import torch

from tests.fp4_reference import rope_table, rotate
from tests.test_gpu_rope import BF16, DEV, F16, pkg, rows  # noqa: F401

pytestmark = pytest.mark.gpu


def made(seed, n, H, D, rot, dtype):
    x, g = rows(seed, n, H, D, dtype), rows(seed + 1, n, H, D, dtype)
    pos = torch.randint(0, 300, (n,), generator=torch.Generator().manual_seed(seed)).int()
    return x, g, pos, rope_table(rot, 300, amplitude=1.1)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("interleaved,backward", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("n,H,D,rot", [(1, 1, 16, 16), (9, 3, 128, 48), (33, 5, 64, 64),
                                       (0, 2, 64, 32)])
@pytest.mark.parametrize("quick", [True, False], ids=["quick", "python"])
def test_gradient(pkg, monkeypatch, quick, n, H, D, rot, interleaved, backward, dtype):  # noqa: F811
    assert pkg._quick() is not None
    monkeypatch.setattr(pkg, "_quick_module", pkg._quick() if quick else None)
    x, g, pos, table = made(40, n, H, D, rot, dtype)
    leaf = x.to(DEV).requires_grad_()
    a = (pos.to(DEV), table.to(DEV), interleaved, backward)
    y = pkg.decode_rope(leaf, *a)
    assert y.requires_grad and torch.equal(y, pkg.decode_rope(x.to(DEV), *a))
    y.backward(g.to(DEV))
    # to the bit of the definition in 32 bits
    want = rotate(g.float(), pos, table, interleaved, not backward).to(dtype)
    assert torch.equal(leaf.grad.cpu(), want)
    # and of the formula's gradient in 64 bits, one rounding and the 32-bit sums away
    x64 = x.double().requires_grad_()
    rotate(x64, pos, table, interleaved, backward).backward(g.double())
    size = g.double().norm(dim=-1, keepdim=True) * 1.1
    tol = torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -20) * x64.grad.abs() + 2.0 ** -22 * size + \
        torch.finfo(dtype).smallest_normal
    assert bool(((leaf.grad.double().cpu() - x64.grad).abs() <= tol).all())


def test_gradient_against_differences(pkg):  # noqa: F811
    """<g, y(x + h e) - y(x - h e)> / 2 h, on values that the result holds to
    half a step of fp16, 2^-6 at most."""
    n, H, D, rot = 4, 2, 32, 32
    x, g, pos, table = made(41, n, H, D, rot, F16)
    x, g = torch.randn(x.shape, generator=torch.Generator().manual_seed(5)).half(), g.sign().half()
    a = (pos.to(DEV), table.to(DEV))
    leaf = x.to(DEV).requires_grad_()
    pkg.decode_rope(leaf, *a).backward(g.to(DEV))
    h = 16.0
    for r, hd, dim in ((0, 0, 0), (1, 1, 5), (2, 0, 16), (3, 1, 31)):
        e = torch.zeros_like(x)
        e[r, hd, dim] = h
        up, down = (pkg.decode_rope((x + s * e).to(DEV), *a).double().cpu() for s in (1, -1))
        slope = float((g.double() * (up - down)).sum()) / (2 * h)
        # two outputs depend on it, each at most 1.1 (16 + 5) * 1.5 and so held to 2^-6,
        # and x + e to the same
        assert abs(slope - float(leaf.grad[r, hd, dim])) <= 8 * 2.0 ** -6 / (2 * h) + 2.0 ** -9


def test_gradients_that_are_views_and_second_gradients(pkg):  # noqa: F811
    x, _, pos, table = made(42, 6, 3, 64, 64, F16)
    a = (pos.to(DEV), table.to(DEV))
    one = rotate(torch.ones(6, 3, 64), pos, table, backward=True).half()
    leaf = x.to(DEV).requires_grad_()
    pkg.decode_rope(leaf, *a).sum().backward()  # an expanded gradient
    assert torch.equal(leaf.grad.cpu(), one)
    wide = torch.ones(6 * 3 * 64 + 4, device=DEV, dtype=F16)[4:].view(6, 3, 64)  # 8 bytes on
    leaf.grad = None
    pkg.decode_rope(leaf, *a).backward(wide)
    assert torch.equal(leaf.grad.cpu(), one)
    leaf.grad = None
    across = torch.ones(3, 6, 64, device=DEV, dtype=F16).transpose(0, 1)
    pkg.decode_rope(leaf, *a).backward(across)
    assert torch.equal(leaf.grad.cpu(), one)
    # the gradient's own gradient is the rotation again
    g = torch.randn(6, 3, 64, generator=torch.Generator().manual_seed(1)).half().to(DEV)
    v = torch.randn(6, 3, 64, generator=torch.Generator().manual_seed(2)).half().to(DEV)
    g.requires_grad_()
    dx, = torch.autograd.grad(pkg.decode_rope(leaf, *a), leaf, g, create_graph=True)
    gg, = torch.autograd.grad(dx, g, v)
    assert torch.equal(gg, pkg.decode_rope(v, *a))
    # a slice of a fused projection: its gradient lands in the projection's
    fused = torch.randn(6, 7, 64, generator=torch.Generator().manual_seed(3)).half().to(DEV)
    fused.requires_grad_()
    pkg.decode_rope(fused[:, 2:5], *a).backward(torch.ones(6, 3, 64, device=DEV, dtype=F16))
    assert torch.equal(fused.grad[:, 2:5].cpu(), one)
    assert not fused.grad[:, :2].any() and not fused.grad[:, 5:].any()


def test_what_a_gradient_refuses_and_what_it_leaves_alone(pkg):  # noqa: F811
    x, _, pos, table = made(43, 6, 3, 64, 64, F16)
    a = (pos.to(DEV), table.to(DEV))
    leaf = x.to(DEV).requires_grad_()
    for out in (leaf, torch.empty_like(leaf)):
        with pytest.raises(ValueError, match="out"):
            pkg.decode_rope(leaf, *a, out=out)
    for bad, exc in ((dict(positions=None), TypeError), (dict(positions=a[0].long()), TypeError),
                     (dict(table=a[1][0]), ValueError), (dict(positions=a[0][:2]), ValueError)):
        with pytest.raises(exc):
            pkg.decode_rope(leaf, **{**dict(positions=a[0], table=a[1]), **bad})
    plain = pkg.decode_rope(x.to(DEV), *a)
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            y = pkg.decode_rope(leaf, *a)
            assert not y.requires_grad and torch.equal(y, plain)
            out = torch.empty_like(y)
            assert pkg.decode_rope(leaf, *a, out=out) is out
    # a table or positions changed between the call and its gradient are noticed
    t = table.to(DEV)
    y = pkg.decode_rope(leaf, a[0], t)
    t.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()
    # a table and positions made where nothing is recorded
    with torch.inference_mode():
        made_there = (pos.to(DEV), table.to(DEV))
    leaf.grad = None
    pkg.decode_rope(leaf, *made_there).sum().backward()
    one = rotate(torch.ones(6, 3, 64), pos, table, backward=True).half()
    assert torch.equal(leaf.grad.cpu(), one)
    # a position outside the table: a zero row, and no gradient through it
    p = a[0].clone()
    p[2] = 10 ** 6
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    leaf.grad = None
    pkg.decode_rope(leaf, p, a[1], err_flag=err).sum().backward()
    assert int(err.item()) == pkg.DEV_BAD_LEN and not leaf.grad[2].any() and leaf.grad[1].any()


def test_gradient_on_another_stream_and_in_a_graph(pkg):  # noqa: F811
    x, g, pos, table = made(44, 65, 4, 128, 128, BF16)
    a = (pos.to(DEV), table.to(DEV))
    want = rotate(g.float(), pos, table, False, True).to(BF16)
    leaf, gd = x.to(DEV).requires_grad_(), g.to(DEV)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    y = pkg.decode_rope(leaf, *a, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    y.backward(gd)
    torch.cuda.synchronize()
    assert torch.equal(leaf.grad.cpu(), want)
    # forward and gradient captured, leaves of the graph's own
    static = x.to(DEV).requires_grad_()
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(pkg.decode_rope(static, *a), static, gd)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, = torch.autograd.grad(pkg.decode_rope(static, *a), static, gd)
    dx.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx.cpu(), want)
