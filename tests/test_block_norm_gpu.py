"""The block norm on the GPU against the formulas in 64 bits, and its gradients against
automatic differentiation and against differences.

Tolerances (2-norm of the difference over 2-norm of the reference): an output in bf16 is off
by its rounding, at most 2^-8 of each value; an output in fp32 by the fp32 steps to it.  A row
sum over D values has at most D / 256 + 16 additions in sequence, each off by 2^-24 at most,
and a dozen further steps follow; gradients subtract terms of their own size, a factor of 4:
2^-24 (D / 256 + 32) x 4.  A weight's gradient adds up to rows / 296 + 64 terms in sequence on
top of that.

dx and dy are differences that can cancel further: r (z - u r^2 sum(z u) / D) with z = gx or gy
and u the normed vector.  By Cauchy and Schwarz the second term's norm is at most
|z| |u|^2 r^2 / D <= |z|, so both terms are at most r |z|, each is off by its fp32 steps relative
to that, and the difference by 2 r |z| times them.  With D = 1 the difference is eps / (u^2 + eps)
of the terms, nearly nothing.  The fp32 part of the bar is therefore taken times `cancel`, the
terms' norm over the result's (and for what is a product with dx, times that of dx)."""
import pytest
import torch

from kda_delta_rule_chunkwise_b200 import binding

BF, F32 = torch.bfloat16, torch.float32
pytestmark = pytest.mark.gpu
TYPES = [(BF, BF), (F32, BF), (F32, F32)]


def formulas(x, y, gate, wo, wi, scale, eps):
    n = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps) * wo
    xn = x + scale * (n if gate is None else n * torch.sigmoid(gate))
    return xn, xn / torch.sqrt(xn.pow(2).mean(-1, keepdim=True) + eps) * wi


def make(rows, D, tx, t, gate, seed=0, y_std=3.0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    return [rn(rows, D).to(tx), (rn(rows, D) * y_std).to(t), rn(rows, D).to(t) if gate else None,
            (1 + 0.2 * rn(D)).to(t), (1 + 0.2 * rn(D)).to(t), rn(rows, D).to(tx), rn(rows, D).to(t)]


def off(got, want):
    got, want = got.detach().cpu().double(), want.detach().double()
    assert torch.isfinite(got).all()
    d = float((got - want).norm())
    return d / float(want.norm()) if float(want.norm()) else d


def bar(dtype, D, rows=0, cancel=1.0):
    f32 = 2.0 ** -24 * (D / 256 + 32 + (rows / 296 + 64 if rows else 0)) * 4 * max(1.0, cancel)
    return f32 if dtype == F32 else 2.0 ** -8 + f32


def cancellations(x, y, g, wo, wi, dxn, dh, scale, eps, dx, dy):
    """The terms' norms over the result's norm, for dx and for dy."""
    xn, _ = formulas(x, y, g, wo, wi, scale, eps)
    rx, ry = (torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + eps) for t in (xn, y))
    gy = scale * dx * wo * (1 if g is None else torch.sigmoid(g))
    ax = float(dxn.norm() + 2 * (rx * dh * wi).norm()) / float(dx.norm())
    return ax, ax * 2 * float((ry * gy).norm()) / float(dy.norm())


def cuda(ts):
    return [None if t is None else t.cuda() for t in ts]


SIZES = [(1, 1), (3, 7), (9, 64), (17, 100), (5, 256), (33, 257), (4, 1000), (7, 2048), (301, 512), (2, 4096), (3, 5000),
         (2, 8191), (2, 8192), (2, 16384), (1, 16383)]


@pytest.mark.parametrize("tx,t", TYPES, ids=["bf16", "f32x", "f32"])
@pytest.mark.parametrize("rows,D", SIZES, ids=lambda v: str(v))
def test_block_norm_and_its_gradients(rows, D, tx, t):
    for gate in (True, False):
        x, y, g, wo, wi, dxn, dh = make(rows, D, tx, t, gate, seed=D)
        leaves = [v.double().requires_grad_(True) for v in (x, y, g, wo, wi) if v is not None]
        full = leaves if gate else [leaves[0], leaves[1], None, *leaves[2:]]
        want = formulas(*full, 0.5, 1e-6)
        grads = list(torch.autograd.grad(want, leaves, [dxn.double(), dh.double()]))
        if not gate:
            grads.insert(2, None)
        d = cuda([x, y, g, wo, wi])
        got = binding.kda_block_norm(*d, scale=0.5, eps=1e-6)
        for a, b in zip(got, want):
            assert off(a, b) <= bar(a.dtype, D)
        back = binding.kda_block_norm_backward(*d, *cuda([dxn, dh]), scale=0.5, eps=1e-6)
        assert (back[2] is None) == (not gate)
        ax, ay = cancellations(*(None if t is None else t.detach().double() for t in (x, y, g, wo, wi, dxn, dh)),
                               0.5, 1e-6, grads[0], grads[1])
        for i, (a, b) in enumerate(zip(back, grads)):
            if a is not None:
                assert off(a, b) <= bar(a.dtype, D, rows if i > 2 else 0, ay if i == 1 else ax), i


def test_unaligned_tensors_take_the_scalar_path():
    x, y, g, wo, wi, _, _ = cuda(make(6, 64, BF, BF, True))
    want = binding.kda_block_norm(x, y, g, wo, wi)
    shifted = torch.empty(6 * 64 + 1, dtype=BF, device="cuda")[1:].view(6, 64)
    shifted.copy_(y)
    got = binding.kda_block_norm(x, shifted, g, wo, wi)
    for a, b in zip(got, want):      # another order of the row sum: the last bit may differ
        assert off(a, b.cpu()) <= 2.0 ** -8


def test_missing_gradients_count_as_zeros():
    x, y, g, wo, wi, dxn, dh = cuda(make(20, 300, BF, BF, True))
    for a, b in ((dxn, None), (None, dh)):
        zeros = [torch.zeros_like(p) if q is None else q for p, q in ((dxn, a), (dh, b))]
        want = binding.kda_block_norm_backward(x, y, g, wo, wi, *zeros)
        got = binding.kda_block_norm_backward(x, y, g, wo, wi, a, b)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_in_place_residual_and_determinism():
    x, y, g, wo, wi, dxn, dh = cuda(make(700, 512, F32, BF, True))
    want = binding.kda_block_norm(x, y, g, wo, wi, scale=0.3)
    again = binding.kda_block_norm_backward(x, y, g, wo, wi, dxn, dh, scale=0.3)
    for a, b in zip(again, binding.kda_block_norm_backward(x, y, g, wo, wi, dxn, dh, scale=0.3)):
        assert torch.equal(a, b)
    h = y.clone()
    got = binding.kda_block_norm(x, h, g, wo, wi, scale=0.3, x_new=x, h=h)
    assert got[0] is x and torch.equal(x, want[0]) and torch.equal(h, want[1])


def test_zero_rows_large_values_and_nan():
    x, y, g, wo, wi, dxn, dh = cuda(make(4, 128, F32, BF, True))
    x[0], y[0] = 0, 0                     # a row of zeros: rms is sqrt(eps)
    g[1], g[2, :64], g[2, 64:] = 0, 1e4, -1e4
    y[3, 5] = float("nan")
    xn, h = binding.kda_block_norm(x, y, g, wo, wi)
    assert (xn[0] == 0).all() and (h[0] == 0).all()
    assert torch.isfinite(xn[:3]).all() and torch.isnan(xn[3]).all() and torch.isnan(h[3]).all()
    assert torch.equal(xn[2, 64:], x[2, 64:])        # a closed gate adds nothing
    back = binding.kda_block_norm_backward(x, y, g, wo, wi, dxn, dh)
    assert all(torch.isfinite(t[:3]).all() for t in back[:3])


def test_no_rows():
    x = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert [tuple(t.shape) for t in binding.kda_block_norm(x, x, None, w, w)] == [(0, 64)] * 2
    back = binding.kda_block_norm_backward(x, x, None, w, w, x, x)
    assert (back[3] == 0).all() and (back[4] == 0).all()


def test_autograd_and_differences():
    """The autograd op's gradients are the call's, and agree with central differences in the loss."""
    x, y, g, wo, wi, dxn, dh = [t.cuda() for t in make(3, 40, F32, F32, True, y_std=1.0)]
    leaves = [t.clone().requires_grad_(True) for t in (x, y, g, wo, wi)]
    a, b = binding.kda_block_norm_autograd(*leaves, 0.7)
    ((a * dxn).sum() + (b * dh).sum()).backward()
    call = binding.kda_block_norm_backward(x, y, g, wo, wi, dxn, dh, scale=0.7)
    gen = torch.Generator().manual_seed(5)
    for leaf, c in zip(leaves, call):
        assert torch.equal(leaf.grad, c)
        # the formulas' directional difference in 64 bits against the kernel's gradient: the
        # step's own error is about its square, the gradient's bar that of fp32
        way = torch.randn(leaf.shape, generator=gen).double()
        base = [t.detach().cpu().double() for t in leaves]
        i = [l is leaf for l in leaves].index(True)
        loss = []
        for sgn in (1, -1):
            moved = list(base)
            moved[i] = base[i] + sgn * 1e-5 * way
            p, q = formulas(*moved, 0.7, 1e-6)
            loss.append(float((p * dxn.cpu().double()).sum() + (q * dh.cpu().double()).sum()))
        diff = (loss[0] - loss[1]) / 2e-5
        have = float((c.cpu().double() * way).sum())
        size = float(c.cpu().double().norm() * way.norm())
        assert abs(diff - have) <= bar(F32, 40, 3) * size + 1e-8 * size
    only_h = binding.kda_block_norm_autograd(*[t.clone().requires_grad_(True) for t in (x, y, g, wo, wi)])[1]
    only_h.sum().backward()              # the other output's gradient is missing


def test_captured_beside_another_stream():
    x, y, g, wo, wi, dxn, dh = cuda(make(64, 1024, BF, BF, True))
    want = binding.kda_block_norm(x, y, g, wo, wi)
    xn, h = torch.zeros_like(x), torch.zeros_like(y)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            binding.kda_block_norm(x, y, g, wo, wi, x_new=xn, h=h)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(xn, want[0]) and torch.equal(h, want[1])


@pytest.mark.parametrize("D", [64, 66, 65, 8192, 8191])
def test_outputs_may_lie_on_inputs(D):
    """Through the C ABI: each output on an input of its own, in both directions and on every path."""
    lib, P = binding.load(), binding._addr
    x, y, g, wo, wi, dxn, dh = cuda(make(5, D, F32, BF, True, seed=D))
    want = binding.kda_block_norm(x, y, g, wo, wi, scale=0.5, eps=1e-6)
    back = binding.kda_block_norm_backward(x, y, g, wo, wi, dxn, dh, scale=0.5, eps=1e-6)
    st = torch.cuda.current_stream().cuda_stream
    a, b = x.clone(), g.clone()
    assert lib.kda_block_norm(P(a), P(y), P(b), P(wo), P(wi), 5, D, 0.5, 1e-6, 0, 1, P(a), P(b), st) == binding.KDA_OK
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    a, b, c = dxn.clone(), dh.clone(), g.clone()
    dw = torch.zeros(2, D, device="cuda")
    need = lib.kda_block_norm_backward_workspace_bytes(5, D)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    assert lib.kda_block_norm_backward(P(x), P(y), P(c), P(wo), P(wi), P(a), P(b), 5, D, 0.5, 1e-6, 0, 1, P(a), P(b), P(c),
                                       P(dw[0]), P(dw[1]), P(ws), need, st) == binding.KDA_OK
    torch.cuda.synchronize()
    for got, w in zip((a, b, c, dw[0], dw[1]), back):
        assert torch.equal(got, w)


def test_more_rows_than_ctas_and_rows_side_by_side():
    for rows, D in ((1000, 40), (700, 200), (333, 1001), (5000, 24)):
        x, y, g, wo, wi, dxn, dh = make(rows, D, BF, BF, True, seed=rows)
        leaves = [t.double().requires_grad_(True) for t in (x, y, g, wo, wi)]
        want = formulas(*leaves, 0.5, 1e-6)
        grads = torch.autograd.grad(want, leaves, [dxn.double(), dh.double()])
        d = cuda([x, y, g, wo, wi])
        for a, b in zip(binding.kda_block_norm(*d, scale=0.5, eps=1e-6), want):
            assert off(a, b) <= bar(BF, D)
        back = binding.kda_block_norm_backward(*d, *cuda([dxn, dh]), scale=0.5, eps=1e-6)
        for i, (a, b) in enumerate(zip(back, grads)):
            assert off(a, b) <= bar(a.dtype, D, rows if i > 2 else 0), (rows, D, i)


@pytest.mark.parametrize("D", [64, 66, 65, 16383])
@pytest.mark.parametrize("size,eps", [(0.0, 1e-30), (0.0, 1e-36), (2.0 ** 50, 1e-6), (2.0 ** -50, 1e-36)])
def test_gradients_of_zero_tiny_and_huge_rows(D, size, eps):
    """rms factors whose cube is no fp32 number: 1e15 and 1e18 for rows of zeros beside a small eps, 2^-50 and
    2^50 for huge and tiny rows (powers of two, so that the rows' digits are those of ordinary ones)."""
    x, y, g, wo, wi, dxn, dh = make(3, D, F32, F32, True, seed=D, y_std=1.0)
    x, y = x * size, y * size
    small = 1e-3 if size == 0.0 else 1.0     # dy grows with the factor squared: keep it a number
    dh = dh * small
    scale = 0.5 * size if size else 0.5      # the block's share of x' is of x's size
    leaves = [t.double().requires_grad_(True) for t in (x, y, g, wo, wi)]
    want = torch.autograd.grad(formulas(*leaves, scale, eps), leaves, [torch.zeros_like(dxn).double(), dh.double()])
    got = binding.kda_block_norm_backward(*cuda([x, y, g, wo, wi]), None, dh.cuda(), scale=scale, eps=eps)
    _, ay = cancellations(*(t.double() for t in (x, y, g, wo, wi, torch.zeros_like(dxn), dh)), scale, eps, want[0], want[1])
    for i, (a, b) in enumerate(zip(got, want)):
        if float(b.abs().max()) == 0:
            assert (a == 0).all(), i
        else:
            assert off(a, b) <= bar(F32, D, 3 if i > 2 else 0, max(4.0, ay)), i


def test_second_derivatives_are_refused_not_dropped():
    """The gradients say so when a second derivative is taken through them; alone they can be used on."""
    leaves = [t.cuda().requires_grad_(True) for t in make(3, 40, F32, F32, True)[:5]]
    a, b = binding.kda_block_norm_autograd(*leaves)
    grads = torch.autograd.grad(a.sum() + b.sum(), leaves, create_graph=True)
    plain = torch.autograd.grad(sum(t.sum() for t in binding.kda_block_norm_autograd(*leaves)), leaves)
    assert all(torch.equal(p, q) for p, q in zip(grads, plain))
    with pytest.raises(RuntimeError, match="second derivative"):
        (a.sum() + grads[1].square().sum()).backward()


@pytest.mark.parametrize("D", [64, 66, 65])
def test_gates_in_fp32_are_fp32s(D):
    """Logits from -80 to 80, each value alone: the gate's own digits show in x' where x is 0 and in dgate.  Steps of
    2^-24 at most: the row sum D / 32 + 8 and half of it in the factor, its square root 2, the exponential 4 (two
    units), the gate's sum and quotient 4, four products; in dgate the gate twice and 1 - a, which is off by 2^-24 / (1 - a)
    where a is near 1: compare it there as an absolute share."""
    x, y, _, wo, wi, dxn, _ = make(161, D, F32, F32, True, seed=D, y_std=1.0)
    g = torch.linspace(-80, 80, 161)[:, None].expand(161, D).contiguous()
    x = torch.zeros_like(x)
    got = binding.kda_block_norm(*cuda([x, y, g, wo, wi]))[0].cpu().double()
    want = formulas(*(t.double() for t in (x, y, g, wo, wi)), 1.0, 1e-6)[0]
    assert float(((got - want) / want).abs().max()) <= 2.0 ** -24 * (D / 64 + 4 + 2 + 4 + 4 + 4)
    leaves = [t.double().requires_grad_(True) for t in (x, y, g, wo, wi)]
    want = torch.autograd.grad(formulas(*leaves, 1.0, 1e-6)[0], leaves[2], dxn.double())[0]
    got = binding.kda_block_norm_backward(*cuda([x, y, g, wo, wi]), dxn.cuda(), None)[2].cpu().double()
    n = formulas(*(t.double() for t in (x, y)), None, wo.double(), wi.double(), 1.0, 1e-6)[0]
    a = torch.sigmoid(g.double())
    steps = 2.0 ** -24 * (D / 64 + 4 + 2 + 2 * (4 + 4) + 6)
    assert ((got - want).abs() <= steps * want.abs() + 2.0 ** -24 * 2 * (dxn.double() * n * a).abs()).all()
