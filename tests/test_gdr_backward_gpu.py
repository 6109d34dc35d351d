"""Gradients of the gated delta rule on the GPU against automatic differentiation of the
recurrence in 64 bits, and against differences.

Tolerances (2-norm of the difference over 2-norm of the reference).  A bf16 gradient is off by its
rounding, 2^-8 of each value at most, and by the block kernel's fp16 operands: a product's two
operands are off by 2^-11 each, and the up to six products that a gradient adds may cancel by a
factor of two: 2^-8 + 6 x 2 x 2 x 2^-11 = 4 x 2^-8.  fp32 gradients and dstate_in: a random walk of
16 roundings a token, 2^-24 x 16 sqrt(T), times the same cancellation, and at least 2e-6."""
import math

import pytest
import torch

import _gdr_reference as ref
from kda_delta_rule_chunkwise_b200 import binding

BF, F32 = torch.bfloat16, torch.float32
pytestmark = pytest.mark.gpu
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dstate_in")


def bar(dtype, T):
    return 4 * 2.0 ** -8 if dtype == BF else max(2e-6, 2 * 2.0 ** -24 * 16 * math.sqrt(T))


def off(got, want):
    got, want = got.detach().cpu().double(), want.double()
    assert torch.isfinite(got).all()
    d = float((got - want).norm())
    return d / float(want.norm()) if float(want.norm()) else d


def gpu(ts):
    return [None if t is None else t.cuda() for t in ts]


def case(B, T, Hk, H, dk, dv, dtype, seed, lengths=None, **kw):
    x = ref.inputs(B, T, Hk, H, dk, dv, dtype, seed=seed, lengths=lengths, **kw)
    gen = torch.Generator().manual_seed(seed + 1000)
    n = B if lengths is None else len(lengths)
    dout = torch.randn(B, T, H, dv, generator=gen).to(dtype)
    ds = torch.randn(n, H, dk, dv, generator=gen) * 0.3
    return x, dout, ds


CASES = [
    (1, 1, 1, 1, 64, 64, None), (1, 31, 1, 2, 128, 128, None), (2, 64, 2, 2, 64, 128, None), (1, 65, 1, 3, 128, 64, None),
    (2, 130, 2, 4, 128, 128, None), (1, 200, 3, 6, 64, 64, None),
    (1, 300, 2, 4, 128, 128, [0, 1, 31, 32, 33, 0, 64, 139]), (1, 211, 1, 2, 64, 128, [100, 0, 110]),
    (1, 260, 1, 2, 128, 128, [63, 65, 1, 1, 130]),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", CASES, ids=lambda c: "x".join(map(str, c[:6])) + ("p" if c[6] else ""))
def test_backward_matches_the_recurrence(shape, dtype):
    B, T, Hk, H, dk, dv, lengths = shape
    x, dout, ds = case(B, T, Hk, H, dk, dv, dtype, T, lengths)
    want = ref.backward(*x[:5], x[5], x[6], dout, ds)
    got = binding.kda_gdr_backward(*gpu(x), dout.cuda(), ds.cuda())
    assert binding.kda_check_device_error() == binding.KDA_OK
    for name, a, b in zip(NAMES, got, want):
        assert off(a, b) <= (bar(F32, T) if name == "dstate_in" else bar(dtype, T)), name


@pytest.mark.parametrize("H,dv", [(1, 128), (38, 128), (80, 128), (150, 128), (160, 64)])
def test_backward_variants_by_unit_count(H, dv):
    x, dout, ds = case(1, 70, 1, H, 128, dv, BF, H)
    want = ref.backward(*x[:5], x[5], x[6], dout, ds)
    got = binding.kda_gdr_backward(*gpu(x), dout.cuda(), ds.cuda())
    for name, a, b in zip(NAMES, got, want):
        assert off(a, b) <= (bar(F32, 70) if name == "dstate_in" else bar(BF, 70)), name


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_missing_states_and_gradients(dtype):
    x, dout, _ = case(2, 50, 1, 2, 64, 64, dtype, 4, state=False)
    want = ref.backward(*x[:5], None, None, dout, None)
    got = binding.kda_gdr_backward(*gpu(x[:5]), None, None, dout.cuda(), None, want_dstate_in=False)
    assert got[5] is None
    for name, a, b in zip(NAMES[:5], got, want):
        assert off(a, b) <= bar(dtype, 50), name


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("g", [0.0, -3.0, -60.0, -math.inf])
def test_backward_decays_from_none_to_full(g, dtype):
    x, dout, ds = case(1, 90, 1, 2, 128, 128, dtype, 8, g=g)
    want = ref.backward(*x[:5], x[5], None, dout, ds)
    got = binding.kda_gdr_backward(*gpu(x[:6]), None, dout.cuda(), ds.cuda())
    for name, a, b in zip(NAMES, got, want):
        assert torch.isfinite(a).all(), name
        if name == "dg" and g < -10:      # exp(g) of anything: nothing to fp32
            assert float(a.abs().max()) <= 1e-6
        elif g > -10 or name != "dstate_in":
            assert off(a, b) <= (bar(F32, 90) if name == "dstate_in" else bar(dtype, 90)), name


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_zero_beta_and_zero_keys(dtype):
    """beta = 0 needs no division: its gradient is that of the formula."""
    x, dout, ds = case(1, 80, 1, 2, 64, 64, dtype, 6)
    x[4][:, ::3] = 0
    x[1][:, 10] = 0
    want = ref.backward(*x[:5], x[5], None, dout, ds)
    got = binding.kda_gdr_backward(*gpu(x[:6]), None, dout.cuda(), ds.cuda())
    for name, a, b in zip(NAMES, got, want):
        assert off(a, b) <= (bar(F32, 80) if name == "dstate_in" else bar(dtype, 80)), name
    assert (got[2][:, ::3] == 0).all()


@pytest.mark.parametrize("beta,length", [(2.0, 1.0), (4.0, 0.5)])
def test_backward_at_the_edge_of_stability(beta, length):
    """The largest beta |k|^2 (2, equal keys, no decay) and the largest beta that the bf16 call takes."""
    x, dout, ds = case(1, 96, 1, 2, 128, 128, BF, 7, g=0.0)
    x[1] = torch.zeros_like(x[1])
    x[1][..., 0] = length
    x[4] = torch.full_like(x[4], beta)
    want = ref.backward(*x[:5], x[5], None, dout, ds)
    got = binding.kda_gdr_backward(*gpu(x[:6]), None, dout.cuda(), ds.cuda())
    for name, a, b in zip(NAMES, got, want):
        assert off(a, b) <= (bar(F32, 96) if name == "dstate_in" else bar(BF, 96)), name


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 30])
def test_backward_is_independent_of_the_gradients_magnitude(scale):
    x, dout, ds = case(1, 75, 1, 2, 128, 128, BF, 7)
    base = binding.kda_gdr_backward(*gpu(x[:6]), None, dout.cuda(), ds.cuda())
    got = binding.kda_gdr_backward(*gpu(x[:6]), None, (dout * scale).cuda(), (ds * scale).cuda())
    for a, b in zip(got, base):
        assert torch.equal(a.float(), b.float() * scale)


def test_rows_outside_every_sequence_and_repeated_calls():
    x, dout, ds = case(1, 128, 2, 4, 128, 128, BF, 9, [40, 0, 50])
    first = binding.kda_gdr_backward(*gpu(x), dout.cuda(), ds.cuda())
    y = [t if i > 4 else t.clone() for i, t in enumerate(x)]
    for t in y[:5] + [dout]:
        t[:, 90:] = float("nan")
    again = binding.kda_gdr_backward(*gpu(y), dout.cuda(), ds.cuda())
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    for a in first[:5]:
        assert (a[:, 90:] == 0).all()


def test_gradients_against_differences():
    """Central differences of the loss, formed from the recurrence in 64 bits, along random directions."""
    x, dout, ds = case(1, 40, 1, 2, 64, 64, F32, 12)
    got = binding.kda_gdr_backward(*gpu(x[:6]), None, dout.cuda(), ds.cuda())
    gen = torch.Generator().manual_seed(3)
    base = [t.double() for t in x[:6]]

    def loss(v):
        o, s = ref.forward(*v)
        return float((o * dout.double()).sum() + (s * ds.double()).sum())

    for i, gr in enumerate(got):
        way = torch.randn(base[i].shape, generator=gen).double()
        ends = [loss([b + sgn * 1e-5 * way if j == i else b for j, b in enumerate(base)]) for sgn in (1, -1)]
        diff, have = (ends[0] - ends[1]) / 2e-5, float((gr.cpu().double() * way).sum())
        size = float(gr.cpu().double().norm() * way.norm())
        # the difference's own error: its third derivative times (1e-5)^2, and 2^-52 of the loss over 1e-5
        assert abs(diff - have) <= (bar(F32, 40) + 1e-7) * size, NAMES[i]


def test_autograd_and_one_training_run():
    """The ops as a model uses them: gated delta rule, then block norm, gradients to every leaf."""
    x, _, _ = case(1, 66, 1, 2, 64, 64, F32, 14)
    leaves = [t.cuda().requires_grad_(True) for t in x[:6]]
    gen = torch.Generator().manual_seed(2)
    res, gate = (torch.randn(1, 66, 128, generator=gen).cuda().requires_grad_(True) for _ in range(2))
    w = [torch.ones(128, device="cuda", requires_grad=True) for _ in range(2)]
    o, s = binding.kda_gdr_autograd(*leaves)
    xn, h = binding.kda_block_norm_autograd(res, o.flatten(2), gate, *w, 0.5)
    (xn.square().sum() + h.sum() + s.sum()).backward()

    cpu = [t.detach().cpu().double().requires_grad_(True) for t in leaves]
    rest = [t.detach().cpu().double().requires_grad_(True) for t in (res, gate, *w)]
    oo, ss = ref.forward(*cpu)
    y = oo.flatten(2)
    n = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6) * rest[2]
    x2 = rest[0] + 0.5 * n * torch.sigmoid(rest[1])
    h2 = x2 / torch.sqrt(x2.pow(2).mean(-1, keepdim=True) + 1e-6) * rest[3]
    (x2.square().sum() + h2.sum() + ss.sum()).backward()
    for a, b in zip(leaves + [res, gate, *w], cpu + rest):
        assert off(a.grad, b.grad) <= 10 * bar(F32, 66)


def test_backward_captured_and_replayed():
    x, dout, ds = case(1, 150, 1, 2, 128, 128, BF, 15, [90, 60])
    d, do, dso = gpu(x), dout.cuda(), ds.cuda()
    want = binding.kda_gdr_backward(*d, do, dso)
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):                 # two graphs, each with a workspace of its own
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = binding.kda_gdr_backward(*d, do, dso)
            graphs.append((graph, out))
    torch.cuda.synchronize()
    for _ in range(2):
        for graph, out in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_backward_of_no_tokens_passes_the_state_gradient():
    x, dout, ds = case(2, 0, 1, 2, 64, 64, BF, 1)
    got = binding.kda_gdr_backward(*gpu(x[:6]), None, dout.cuda(), ds.cuda())
    assert torch.equal(got[5].cpu(), ds) and got[0].numel() == 0
    x, dout, ds = case(1, 4, 1, 2, 64, 64, F32, 1, [0, 0])
    got = binding.kda_gdr_backward(*gpu(x), dout.cuda(), ds.cuda())
    assert torch.equal(got[5].cpu(), ds) and (got[0] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_backward_of_many_short_sequences(dtype):
    lengths = [i % 3 for i in range(700)]
    x, dout, ds = case(1, sum(lengths), 1, 1, 64, 64, dtype, 5, lengths)
    want = ref.backward(*x[:5], x[5], x[6], dout, ds)
    got = binding.kda_gdr_backward(*gpu(x), dout.cuda(), ds.cuda())
    for name, a, b in zip(NAMES, got, want):
        assert off(a, b) <= (bar(F32, 2) if name == "dstate_in" else bar(dtype, 2)), name


def test_backward_of_bad_offsets_stays_inside_the_tensors():
    x, dout, ds = case(1, 128, 1, 2, 64, 64, BF, 6, [40, 40, 48])
    d = gpu(x)
    d[6] = torch.tensor([0, 90, 30, 500], dtype=torch.int32).cuda()
    got = binding.kda_gdr_backward(*d, dout.cuda(), ds.cuda())
    d[6] = torch.tensor([0, 90, 90, 128], dtype=torch.int32).cuda()
    want = binding.kda_gdr_backward(*d, dout.cuda(), ds.cuda())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_one_token_without_a_state_has_no_decay_gradient(dtype):
    """The decay of a sequence's first token multiplies a state of zeros: its gradient is exactly zero,
    and dg is not formed as a difference that would leave roundings there."""
    x, dout, ds = case(3, 1, 2, 4, 128, 128, dtype, 31, state=False)
    got = binding.kda_gdr_backward(*gpu(x), dout.cuda(), ds.cuda())
    assert (got[3] == 0).all()
    want = ref.backward(*x[:5], None, None, dout, ds)
    for name, a, b in zip(NAMES, got, want):
        assert off(a, b) <= (bar(F32, 1) if name == "dstate_in" else bar(dtype, 1)), name


def test_second_derivatives_are_refused_not_dropped():
    """The gradients say so when a second derivative is taken through them; alone they can be used on."""
    x, _, _ = case(1, 20, 1, 2, 64, 64, F32, 42)
    leaves = [t.cuda().requires_grad_(True) for t in x[:6]]
    o, s = binding.kda_gdr_autograd(*leaves)
    grads = torch.autograd.grad(o.sum() + s.sum(), leaves, create_graph=True)
    plain = torch.autograd.grad(sum(t.sum() for t in binding.kda_gdr_autograd(*leaves)), leaves)
    assert all(torch.equal(p, q) for p, q in zip(grads, plain))
    with pytest.raises(RuntimeError, match="second derivative"):
        (o.sum() + grads[0].square().sum()).backward()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gradients_that_arrive_at_odd_addresses(dtype):
    """What autograd hands over may be a slice of a larger gradient, at any element."""
    x, dout, ds = case(1, 40, 1, 2, 64, 64, dtype, 41)
    leaves = [t.cuda().requires_grad_(True) for t in x[:6]]
    o, s = binding.kda_gdr_autograd(*leaves)
    head = torch.ones(3, dtype=dtype, device="cuda", requires_grad=True)
    both, states = torch.cat([head, o.flatten()]), torch.cat([head.float(), s.flatten()])
    torch.autograd.backward([both, states], [torch.cat([torch.zeros(3, dtype=dtype), dout.flatten()]).cuda(),
                                             torch.cat([torch.zeros(3), ds.flatten()]).cuda()])
    want = binding.kda_gdr_backward(*gpu(x[:6]), None, dout.cuda(), ds.cuda())
    assert all(torch.equal(a.grad, b) for a, b in zip(leaves, want))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("g", [-100.0, -math.inf])
def test_backward_through_full_forgetting_is_exactly_nothing(g, dtype):
    """Nothing passes a token that forgets: not the state gradient behind it, however large, and not the state
    before it; and its decay has no gradient."""
    x, dout, ds = case(1, 40, 1, 2, 64, 64, dtype, 43)
    x[3][:, 20] = g
    x[5] = x[5] * 1e18                             # <S, Z> stays a number
    got = binding.kda_gdr_backward(*gpu(x[:6]), None, torch.zeros_like(dout).cuda(), (ds * 1e18).cuda())
    assert (got[5] == 0).all()
    if dtype == F32:      # in bf16 dg is a sum over the block, whose other tokens' shares cancel to their roundings
        assert (got[3][:, :21] == 0).all()
    for a in (got[1], got[2], got[4]):
        assert (a[:, :20] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_backward_of_a_nan_decay_shows_it(dtype):
    x, dout, ds = case(1, 100, 2, 4, 64, 64, dtype, 44, [50, 50])
    clean = binding.kda_gdr_backward(*gpu(x), dout.cuda(), ds.cuda())
    x[3][0, 60, 1] = float("nan")
    got = binding.kda_gdr_backward(*gpu(x), dout.cuda(), ds.cuda())
    assert torch.isnan(got[3][0, 50:61, 1]).any() and torch.isnan(got[5][1, 1]).any()
    keep = [0, 2, 3]                               # other heads, and the other sequence
    for i in (2, 3, 4):
        assert torch.equal(got[i][0, :50], clean[i][0, :50]) and torch.equal(got[i][0, :, keep], clean[i][0, :, keep])
    assert torch.equal(got[5][0], clean[5][0]) and torch.equal(got[5][1, keep], clean[5][1, keep])
    for i in (0, 1):                               # key head 1 has value heads 2 and 3
        assert torch.equal(got[i][0, :50], clean[i][0, :50]) and torch.equal(got[i][0, :, 1], clean[i][0, :, 1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("g", [-60.0, -math.inf])
def test_state_gradient_through_strong_decay(g, dtype):
    """What reaches the state before 90 tokens: a share of exp(-60) of the first token's, or nothing."""
    x, dout, ds = case(1, 90, 1, 2, 128, 128, dtype, 8, g=g)
    want = ref.backward(*x[:5], x[5], None, dout, ds)[5]
    got = binding.kda_gdr_backward(*gpu(x[:6]), None, dout.cuda(), ds.cuda())[5]
    assert off(got, want) <= bar(F32, 90) and float(got.abs().max()) <= 1e-20


@pytest.mark.parametrize("shape", [(1, 300, 2, 4, 128, 128), (2, 130, 1, 2, 64, 128), (1, 200, 2, 2, 128, 64)],
                         ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("dout_size,ds_size,g", [(1.0, 0.3, None), (2.0 ** -10, 1.0, -0.01), (1.0, 0.0, None), (0.0, 1.0, -0.01)])
def test_bf16_gradients_are_off_by_their_rounding(shape, dout_size, ds_size, g):
    """A bar for sums of many independent roundings, also where dg is the state's share alone (little or no dout,
    slow decay).  A rounding to bf16 is uniform in half a step, 2^-8 of a value at most: its RMS is 2^-8 / sqrt 3 at
    most.  The six products of a gradient have two operands each with fp16 roundings of RMS 2^-11 / sqrt 3, and may
    cancel by a factor of two: sqrt(12) x 2 x 2^-11 / sqrt 3.  Together sqrt(2^-16 / 3 + 48 x 2^-22 / 3) = 3.0e-3."""
    B, T, Hk, H, dk, dv = shape
    x, dout, ds = case(B, T, Hk, H, dk, dv, BF, T + 1, **({} if g is None else dict(g=g)))
    dout, ds = dout * dout_size, ds * ds_size
    want = ref.backward(*x[:5], x[5], None, dout, ds)
    got = binding.kda_gdr_backward(*gpu(x[:6]), None, dout.cuda(), ds.cuda())
    for name, a, b in zip(NAMES, got, want):
        limit = bar(F32, T) if name == "dstate_in" else math.sqrt(2.0 ** -16 / 3 + 48 * 2.0 ** -22 / 3)
        assert off(a, b) <= limit, (name, off(a, b))
