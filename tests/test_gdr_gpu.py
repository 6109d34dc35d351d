"""The gated delta rule on the GPU against the recurrence in 64 bits.

Tolerances, in units of the reference's RMS over the tensor (2-norm of the difference over
2-norm of the reference):
 * o in bf16: rounding to bf16 is off by at most torch.finfo(bf16).eps / 2 = 2^-8 of each
   value; what the kernel rounds before (S, beta N and P to fp16, 2^-11 each at most)
   adds at most 3 x 2^-11 of the terms' magnitude, and the terms of o are at most a few times
   o itself: 2^-8 + 4 x 3 x 2^-11 = 2.5 x 2^-8.
 * o in fp32 and the states: each token's step rounds a few times to 2^-24, errors decay with
   the state; over T tokens they add up like a random walk at worst: 2^-24 x 8 sqrt(T) with
   8 roundings a token, but never below 1e-6 (the split operands' 2^-22).
"""
import math

import pytest
import torch

import _gdr_reference as ref
from kda_delta_rule_chunkwise_b200 import binding

BF, F32 = torch.bfloat16, torch.float32
pytestmark = pytest.mark.gpu


def off(got, want):
    got, want = got.detach().cpu().double(), want.double()
    live = ~torch.isnan(want)
    got, want = got[live], want[live]
    assert torch.isfinite(got).all()
    d = (got - want).norm()
    return float(d / want.norm()) if float(want.norm()) else float(d)


def tol_o(dtype, T):
    return 2.5 * 2.0 ** -8 if dtype == BF else tol_state(T)


def tol_state(T):
    return max(1e-6, 2.0 ** -24 * 8 * math.sqrt(max(T, 1)))


def gpu(ts):
    return [None if t is None else t.cuda() for t in ts]


CASES = [  # B, T, Hk, H, dk, dv, lengths
    (1, 1, 1, 1, 64, 64, None), (1, 31, 2, 2, 128, 128, None), (2, 32, 1, 4, 64, 128, None),
    (3, 33, 2, 4, 128, 64, None), (1, 257, 2, 6, 128, 128, None), (2, 100, 3, 3, 64, 64, None),
    (1, 300, 2, 4, 128, 128, [0, 1, 31, 32, 33, 0, 64, 139]),
    (1, 211, 1, 2, 64, 128, [100, 0, 110]),            # one row behind the last sequence
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:6])) + ("p" if c[6] else ""))
def test_prefill_matches_the_recurrence(case, dtype):
    B, T, Hk, H, dk, dv, lengths = case
    x = ref.inputs(B, T, Hk, H, dk, dv, dtype, seed=T, lengths=lengths)
    want_o, want_s = ref.forward(*x)
    d = gpu(x)
    o = torch.full((B, T, H, dv), 7.0, dtype=dtype, device="cuda")
    got_o, got_s = binding.kda_gdr_chunk_prefill(*d, o=o)
    assert binding.kda_check_device_error() == binding.KDA_OK
    assert off(got_o, want_o) <= tol_o(dtype, T)
    assert off(got_s, want_s) <= tol_state(T)
    outside = torch.isnan(want_o)
    assert (got_o.cpu()[outside] == 7.0).all()             # rows of no sequence stay as they were


@pytest.mark.parametrize("H,dv", [(1, 128), (37, 128), (38, 128), (75, 128), (148, 128), (150, 128), (75, 64), (160, 64)])
def test_prefill_variants_by_unit_count(H, dv):
    """Each split of the columns over CTAs and warps (the choice goes by N H and dv)."""
    x = ref.inputs(1, 70, 1, H, 128, dv, BF, seed=H)
    want_o, want_s = ref.forward(*x)
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    assert off(o, want_o) <= tol_o(BF, 70) and off(s, want_s) <= tol_state(70)


def test_prefill_without_states_and_in_place():
    x = ref.inputs(2, 65, 2, 4, 128, 128, BF, seed=5, state=False)
    want_o, want_s = ref.forward(*x)
    d = gpu(x)
    o, none = binding.kda_gdr_chunk_prefill(*d, want_state=False)
    assert none is None and off(o, want_o) <= tol_o(BF, 65)
    state = torch.zeros(2, 4, 128, 128, device="cuda")
    d[5] = state
    o2, s = binding.kda_gdr_chunk_prefill(*d, state_out=state)
    assert s is state and torch.equal(o, o2) and off(state, want_s) <= tol_state(65)


@pytest.mark.parametrize("g", [0.0, -1e-6, -5.0, -30.0, -100.0, -1e4, -math.inf])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_prefill_decays_from_none_to_full(g, dtype):
    """Any decay down to -infinity, which forgets all before the token."""
    x = ref.inputs(1, 90, 1, 2, 128, 128, dtype, seed=9, g=g)
    want_o, want_s = ref.forward(*x)
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    assert off(o, want_o) <= tol_o(dtype, 90) and off(s, want_s) <= tol_state(90)


def test_prefill_full_forgetting_among_slow_tokens():
    """Single tokens of g = -100 and -infinity between slow ones: decays of rows behind them stay exact."""
    x = ref.inputs(1, 130, 1, 2, 128, 128, BF, seed=10)
    x[3][:, 5::17] = -math.inf
    x[3][:, 9::23] = -100.0
    want_o, want_s = ref.forward(*x)
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    assert off(o, want_o) <= tol_o(BF, 130) and off(s, want_s) <= tol_state(130)


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -20, 2.0 ** 40])
def test_prefill_is_independent_of_the_values_magnitude(scale):
    """Values and state times a power of two: o and the state times it, since operands are scaled per row."""
    x = ref.inputs(1, 77, 1, 2, 128, 128, BF, seed=11)
    base_o, base_s = binding.kda_gdr_chunk_prefill(*gpu(x))
    x[2], x[5] = x[2] * scale, x[5] * scale
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    assert torch.equal(o.float(), base_o.float() * scale) and torch.equal(s, base_s * scale)


def test_prefill_of_long_small_and_large_keys():
    """Keys that are not unit vectors (beta |k|^2 < 2 keeps the rule stable), zero keys among them."""
    x = ref.inputs(1, 96, 1, 2, 128, 128, BF, seed=12)
    x[1] = (x[1].float() * torch.rand(1, 96, 1, 1, generator=torch.Generator().manual_seed(1)) * 1.3).to(BF)
    x[1][:, 7] = 0
    x[0] = x[0] * 1000
    x[0][:, 11] = 0
    want_o, want_s = ref.forward(*x)
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    assert off(o, want_o) <= tol_o(BF, 96) and off(s, want_s) <= tol_state(96)
    assert (o[:, 11] == 0).all()


@pytest.mark.parametrize("keys", ["equal", "unequal lengths"])
def test_prefill_at_the_edge_of_stability(keys):
    """beta |k|^2 = 2 without decay (each step a reflection), where (I + A)^-1 is largest: equal keys
    e_0, and unit axes of lengths 2^-3 to 2^3 (beta |k_r| |k_s| up to 2^7).  The states' errors are
    2^-22 of elements that sum to N itself, so the tolerance is that of any states."""
    x = ref.inputs(1, 96, 1, 2, 128, 128, BF, seed=21, g=0.0)
    length = torch.ones(96) if keys == "equal" else 2.0 ** ((torch.arange(96) * 5) % 7 - 3)
    x[1] = torch.zeros_like(x[1])
    x[1][0, torch.arange(96), 0, 0 if keys == "equal" else torch.arange(96) % 3] = length.to(BF)
    x[4] = (2.0 / length ** 2)[None, :, None].expand(1, 96, 2).to(BF).contiguous()
    x[2] = (x[2].float() * length[None, :, None, None]).to(BF)
    want_o, want_s = ref.forward(*x)
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    assert off(o, want_o) <= tol_o(BF, 96) and off(s, want_s) <= tol_state(96)


def test_prefill_nan_stays_in_its_sequence_and_head():
    x = ref.inputs(1, 120, 2, 4, 128, 128, BF, seed=13, lengths=[50, 70])
    clean = binding.kda_gdr_chunk_prefill(*gpu(x))
    y = [None if t is None else t.clone() for t in x]
    y[2][0, 60, 1] = float("nan")
    o, s = binding.kda_gdr_chunk_prefill(*gpu(y))
    keep = torch.ones(1, 120, 4, dtype=torch.bool)
    keep[0, 50:, 1] = False
    assert torch.equal(o[keep.cuda()], clean[0][keep.cuda()])
    assert torch.isnan(s[1, 1]).any() and torch.equal(s[0], clean[1][0]) and torch.equal(s[1, 0], clean[1][1, 0])


def test_prefill_ignores_what_lies_behind_a_sequence():
    """NaN rows behind the last sequence, inside its last chunk, reach nothing."""
    x = ref.inputs(1, 64, 1, 2, 128, 128, BF, seed=14, lengths=[33])
    want = binding.kda_gdr_chunk_prefill(*gpu(x))
    y = [t if i > 4 or t is None else t.clone() for i, t in enumerate(x)]
    for t in y[:5]:
        t[:, 33:] = float("nan")
    got = binding.kda_gdr_chunk_prefill(*gpu(y))
    assert torch.equal(got[0][:, :33], want[0][:, :33]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("cu", [[0, 40, 20, 90], [-5, 30, 500, 60], [90, 10, 0, 64]])
def test_prefill_bad_offsets_stay_inside_the_tensors(cu):
    """Offsets are clamped and made non-decreasing; the good prefix keeps its results."""
    x = ref.inputs(1, 64, 1, 2, 64, 64, BF, seed=15, lengths=[20, 20, 24])
    x[6] = torch.tensor(cu, dtype=torch.int32)
    fixed, top = [], 0
    for c in cu:
        top = max(top, min(max(c, 0), 64))
        fixed.append(top)
    d = gpu(x)
    got = binding.kda_gdr_chunk_prefill(*d)
    d[6] = torch.tensor(fixed, dtype=torch.int32).cuda()
    want = binding.kda_gdr_chunk_prefill(*d)
    torch.cuda.synchronize()
    rows = slice(fixed[0], fixed[-1])
    assert torch.equal(got[1], want[1]) and torch.equal(got[0][:, rows], want[0][:, rows])


def test_prefill_two_calls_are_equal_and_can_be_captured():
    x = gpu(ref.inputs(1, 200, 2, 4, 128, 128, BF, seed=16, lengths=[150, 50]))
    want = binding.kda_gdr_chunk_prefill(*x)
    again = binding.kda_gdr_chunk_prefill(*x)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    o, s = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            binding.kda_gdr_chunk_prefill(*x, o=o, state_out=s)
    for _ in range(2):
        o.zero_(), s.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(s, want[1])


def test_prefill_on_two_streams_at_once():
    xs = [gpu(ref.inputs(1, 400, 1, 8, 128, 128, BF, seed=20 + i)) for i in range(2)]
    want = [binding.kda_gdr_chunk_prefill(*x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for x, st in zip(xs, streams):
        with torch.cuda.stream(st):
            got.append(binding.kda_gdr_chunk_prefill(*x))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


# ------------------------------------------------------------------------- decode

def decode_reference(x, state, slots=None, lens=None):
    q, k, v, g, beta = x[:5]
    N, L = q.shape[:2]
    pool, o = state.double().clone(), torch.full(v.shape, float("nan"), dtype=torch.float64)
    for n in range(N):
        at = n if slots is None else int(slots[n])
        m = L if lens is None else max(0, min(L, int(lens[n])))
        if m == 0 or not 0 <= at < pool.shape[0]:
            continue
        on, s = ref.forward(*(t[n:n + 1, :m] for t in x[:5]), pool[at:at + 1])
        o[n, :m], pool[at] = on[0], s[0]
    return o, pool


DECODES = [  # N, L, Hk, H, dk, dv, pool, lens
    (1, 1, 1, 1, 64, 64, 0, None), (1, 1, 4, 16, 128, 128, 0, None), (40, 1, 2, 8, 128, 128, 0, None),
    (5, 1, 2, 2, 64, 128, 9, None), (3, 4, 1, 4, 128, 64, 0, None), (30, 5, 4, 8, 128, 128, 37, [0, 1, 5, 9, -3, 2]),
    (2, 33, 1, 2, 128, 128, 0, [33, 17]),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", DECODES, ids=lambda c: "x".join(map(str, c[:6])))
def test_decode_matches_the_recurrence(case, dtype):
    N, L, Hk, H, dk, dv, P, lens = case
    x = ref.inputs(N, L, Hk, H, dk, dv, dtype, seed=N + L, state=False)[:5]
    gen = torch.Generator().manual_seed(3)
    state = torch.randn(P or N, H, dk, dv, generator=gen) * 0.1
    slots = torch.randperm(P, generator=gen)[:N].to(torch.int32) if P else None
    lens = None if lens is None else torch.tensor([lens[i % len(lens)] for i in range(N)], dtype=torch.int32)
    want_o, want_s = decode_reference(x, state, slots, lens)
    s = state.cuda()
    o = torch.full((N, L, H, dv), 7.0, dtype=dtype, device="cuda")
    kw = dict(slots=None if slots is None else slots.cuda(), lens=None if lens is None else lens.cuda())
    scored = binding.kda_gdr_decode(*gpu(x), s, o=o.clone(), update_state=False, **kw)
    assert torch.equal(s.cpu(), state)                      # nothing updated
    got = binding.kda_gdr_decode(*gpu(x), s, o=o, **kw)
    assert torch.equal(scored, got)
    # one rounding to bf16 of a sum that is exact to fp32: 2^-8 of each value at most
    assert off(got, want_o) <= (2.0 ** -8 if dtype == BF else tol_state(L))
    assert off(s, want_s) <= tol_state(L)
    outside = torch.isnan(want_o)
    assert (got.cpu()[outside] == 7.0).all()
    untouched = (want_s == state.double()).all(-1).all(-1).all(-1)
    assert torch.equal(s.cpu()[untouched], state[untouched])


def test_decode_skips_slots_outside_the_pool():
    x = ref.inputs(4, 1, 1, 2, 128, 128, BF, seed=1, state=False)[:5]
    state = torch.randn(6, 2, 128, 128, generator=torch.Generator().manual_seed(2))
    slots = torch.tensor([5, -1, 6, 0], dtype=torch.int32)
    want_o, want_s = decode_reference(x, state, slots)
    s, o = state.cuda(), torch.full((4, 1, 2, 128), 7.0, dtype=BF, device="cuda")
    binding.kda_gdr_decode(*gpu(x), s, slots=slots.cuda(), o=o)
    assert binding.kda_check_device_error() == binding.KDA_ERR_INVALID_ARG
    assert binding.kda_check_device_error() == binding.KDA_OK
    assert (o[1:3] == 7.0).all() and off(o[[0, 3]], want_o[[0, 3]]) <= 2.0 ** -8
    assert off(s, want_s) <= 1e-6 and torch.equal(s[1:5].cpu(), state[1:5])


def test_prefill_then_decode_is_one_long_prefill():
    """Serving: a prompt, three tokens, a drafted run scored and then committed in part."""
    x = ref.inputs(2, 80, 2, 4, 128, 128, BF, seed=30)
    want_o, want_s = ref.forward(*x)
    d = gpu(x)
    cut = lambda a, e: [t[:, a:e].contiguous() for t in d[:5]]
    o, s = binding.kda_gdr_chunk_prefill(*cut(0, 70), d[5])
    parts = [o]
    for t in range(70, 73):
        parts.append(binding.kda_gdr_decode(*cut(t, t + 1), s))
    draft = cut(73, 80)
    scored = binding.kda_gdr_decode(*draft, s, update_state=False)
    parts.append(scored)
    taken = torch.tensor([7, 4], dtype=torch.int32, device="cuda")
    binding.kda_gdr_decode(*draft, s, lens=taken)
    assert off(torch.cat(parts, 1), want_o) <= tol_o(BF, 80)
    short = ref.forward(*(t[1:, :77] for t in x[:5]), x[5][1:])[1]
    assert off(s[0], want_s[0]) <= tol_state(80) and off(s[1], short[0]) <= tol_state(77)


def test_prefill_of_no_tokens_keeps_the_states():
    x = ref.inputs(2, 0, 1, 2, 64, 64, BF, seed=1)
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    assert o.shape == (2, 0, 2, 64) and torch.equal(s.cpu(), x[5])
    x = ref.inputs(1, 5, 1, 2, 64, 64, BF, seed=1, lengths=[0, 0, 0])
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    assert torch.equal(s.cpu(), x[5])
    assert (binding.kda_gdr_autograd(*gpu(x))[0] == 0).all()      # no row belongs to a sequence


def test_prefill_of_many_short_sequences():
    """More sequences than are sorted by length (4096), zero to two tokens each."""
    lengths = [i % 3 for i in range(4200)]
    x = ref.inputs(1, sum(lengths), 1, 1, 64, 64, BF, seed=2, lengths=lengths)
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    want_o, want_s = ref.forward(*x)
    assert off(o, want_o) <= tol_o(BF, 2) and off(s, want_s) <= tol_state(2)


@pytest.mark.parametrize("lengths", [[5, 300, 40, 300, 0, 1], [1] * 33 + [200]])
def test_prefill_result_does_not_depend_on_the_neighbours(lengths):
    """A sequence alone and packed among others: the same bits, whatever order they run in."""
    x = ref.inputs(1, sum(lengths), 1, 2, 128, 128, BF, seed=3, lengths=lengths)
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    at = 0
    for n, m in enumerate(lengths):
        alone = gpu([t[:, at:at + m].contiguous() for t in x[:5]] + [x[5][n:n + 1].contiguous(), None])
        oo, ss = binding.kda_gdr_chunk_prefill(*alone)
        # the columns may be split over another number of warps: sums of channel halves differ in order
        if m:
            assert off(o[:, at:at + m], oo.cpu().double()) <= 2.0 ** -8
        assert off(s[n], ss[0].cpu().double()) <= 1e-6
        at += m


def test_prefill_with_a_given_workspace_and_on_a_given_stream():
    x = gpu(ref.inputs(1, 100, 2, 4, 128, 64, BF, seed=4, lengths=[60, 40]))
    want = binding.kda_gdr_chunk_prefill(*x)
    need = binding.load().kda_gdr_prefill_workspace_bytes(100, 2, 2, 4, 128, 64, binding.KDA_BF16)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")     # NaN patterns; a larger one
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.kda_gdr_chunk_prefill(*x, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (ws[need:] == 255).all()


def test_decode_captured_and_replayed_moves_the_states_on():
    x = gpu(ref.inputs(3, 1, 1, 2, 128, 128, BF, seed=5, state=False)[:5])
    a = torch.randn(3, 2, 128, 128, generator=torch.Generator().manual_seed(1)).cuda()
    b = a.clone()
    o = torch.zeros(3, 1, 2, 128, dtype=BF, device="cuda")
    want = [binding.kda_gdr_decode(*x, a).clone() for _ in range(3)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            binding.kda_gdr_decode(*x, b, o=o)
    torch.cuda.synchronize()
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, w)
    assert torch.equal(a, b)


@pytest.mark.parametrize("N,L,dv", [(200, 8, 128), (2, 64, 128), (300, 16, 64), (9, 31, 64)])
def test_decode_of_many_tokens_is_decode_of_one_after_another(N, L, dv):
    """All tokens in one call, many CTAs on an SM, and each in a call of its own: the same bits, every time."""
    x = gpu(ref.inputs(N, L, 2, 4, 128, dv, BF, seed=N, state=False)[:5])
    start = torch.randn(N, 4, 128, dv, generator=torch.Generator().manual_seed(L)).cuda()
    one = start.clone()
    parts = [binding.kda_gdr_decode(*[t[:, i:i + 1].contiguous() for t in x], one) for i in range(L)]
    want = torch.cat(parts, 1)
    for _ in range(5):
        state = start.clone()
        o = binding.kda_gdr_decode(*x, state)
        assert torch.equal(o, want) and torch.equal(state, one)


def test_lens_and_slots_on_the_host_are_refused():
    x = gpu(ref.inputs(2, 1, 1, 2, 64, 64, BF, seed=6, state=False)[:5])
    s = torch.zeros(2, 2, 64, 64, device="cuda")
    for kw in (dict(slots=torch.zeros(2, dtype=torch.int32)), dict(lens=torch.zeros(2, dtype=torch.int64, device="cuda")),
               dict(slots=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(o=torch.zeros(2, 1, 2, 64, device="cuda"))):
        with pytest.raises(ValueError):
            binding.kda_gdr_decode(*x, s, **kw)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("g", [-100.0, -1e4, -math.inf])
def test_full_forgetting_leaves_nothing_of_any_state(g, dtype):
    """exp(-100) is 3.7e-44, which is something beside a large state: a token of -100 or less leaves zeros."""
    x = ref.inputs(1, 40, 1, 2, 128, 64, dtype, seed=17)
    x[2], x[5] = torch.zeros_like(x[2]), torch.full_like(x[5], 1e36)
    x[3][:, 20] = g
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    assert (s == 0).all() and (o[:, 20:] == 0).all()
    d, state = gpu([t[:, 20:23].contiguous() for t in x[:5]]), x[5].cuda()
    assert (binding.kda_gdr_decode(*d, state) == 0).all() and (state == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_nan_decay_shows_in_its_sequence_and_head(dtype):
    x = ref.inputs(1, 100, 1, 3, 128, 64, dtype, seed=18, lengths=[40, 60])
    clean = binding.kda_gdr_chunk_prefill(*gpu(x))
    x[3][0, 75, 1] = float("nan")
    o, s = binding.kda_gdr_chunk_prefill(*gpu(x))
    assert torch.isnan(o[0, 75:, 1]).all() and torch.isnan(s[1, 1]).all()
    keep = torch.ones(1, 100, 3, dtype=torch.bool)
    keep[0, 72:, 1] = False                       # 72: the start of the token's chunk
    assert torch.equal(o[keep.cuda()], clean[0][keep.cuda()])
    assert torch.equal(s[0], clean[1][0]) and torch.equal(s[1, [0, 2]], clean[1][1, [0, 2]])
    d, state = gpu([t[:, 74:77].contiguous() for t in x[:5]]), torch.ones(1, 3, 128, 64, device="cuda")
    o = binding.kda_gdr_decode(*d, state)
    assert torch.isnan(o[0, 1:, 1]).all() and torch.isnan(state[0, 1]).all()
    assert torch.isfinite(o[0, :, [0, 2]]).all() and torch.isfinite(state[0, [0, 2]]).all() and torch.isfinite(o[0, 0]).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_the_debug_scan_reports_inputs_outside_the_contract(monkeypatch, dtype):
    """Positive and NaN decays in any call; keys and beta beyond the bf16 limits where they hold."""
    while binding.kda_check_device_error() != binding.KDA_OK:
        pass
    base = gpu(ref.inputs(1, 100, 2, 4, 128, 128, dtype, seed=51, lengths=[30, 0, 60]))
    dout = torch.randn(1, 100, 4, 128, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    want = binding.kda_gdr_chunk_prefill(*base)
    want_back = binding.kda_gdr_backward(*base, dout)
    monkeypatch.setenv("KDA_DEBUG_CHECKS", "1")

    def reports(which, value, at, back=False):
        x = [None if t is None else t.clone() for t in base]
        x[which][at] = value
        binding.kda_gdr_backward(*x, dout) if back else binding.kda_gdr_chunk_prefill(*x)
        code = binding.kda_check_device_error()
        assert code in (binding.KDA_OK, binding.KDA_ERR_INPUT_RANGE)
        assert binding.kda_check_device_error() == binding.KDA_OK
        return code == binding.KDA_ERR_INPUT_RANGE

    got, back = binding.kda_gdr_chunk_prefill(*base), binding.kda_gdr_backward(*base, dout)
    assert binding.kda_check_device_error() == binding.KDA_OK
    assert torch.equal(got[0][:, :90], want[0][:, :90]) and torch.equal(got[1], want[1])      # nothing changes
    assert all(torch.equal(a, b) for a, b in zip(back, want_back))
    for back in (False, True):
        for bad in (1e-3, float("nan"), math.inf):
            assert reports(3, bad, (0, 89, 3), back) and not reports(3, bad, (0, 90, 3), back)   # 90: of no sequence
        assert not reports(3, -math.inf, (0, 5, 0), back)
        # a unit key times 1.4 is |k|^2 = 1.96, times 1.5 2.25; beta = 1
        one = lambda f: base[1][0, 40, 1] / base[1][0, 40, 1].float().norm().to(dtype) * f
        base[4][0, 40] = 1.0
        assert not reports(1, one(1.4), (0, 40, 1), back) and reports(1, one(1.5), (0, 40, 1), back) == (dtype == BF)
        assert reports(4, -0.1, (0, 40, 2), back) == (dtype == BF)
        # beta_r |k_r| |k_s| = 2^-16 2^8 2^23: each beta |k|^2 is at most 1, their cross term 2^15
        x = [None if t is None else t.clone() for t in base]
        for row, size, b in ((30, 2.0 ** 8, 2.0 ** -16), (31, 2.0 ** 23, 2.0 ** -46)):
            x[1][0, row] = 0
            x[1][0, row, :, 0], x[4][0, row] = size, b
        binding.kda_gdr_chunk_prefill(*x)
        assert (binding.kda_check_device_error() == binding.KDA_ERR_INPUT_RANGE) == (dtype == BF)
    x = [None if t is None else t.clone() for t in base]
    x[1][0, 40], x[4][0, 40] = x[1][0, 40] * 0.1, 5.0
    binding.kda_gdr_chunk_prefill(*x)
    assert binding.kda_check_device_error() == binding.KDA_OK
    binding.kda_gdr_backward(*x, dout)
    assert (binding.kda_check_device_error() == binding.KDA_ERR_INPUT_RANGE) == (dtype == BF)

    d = [t[:, :8].reshape(2, 4, *t.shape[2:]).contiguous() for t in base[:5]]
    state = torch.zeros(2, 4, 128, 128, device="cuda")
    d[3][1, 2, 3] = 0.5
    for lens, code in ((None, binding.KDA_ERR_INPUT_RANGE), ([4, 3], binding.KDA_ERR_INPUT_RANGE), ([4, 2], binding.KDA_OK)):
        binding.kda_gdr_decode(*d, state, lens=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda())
        assert binding.kda_check_device_error() == code
