"""Measured cases of the gated delta rule and the block norm.

The gated delta rule is the delta rule with one retention factor per value head
and token (KDA has one per key channel):

    S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t

with q and k in Hk heads shared by groups of H / Hk value heads.  The block norm
closes one block of a model and opens the next: RMS norm of the block's output y,
its gate, the scaled residual sum, and the RMS norm of that sum:

    x' = x + scale * sigmoid(gate) * norm(y) * w_post,   h = norm(x') * w_pre

Each case is one pass through one operator: `run` with `own` false computes it in
its plain form, with `own` true through this package.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
CHUNK = 64
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one long prompt with the benchmark's head count, q and k shared by pairs of value heads
        dict(name="prefill_h32_t8192", op="prefill", seqs=1, tokens=8192, hk=16, h=32, dk=128, dv=128, dtype="bf16", packed=False),
        # the benchmark's longest prompt
        dict(name="prefill_h32_t65536", op="prefill", seqs=1, tokens=65536, hk=32, h=32, dk=128, dv=128, dtype="bf16", packed=False),
        # a serving step over ragged prompts, each resumed from its own state
        dict(name="prefill_packed_16", op="prefill", seqs=16, tokens=30011, hk=8, h=32, dk=128, dv=128, dtype="bf16", packed=True),
        # the smallest model of the tests, in full precision
        dict(name="prefill_f32_t256", op="prefill", seqs=1, tokens=256, hk=2, h=2, dk=64, dv=64, dtype="f32", packed=False),
        # a full decode batch: one token for each of 256 requests
        dict(name="decode_n256", op="decode", seqs=256, steps=1, hk=16, h=32, dk=128, dv=128, dtype="bf16", pool=0),
        # one user alone: latency counts
        dict(name="decode_n1", op="decode", seqs=1, steps=1, hk=16, h=32, dk=128, dv=128, dtype="bf16", pool=0),
        # up to five accepted tokens for each request, states in a pool
        dict(name="decode_n48_l5_pool", op="decode", seqs=48, steps=5, hk=16, h=32, dk=128, dv=128, dtype="bf16", pool=64),
        # a training step's backward at the benchmark's prefill size
        dict(name="backward_h32_t8192", op="backward", seqs=1, tokens=8192, hk=16, h=32, dk=128, dv=128, dtype="bf16", packed=False),
        # fine-tuning on short packed samples with small heads
        dict(name="backward_packed_9", op="backward", seqs=9, tokens=3001, hk=4, h=8, dk=64, dv=64, dtype="bf16", packed=True),
        # between two blocks, at the prefill's row count and width (32 heads of 128)
        dict(name="norm_8192x4096", op="norm", rows=8192, width=4096, dtype="bf16", xtype="bf16", gate=True),
        # the same for a decode batch, with the residual kept in fp32
        dict(name="norm_256x4096", op="norm", rows=256, width=4096, dtype="bf16", xtype="f32", gate=True),
        # its backward in training
        dict(name="norm_backward_8192x4096", op="norm_backward", rows=8192, width=4096, dtype="bf16", xtype="bf16", gate=True),
    ]


def _log_uniform(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "backward", "norm", "norm_backward"])
    if op in ("norm", "norm_backward"):
        width = rng.choice([_log_uniform(rng, 64, 8192), 8 * _log_uniform(rng, 8, 1024)])
        dtype, xtype = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        return dict(op=op, rows=_log_uniform(rng, 1, min(16384, (1 << 25) // width)), width=width,
                    dtype=dtype, xtype=xtype, gate=rng.random() < 0.7)
    hk = _log_uniform(rng, 1, 16)
    h = hk * rng.choice([1, 2, 4]) if hk <= 8 else hk * rng.choice([1, 2])
    heads = dict(hk=hk, h=h, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                 dtype="f32" if rng.random() < 0.25 else "bf16")
    if op == "decode":
        seqs = _log_uniform(rng, 1, 256)
        return dict(op=op, seqs=seqs, steps=rng.choice([1, 1, 1, rng.randint(2, 8)]),
                    pool=rng.choice([0, seqs + rng.randint(0, 40)]), **heads)
    most = 16384 if op == "prefill" else 6000
    if heads["dtype"] == "f32":
        most //= 8
    packed = rng.random() < 0.5
    if packed:
        return dict(op=op, seqs=rng.randint(2, 24), tokens=_log_uniform(rng, 40, most), packed=True, **heads)
    return dict(op=op, seqs=rng.choice([1, 1, 2, 3]), tokens=_log_uniform(rng, 1, most // 2), packed=False, **heads)


def _lengths(case):
    """Tokens of each sequence: equal for a dense batch, ragged (zero and one among them) when packed."""
    n, tokens = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [tokens] * n
    rng = random.Random(n * 1000003 + tokens)
    cuts = sorted(rng.randint(0, tokens) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
    if n >= 4:  # one empty sequence and one of a single token
        i, j, k = rng.sample(range(n), 3)
        lens[k] += lens[i] + max(0, lens[j] - 1)
        lens[i], lens[j] = 0, min(1, lens[j])
    return lens


# ------------------------------------------------------------------ the inputs

class _Inputs:
    def __init__(self, seed):
        self.gen = torch.Generator(device=DEVICE)
        self.gen.manual_seed(int(seed))

    def normal(self, *shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=self.gen, device=DEVICE) * std).to(dtype)

    def unit(self, *shape, dtype=torch.float32):
        x = torch.randn(*shape, generator=self.gen, device=DEVICE)
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    def tokens(self, rows, case):
        """q, k, v, g, beta of `rows` tokens (a tuple of leading sizes)."""
        t, hk, h = DTYPES[case["dtype"]], case["hk"], case["h"]
        q = self.unit(*rows, hk, case["dk"], dtype=t)
        k = self.unit(*rows, hk, case["dk"], dtype=t)
        v = self.normal(*rows, h, case["dv"], dtype=t)
        # g = -a softplus(x): heads from slow to fast decay, as a gate projection gives it
        a = torch.exp(torch.linspace(math.log(0.02), math.log(2.0), h, device=DEVICE))
        g = (-a * torch.nn.functional.softplus(self.normal(*rows, h))).to(t)
        beta = torch.sigmoid(self.normal(*rows, h)).to(t)
        return q, k, v, g, beta


def prepare(case, seed):
    make, op = _Inputs(seed), case["op"]
    s = dict(case=case)
    if op in ("norm", "norm_backward"):
        rows, d, t, tx = case["rows"], case["width"], DTYPES[case["dtype"]], DTYPES[case["xtype"]]
        s.update(x=make.normal(rows, d, dtype=tx), y=make.normal(rows, d, dtype=t, std=3.0),
                 gate=make.normal(rows, d, dtype=t) if case["gate"] else None,
                 w_post=(1 + make.normal(d, std=0.2)).to(t), w_pre=(1 + make.normal(d, std=0.2)).to(t), scale=0.5)
        if op == "norm_backward":
            s.update(dx_new=make.normal(rows, d, dtype=tx), dh=make.normal(rows, d, dtype=t))
        return s
    n, h, dk, dv = case["seqs"], case["h"], case["dk"], case["dv"]
    if op == "decode":
        s["q"], s["k"], s["v"], s["g"], s["beta"] = make.tokens((n, case["steps"]), case)
        s["state"] = make.normal(case["pool"] or n, h, dk, dv, std=0.1)
        s["slots"] = s["lens"] = None
        if case["pool"]:
            s["slots"] = torch.randperm(case["pool"], generator=make.gen, device=DEVICE)[:n].to(torch.int32)
        if case["steps"] > 1:
            s["lens"] = torch.randint(0, case["steps"] + 1, (n,), generator=make.gen, device=DEVICE).to(torch.int32)
        s["o"] = torch.zeros(n, case["steps"], h, dv, dtype=DTYPES[case["dtype"]], device=DEVICE)
        return s
    lens = _lengths(case)
    rows = (1, sum(lens)) if case["packed"] else (n, case["tokens"])
    s["q"], s["k"], s["v"], s["g"], s["beta"] = make.tokens(rows, case)
    s["cu_seqlens"] = s["state_in"] = s["place"] = None
    if case["packed"]:
        s["state_in"] = make.normal(n, h, dk, dv, std=0.1)
        at = [0]
        for m in lens:
            at.append(at[-1] + m)
        s["cu_seqlens"] = torch.tensor(at, dtype=torch.int32, device=DEVICE)
        s["place"] = _places(lens)
    if op == "backward":
        s["dout"] = make.normal(*rows, h, dv, dtype=DTYPES[case["dtype"]])
        s["dstate_out"] = make.normal(n, h, dk, dv, std=0.3)
    return s


def _places(lens):
    """Row of each packed token in a batch padded to the longest sequence."""
    longest = max(lens)
    return torch.cat([torch.arange(m, device=DEVICE) + i * longest for i, m in enumerate(lens)])


# ------------------------------------------------- plain form: gated delta rule

def _heads_first(s, name, longest, dtype):
    """One input as [N, H, T, ...]: padded with zeros to a multiple of the chunk, key heads repeated for their group."""
    t, case = s[name], s["case"]
    n, h = case["seqs"], case["h"]
    t = t.to(dtype)
    rest = t.shape[2:]
    padded = -(-longest // CHUNK) * CHUNK
    out = torch.zeros(n, padded, *rest, dtype=dtype, device=t.device)
    if s["place"] is None:
        out[:, :longest] = t
    else:
        dense = torch.zeros(n * longest, *rest, dtype=dtype, device=t.device)
        dense[s["place"]] = t[0]
        out[:, :longest] = dense.view(n, longest, *rest)
    out = out.transpose(1, 2)
    return out.repeat_interleave(h // rest[0], dim=1) if rest[0] != h else out


def _tokens_first(s, t, longest, dtype):
    """[N, H, T, ...] back to the layout of the inputs."""
    t = t.transpose(1, 2)[:, :longest]
    if s["place"] is not None:
        t = t.reshape(-1, *t.shape[2:])[s["place"]][None]
    return t.to(dtype).contiguous()


def _chunked(s):
    """The chunks' own terms, all chunks at once: tensors [N, H, chunks, 64, ...] in 32 bits."""
    case = s["case"]
    longest = max(1, max(_lengths(case)))
    c = dict(longest=longest)
    for name in ("q", "k", "v", "g", "beta"):
        t = _heads_first(s, name, longest, torch.float32)
        c[name] = t.reshape(t.shape[0], t.shape[1], -1, CHUNK, *t.shape[3:])
    big = torch.cumsum(c["g"].double(), dim=-1)  # decays of far rows are differences of long sums
    c["G"] = big
    c["into"] = torch.exp(big).float()                      # from the chunk's start to a row
    c["out"] = torch.exp(big[..., -1:] - big).float()       # from a row to the chunk's end
    c["all"] = torch.exp(big[..., -1]).float()
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=big.device).tril()
    c["D"] = torch.exp((big[..., :, None] - big[..., None, :]).masked_fill(~low, -math.inf)).float()
    c["kk"] = c["k"] @ c["k"].transpose(-1, -2)
    c["P"] = c["D"] * (c["q"] @ c["k"].transpose(-1, -2))
    # (I + A)^-1 for the strictly lower A: A^64 = 0, so a product of six factors, in 64 bits
    a = -(c["beta"][..., None] * c["D"] * c["kk"]).tril(-1).double()
    x = a + torch.eye(CHUNK, dtype=a.dtype, device=a.device)
    for _ in range(5):
        a = a @ a
        x = x + x @ a
    c["T"] = (x * c["beta"].double()[..., None, :]).float()
    c["X"] = x.float()
    return c


def _start(s):
    case = s["case"]
    shape = (case["seqs"], case["h"], case["dk"], case["dv"])
    return torch.zeros(shape, device=DEVICE) if s["state_in"] is None else s["state_in"].clone()


def _pass_over_chunks(c, state):
    """U and the read R = v - decayed prediction of each chunk, the state before each chunk, and the last state."""
    us, rs, states = [], [], []
    for i in range(c["k"].shape[2]):
        states.append(state)
        r = c["v"][:, :, i] - c["into"][:, :, i, :, None] * (c["k"][:, :, i] @ state)
        u = c["T"][:, :, i] @ r
        rs.append(r)
        us.append(u)
        state = c["all"][:, :, i, None, None] * state + (c["out"][:, :, i, :, None] * c["k"][:, :, i]).transpose(-1, -2) @ u
    return torch.stack(us, 2), torch.stack(rs, 2), torch.stack(states, 2), state


def _prefill(s):
    c = _chunked(s)
    u, _, states, last = _pass_over_chunks(c, _start(s))
    o = c["into"][..., None] * (c["q"] @ states) + c["P"] @ u
    return _tokens_first(s, o.flatten(2, 3), c["longest"], s["v"].dtype), last


def _backward(s):
    case, c = s["case"], _chunked(s)
    u, r, states, last = _pass_over_chunks(c, _start(s))
    t = _heads_first(s, "dout", c["longest"], torch.float32)
    do = t.reshape(u.shape)
    q, k, into, out, T, P = c["q"], c["k"], c["into"][..., None], c["out"][..., None], c["T"], c["P"]
    z, zs, drs, es = s["dstate_out"], [], [], []
    for i in reversed(range(u.shape[2])):
        zs.append(z)
        du = P[:, :, i].transpose(-1, -2) @ do[:, :, i] + out[:, :, i] * (k[:, :, i] @ z)
        e = c["X"][:, :, i].transpose(-1, -2) @ du
        dr = c["beta"][:, :, i, :, None] * e
        z = c["all"][:, :, i, None, None] * z + (into[:, :, i] * q[:, :, i]).transpose(-1, -2) @ do[:, :, i] \
            - (into[:, :, i] * k[:, :, i]).transpose(-1, -2) @ dr
        drs.append(dr)
        es.append(e)
    zs, dr, e = torch.stack(zs[::-1], 2), torch.stack(drs[::-1], 2), torch.stack(es[::-1], 2)
    dp = c["D"] * (do @ u.transpose(-1, -2))
    eu = (e @ u.transpose(-1, -2)).tril(-1)
    da = -c["beta"][..., None] * c["D"] * eu
    dq = into * (do @ states.transpose(-1, -2)) + dp @ k
    read = -into * (dr @ states.transpose(-1, -2)) + da @ k           # k as the row that reads
    write = out * (u @ zs.transpose(-1, -2)) + dp.transpose(-1, -2) @ q + da.transpose(-1, -2) @ k
    dbeta = (e * r).sum(-1) - (c["D"] * c["kk"] * eu).sum(-1)
    # decays: + at the row that reads, - at the row that writes, and the state at the chunk's end,
    # summed from the end in 64 bits, since these nearly cancel
    per_row = (q.double() * dq).sum(-1) + (k.double() * (read.double() - write.double())).sum(-1)
    after = torch.cat([states[:, :, 1:], last[:, :, None]], 2)
    end = (after.double() * zs).sum((-1, -2))
    dg = per_row.flip(-1).cumsum(-1).flip(-1) + end[..., None]
    n, h, dtype = case["seqs"], case["h"], s["q"].dtype

    def back(x, heads):
        x = x.flatten(2, 3)
        if heads != h:
            x = x.reshape(n, heads, h // heads, *x.shape[2:]).sum(2)
        return _tokens_first(s, x, c["longest"], dtype)

    return back(dq, case["hk"]), back(read + write, case["hk"]), back(dr, h), back(dg, h), back(dbeta, h), z


def _decode(s):
    case = s["case"]
    group, state, o = case["h"] // case["hk"], s["state"], s["o"]
    S = state if s["slots"] is None else state[s["slots"].long()]
    for t in range(case["steps"]):
        q, k = (s[x][:, t].float().repeat_interleave(group, dim=1) for x in ("q", "k"))
        v, a, b = s["v"][:, t].float(), torch.exp(s["g"][:, t].float()), s["beta"][:, t].float()
        new = a[..., None, None] * S
        new = new + k[..., :, None] * (b[..., None] * (v - (new * k[..., :, None]).sum(-2)))[..., None, :]
        out = (new * q[..., :, None]).sum(-2)
        if s["lens"] is not None:
            live = s["lens"] > t
            new = torch.where(live[:, None, None, None], new, S)
            out = torch.where(live[:, None, None], out, o[:, t].float())
        S = new
        o[:, t] = out.to(o.dtype)
    if s["slots"] is None:
        state.copy_(S)
    else:
        state[s["slots"].long()] = S
    return o, state


# ------------------------------------------------------- plain form: block norm

def _norm_parts(s):
    x, y = s["x"].float(), s["y"].float()
    ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    a = torch.sigmoid(s["gate"].float()) if s["gate"] is not None else torch.ones_like(y)
    n = y * ry * s["w_post"].float()
    xn = x + s["scale"] * a * n
    rx = torch.rsqrt((xn * xn).mean(-1, keepdim=True) + EPS)
    return y, ry, a, n, xn, rx


def _norm(s):
    _, _, _, _, xn, rx = _norm_parts(s)
    return xn.to(s["x"].dtype), (xn * rx * s["w_pre"].float()).to(s["y"].dtype)


def _norm_backward(s):
    y, ry, a, n, xn, rx = _norm_parts(s)
    dh, scale = s["dh"].float(), s["scale"]
    gx = dh * s["w_pre"].float()
    dx = s["dx_new"].float() + rx * (gx - xn * (rx * rx * (gx * xn).mean(-1, keepdim=True)))
    dn = scale * a * dx
    gy = dn * s["w_post"].float()
    dy = ry * (gy - y * (ry * ry * (gy * y).mean(-1, keepdim=True)))
    dw_post, dw_pre = (dn * y * ry).double().sum(0).float(), (dh * xn * rx).double().sum(0).float()
    dgate = (scale * dx * n * a * (1 - a)).to(s["gate"].dtype) if s["gate"] is not None else None
    return dx.to(s["x"].dtype), dy.to(s["y"].dtype), dgate, dw_post, dw_pre


# --------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        from kda_delta_rule_chunkwise_b200 import binding as kda
        if op == "prefill":
            return kda.kda_gdr_chunk_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state_in"], s["cu_seqlens"])
        if op == "decode":
            o = kda.kda_gdr_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"], lens=s["lens"], o=s["o"])
            return o, s["state"]
        if op == "backward":
            return kda.kda_gdr_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state_in"], s["cu_seqlens"], s["dout"], s["dstate_out"])
        if op == "norm":
            return kda.kda_block_norm(s["x"], s["y"], s["gate"], s["w_post"], s["w_pre"], scale=s["scale"], eps=EPS)
        return kda.kda_block_norm_backward(s["x"], s["y"], s["gate"], s["w_post"], s["w_pre"], s["dx_new"], s["dh"], scale=s["scale"], eps=EPS)
    return {"prefill": _prefill, "decode": _decode, "backward": _backward, "norm": _norm, "norm_backward": _norm_backward}[op](s)


def work(case):
    op, el = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_backward"):
        n, d = case["rows"], case["width"]
        ex = 2 if case["xtype"] == "bf16" else 4
        g = el if case["gate"] else 0
        if op == "norm":   # x, y, gate in; x', h out; the weights
            return {"bytes": n * d * (2 * ex + 2 * el + g) + 2 * d * el, "flops": n * d * 14}
        return {"bytes": n * d * (3 * ex + 3 * el + 2 * g) + 2 * d * (el + 4), "flops": n * d * 34}
    hk, h, dk, dv, n = case["hk"], case["h"], case["dk"], case["dv"], case["seqs"]
    if op == "decode":  # `lens` is uniform in 0..steps
        steps = case["steps"]
        rows = n * steps if steps == 1 else n * steps / 2
        return {"bytes": rows * el * (2 * hk * dk + 2 * h * dv + 2 * h) + 2 * n * h * dk * dv * 4, "flops": rows * h * 6 * dk * dv}
    rows = sum(_lengths(case))
    states = n * h * dk * dv * 4
    if op == "prefill":  # q, k, v, g, beta in; o out; last states out, first states in when given
        return {"bytes": rows * el * (2 * hk * dk + 2 * h * dv + 2 * h) + states * (2 if case["packed"] else 1), "flops": rows * h * 6 * dk * dv}
    # q, k, v, g, beta, dout in; a gradient out for each input; dstate_out in, dstate_in out
    return {"bytes": rows * el * (4 * hk * dk + 3 * h * dv + 4 * h) + states * (3 if case["packed"] else 2), "flops": rows * h * 18 * dk * dv}


# ------------------------------------------------------ the definition, 64 bits

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("norm", "norm_backward"):
        return _exact_norm(s, op)
    if op == "decode":
        return _exact_decode(s)
    lens = _lengths(case)
    n, h, longest = case["seqs"], case["h"], max(lens)
    dk, dv, group = case["dk"], case["dv"], h // case["hk"]
    if op == "backward" and n * h * dk * dv * longest * 8 > 60e9:
        return None
    ragged = s["cu_seqlens"] is not None

    def steps(name):
        """[T, N, H or Hk, ...] in 64 bits, zeros behind each sequence's end: such a step changes no state."""
        t = s[name].double()
        if not ragged:
            return t.transpose(0, 1)
        out = torch.zeros(longest, n, *t.shape[2:], dtype=t.dtype, device=t.device)
        at = 0
        for i, m in enumerate(lens):
            out[:m, i] = t[0, at:at + m]
            at += m
        return out

    def rows(t, dtype):
        if not ragged:
            return t.transpose(0, 1).to(dtype).double()
        return torch.cat([t[:m, i] for i, m in enumerate(lens)])[None].double()

    q, k, v, g, beta = (steps(x) for x in ("q", "k", "v", "g", "beta"))
    S = torch.zeros(n, h, dk, dv, dtype=torch.float64, device=DEVICE)
    if s["state_in"] is not None:
        S += s["state_in"]
    wide = lambda x: x.repeat_interleave(group, dim=1)  # noqa: E731
    if op == "prefill":
        o = torch.zeros(longest, n, h, dv, dtype=torch.float64, device=DEVICE)
        for t in range(longest):
            kt = wide(k[t])
            S = S * torch.exp(g[t])[..., None, None]
            delta = beta[t][..., None] * (v[t] - (kt[..., None, :] @ S)[..., 0, :])
            S = S + kt[..., :, None] * delta[..., None, :]
            o[t] = (wide(q[t])[..., None, :] @ S)[..., 0, :]
        return rows(o, torch.float64), S
    before = torch.zeros(longest, n, h, dk, dv, dtype=torch.float64, device=DEVICE)
    errs = torch.zeros(longest, n, h, dv, dtype=torch.float64, device=DEVICE)
    for t in range(longest):
        kt = wide(k[t])
        before[t] = S
        S = S * torch.exp(g[t])[..., None, None]
        errs[t] = v[t] - (kt[..., None, :] @ S)[..., 0, :]
        S = S + kt[..., :, None] * (beta[t][..., None] * errs[t])[..., None, :]
    do = steps("dout")
    grads = [torch.zeros(longest, n, h, m, dtype=torch.float64, device=DEVICE) for m in (dk, dk, dv)]
    dgs, dbs = (torch.zeros(longest, n, h, dtype=torch.float64, device=DEVICE) for _ in range(2))
    Z = s["dstate_out"].double()
    for t in reversed(range(longest)):
        qt, kt, a, b = wide(q[t]), wide(k[t]), torch.exp(g[t])[..., None, None], beta[t][..., None]
        kept = before[t] * a                                        # decayed state that the step corrects
        delta = b * errs[t]
        after = kept + kt[..., :, None] * delta[..., None, :]
        grads[0][t] = (after @ do[t][..., :, None])[..., 0]
        Z = Z + qt[..., :, None] * do[t][..., None, :]
        ddelta = (kt[..., None, :] @ Z)[..., 0, :]
        derr = b * ddelta
        grads[1][t] = (Z @ delta[..., :, None])[..., 0] - (kept @ derr[..., :, None])[..., 0]
        grads[2][t] = derr
        dbs[t] = (ddelta * errs[t]).sum(-1)
        Z = Z - kt[..., :, None] * derr[..., None, :]
        dgs[t] = (Z * kept).sum((-1, -2))
        Z = Z * a
    fold = lambda x: x.reshape(longest, n, case["hk"], group, dk).sum(3)  # noqa: E731
    f64 = torch.float64
    return (rows(fold(grads[0]), f64), rows(fold(grads[1]), f64), rows(grads[2], f64), rows(dgs, f64), rows(dbs, f64), Z)


def _exact_decode(s):
    case = s["case"]
    group, pool, out = case["h"] // case["hk"], s["state"].double(), s["o"].double()
    for i in range(case["seqs"]):
        at = i if s["slots"] is None else int(s["slots"][i])
        for t in range(case["steps"] if s["lens"] is None else int(s["lens"][i])):
            q, k = (s[x][i, t].double().repeat_interleave(group, dim=0) for x in ("q", "k"))
            S = pool[at] * torch.exp(s["g"][i, t].double())[:, None, None]
            err = s["v"][i, t].double() - torch.einsum("hc,hcj->hj", k, S)
            S = S + torch.einsum("hc,hj->hcj", k, s["beta"][i, t].double()[:, None] * err)
            pool[at] = S
            out[i, t] = torch.einsum("hc,hcj->hj", q, S)
    return out, pool


def _exact_norm(s, op):
    x, y, wo, wi = (s[n].double() for n in ("x", "y", "w_post", "w_pre"))
    gate = None if s["gate"] is None else s["gate"].double()
    leaves = [t.requires_grad_() for t in (x, y, gate, wo, wi) if t is not None]
    normed = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + EPS) * wo
    xn = x + s["scale"] * (normed if gate is None else normed / (1 + torch.exp(-gate)))
    h = xn / torch.sqrt(xn.pow(2).mean(-1, keepdim=True) + EPS) * wi
    if op == "norm":
        return xn.detach(), h.detach()
    got = list(torch.autograd.grad([xn, h], leaves, [s["dx_new"].double(), s["dh"].double()]))
    return (got[0], got[1], None, *got[2:]) if gate is None else tuple(got)
