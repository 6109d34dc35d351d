"""Gated delta rule, token by token in 64 bits on the CPU: the definition that the tests compare with.

    S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t

Nothing here is shared with the package."""
from __future__ import annotations

import torch


def spans(B, T, cu):
    """(first row, end row) of each sequence in the flattened rows."""
    if cu is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    return [(int(a), int(e)) for a, e in zip(cu[:-1], cu[1:])]


def forward(q, k, v, g, beta, state_in=None, cu=None):
    """o [B, T, H, dv] (rows outside every sequence NaN) and the last states, in 64 bits."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    q, k, v, g, beta = (x.double().reshape((B * T,) + tuple(x.shape[2:])) for x in (q, k, v, g, beta))
    q, k = (x.repeat_interleave(H // Hk, dim=1) for x in (q, k))
    rows = spans(B, T, cu)
    o = torch.full((B * T, H, dv), float("nan"), dtype=torch.float64)
    last = torch.zeros(len(rows), H, dk, dv, dtype=torch.float64)
    for n, (a, e) in enumerate(rows):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if state_in is None else state_in[n].double()
        for t in range(a, e):
            S = torch.exp(g[t])[:, None, None] * S
            delta = beta[t][:, None] * (v[t] - torch.einsum("hc,hcj->hj", k[t], S))
            S = S + k[t][:, :, None] * delta[:, None, :]
            o[t] = torch.einsum("hc,hcj->hj", q[t], S)
        last[n] = S
    return o.reshape(B, T, H, dv), last


def backward(q, k, v, g, beta, state_in, cu, dout, dstate_out):
    """Gradients of <o, dout> + <last states, dstate_out> by automatic differentiation of `forward`."""
    leaves = [x.double().clone().requires_grad_(True) for x in (q, k, v, g, beta)]
    n = q.shape[0] if cu is None else len(cu) - 1
    H, dk, dv = v.shape[2], q.shape[3], v.shape[3]
    s0 = (torch.zeros(n, H, dk, dv) if state_in is None else state_in).double().clone().requires_grad_(True)
    o, last = forward(*leaves, s0, cu)
    live = ~torch.isnan(o.detach())
    loss = (torch.where(live, o, torch.zeros_like(o)) * torch.where(live, dout.double(), torch.zeros_like(o))).sum()
    if dstate_out is not None:
        loss = loss + (last * dstate_out.double()).sum()
    grads = torch.autograd.grad(loss, leaves + [s0], allow_unused=True)
    return [torch.zeros_like(x) if gr is None else gr for x, gr in zip(leaves + [s0], grads)]


def inputs(B, T, Hk, H, dk, dv, dtype, seed, lengths=None, state=True, g=None, unit=True):
    """Seeded CPU inputs: unit keys and queries, decays from slow to fast heads."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    q, k = rn(B, T, Hk, dk), rn(B, T, Hk, dk)
    if unit:
        q, k = (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12) for x in (q, k))
    v, beta = rn(B, T, H, dv), torch.sigmoid(rn(B, T, H))
    a = torch.exp(torch.linspace(-4.0, 0.7, H))
    gg = -a * torch.nn.functional.softplus(rn(B, T, H)) if g is None else torch.full((B, T, H), float(g))
    cu = None
    if lengths is not None:
        cu = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32)
    n = B if lengths is None else len(lengths)
    s0 = rn(n, H, dk, dv) * 0.1 if state else None
    return [x.to(dtype) for x in (q, k, v, gg, beta)] + [s0, cu]
