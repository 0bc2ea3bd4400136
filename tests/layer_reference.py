"""The operators of kda_layer.h from their definitions, in 64 bits and token by
token, for the tests."""

from __future__ import annotations

import torch


def log_decay(gate, a_log, dt_bias):
    """(tokens, heads, head_dim or 1) fp64 log decays."""
    g = gate.double()
    if g.dim() == 2:
        g = g.unsqueeze(-1)
    if a_log is None:
        return g
    if dt_bias is not None:
        g = g + dt_bias.double().reshape(g.shape[1], -1)
    return -a_log.double().exp()[:, None] * torch.logaddexp(g, torch.zeros_like(g))


def delta_rule(q, k, v, gate, beta, states, lens, starts, lines, reads, scale, a_log=None,
               dt_bias=None, beta_logits=False):
    """Returns out (rows no sequence owns are NaN), the new states, and, per output
    element, scale * |S_t row| |q_t|: what the sum's error is measured against.
    lines[s] < 0 is a padding sequence."""
    g = log_decay(gate, a_log, dt_bias).exp()
    q, k, v, b = q.double(), k.double(), v.double(), beta.double()
    if beta_logits:
        b = torch.sigmoid(b)
    out = torch.full_like(q, float("nan"))
    size = torch.zeros_like(q)
    new = states.double().clone()
    for s, n in enumerate(lens):
        if n == 0:
            continue
        S = states[lines[s]].double() if lines[s] >= 0 and reads[s] else \
            torch.zeros_like(new[0])
        for t in range(starts[s], starts[s] + n):
            S = S * g[t][:, None, :]
            u = b[t][:, None] * (v[t] - (S @ k[t][..., None])[..., 0])
            S = S + u[:, :, None] * k[t][:, None, :]
            out[t] = scale * (S @ q[t][..., None])[..., 0]
            size[t] = scale * S.norm(dim=-1) * q[t].norm(dim=-1, keepdim=True)
        if lines[s] >= 0:
            new[lines[s]] = S
    return out, new, size


def gate_act(z, name):
    if name == "none":
        return torch.ones_like(z)
    return torch.sigmoid(z) * (z if name == "silu" else 1)


def rmsnorm(x, weight, eps):
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if weight is None else y * weight.double()


def gated_rmsnorm(x, gate, weight, eps, act):
    y = rmsnorm(x.double(), weight, eps)
    return y if gate is None else y * gate_act(gate.double(), act)


def residual_rmsnorm(y, residual, weight, scale, gate, act, post_weight, eps):
    p = y.double()
    if post_weight is not None:
        p = rmsnorm(p, post_weight, eps)
    if gate is not None:
        p = p * gate_act(gate.double(), act)
    r = residual.double() + scale * p
    return rmsnorm(r, weight, eps), r
