"""One KDA linear-attention layer from this package's operators, as a serving loop
runs it: a prefill of packed prompts, then decode steps through a CUDA graph.

    python examples/kda_layer.py [--heads 12] [--steps 4]

Random weights.  The layer is
    x, n   = residual_rmsnorm(previous block's output, x)          norm before the block
    q|k|v  = short conv of n W_qkv, SiLU, q and k normed per head
    o      = gated delta rule of q, k, v with decays from n W_f, beta from n W_b
    y      = gated_rmsnorm(o, n W_g) W_o                           norm after it, with its gate
and the decode steps continue the prompts' conv and delta-rule states.  At the end the
decoded rows are compared with one prefill over prompt and decoded tokens together.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_prefill_varlen_gb300 as kda  # noqa: E402

HEAD = 128


class Layer:
    def __init__(self, width: int, heads: int, lines: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, std):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

        self.heads, self.part = heads, heads * HEAD
        # one projection: q|k|v, decay, output gate, beta (padded to 16 bytes per row)
        self.cols = 5 * self.part + (heads + 7) // 8 * 8
        self.w_in = weight(width, self.cols, std=width ** -0.5)
        self.w_out = weight(self.part, width, std=self.part ** -0.5)
        self.w_conv = torch.rand(3 * self.part, 4, generator=gen, device="cuda") - 0.5
        self.a_log = torch.rand(heads, generator=gen, device="cuda").mul_(15).add_(1).log_()
        self.dt_bias = torch.randn(heads, HEAD, generator=gen, device="cuda") - 4
        self.norm, self.norm_out = torch.ones(width, device="cuda"), torch.ones(HEAD, device="cuda")
        self.conv_states = torch.zeros(lines, 3 * self.part, 3, device="cuda")
        self.states = torch.zeros(lines, heads, HEAD, HEAD, device="cuda")

    def project(self, n: torch.Tensor):
        z, p = n @ self.w_in, self.part
        per_head = lambda t: t.unflatten(1, (self.heads, HEAD))  # noqa: E731
        return (z[:, :3 * p], per_head(z[:, 3 * p:4 * p]), per_head(z[:, 4 * p:5 * p]),
                z[:, 5 * p:5 * p + self.heads])

    def after(self, o: torch.Tensor, gate: torch.Tensor) -> torch.Tensor:
        return kda.gated_rmsnorm(o, gate, self.norm_out).flatten(1) @ self.w_out

    def prefill(self, y, x, query_start_loc, lines, has_initial_state):
        """y: the previous block's output, x: the residual stream (updated in place)."""
        n, _ = kda.residual_rmsnorm(y, x, self.norm)
        qkv, decay, gate, beta = self.project(n)
        planes = kda.packed_causal_conv1d_fn(
            qkv, self.w_conv, None, self.conv_states, query_start_loc, lines, has_initial_state,
            self.part, use_qk_l2norm=True, head_dim=HEAD)
        q, k, v = (t.unflatten(1, (self.heads, HEAD)) for t in planes)
        o = kda.packed_delta_rule_fn(q, k, v, decay, beta, self.states, query_start_loc, lines,
                                     has_initial_state, a_log=self.a_log, dt_bias=self.dt_bias,
                                     beta_logits=True)
        return self.after(o, gate)

    def decode(self, y, x, lines):
        n, _ = kda.residual_rmsnorm(y, x, self.norm)
        qkv, decay, gate, beta = self.project(n)
        planes = kda.causal_conv1d_update(qkv, self.conv_states, self.w_conv, None, lines,
                                          self.part, use_qk_l2norm=True, head_dim=HEAD)
        q, k, v = (t.unflatten(1, (self.heads, HEAD)) for t in planes)
        o = kda.delta_rule_update(q, k, v, decay, beta, self.states, lines, a_log=self.a_log,
                                  dt_bias=self.dt_bias, beta_logits=True)
        return self.after(o, gate)


def run(heads: int = 12, steps: int = 4, width: int = 1536, prompts=(700, 1, 90, 1300)) -> float:
    """The largest difference between decoded rows and one prefill of everything,
    relative to the largest output."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    count, lens = len(prompts), [p + steps for p in prompts]
    start = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32).cuda()
    y = torch.randn(sum(lens), width, generator=gen, device="cuda").bfloat16()
    lines = torch.arange(count, dtype=torch.int32, device="cuda")
    fresh = torch.zeros(count, dtype=torch.bool, device="cuda")

    whole = Layer(width, heads, count).prefill(y, torch.zeros_like(y), start, lines, fresh)

    layer = Layer(width, heads, count)
    first = [int(s) for s in start[:-1]]
    rows = torch.cat([torch.arange(f, f + p) for f, p in zip(first, prompts)]).cuda()
    begin = torch.tensor([0, *torch.tensor(prompts).cumsum(0).tolist()], dtype=torch.int32).cuda()
    out = layer.prefill(y[rows], torch.zeros_like(y[rows]), begin, lines, fresh)
    worst = (out.float() - whole[rows].float()).abs().max()

    step_y = torch.zeros(count, width, dtype=torch.bfloat16, device="cuda")
    step_x = torch.zeros_like(step_y)
    kept = layer.conv_states.clone(), layer.states.clone()
    layer.decode(step_y, step_x, lines)  # warm up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_out = layer.decode(step_y, step_x, lines)
    layer.conv_states.copy_(kept[0])
    layer.states.copy_(kept[1])
    for t in range(steps):
        at = torch.tensor([f + p + t for f, p in zip(first, prompts)], device="cuda")
        step_y.copy_(y[at])
        step_x.zero_()
        graph.replay()
        worst = torch.maximum(worst, (step_out.float() - whole[at].float()).abs().max())
    return float(worst / whole.float().abs().max())


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--heads", type=int, default=12)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    print(f"decode against one prefill: largest difference {run(a.heads, a.steps):.2e} of the "
          "largest output")
