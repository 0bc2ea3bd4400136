"""What a linear-attention layer runs around its short conv, as measurable cases.

Four operators: the gated delta rule over packed sequences of any length
("prefill") and for one token per sequence ("decode"), the per-head RMS norm
with the layer's gate that follows it ("gated_norm"), and the norms before and
after a block with its gate and residual scale ("residual_norm").

`run` computes each in its plain form from elementary torch operations, or,
where `own` is set, through the package's entry points.  `exact` restates each
from its definition in 64 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_CHUNK = 32  # tokens per step of the plain form's chunk loop


# --------------------------------------------------------------------------- cases


def _prefill(name, dtype="bf16", heads=12, head_dim=128, n_long=0, long=0, n_short=0,
             short_max=0, n_one=0, gate="raw", init=0.8, null=0, lay=0):
    """A packed batch: n_long sequences of `long` tokens, n_short of U[1, short_max], n_one of a
    single token, shuffled.  gate "raw": the projection's output, one value per channel, in the
    inputs' type, with A_log, dt_bias and logit beta; "log": one fp32 log decay per head, plain
    beta.  init: share of the sequences that continue a cached state; null: padding sequences;
    lay: seed of the layout."""
    c = dict(op="prefill", dtype=dtype, heads=heads, head_dim=head_dim, n_long=n_long, long=long,
             n_short=n_short, short_max=short_max, n_one=n_one, gate=gate, init=init, null=null,
             lay=lay)
    return {"name": name, **c} if name else c


def _decode(name, batch, dtype="bf16", heads=12, head_dim=128, gate="raw", null=0):
    c = dict(op="decode", dtype=dtype, heads=heads, head_dim=head_dim, batch=batch, gate=gate,
             null=null)
    return {"name": name, **c} if name else c


def _gated_norm(name, rows, dtype="bf16", heads=12, head_dim=128, act="sigmoid"):
    c = dict(op="gated_norm", dtype=dtype, rows=rows, heads=heads, head_dim=head_dim, act=act)
    return {"name": name, **c} if name else c


def _residual_norm(name, rows, width, dtype="bf16", res="same", post=True, act="sigmoid",
                   scale=0.5):
    c = dict(op="residual_norm", dtype=dtype, rows=rows, width=width, res=res, post=post, act=act,
             scale=scale)
    return {"name": name, **c} if name else c


def listed():
    return [
        # one long prompt, the benchmark's 16K chunk of 3 x 1536 channels
        _prefill("prefill 1x16384", n_long=1, long=16384, init=1.0),
        # one long prompt among many short ones (the benchmark's skewed batch)
        _prefill("prefill 8192+99x80", n_long=1, long=8192, n_short=99, short_max=80, lay=1),
        # short prompts mixed with decode tokens (the benchmark's short_decode batch)
        _prefill("prefill 256 short+1024x1", n_short=256, short_max=128, n_one=1024, lay=2),
        # the varlen mixed batch: 8 prompts of up to 512 tokens, one of them padding
        _prefill("prefill 8xU512", n_short=8, short_max=512, null=1, init=0.5, lay=3),
        # a first prompt of one head: latency
        _prefill("prefill 1x64 1 head", heads=1, n_long=1, long=64, init=1.0),
        # four long prompts, 17 heads of 64 (1088 channels), fp16, one decay per head
        _prefill("prefill 4x8192 17x64 fp16", dtype="fp16", heads=17, head_dim=64, n_long=4,
                 long=8192, gate="log", init=0.5, lay=5),
        # one user's next token
        _decode("decode 1", 1),
        # the benchmark's decode step of 1024 sequences
        _decode("decode 1024", 1024),
        # after the 16K chunk: norm and gate of 12 heads
        _gated_norm("gated norm 16384x12x128", 16384),
        # after a small decode step, 17 heads of 64, SiLU gate
        _gated_norm("gated norm 33x17x64 fp16", 33, dtype="fp16", heads=17, head_dim=64,
                    act="silu"),
        # around a block of the 16K chunk: post-norm, gate, scaled residual, next pre-norm
        _residual_norm("residual norm 16384x4608", 16384, 4608),
        # the same join on a few decode tokens, fp32 residual stream, no post-norm or gate
        _residual_norm("residual norm 7x1536", 7, 1536, res="fp32", post=False, act="none",
                       scale=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "prefill", "decode", "gated_norm", "residual_norm"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    heads = rng.randint(1, 17)
    head_dim = rng.choice((64, 128, 128))
    gate = rng.choice(("raw", "raw", "log"))
    if op == "prefill":
        most = 16384 * 12 * 128 // (heads * head_dim)  # channels x tokens of the 16K chunk
        tokens = min(_log_int(rng, 16, 32768), most)
        kind = rng.choice(("long", "short", "mixed"))
        n_long = rng.randint(1, 4) if kind != "short" else 0
        long = max(1, tokens // n_long - rng.randint(0, 5)) if n_long else 0
        long = long // 2 if kind == "mixed" and long > 1 else long
        short_max = _log_int(rng, 1, 512) if kind != "long" else 0
        n_short = max(1, min(512, tokens // max(1, short_max))) if short_max else 0
        n_one = rng.choice((0, rng.randint(1, 256))) if kind == "mixed" else 0
        return _prefill(None, dtype, heads, head_dim, n_long, long, n_short, short_max, n_one,
                        gate, rng.choice((0.0, 0.5, 1.0)), rng.randint(0, 1),
                        rng.randint(0, 1 << 20))
    if op == "decode":
        return _decode(None, _log_int(rng, 1, 1024), dtype, heads if head_dim == 64 else
                       min(heads, 12), head_dim, gate, rng.randint(0, 1))
    if op == "gated_norm":
        return _gated_norm(None, _log_int(rng, 1, 16384), dtype, min(heads, 12),
                           rng.choice((64, 128)), rng.choice(("sigmoid", "silu")))
    return _residual_norm(None, _log_int(rng, 1, 8192), 8 * _log_int(rng, 16, 576), dtype,
                          rng.choice(("same", "fp32")), rng.random() < 0.5,
                          rng.choice(("none", "sigmoid", "silu")), rng.choice((1.0, 0.25)))


def _layout(case):
    """Lengths, has_initial_state and padding of a packed batch, from the case alone."""
    r = np.random.RandomState(case["lay"])
    lens = np.concatenate([np.full(case["n_long"], case["long"], np.int64),
                           r.randint(1, case["short_max"] + 1, case["n_short"])
                           if case["n_short"] else np.zeros(0, np.int64),
                           np.ones(case["n_one"], np.int64)]).astype(np.int64)
    lens = r.permutation(lens)
    init = r.rand(len(lens)) < case["init"]
    null = np.zeros(len(lens), bool)
    null[r.permutation(len(lens))[:min(case["null"], len(lens) - 1)]] = True
    return lens, init, null


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] in ("prefill", "decode"):
        h, d = case["heads"], case["head_dim"]
        if case["op"] == "prefill":
            lens, init, null = _layout(case)
            tokens = int(lens.sum())
            lines = int((init & ~null).sum() + (~null).sum())  # states read + written
        else:
            tokens = case["batch"]
            lines = 2 * (tokens - min(case["null"], tokens - 1))
        gate = d * e if case["gate"] == "raw" else 4
        beta = e if case["gate"] == "raw" else 4
        return {"bytes": tokens * h * (4 * d * e + gate + beta) + 4 * lines * h * d * d,
                "flops": 7 * tokens * h * d * d}
    if case["op"] == "gated_norm":
        n = case["rows"] * case["heads"] * case["head_dim"]
        return {"bytes": 3 * n * e, "flops": 8 * n}
    n = case["rows"] * case["width"]
    r = 4 if case["res"] == "fp32" else e
    return {"bytes": n * (2 * e + 2 * r + (e if case["act"] != "none" else 0)), "flops": 10 * n}


# --------------------------------------------------------------------------- inputs


def _unit(x):
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)


def _delta_inputs(case, gen, tokens, lines, s):
    h, d, dt = case["heads"], case["head_dim"], _DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    # three planes as the conv leaves them: SiLU outputs, q and k normalised per head
    planes = torch.empty(3, tokens, h * d, dtype=dt, device="cuda")
    for i in range(3):
        y = torch.nn.functional.silu(randn(tokens, h, d))
        planes[i] = (_unit(y) if i < 2 else y).reshape(tokens, h * d).to(dt)
    s["q"], s["k"], s["v"] = (planes[i].view(tokens, h, d) for i in range(3))
    if case["gate"] == "raw":
        s["gate"] = randn(tokens, h, d).to(dt)
        s["beta"] = randn(tokens, h).to(dt)
        s["a_log"] = torch.rand(h, generator=gen, device="cuda").mul_(15).add_(1).log_()
        step = torch.rand(h, d, generator=gen, device="cuda")
        step = torch.exp(step * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(dt_bias) = step
    else:
        s["gate"] = -torch.rand(tokens, h, generator=gen, device="cuda").square()
        s["beta"] = torch.rand(tokens, h, generator=gen, device="cuda")
        s["a_log"] = s["dt_bias"] = None
    s["scale"] = d ** -0.5
    s["states"] = randn(lines, h, d, d).mul_(0.1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]
    s = {"case": case}

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] == "prefill":
        lens, init, null = _layout(case)
        n, tokens = len(lens), int(lens.sum())
        _delta_inputs(case, gen, tokens, n + 3, s)
        lines = torch.randperm(n + 3, generator=gen, device="cuda")[:n].to(torch.int32)
        lines[torch.from_numpy(np.flatnonzero(null)).cuda()] = -1
        qsl = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        s["cache_indices"], s["query_start_loc"] = lines, torch.from_numpy(qsl).cuda()
        s["has_initial_state"] = torch.from_numpy(init).cuda()
        s["plan"] = _plan(lens, qsl, init, null)
    elif case["op"] == "decode":
        b = case["batch"]
        _delta_inputs(case, gen, b, b + 3, s)
        lines = torch.randperm(b + 3, generator=gen, device="cuda")[:b].to(torch.int32)
        lines[b - min(case["null"], b - 1):] = -1
        s["cache_indices"] = lines
        live = np.arange(b - min(case["null"], b - 1))
        s["live"] = torch.from_numpy(live).cuda()
    elif case["op"] == "gated_norm":
        shape = (case["rows"], case["heads"], case["head_dim"])
        s["x"], s["gate"] = randn(*shape).to(dt), randn(*shape).to(dt)
        s["weight"] = 1 + 0.1 * randn(case["head_dim"])
    else:
        shape = (case["rows"], case["width"])
        s["y"] = randn(*shape).to(dt)
        s["residual"] = (2 * randn(*shape)).to(torch.float32 if case["res"] == "fp32" else dt)
        s["gate"] = randn(*shape).to(dt) if case["act"] != "none" else None
        s["weight"] = 1 + 0.1 * randn(case["width"])
        s["post_weight"] = 1 + 0.1 * randn(case["width"]) if case["post"] else None
    return s


def _plan(lens, qsl, init, null):
    """Index tables of the plain form: sequences by falling length; for its step i, the chunk i of
    every sequence that has one (a contiguous run of table rows, as they are sorted)."""
    order = np.argsort(-lens, kind="stable")
    chunks = -(-lens[order] // _CHUNK)
    counts = [int(np.searchsorted(-chunks, -i, side="left")) for i in range(int(chunks[0]))]
    first = np.concatenate([[0], np.cumsum(counts)])
    at = np.empty((int(first[-1]), _CHUNK), np.int64)
    for i, n in enumerate(counts):
        at[first[i]:first[i + 1]] = (i * _CHUNK + np.arange(_CHUNK))[None]
    seq = np.concatenate([np.arange(n) for n in counts])
    inside = at < lens[order][seq][:, None]
    rows = np.where(inside, at + qsl[:-1][order][seq][:, None], 0)
    cuda = {k: torch.from_numpy(v).cuda() for k, v in
            {"order": order, "rows": rows, "inside": inside, "reads": (init & ~null)[order],
             "kept": np.flatnonzero(~null[order]), "zero": np.zeros(1, np.int64)}.items()}
    return {"counts": counts, "first": [int(v) for v in first], "lens": lens[order].tolist(),
            "starts": qsl[:-1][order].tolist(), **cuda}


# --------------------------------------------------------------------------- plain forms


def _log_decay(s, wide):
    """The log decay, (tokens, heads, head_dim or 1)."""
    g = s["gate"].to(wide)
    if s["a_log"] is None:
        return g.unsqueeze(-1)
    z = g + s["dt_bias"].to(wide)
    soft = torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))
    return -torch.exp(s["a_log"].to(wide))[:, None] * soft


def _beta(s, wide):
    b = s["beta"].to(wide)
    return b if s["a_log"] is None else 1 / (1 + torch.exp(-b))


def _plain_prefill(s):
    """Chunks of 32 tokens: all products inside a chunk at once for every chunk, with the decay
    between each two of its tokens written out per channel, then one step per chunk for the state."""
    p, c = s["plan"], _CHUNK
    inside = p["inside"][:, :, None]

    def rows(x, fill):  # (chunks, heads, 32, ...)
        x = x[p["rows"]]
        mask = inside if x.dim() == 3 else inside[..., None]
        return torch.where(mask, x, torch.full((), fill, device=x.device)).transpose(1, 2)

    q, k, v = (rows(s[n].float(), 0.0) for n in ("q", "k", "v"))
    g, b = rows(_log_decay(s, torch.float32), 0.0), rows(_beta(s, torch.float32), 0.0)
    run = g.double().cumsum(2)  # 64 bits: differences of neighbours late in a chunk
    low = torch.ones(c, c, dtype=torch.bool, device=q.device).tril()
    gap = (run[:, :, :, None] - run[:, :, None]).float()
    gap = torch.where(low[:, :, None], gap, torch.full((), -math.inf, device=q.device))
    kd = torch.exp(gap) * k[:, :, None]  # [i, j]: k_j decayed to token i
    att = (kd @ q[..., None]).squeeze(-1)
    mix = b[..., None] * (kd @ k[..., None]).squeeze(-1)
    del gap, kd
    inv = torch.zeros_like(mix) + torch.eye(c, device=q.device)
    for i in range(1, c):  # forward substitution
        inv[:, :, i, :i] = -(mix[:, :, i, None, :i] @ inv[:, :, :i, :i]).squeeze(-2)
    grow = torch.exp(run).float()
    last = run[:, :, -1:]
    w, u = inv @ (b[..., None] * k * grow), inv @ (b[..., None] * v)
    q, k, end = q * grow, k * torch.exp(last - run).float(), torch.exp(last).float()

    lines = s["cache_indices"].long()[p["order"]]
    state = s["states"][lines.clamp(min=0)]
    state = torch.where(p["reads"][:, None, None, None], state, torch.zeros((), device=q.device))
    outs = []
    for i, n in enumerate(p["counts"]):
        at = slice(p["first"][i], p["first"][i + 1])
        sT = state[:n].transpose(-1, -2)
        new = u[at] - w[at] @ sT
        outs.append(q[at] @ sT + att[at] @ new)
        state[:n] = state[:n] * end[at] + new.transpose(-1, -2) @ k[at]
    o = (torch.cat(outs) * s["scale"]).transpose(1, 2)
    out = torch.empty_like(s["q"], memory_format=torch.contiguous_format)
    out[p["rows"][p["inside"]]] = o[p["inside"]].to(out.dtype)
    s["states"][lines[p["kept"]]] = state[p["kept"]]
    return {"out": out, "states": s["states"]}


def _plain_decode(s):
    lines = s["cache_indices"].long()
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    state = s["states"][lines.clamp(min=0)]
    state = torch.where((lines >= 0)[:, None, None, None], state,
                        torch.zeros((), device=q.device))
    state = state * torch.exp(_log_decay(s, torch.float32))[:, :, None]
    u = _beta(s, torch.float32)[..., None] * (v - (state * k[:, :, None]).sum(-1))
    state = state + u[..., None] * k[:, :, None]
    out = s["scale"] * (state * q[:, :, None]).sum(-1)
    s["states"][lines[s["live"]]] = state[s["live"]]
    return {"out": out.to(s["q"].dtype), "states": s["states"]}


def _act(z, name):
    if name == "none":
        return torch.ones_like(z)
    sig = 1 / (1 + torch.exp(-z))
    return sig * z if name == "silu" else sig


_EPS = 1e-5


def _plain_gated_norm(s):
    x = s["x"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * s["weight"]
    return (y * _act(s["gate"].float(), s["case"]["act"])).to(s["x"].dtype)


def _plain_residual_norm(s):
    y = s["y"].float()
    if s["post_weight"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + _EPS) * s["post_weight"]
    if s["gate"] is not None:
        y = y * _act(s["gate"].float(), s["case"]["act"])
    r = s["residual"].float() + s["case"]["scale"] * y
    n = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS) * s["weight"]
    return n.to(s["y"].dtype), r.to(s["residual"].dtype)


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"prefill": _plain_prefill, "decode": _plain_decode,
                "gated_norm": _plain_gated_norm, "residual_norm": _plain_residual_norm}[op](s)
    import linear_attention_prefill_varlen_gb300 as kda

    if op == "prefill":
        out = kda.packed_delta_rule_fn(
            s["q"], s["k"], s["v"], s["gate"], s["beta"], s["states"], s["query_start_loc"],
            s["cache_indices"], s["has_initial_state"], scale=s["scale"], a_log=s["a_log"],
            dt_bias=s["dt_bias"], beta_logits=s["a_log"] is not None, null_block_id=-1)
        return {"out": out, "states": s["states"]}
    if op == "decode":
        out = kda.delta_rule_update(
            s["q"], s["k"], s["v"], s["gate"], s["beta"], s["states"], s["cache_indices"],
            scale=s["scale"], a_log=s["a_log"], dt_bias=s["dt_bias"],
            beta_logits=s["a_log"] is not None, null_block_id=-1)
        return {"out": out, "states": s["states"]}
    if op == "gated_norm":
        return kda.gated_rmsnorm(s["x"], s["gate"], s["weight"], eps=_EPS,
                                 activation=s["case"]["act"])
    return kda.residual_rmsnorm(s["y"], s["residual"], s["weight"], scale=s["case"]["scale"],
                                gate=s["gate"], activation=s["case"]["act"],
                                post_weight=s["post_weight"], eps=_EPS,
                                residual_out=torch.empty_like(s["residual"]))


# --------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("prefill", "decode"):
        return _exact_delta(case, s)
    if case["op"] == "gated_norm":
        x, z = s["x"].double(), s["gate"].double()
        gate = torch.sigmoid(z) * (z if case["act"] == "silu" else 1)
        return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS) \
            * s["weight"].double() * gate
    y, r = s["y"].double(), s["residual"].double()
    if s["post_weight"] is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + _EPS)
        y = y * s["post_weight"].double()
    if s["gate"] is not None:
        z = s["gate"].double()
        y = y * torch.sigmoid(z) * (z if case["act"] == "silu" else 1)
    r = r + case["scale"] * y
    n = r / torch.sqrt((r * r).sum(-1, keepdim=True) / r.shape[-1] + _EPS) * s["weight"].double()
    return n, r


def _exact_delta(case, s):
    """Token by token, as the recurrence is written, on all sequences that still have a token."""
    q, k, v, g, b = (s[n].double() for n in ("q", "k", "v", "gate", "beta"))
    if case["gate"] == "raw":
        z = g + s["dt_bias"].double()
        g = -s["a_log"].double().exp()[:, None] * torch.logaddexp(z, torch.zeros_like(z))
        b = torch.sigmoid(b)
    else:
        g = g[..., None]
    if case["op"] == "prefill":
        p = s["plan"]
        order, lens, starts = p["order"], p["lens"], torch.tensor(p["starts"], device="cuda")
        reads = p["reads"]
    else:
        order = torch.arange(case["batch"], device="cuda")
        lens, starts = [1] * case["batch"], order
        reads = s["cache_indices"] >= 0
    lines = s["cache_indices"].long()[order]
    state = s["states"][lines.clamp(min=0)].double()
    state[~reads] = 0
    out = torch.empty_like(q)
    n = len(lens)
    for t in range(lens[0]):
        while lens[n - 1] <= t:
            n -= 1
        at = starts[:n] + t
        S = state[:n]  # [sequence, head, v, k]
        S *= g[at].exp()[:, :, None, :]
        u = b[at][..., None] * (v[at] - torch.matmul(S, k[at][..., None])[..., 0])
        S += u[..., :, None] * k[at][..., None, :]
        out[at] = case["head_dim"] ** -0.5 * torch.matmul(S, q[at][..., None])[..., 0]
    whole = s["states"].double()
    kept = lines >= 0
    whole[lines[kept]] = state[kept]
    return {"out": out, "states": whole}
