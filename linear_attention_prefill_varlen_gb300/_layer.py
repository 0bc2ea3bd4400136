"""The operators around the short conv (include/kda_layer.h) on torch tensors:
the gated delta rule, the gated per-head norm and the residual norm.  Argument
conversion only; every step runs in the library's CUDA kernels."""

from __future__ import annotations

import ctypes

import torch

from ._binding import KDA_ERR_CUDA, KDA_OK, KdaError, _DTYPES, _check_vector, _ptr, lib

KDA_GATE_LOG = 0
KDA_GATE_SOFTPLUS = 1
KDA_BETA_PLAIN = 0
KDA_BETA_SIGMOID = 1
KDA_NORM_GATE_NONE = 0
KDA_NORM_GATE_SIGMOID = 1
KDA_NORM_GATE_SILU = 2

_P, _I64, _I32, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_Pair = _I64 * 2


class KdaDelta(ctypes.Structure):
    """kda_delta_t: the tensors of the gated delta rule and how they are read."""

    _fields_ = [("version", _I32), ("x_dtype", _I32), ("gate_dtype", _I32), ("beta_dtype", _I32),
                ("gate_kind", _I32), ("gate_per_channel", _I32), ("beta_kind", _I32),
                ("head_dim", _I32), ("heads", _I64), ("scale", _F), ("reserved", _I32),
                ("q", _P), ("k", _P), ("v", _P), ("gate", _P), ("beta", _P), ("a_log", _P),
                ("dt_bias", _P), ("states", _P), ("out", _P), ("q_stride", _Pair),
                ("k_stride", _Pair), ("v_stride", _Pair), ("gate_stride", _Pair),
                ("beta_stride", _Pair), ("out_stride", _Pair), ("state_stride", _Pair),
                ("cache_index_stride", _I64)]


_declared = None


def _lib() -> ctypes.CDLL:
    global _declared
    h = lib()
    if _declared is not h:
        D = ctypes.POINTER(KdaDelta)
        h.kda_delta_check.argtypes = [D]
        h.kda_packed_delta_rule_workspace.argtypes = [_I64, _I64, _I64, _I32, _I32, _I32,
                                                      ctypes.POINTER(_I64)]
        h.kda_packed_delta_rule.argtypes = [D, _I64, _P, _P, _P, _I64, _I64, _P, _I64, _P]
        h.kda_delta_rule_update.argtypes = [D, _I64, _P, _I64, _P]
        h.kda_gated_rmsnorm.argtypes = [_P, _P, _P, _P, _P, _F, ctypes.c_int, _I64, _I64, _I64,
                                        ctypes.c_int, _P, _P, _P]
        h.kda_residual_rmsnorm.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _P, _F, _F,
                                           ctypes.c_int, _I64, _I64, ctypes.c_int, ctypes.c_int,
                                           _P, _I64, _P, _I64, _P]
        for name in ("kda_delta_check", "kda_packed_delta_rule_workspace", "kda_packed_delta_rule",
                     "kda_delta_rule_update", "kda_gated_rmsnorm", "kda_residual_rmsnorm"):
            getattr(h, name).restype = ctypes.c_int
        h.kda_layer_error_string.argtypes = []
        h.kda_layer_error_string.restype = ctypes.c_char_p
        _declared = h
    return h


def _check(status: int) -> None:
    if status != KDA_OK:
        h = _lib()
        what = h.kda_status_string(status).decode()
        if status == KDA_ERR_CUDA:
            what += ": " + h.kda_layer_error_string().decode()
        raise KdaError(status, what)


def _stream_of(stream, device) -> int:
    """The raw handle: `stream`, or torch's current stream of the tensors' device."""
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty_on(stream, shape, dtype, device) -> torch.Tensor:
    """torch.empty in the memory pool of the stream that will use it, so that the
    block is not handed out again while that stream still works on it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=device)


def _same_device(lead: str, **tensors) -> torch.device:
    """Every tensor on the CUDA device of `lead` (there is no CPU path)."""
    dev = tensors[lead].device
    if dev.type != "cuda":
        raise ValueError(f"{lead} must be a CUDA tensor: the library has no CPU path")
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, {lead} on {dev}")
    return dev


def _strides(t: torch.Tensor, n: int):
    """The first n strides; 0 for an axis of one entry, whose stride is never used."""
    return [t.stride(i) if t.size(i) > 1 else 0 for i in range(n)]


def _written(name: str, t) -> None:
    """A tensor the call writes has no expanded axis: its elements would overlap."""
    if t is not None and any(t.stride(i) == 0 for i in range(t.dim()) if t.size(i) > 1):
        raise ValueError(f"the elements of {name} overlap")


def _vector32(name: str, t, shapes) -> None:
    if t is None:
        return
    if t.dtype != torch.float32 or tuple(t.shape) not in shapes or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape "
                         f"{' or '.join(str(s) for s in shapes)}, not {t.dtype} {tuple(t.shape)}")


def _delta(q, k, v, gate, beta, states, scale, a_log, dt_bias, beta_logits, out):
    """The checked KdaDelta of these tensors (out's pointer and strides left out)."""
    if q.dim() != 3 or q.dtype not in _DTYPES:
        raise ValueError("q must be (tokens, heads, head_dim) in bf16, fp16 or fp32")
    tokens, heads, dim = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t is None:
            continue
        if t.dtype != q.dtype or t.shape != q.shape:
            raise ValueError(f"{name} must be {q.dtype} {tuple(q.shape)}, not {t.dtype} "
                             f"{tuple(t.shape)}")
        if t.numel() and t.stride(2) != 1:
            raise ValueError(f"{name} must have unit channel stride")
    _written("out", out)
    _written("states", states)
    channel = gate.dim() == 3
    if gate.dtype not in _DTYPES or tuple(gate.shape) not in ((tokens, heads, dim),
                                                             (tokens, heads)):
        raise ValueError(f"gate must be (tokens, heads, head_dim) or (tokens, heads) in bf16, "
                         f"fp16 or fp32, not {gate.dtype} {tuple(gate.shape)}")
    if channel and gate.numel() and gate.stride(2) != 1:
        raise ValueError("gate must have unit channel stride")
    if beta.dtype not in _DTYPES or tuple(beta.shape) != (tokens, heads):
        raise ValueError(f"beta must be ({tokens}, {heads}) in bf16, fp16 or fp32, not "
                         f"{beta.dtype} {tuple(beta.shape)}")
    if (states.dtype != torch.float32 or states.dim() != 4
            or tuple(states.shape[1:]) != (heads, dim, dim)):
        raise ValueError(f"states must be fp32 (lines, {heads}, {dim}, {dim}), not "
                         f"{states.dtype} {tuple(states.shape)}")
    if states.numel() and (states.stride(3) != 1 or states.stride(2) != dim):
        raise ValueError("a head's state must be a contiguous (head_dim, head_dim) matrix")
    if dt_bias is not None and a_log is None:
        raise ValueError("dt_bias needs a_log")
    _vector32("a_log", a_log, [(heads,)])
    _vector32("dt_bias", dt_bias, [(heads, dim), (heads * dim,)] if channel else [(heads,)])
    d = KdaDelta()
    d.x_dtype, d.gate_dtype, d.beta_dtype = (_DTYPES[t.dtype] for t in (q, gate, beta))
    d.gate_kind = KDA_GATE_LOG if a_log is None else KDA_GATE_SOFTPLUS
    d.gate_per_channel = int(channel)
    d.beta_kind = KDA_BETA_SIGMOID if beta_logits else KDA_BETA_PLAIN
    d.heads, d.head_dim = heads, dim
    d.scale = dim ** -0.5 if scale is None else float(scale)
    d.q, d.k, d.v, d.gate, d.beta = (t.data_ptr() for t in (q, k, v, gate, beta))
    d.a_log, d.dt_bias, d.states = _ptr(a_log), _ptr(dt_bias), states.data_ptr()
    for name, t in (("q_stride", q), ("k_stride", k), ("v_stride", v), ("gate_stride", gate),
                    ("beta_stride", beta), ("state_stride", states)):
        setattr(d, name, _Pair(*_strides(t, 2)))
    return d


def _set_out(d: KdaDelta, out: torch.Tensor) -> None:
    d.out, d.out_stride = out.data_ptr(), _Pair(*_strides(out, 2))


def _null(null_block_id) -> int:
    return -(2 ** 62) if null_block_id is None else int(null_block_id)


def delta_rule_workspace(tokens: int, num_seqs: int, heads: int, head_dim: int,
                         dtype: torch.dtype = torch.bfloat16, sm_count: int = 0) -> int:
    """Bytes of workspace packed_delta_rule_fn uses for these sizes (sm_count 0:
    the current device)."""
    n = _I64()
    _check(_lib().kda_packed_delta_rule_workspace(tokens, num_seqs, heads, head_dim,
                                                  _DTYPES[dtype], sm_count, ctypes.byref(n)))
    return n.value


def packed_delta_rule_fn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gate: torch.Tensor,
                         beta: torch.Tensor, states: torch.Tensor, query_start_loc: torch.Tensor,
                         cache_indices: torch.Tensor, has_initial_state: torch.Tensor,
                         scale: float | None = None, a_log: torch.Tensor | None = None,
                         dt_bias: torch.Tensor | None = None, beta_logits: bool = False,
                         null_block_id: int | None = None, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gated delta rule over a packed varlen batch.

    q, k, v are (tokens, heads, head_dim) bf16, fp16 or fp32 with unit channel
    stride, such as the planes packed_causal_conv1d_fn returns, viewed per head;
    head_dim is 64 or 128.  `gate` is (tokens, heads, head_dim), a decay per
    channel, or (tokens, heads), one per head: the log decay itself, or, with
    `a_log` (heads) given, raw values r for -exp(a_log) * softplus(r + dt_bias).
    `beta` (tokens, heads) is used as it is, or through a sigmoid with
    `beta_logits`.  `states` (lines, heads, head_dim, head_dim) fp32, [v][k],
    is updated in place; query_start_loc, cache_indices (may be strided),
    has_initial_state and null_block_id are those of packed_causal_conv1d_fn.
    `scale` defaults to head_dim ** -0.5.  `workspace` may be a contiguous uint8 CUDA
    tensor of delta_rule_workspace bytes; else it is allocated.  Returns out
    (tokens, heads, head_dim) in q's dtype."""
    d = _delta(q, k, v, gate, beta, states, scale, a_log, dt_bias, beta_logits, out)
    tokens, heads, dim = q.shape
    num_seqs = max(query_start_loc.numel() - 1, 0)
    _check_vector("query_start_loc", query_start_loc, 0, (torch.int32,))
    _check_vector("cache_indices", cache_indices, num_seqs, (torch.int32,), strided=True)
    _check_vector("has_initial_state", has_initial_state, num_seqs, (torch.bool, torch.uint8))
    dev = _same_device("q", q=q, k=k, v=v, gate=gate, beta=beta, states=states, a_log=a_log,
                       dt_bias=dt_bias, query_start_loc=query_start_loc,
                       cache_indices=cache_indices, has_initial_state=has_initial_state, out=out,
                       workspace=workspace)
    with torch.cuda.device(dev):
        if out is None:
            out = _empty_on(stream, q.shape, q.dtype, dev)
        _set_out(d, out)
        d.cache_index_stride = cache_indices.stride(0) if cache_indices.numel() > 1 else 1
        need = delta_rule_workspace(tokens, num_seqs, heads, dim, q.dtype)
        if workspace is None:
            workspace = _empty_on(stream, (need,), torch.uint8, dev) if need else None
        elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        _check(_lib().kda_packed_delta_rule(
            ctypes.byref(d), tokens, cache_indices.data_ptr(), has_initial_state.data_ptr(),
            query_start_loc.data_ptr(), num_seqs, _null(null_block_id), _ptr(workspace),
            0 if workspace is None else workspace.numel(), _stream_of(stream, dev)))
    return out


def delta_rule_update(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gate: torch.Tensor,
                      beta: torch.Tensor, states: torch.Tensor, cache_indices: torch.Tensor,
                      scale: float | None = None, a_log: torch.Tensor | None = None,
                      dt_bias: torch.Tensor | None = None, beta_logits: bool = False,
                      null_block_id: int | None = None, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """One decode step of the gated delta rule: row i of q, k, v, gate, beta is the
    next token of the sequence at line cache_indices[i]; arguments as for
    packed_delta_rule_fn.  Returns out (batch, heads, head_dim)."""
    d = _delta(q, k, v, gate, beta, states, scale, a_log, dt_bias, beta_logits, out)
    batch = q.size(0)
    _check_vector("cache_indices", cache_indices, batch, (torch.int32,), strided=True)
    dev = _same_device("q", q=q, k=k, v=v, gate=gate, beta=beta, states=states, a_log=a_log,
                       dt_bias=dt_bias, cache_indices=cache_indices, out=out)
    with torch.cuda.device(dev):
        if out is None:
            out = _empty_on(stream, q.shape, q.dtype, dev)
        _set_out(d, out)
        d.cache_index_stride = cache_indices.stride(0) if cache_indices.numel() > 1 else 1
        _check(_lib().kda_delta_rule_update(ctypes.byref(d), batch, cache_indices.data_ptr(),
                                            _null(null_block_id), _stream_of(stream, dev)))
    return out


_NORM_GATES = {"sigmoid": KDA_NORM_GATE_SIGMOID, "silu": KDA_NORM_GATE_SILU,
               "swish": KDA_NORM_GATE_SILU, "none": KDA_NORM_GATE_NONE}


def _norm_gate(gate, activation) -> int:
    """The kda_norm_gate_t of a wrapper's gate and `activation`."""
    name = "none" if activation is None else activation
    if not isinstance(name, str) or name not in _NORM_GATES:
        raise ValueError(f"activation must be 'sigmoid', 'silu', 'swish', 'none' or None, not "
                         f"{activation!r}")
    if gate is None:
        return KDA_NORM_GATE_NONE
    if _NORM_GATES[name] == KDA_NORM_GATE_NONE:
        raise ValueError("a gate needs an activation")
    return _NORM_GATES[name]


def _like(name: str, t, x: torch.Tensor, dtypes) -> None:
    if t is None:
        return
    if t.dtype not in dtypes or t.shape != x.shape:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)} "
                         f"{tuple(x.shape)}, not {t.dtype} {tuple(t.shape)}")
    if t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit channel stride")


def gated_rmsnorm(x: torch.Tensor, gate: torch.Tensor | None, weight: torch.Tensor | None,
                  eps: float = 1e-5, activation="sigmoid", out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) * weight * act(gate) over the channels of each
    head.  x, gate, out (rows, heads, head_dim) in bf16, fp16 or fp32 with unit
    channel stride; weight fp32 (head_dim) or None.  `activation` "sigmoid" or
    "silu" ("swish"); gate None: no gate.  `out` may be x or gate."""
    if x.dim() != 3 or x.dtype not in _DTYPES:
        raise ValueError("x must be (rows, heads, head_dim) in bf16, fp16 or fp32")
    act = _norm_gate(gate, activation)
    for name, t in (("x", x), ("gate", gate), ("out", out)):
        _like(name, t, x, (x.dtype,))
    _written("out", out)
    rows, heads, dim = x.shape
    _vector32("weight", weight, [(dim,)])
    dev = _same_device("x", x=x, gate=gate, weight=weight, out=out)
    with torch.cuda.device(dev):
        if out is None:
            out = _empty_on(stream, x.shape, x.dtype, dev)
        _check(_lib().kda_gated_rmsnorm(
            _ptr(x), _Pair(*_strides(x, 2)), _ptr(gate),
            None if gate is None else _Pair(*_strides(gate, 2)), _ptr(weight), eps, act, rows,
            heads, dim, _DTYPES[x.dtype], _ptr(out), _Pair(*_strides(out, 2)),
            _stream_of(stream, dev)))
    return out


def residual_rmsnorm(y: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor | None,
                     scale: float = 1.0, gate: torch.Tensor | None = None, activation="sigmoid",
                     post_weight: torch.Tensor | None = None, eps: float = 1e-5,
                     out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The join between two blocks: r = residual + scale * act(gate) * p with p = y,
    or y normed and weighted by `post_weight` when that is given, and out = r
    normed and weighted by `weight`.  y, gate (rows, width) in bf16, fp16 or
    fp32; residual in y's dtype or fp32; weights fp32 (width).  Returns (out,
    residual_out); residual_out defaults to `residual` itself (updated in
    place).  The norm is taken of r before its rounding."""
    if y.dim() != 2 or y.dtype not in _DTYPES:
        raise ValueError("y must be (rows, width) in bf16, fp16 or fp32")
    act = _norm_gate(gate, activation)
    for name, t in (("y", y), ("gate", gate), ("out", out)):
        _like(name, t, y, (y.dtype,))
    _like("residual", residual, y, (y.dtype, torch.float32))
    _like("residual_out", residual_out, y, (residual.dtype,))
    _written("out", out)
    _written("residual_out", residual if residual_out is None else residual_out)
    rows, width = y.shape
    _vector32("weight", weight, [(width,)])
    _vector32("post_weight", post_weight, [(width,)])
    dev = _same_device("y", y=y, residual=residual, gate=gate, weight=weight,
                       post_weight=post_weight, out=out, residual_out=residual_out)
    with torch.cuda.device(dev):
        if out is None:
            out = _empty_on(stream, y.shape, y.dtype, dev)
        if residual_out is None:
            residual_out = residual
        stride = {n: _strides(t, 1)[0] if t is not None else 0
                  for n, t in (("y", y), ("r", residual), ("g", gate), ("o", out),
                               ("ro", residual_out))}
        _check(_lib().kda_residual_rmsnorm(
            _ptr(y), stride["y"], _ptr(residual), stride["r"], _ptr(gate), stride["g"],
            _ptr(weight), _ptr(post_weight), scale, eps, act, rows, width, _DTYPES[y.dtype],
            int(residual.dtype == torch.float32), _ptr(out), stride["o"], _ptr(residual_out),
            stride["ro"], _stream_of(stream, dev)))
    return out, residual_out
