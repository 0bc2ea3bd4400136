"""The operators of kda_layer.h without a GPU: exported symbols, argument
checks of the C ABI (addresses are never dereferenced) and of the wrappers,
empty calls, workspace sizes.  No kernel is launched."""

from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A16 = 1 << 20
INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3


@pytest.fixture(scope="module")
def layer():
    from linear_attention_prefill_varlen_gb300 import _build, _layer

    _build.build()
    _layer._lib()
    return _layer


def test_library_exports_every_declared_symbol(layer):
    text = open(os.path.join(ROOT, "include", "kda_layer.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(kda_[a-z0-9_]+)\s*\(", text)))
    assert len(names) >= 7
    assert [n for n in names if not hasattr(layer._lib(), n)] == []


def delta(layer, **over):
    d = layer.KdaDelta()
    base = dict(gate_kind=1, gate_per_channel=1, beta_kind=1, head_dim=128, heads=12, scale=0.1,
                q=A16, k=A16, v=A16, gate=A16, beta=A16, a_log=A16, dt_bias=A16, states=A16,
                out=A16)
    for name in ("q", "k", "v", "gate", "out"):
        base[name + "_stride"] = (1536, 128)
    base["beta_stride"], base["state_stride"] = (12, 1), (12 * 16384, 16384)
    for key, value in {**base, **over}.items():
        setattr(d, key, layer._Pair(*value) if isinstance(value, tuple) else value)
    return d


@pytest.mark.parametrize("over,status", [
    ({}, 0),
    ({"dt_bias": None}, 0),
    ({"head_dim": 64}, 0),
    ({"beta": A16 + 2}, 0),
    ({"version": 1}, INVALID),
    ({"reserved": 1}, INVALID),
    ({"x_dtype": 3}, INVALID),
    ({"gate_dtype": -1}, INVALID),
    ({"beta_dtype": 7}, INVALID),
    ({"gate_kind": 2}, INVALID),
    ({"beta_kind": 2}, INVALID),
    ({"gate_per_channel": 2}, INVALID),
    ({"heads": 0}, INVALID),
    ({"scale": float("nan")}, INVALID),
    ({"scale": float("inf")}, INVALID),
    ({"cache_index_stride": -1}, INVALID),
    ({"a_log": None, "dt_bias": None}, INVALID),  # softplus needs a_log
    ({"gate_kind": 0}, INVALID),                  # a log gate takes neither
    ({"gate_kind": 0, "a_log": None}, INVALID),
    ({"gate_kind": 0, "a_log": None, "dt_bias": None}, 0),
    ({"q": None}, INVALID), ({"k": None}, INVALID), ({"v": None}, INVALID),
    ({"gate": None}, INVALID), ({"beta": None}, INVALID), ({"states": None}, INVALID),
    ({"out": None}, INVALID),
    ({"beta_stride": (-1, 1)}, INVALID),
    ({"gate_stride": (1536, -128)}, INVALID),
    ({"head_dim": 96}, UNSUPPORTED),
    ({"head_dim": 256}, UNSUPPORTED),
    ({"heads": 1 << 17}, UNSUPPORTED),
    ({"q": A16 + 8}, MISALIGNED), ({"k": A16 + 2}, MISALIGNED), ({"v": A16 + 4}, MISALIGNED),
    ({"out": A16 + 8}, MISALIGNED), ({"states": A16 + 4}, MISALIGNED),
    ({"gate": A16 + 8}, MISALIGNED), ({"beta": A16 + 1}, MISALIGNED),
    ({"a_log": A16 + 2}, MISALIGNED),
    ({"q_stride": (1540, 128)}, MISALIGNED), ({"out_stride": (1536, 130)}, MISALIGNED),
    ({"k_stride": (-1536, 128)}, MISALIGNED), ({"state_stride": (16384, 16386)}, MISALIGNED),
    ({"gate_stride": (1536, 132)}, MISALIGNED),
    ({"gate_per_channel": 0, "gate": A16 + 2, "gate_stride": (13, 1)}, 0),
    ({"gate_per_channel": 0, "gate": A16 + 1}, MISALIGNED),
])
def test_delta_checks(layer, over, status):
    assert layer._lib().kda_delta_check(ctypes.byref(delta(layer, **over))) == status


def test_delta_calls_reject_before_any_cuda_call(layer):
    h = layer._lib()
    assert h.kda_delta_check(None) == INVALID
    bad = ctypes.byref(delta(layer, head_dim=96))
    good = ctypes.byref(delta(layer))
    assert h.kda_packed_delta_rule(bad, 10, A16, A16, A16, 2, -1, None, 0, None) == UNSUPPORTED
    assert h.kda_packed_delta_rule(good, 10, None, A16, A16, 2, -1, None, 0, None) == INVALID
    assert h.kda_packed_delta_rule(good, 10, A16, None, A16, 2, -1, None, 0, None) == INVALID
    assert h.kda_packed_delta_rule(good, 10, A16, A16, None, 2, -1, None, 0, None) == INVALID
    assert h.kda_packed_delta_rule(good, -1, A16, A16, A16, 2, -1, None, 0, None) == INVALID
    assert h.kda_packed_delta_rule(good, 10, A16, A16, A16, -2, -1, None, 0, None) == INVALID
    assert h.kda_packed_delta_rule(good, 1 << 31, A16, A16, A16, 2, -1, None, 0, None) == INVALID
    assert h.kda_packed_delta_rule(good, 0, None, None, None, 2, -1, None, 0, None) == 0
    assert h.kda_packed_delta_rule(good, 10, None, None, None, 0, -1, None, 0, None) == 0
    assert h.kda_delta_rule_update(bad, 4, A16, -1, None) == UNSUPPORTED
    assert h.kda_delta_rule_update(good, 4, None, -1, None) == INVALID
    assert h.kda_delta_rule_update(good, -4, A16, -1, None) == INVALID
    assert h.kda_delta_rule_update(good, 0, None, -1, None) == 0


def test_workspace_arguments(layer):
    h, n = layer._lib(), ctypes.c_int64(-1)
    ref = ctypes.byref(n)
    assert h.kda_packed_delta_rule_workspace(16384, 1, 12, 128, 0, 152, ref) == 0 and n.value >= 0
    assert h.kda_packed_delta_rule_workspace(-1, 1, 12, 128, 0, 152, ref) == INVALID
    assert h.kda_packed_delta_rule_workspace(1, 1, 0, 128, 0, 152, ref) == INVALID
    assert h.kda_packed_delta_rule_workspace(1, 1, 12, 100, 0, 152, ref) == UNSUPPORTED
    assert h.kda_packed_delta_rule_workspace(1, 1, 12, 128, 5, 152, ref) == INVALID
    assert h.kda_packed_delta_rule_workspace(1, 1, 12, 128, 0, -1, ref) == INVALID
    assert h.kda_packed_delta_rule_workspace(1, 1, 12, 128, 0, 152, None) == INVALID


def gated(layer, **over):
    P = layer._Pair
    a = dict(x=A16, xs=(1536, 128), gate=A16, gs=(1536, 128), weight=A16, eps=1e-5, act=1, rows=4,
             heads=12, dim=128, dtype=0, out=A16, os=(1536, 128))
    a.update(over)
    pair = lambda v: None if v is None else P(*v)  # noqa: E731
    return layer._lib().kda_gated_rmsnorm(a["x"], pair(a["xs"]), a["gate"], pair(a["gs"]),
                                          a["weight"], a["eps"], a["act"], a["rows"], a["heads"],
                                          a["dim"], a["dtype"], a["out"], pair(a["os"]), None)


@pytest.mark.parametrize("over,status", [
    ({"rows": 0, "x": None, "gate": None, "out": None}, 0),
    ({"rows": -1}, INVALID), ({"heads": 0}, INVALID), ({"dim": 0}, INVALID),
    ({"dtype": 3}, INVALID), ({"act": 3}, INVALID), ({"act": -1}, INVALID),
    ({"eps": -1e-5}, INVALID), ({"eps": float("nan")}, INVALID), ({"eps": float("inf")}, INVALID),
    ({"x": None}, INVALID), ({"out": None}, INVALID), ({"gate": None}, INVALID),
    ({"xs": None}, INVALID), ({"gs": None}, INVALID), ({"os": None}, INVALID),
    ({"rows": 1 << 40}, INVALID), ({"rows": 1 << 31}, INVALID),
    ({"dim": 100}, UNSUPPORTED), ({"dim": 1032}, UNSUPPORTED),
    ({"dim": 516, "dtype": 2}, UNSUPPORTED),
    ({"x": A16 + 8}, MISALIGNED), ({"out": A16 + 2}, MISALIGNED), ({"gate": A16 + 4}, MISALIGNED),
    ({"weight": A16 + 4}, MISALIGNED), ({"xs": (1540, 128)}, MISALIGNED),
    ({"gs": (1536, 124)}, MISALIGNED), ({"os": (-1536, 128)}, MISALIGNED),
])
def test_gated_norm_checks(layer, over, status):
    assert gated(layer, **over) == status


def residual(layer, **over):
    a = dict(y=A16, ys=4608, r=A16, rs=4608, gate=A16, gs=4608, w=A16, pw=A16, scale=1.0, eps=1e-5,
             act=1, rows=4, width=4608, dtype=0, f32=0, out=A16, os=4608, ro=A16, ros=4608)
    a.update(over)
    return layer._lib().kda_residual_rmsnorm(
        a["y"], a["ys"], a["r"], a["rs"], a["gate"], a["gs"], a["w"], a["pw"], a["scale"], a["eps"],
        a["act"], a["rows"], a["width"], a["dtype"], a["f32"], a["out"], a["os"], a["ro"],
        a["ros"], None)


@pytest.mark.parametrize("over,status", [
    ({"rows": 0, "y": None, "r": None, "gate": None, "out": None, "ro": None}, 0),
    ({"rows": -1}, INVALID), ({"width": 0}, INVALID), ({"dtype": 9}, INVALID),
    ({"f32": 2}, INVALID), ({"act": 3}, INVALID), ({"eps": -1.0}, INVALID),
    ({"y": None}, INVALID), ({"r": None}, INVALID), ({"out": None}, INVALID),
    ({"ro": None}, INVALID), ({"gate": None}, INVALID),
    ({"width": 4604}, UNSUPPORTED), ({"width": 16392}, UNSUPPORTED),
    ({"width": 8196, "dtype": 2}, UNSUPPORTED),
    ({"y": A16 + 2}, MISALIGNED), ({"r": A16 + 8}, MISALIGNED), ({"gate": A16 + 8}, MISALIGNED),
    ({"w": A16 + 4}, MISALIGNED), ({"pw": A16 + 8}, MISALIGNED), ({"out": A16 + 8}, MISALIGNED),
    ({"ro": A16 + 4}, MISALIGNED), ({"ys": 4612}, MISALIGNED), ({"rs": 4612}, MISALIGNED),
    ({"gs": 4610}, MISALIGNED), ({"os": -4608}, MISALIGNED), ({"ros": 4612}, MISALIGNED),
])
def test_residual_norm_checks(layer, over, status):
    assert residual(layer, **over) == status


T, H, D = 6, 2, 64


def call(**over):
    import linear_attention_prefill_varlen_gb300 as pkg

    a = dict(q=torch.zeros(T, H, D), k=torch.zeros(T, H, D), v=torch.zeros(T, H, D),
             gate=torch.zeros(T, H, D), beta=torch.zeros(T, H), states=torch.zeros(3, H, D, D),
             query_start_loc=torch.tensor([0, T], dtype=torch.int32),
             cache_indices=torch.zeros(1, dtype=torch.int32),
             has_initial_state=torch.zeros(1, dtype=torch.bool))
    a.update(over)
    return pkg.packed_delta_rule_fn(**a)


@pytest.mark.parametrize("over,exc,words", [
    ({"q": torch.zeros(T, H * D)}, ValueError, "q must be"),
    ({"q": torch.zeros(T, H, D, dtype=torch.int32)}, ValueError, "q must be"),
    ({"k": torch.zeros(T, H, D).half()}, ValueError, "k must be"),
    ({"v": torch.zeros(T, H, D + 1)}, ValueError, "v must be"),
    ({"q": torch.zeros(T, D, H).transpose(1, 2)}, ValueError, "q must have unit"),
    ({"gate": torch.zeros(T, H, 1)}, ValueError, "gate must be"),
    ({"gate": torch.zeros(T, H, D).double()}, ValueError, "gate must be"),
    ({"gate": torch.zeros(T, H, 1).expand(T, H, D)}, ValueError, "gate must have unit"),
    ({"beta": torch.zeros(T, H, D)}, ValueError, "beta"),
    ({"states": torch.zeros(3, H, D, D).bfloat16()}, ValueError, "states"),
    ({"states": torch.zeros(3, H, D, D).transpose(2, 3)}, ValueError, "contiguous"),
    ({"states": torch.zeros(3, H + 1, D, D)}, ValueError, "states"),
    ({"a_log": torch.zeros(H + 1)}, ValueError, "a_log"),
    ({"dt_bias": torch.zeros(H, D)}, ValueError, "needs a_log"),
    ({"a_log": torch.zeros(H), "dt_bias": torch.zeros(D, H).t()}, ValueError, "dt_bias"),
    ({"out": torch.zeros(T, H, D).half()}, ValueError, "out must be"),
    ({"out": torch.zeros(1, H, D).expand(T, H, D)}, ValueError, "overlap"),
    ({"cache_indices": torch.zeros(1, dtype=torch.int64)}, TypeError, "cache_indices"),
    ({"cache_indices": torch.zeros(0, dtype=torch.int32)}, ValueError, "needed"),
    ({"query_start_loc": torch.tensor([0, T])}, TypeError, "query_start_loc"),
    ({"has_initial_state": torch.zeros(1)}, TypeError, "has_initial_state"),
    ({}, ValueError, "CUDA"),
])
def test_delta_wrapper_rejects(over, exc, words):
    with pytest.raises(exc, match=words):
        call(**over)


def test_norm_wrappers_reject():
    import linear_attention_prefill_varlen_gb300 as pkg

    x = torch.zeros(3, 2, 64)
    for args, kw, words in [
            ((x[0], x[0], None), {}, "x must be"),
            ((x, x.half(), None), {}, "gate must be"),
            ((x, x, torch.zeros(63)), {}, "weight"),
            ((x, x, torch.zeros(64).half()), {}, "weight"),
            ((x, x, None), {"activation": "relu"}, "activation"),
            ((x, x, None), {"activation": "none"}, "needs an activation"),
            ((x, x, None), {"out": torch.zeros(3, 2, 65)}, "out must be"),
            ((x, x, None), {"out": torch.zeros(1, 2, 64).expand(3, 2, 64)}, "overlap"),
            ((x, x, None), {}, "CUDA")]:
        with pytest.raises(ValueError, match=words):
            pkg.gated_rmsnorm(*args, **kw)
    y = torch.zeros(3, 64).half()
    for args, kw, words in [
            ((x, x, None), {}, "y must be"),
            ((y, y.bfloat16(), None), {}, "residual must be"),
            ((y, y, None), {"residual_out": y.float()}, "residual_out must be"),
            ((y, y, None), {"gate": y[:2]}, "gate must be"),
            ((y, y, None), {"post_weight": torch.zeros(3)}, "post_weight"),
            ((y, y[:1].expand(3, 64), None), {}, "overlap"),
            ((y, y, None), {}, "CUDA")]:
        with pytest.raises(ValueError, match=words):
            pkg.residual_rmsnorm(*args, **kw)
