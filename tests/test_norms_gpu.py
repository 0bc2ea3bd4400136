"""The gated per-head norm and the residual norm against their definitions in
64 bits.

Tolerance: the rounding of the result, eps / 2 of its type relative, and the
FP32 arithmetic before it: the sum of squares (relative 2^-24 times a few, all
terms positive), the reciprocal root (2 ulp), the exponential and the quotient
of the gate (a few ulp) and three products: 2^-20 relative covers them with a
factor of two.  The residual's sum may cancel, so its error is taken against
the sum of the absolute values."""

from __future__ import annotations

import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -24, "fp32": 2.0 ** -126}  # fp16 results may be subnormal


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import linear_attention_prefill_varlen_gb300 as pkg

    pkg.lib()
    return pkg


def close(got, want, dtype, size=None):
    got, want = got.cpu().double(), want.cpu()
    eps = torch.finfo(DT[dtype]).eps / 2
    room = eps * want.abs() + (2.0 ** -20) * (1 + eps) * (want.abs() if size is None else size.cpu())
    assert got.shape == want.shape and torch.isfinite(got).all()
    off = (got - want).abs()
    assert (off <= room + TINY[dtype]).all(), f"off by {(off / room).max():.3g} of what is allowed"


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("act", ["sigmoid", "silu", "none"])
@pytest.mark.parametrize("rows,heads,dim", [(1, 1, 8), (3, 2, 24), (5, 3, 64), (33, 17, 64),
                                            (37, 12, 128), (2, 1, 200), (9, 2, 256), (4, 1, 512),
                                            (700, 5, 128)])
def test_gated(kda, dtype, act, rows, heads, dim):
    gen = torch.Generator(device="cuda").manual_seed(rows + dim)
    x = torch.randn(rows, heads, dim, generator=gen, device="cuda").to(DT[dtype])
    gate = (3 * torch.randn(rows, heads, dim, generator=gen, device="cuda")).to(DT[dtype])
    w = torch.randn(dim, generator=gen, device="cuda") if dim != 24 else None
    g = None if act == "none" else gate
    got = kda.gated_rmsnorm(x, g, w, eps=1e-5, activation=act)
    close(got, ref.gated_rmsnorm(x, g, w, 1e-5, act), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated_large_heads(kda, dtype):
    x = torch.randn(3, 2, 1024, device="cuda").to(DT[dtype])
    close(kda.gated_rmsnorm(x, x, None), ref.gated_rmsnorm(x, x, None, 1e-5, "sigmoid"), dtype)


def test_gated_strides_and_in_place(kda):
    """Columns of a wider projection as x and gate, a wider out; guards stay; in place."""
    buf = torch.randn(10, 1000, device="cuda").bfloat16()
    x, gate = buf[:, 8:8 + 384].unflatten(1, (3, 128)), buf[:, 512:896].unflatten(1, (3, 128))
    w = torch.randn(128, device="cuda")
    want = ref.gated_rmsnorm(x, gate, w, 1e-6, "silu")
    wide = torch.full((10, 4, 136), 3.0, device="cuda").bfloat16()
    out = wide[:, :3, :128]
    kda.gated_rmsnorm(x, gate, w, eps=1e-6, activation="silu", out=out)
    close(out, want, "bf16")
    assert (wide[:, 3] == 3).all() and (wide[:, :, 128:] == 3).all()
    keep = buf.clone()
    kda.gated_rmsnorm(x, gate, w, eps=1e-6, activation="silu", out=x)
    close(x, want, "bf16")
    keep[:, 8:392] = buf[:, 8:392]
    assert torch.equal(keep, buf)


def test_gated_zero_rows_and_far_gates(kda):
    x = torch.zeros(4, 2, 64, device="cuda")
    gate = torch.tensor([0.0, 1e4, -1e4, 88.9], device="cuda")[:, None, None].expand(4, 2, 64)
    assert (kda.gated_rmsnorm(x, gate.contiguous(), None) == 0).all()
    x = torch.randn(4, 2, 64, device="cuda")
    for act in ("sigmoid", "silu"):
        got = kda.gated_rmsnorm(x, gate.contiguous(), None, activation=act)
        close(got, ref.gated_rmsnorm(x, gate, None, 1e-5, act), "fp32")
    big = torch.full((1, 1, 64), 1e18, device="cuda")
    close(kda.gated_rmsnorm(big, None, None), ref.gated_rmsnorm(big, None, None, 1e-5, "none"), "fp32")


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                       ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("rows,width", [(1, 8), (3, 264), (7, 1536), (5, 4608), (2, 6400),
                                        (3, 8192), (400, 1088)])
def test_residual(kda, dtype, res, act, post, rows, width):
    gen = torch.Generator(device="cuda").manual_seed(width)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    y, gate = randn(rows, width).to(DT[dtype]), (3 * randn(rows, width)).to(DT[dtype])
    r = (2 * randn(rows, width)).to(DT[res])
    w = randn(width) if width != 264 else None
    pw = randn(width) if post else None
    g = None if act == "none" else gate
    want, want_r = ref.residual_rmsnorm(y, r, w, 0.7, g, act, pw, 1e-5)
    ro = torch.empty_like(r)
    n, r2 = kda.residual_rmsnorm(y, r, w, scale=0.7, gate=g, activation=act, post_weight=pw,
                                 residual_out=ro)
    assert r2 is ro
    size = r.double().abs() + (want_r - r.double()).abs()
    close(ro, want_r, res, size)
    inv = torch.rsqrt((want_r * want_r).mean(-1, keepdim=True) + 1e-5)
    close(n, want, dtype, size * inv * (1 if w is None else w.double().abs()) + want.abs())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_residual_widest_row(kda, dtype):
    y, r = (torch.randn(3, 16384, device="cuda").to(DT[dtype]) for _ in range(2))
    want, want_r = ref.residual_rmsnorm(y, r, None, 1.0, None, "none", y[0].float(), 1e-5)
    n, ro = kda.residual_rmsnorm(y, r.clone(), None, post_weight=y[0].float())
    size = r.double().abs() + (want_r - r.double()).abs()
    close(ro, want_r, dtype, size)
    inv = torch.rsqrt((want_r * want_r).mean(-1, keepdim=True) + 1e-5)
    close(n, want, dtype, size * inv + want.abs())


def test_residual_in_place_and_strided(kda):
    buf = torch.randn(9, 1200, device="cuda").half()
    y, gate = buf[:, :512], buf[:, 520:1032]
    r = torch.randn(9, 520, device="cuda")
    keep = r.clone()
    want, want_r = ref.residual_rmsnorm(y, r[:, :512], None, 0.5, gate, "sigmoid", None, 1e-5)
    out, ro = kda.residual_rmsnorm(y, r[:, :512], None, scale=0.5, gate=gate, out=y)
    assert out.data_ptr() == y.data_ptr()
    close(ro, want_r, "fp32", 4 + want_r.abs())
    close(y, want, "fp16", 4 + want.abs())
    assert torch.equal(r[:, 512:], keep[:, 512:])


def test_no_rows(kda):
    x = torch.zeros(0, 2, 64, device="cuda")
    assert kda.gated_rmsnorm(x, x, None).shape == (0, 2, 64)
    y = torch.zeros(0, 64, device="cuda")
    assert kda.residual_rmsnorm(y, y, None)[0].shape == (0, 64)


def test_graph_and_stream(kda):
    s = torch.cuda.Stream()
    x = torch.randn(100, 4, 128, device="cuda").bfloat16()
    y = torch.randn(100, 512, device="cuda").bfloat16()
    r = torch.randn(100, 512, device="cuda").bfloat16()
    ro, n, o = torch.empty_like(r), torch.empty_like(y), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kda.gated_rmsnorm(x, x, None, out=o)
        with torch.cuda.graph(g, stream=s):
            kda.gated_rmsnorm(x, x, None, out=o)
            kda.residual_rmsnorm(y, r, None, residual_out=ro, out=n)
        x.normal_()
        y.normal_()
        g.replay()
    s.synchronize()
    close(o, ref.gated_rmsnorm(x, x, None, 1e-5, "sigmoid"), "bf16")
    want, want_r = ref.residual_rmsnorm(y, r, None, 1.0, None, "none", None, 1e-5)
    close(ro, want_r, "bf16", y.double().abs() + r.double().abs())
    close(n, want, "bf16", (y.double().abs() + r.double().abs()) * 4 + want.abs())
