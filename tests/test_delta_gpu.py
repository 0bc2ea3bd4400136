"""The gated delta rule (packed and one token) against its definition in 64
bits, at the lengths, types, layouts and values where it can go wrong.

Tolerances.  An output is off by its rounding, eps / 2 of its type relative,
and by its sum: the largest error allowed there is taken against |S row| |q|,
which bounds the sum's size; 2^-10 for 16-bit outputs (the attention products
of the chunked path may round each operand to 11 bits, 2^-11 each) and 2^-18 for
fp32 outputs.  A state is fp32 with operands of at least 22 bits: 2^-18 of its
head's norm, which leaves a factor of 16 for the sums of up to a few hundred
tokens."""

from __future__ import annotations

import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import linear_attention_prefill_varlen_gb300 as pkg

    pkg.lib()
    return pkg


class Batch:
    """A packed batch with guard rows before, between and after what the calls own."""

    def __init__(self, lens, dtype="bf16", heads=2, dim=128, gate="raw", gate_dtype=None,
                 seed=0, lead=3, tail=5, init=None, null=(), k_scale=1.0, packed=False,
                 gate_mul=1.0, v_scale=1.0):
        gen = torch.Generator().manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=gen)

        self.lens, self.heads, self.dim, self.gate_form = list(lens), heads, dim, gate
        n = len(self.lens)
        self.starts = [lead + sum(self.lens[:i]) for i in range(n)]
        self.tokens = T = lead + sum(self.lens) + tail
        dt = DT[dtype]
        self.dtype = dt
        unit = torch.nn.functional.normalize
        qkv = [unit(randn(T, heads, dim), dim=-1), unit(randn(T, heads, dim), dim=-1) * k_scale,
               randn(T, heads, dim) * v_scale]
        if packed:  # columns of one row-strided projection
            buf = torch.zeros(T, 3 * heads * dim + 24, dtype=dt)
            for i in range(3):
                buf[:, 8 + i * heads * dim:8 + (i + 1) * heads * dim] = \
                    qkv[i].reshape(T, -1).to(dt)
            buf = buf.cuda()
            self.q, self.k, self.v = (
                buf[:, 8 + i * heads * dim:8 + (i + 1) * heads * dim].unflatten(1, (heads, dim))
                for i in range(3))
        else:
            self.q, self.k, self.v = (x.to(dt).cuda() for x in qkv)
        gdt = DT[gate_dtype] if gate_dtype else (dt if gate.startswith("raw") else torch.float32)
        per_head = gate.endswith("head")
        shape = (T, heads) if per_head else (T, heads, dim)
        if gate.startswith("raw"):
            self.gate = (randn(*shape) * gate_mul).to(gdt).cuda()
            self.a_log = torch.log(1 + 15 * torch.rand(heads, generator=gen)).cuda()
            self.dt_bias = (randn(heads) if per_head else randn(heads, dim)).sub(3).cuda()
            self.beta, self.logits = randn(T, heads).to(dt).cuda(), True
        else:
            self.gate = -(randn(*shape).square() * 0.3 * gate_mul).to(gdt).cuda()
            self.a_log = self.dt_bias = None
            self.beta, self.logits = torch.rand(T, heads, generator=gen).cuda(), False
        self.scale = dim ** -0.5
        lines = torch.randperm(n + 4, generator=gen)[:n].to(torch.int32)
        for s in null:
            lines[s] = -1
        self.lines = lines
        self.reads = torch.rand(n, generator=gen) < 0.6 if init is None else \
            torch.full((n,), bool(init))
        self.states = (randn(n + 4, heads, dim, dim) * 0.1 * v_scale).cuda()
        self.qsl = torch.tensor([*self.starts, lead + sum(self.lens)], dtype=torch.int32).cuda()
        self.ci, self.his = lines.cuda(), self.reads.cuda()

    def args(self):
        return dict(scale=self.scale, a_log=self.a_log, dt_bias=self.dt_bias,
                    beta_logits=self.logits, null_block_id=-1)

    def run(self, kda, **over):
        out = torch.full((self.tokens, self.heads, self.dim), 7.0, dtype=self.dtype,
                         device="cuda")
        a = {**self.args(), "out": out, **over}
        kda.packed_delta_rule_fn(self.q, self.k, self.v, self.gate, self.beta, self.states,
                                 self.qsl, self.ci, self.his, **a)
        return a["out"]

    def want(self):
        c = lambda t: None if t is None else t.cpu()  # noqa: E731
        return ref.delta_rule(c(self.q), c(self.k), c(self.v), c(self.gate), c(self.beta),
                              c(self.states), self.lens, self.starts, self.lines.tolist(),
                              self.reads.tolist(), self.scale, c(self.a_log), c(self.dt_bias),
                              self.logits)


def compare(b, out, states, want):
    o, s, size = want
    owned = ~torch.isnan(o[:, 0, 0])
    got = out.cpu().double()
    assert (got[~owned] == 7.0).all(), "rows no sequence owns were written"
    eps = torch.finfo(b.dtype).eps / 2
    loose = 2.0 ** -18 if b.dtype == torch.float32 else 2.0 ** -10
    off = (got - o).abs()[owned]
    room = eps * o.abs()[owned] + loose * size[owned] + torch.finfo(b.dtype).tiny
    assert torch.isfinite(got[owned]).all()
    assert (off <= room).all(), f"output off by {(off / room).max():.3g} of what is allowed"
    got = states.cpu().double()
    used = sorted({int(x) for x, n in zip(b.lines, b.lens) if x >= 0 and n})
    others = [i for i in range(got.shape[0]) if i not in used]
    assert torch.equal(got[others], s[others]), "a line that no sequence uses was written"
    off = (got[used] - s[used]).flatten(2).norm(dim=-1)
    room = 2.0 ** -18 * s[used].flatten(2).norm(dim=-1) + 1e-30
    assert torch.isfinite(got[used]).all()
    assert (off <= room).all(), f"state off by {(off / room).max():.3g} of what is allowed"


def check(kda, b, **over):
    want = b.want()
    out = b.run(kda, **over)
    torch.cuda.synchronize()
    compare(b, out, b.states, want)


LENS = [1, 2, 0, 15, 16, 17, 63, 64, 65, 0, 127, 130]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gate", ["raw", "log", "loghead", "rawhead"])
def test_lengths_types_gates(kda, dim, dtype, gate):
    check(kda, Batch(LENS, dtype, 2, dim, gate, null=(4,), seed=dim))


@pytest.mark.parametrize("n", [1, 2, 3, 8, 9, 31, 32, 33, 48, 64, 65, 96, 128, 129, 191, 193, 257])
@pytest.mark.parametrize("init", [False, True])
def test_one_sequence(kda, n, init):
    check(kda, Batch([n], heads=3, init=init, seed=n))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_long_sequence_carries_its_state(kda, dtype, dim):
    check(kda, Batch([1500, 0, 700], dtype, 1, dim, "log", gate_mul=0.05, init=True, seed=11))


@pytest.mark.parametrize("gate_dtype", ["bf16", "fp16", "fp32"])
def test_gate_type_apart_from_x(kda, gate_dtype):
    check(kda, Batch([70, 5], "bf16", gate="raw", gate_dtype=gate_dtype, seed=3))


def test_columns_of_a_projection(kda):
    check(kda, Batch([100, 1, 30], heads=3, packed=True, seed=4))


def test_many_sequences(kda):
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 40, (150,), generator=g).tolist()
    check(kda, Batch(lens, heads=2, dim=64, gate="log", null=(7, 8), seed=5))


@pytest.mark.parametrize("value", [0.0, -40.0, -200.0, float("-inf")])
def test_decays_at_the_ends(kda, value):
    """No decay at all, and decays that underflow inside a few tokens, on some
    channels and tokens only."""
    b = Batch([90, 20], gate="log", seed=6, init=True)
    pick = torch.rand(b.gate.shape, generator=torch.Generator().manual_seed(1)) < 0.3
    b.gate[pick.cuda()] = value
    check(kda, b)
    b = Batch([90, 20], gate="log", seed=6, init=True)
    b.gate[:, :, ::2] = value
    check(kda, b)
    b = Batch([90, 20], gate="log", seed=7, init=True)
    b.gate[20:40] = value
    check(kda, b)


def test_gates_far_out(kda):
    """Raw gates of +-80: a decay of 1 to rounding, and one that is 0."""
    b = Batch([100], seed=8, init=True)
    b.gate[::3] = 80.0
    b.gate[1::3] = -80.0
    check(kda, b)


@pytest.mark.parametrize("k_scale,v_scale", [(1e-3, 1e3), (1.2, 1e-4), (1.0, 1e4)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_magnitudes(kda, k_scale, v_scale, dtype):
    check(kda, Batch([150, 33], dtype, k_scale=k_scale, v_scale=v_scale, seed=10, init=True))


def test_rows_of_zeros_and_repeated_keys(kda):
    b = Batch([130], heads=2, gate="log", gate_mul=0.0, seed=12, init=True)
    b.k[20:60] = b.k[20]          # the same key forty times, no decay
    b.k[70:75] = 0
    b.v[80:90] = 0
    b.beta[20:60] = 1.0
    b.beta[90:100] = 0.0
    check(kda, b)


def test_garbage_where_nothing_is_read(kda):
    """NaN in unowned rows, in lines that are only written, and in the lines of
    no sequence; the padding sequence starts from zero."""
    b = Batch([40, 70, 1, 20, 1], seed=13, null=(3, 4), init=False)
    want = b.want()
    nan = float("nan")
    owned = torch.zeros(b.tokens, dtype=torch.bool)
    for s, n in zip(b.starts, b.lens):
        owned[s:s + n] = True
    for t in (b.q, b.k, b.v, b.gate, b.beta):
        t[~owned.cuda()] = nan
    b.states.fill_(nan)
    out = b.run(kda)
    torch.cuda.synchronize()
    used = [int(x) for x in b.lines if x >= 0]
    rest = [i for i in range(b.states.shape[0]) if i not in used]
    assert torch.isnan(b.states[rest]).all()
    b.states[rest] = want[1][rest].float().cuda()
    compare(b, out, b.states, want)


def test_strides(kda):
    """A state cache with gaps between lines and heads, strided cache_indices and beta."""
    b = Batch([66, 3, 17], heads=2, dim=64, seed=14)
    want = b.want()
    cache = torch.full((7, 3, 65, 64), 5.0, device="cuda")
    cache[:, :2, :64] = b.states
    b.states = cache[:, :2, :64]
    wide = torch.full((3, 4), -9, dtype=torch.int32, device="cuda")
    wide[:, 1] = b.ci
    b.ci = wide[:, 1]
    beta = torch.zeros(b.tokens, 2, 3, dtype=b.beta.dtype, device="cuda")
    beta[..., 1] = b.beta
    b.beta = beta[..., 1]
    out = b.run(kda)
    torch.cuda.synchronize()
    compare(b, out, b.states, want)
    assert (cache[:, 2] == 5.0).all() and (cache[:, :, 64] == 5.0).all()


def test_far_cache_lines(kda):
    """A line whose elements lie past 2^32 of the cache's base."""
    b = Batch([40, 1], heads=1, dim=64, seed=15, init=True)
    want = b.want()
    far = 2 ** 31 + 64
    cache = torch.empty(2 * far + 64 * 64, dtype=torch.float32, device="cuda")
    view = cache.as_strided((3, 1, 64, 64), (far, 64 * 64, 64, 1))
    view[:] = 0
    order = b.lines.tolist()
    view[2], view[1] = b.states[order[0]], b.states[order[1]]
    b.ci = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    out = torch.full((b.tokens, 1, 64), 7.0, dtype=b.dtype, device="cuda")
    kda.packed_delta_rule_fn(b.q, b.k, b.v, b.gate, b.beta, view, b.qsl, b.ci, b.his, out=out,
                             **b.args())
    torch.cuda.synchronize()
    b.states[order[0]], b.states[order[1]] = view[2], view[1]
    compare(b, out, b.states, want)


@pytest.mark.parametrize("gate", ["raw", "loghead"])
def test_split_equals_whole(kda, gate):
    """Two calls with the state carried, against the definition of the whole."""
    b = Batch([150], heads=2, gate=gate, seed=16, init=True, lead=0, tail=0)
    want = b.want()
    outs = []
    for lo, hi in ((0, 70), (70, 150)):
        qsl = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        outs.append(kda.packed_delta_rule_fn(
            b.q[lo:hi], b.k[lo:hi], b.v[lo:hi], b.gate[lo:hi], b.beta[lo:hi], b.states, qsl, b.ci,
            b.his, **b.args()))
    torch.cuda.synchronize()
    compare(b, torch.cat(outs), b.states, want)


def test_same_bits_every_time(kda):
    first = None
    for _ in range(3):
        b = Batch([300, 64, 17, 1], heads=2, seed=17)
        out = b.run(kda)
        torch.cuda.synchronize()
        both = (out.clone(), b.states.clone())
        if first is not None:
            assert torch.equal(first[0], both[0]) and torch.equal(first[1], both[1])
        first = both


def test_graph_replays_with_new_lengths(kda):
    """A captured call follows new metadata and inputs of the same sizes."""
    a = Batch([100, 3, 40], seed=18, lead=0, tail=7)
    b = Batch([1, 80, 69], seed=19, lead=0, tail=0)
    out = torch.full((150, 2, 128), 7.0, dtype=a.dtype, device="cuda")
    a.run(kda, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(kda, out=out)
    want = b.want()
    for name in ("q", "k", "v", "gate", "beta", "states", "qsl", "ci", "his", "a_log", "dt_bias"):
        getattr(a, name).copy_(getattr(b, name))
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    compare(b, out, a.states, want)


def test_own_stream(kda):
    """The call and its workspace live on the given stream."""
    b = Batch([300, 64, 5], seed=20)
    want = b.want()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.full((b.tokens, 2, 128), 7.0, dtype=b.dtype, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    b.run(kda, stream=s, out=out)
    s.synchronize()
    compare(b, out, b.states, want)


def test_empty_calls(kda):
    b = Batch([0, 0], lead=0, tail=0)
    before = b.states.clone()
    assert b.run(kda).shape == (0, 2, 128)
    b = Batch([4], lead=0, tail=0)
    qsl = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.packed_delta_rule_fn(b.q, b.k, b.v, b.gate, b.beta, b.states, qsl, b.ci[:0], b.his[:0])
    torch.cuda.synchronize()
    assert torch.equal(before.shape and b.states, b.states)


# ------------------------------------------------------------------ one token


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gate", ["raw", "log", "loghead", "rawhead"])
@pytest.mark.parametrize("batch", [1, 7, 200])
def test_update(kda, dim, dtype, gate, batch):
    heads = 3 if batch < 100 else 2
    null = (batch // 2,) if batch > 1 else ()
    b = Batch([1] * batch, dtype, heads, dim, gate, init=True, null=null, lead=0, tail=0, seed=21)
    want = b.want()
    out = kda.delta_rule_update(b.q, b.k, b.v, b.gate, b.beta, b.states, b.ci, **b.args())
    torch.cuda.synchronize()
    compare(b, out, b.states, want)


def test_updates_follow_a_prefill(kda):
    """A prompt, then tokens one by one, against the definition of the whole; through
    a captured step, as a serving loop runs it."""
    b = Batch([100], heads=2, seed=22, init=False, lead=0, tail=0)
    want = b.want()
    a = b.args()
    out = torch.empty_like(b.q)
    qsl = torch.tensor([0, 90], dtype=torch.int32, device="cuda")
    kda.packed_delta_rule_fn(b.q[:90], b.k[:90], b.v[:90], b.gate[:90], b.beta[:90], b.states, qsl,
                             b.ci, b.his, out=out[:90], **a)
    step = [x[:1].clone() for x in (b.q, b.k, b.v, b.gate, b.beta)]
    one = torch.empty_like(step[0])
    keep = b.states.clone()
    kda.delta_rule_update(*step, b.states, b.ci, out=one, **a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.delta_rule_update(*step, b.states, b.ci, out=one, **a)
    b.states.copy_(keep)
    for t in range(90, 100):
        for dst, src in zip(step, (b.q, b.k, b.v, b.gate, b.beta)):
            dst.copy_(src[t:t + 1])
        g.replay()
        out[t:t + 1] = one
    torch.cuda.synchronize()
    compare(b, out, b.states, want)


def test_conv_into_the_rule(kda):
    """The layer's own chain: the packed conv with q and k normed per head, the rule on
    its planes, the gated norm; the rule's part against the definition."""
    heads, dim, lens = 2, 128, [90, 1, 20]
    T, part = sum(lens), heads * dim
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, 3 * part + 64, generator=gen, device="cuda").bfloat16()
    w = torch.rand(3 * part, 4, generator=gen, device="cuda") - 0.5
    conv_states = torch.randn(4, 3 * part, 3, generator=gen, device="cuda")
    b = Batch(lens, heads=heads, dim=dim, seed=23, lead=0, tail=0)
    planes = kda.packed_causal_conv1d_fn(x[:, :3 * part], w, None, conv_states, b.qsl,
                                         b.ci.clamp(max=3), b.his, part, use_qk_l2norm=True,
                                         head_dim=dim)
    b.q, b.k, b.v = (planes[i].unflatten(1, (heads, dim)) for i in range(3))
    want = b.want()
    out = b.run(kda)
    y = kda.gated_rmsnorm(out, b.q, torch.ones(dim, device="cuda"))
    torch.cuda.synchronize()
    compare(b, out, b.states, want)
    z = ref.gated_rmsnorm(out.cpu(), b.q.cpu(), None, 1e-5, "sigmoid")
    assert ((y.cpu().double() - z).abs() <= 2.0 ** -8 * z.abs() + 2.0 ** -20).all()
