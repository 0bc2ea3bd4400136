"""The gated delta rule on sequences long enough for its chunked path, and on
batches that mix all of its paths: one-token sequences, short ones (groups of
eight tokens), chunks of 64, and sequences split into segments.  Against the
definition in 64 bits, with the tolerances of test_delta_gpu."""

from __future__ import annotations

import ctypes

import pytest
import torch

from test_delta_gpu import Batch, check, compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import linear_attention_prefill_varlen_gb300 as pkg

    pkg.lib()
    return pkg


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gate", ["raw", "log", "loghead", "rawhead"])
def test_types_and_gates(kda, dim, dtype, gate):
    check(kda, Batch([113, 0, 128, 1, 193, 40], dtype, 2, dim, gate, null=(2,), seed=dim + 1))


@pytest.mark.parametrize("n", [112, 113, 119, 120, 121, 127, 128, 129, 160, 191, 192, 193, 255, 256,
                               257, 300, 383])
@pytest.mark.parametrize("init", [False, True])
def test_one_sequence(kda, n, init):
    check(kda, Batch([n], heads=2, init=init, seed=n))


@pytest.mark.parametrize("n", [1024, 1025, 1030, 1088, 1100, 1537])
def test_segments(kda, n):
    """More than 16 chunks: several segments, whole and ragged last ones."""
    check(kda, Batch([n], "bf16", 1, 64, "raw", seed=n, init=True))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_segments_next_to_short_sequences(kda, dtype):
    check(kda, Batch([700, 3, 0, 1, 1200, 65, 513, 1, 512], dtype, 1, 128, "log", gate_mul=0.02,
                     seed=31, null=(4,)))


@pytest.mark.parametrize("lens_of", ["ones", "short", "mixed"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_pairs(kda, lens_of, dtype):
    """Enough (sequence, head) pairs to fill the GPU: the other length rule, one-token
    sequences apart, slots counted by start row."""
    g = torch.Generator().manual_seed(3)
    if lens_of == "ones":
        lens = [1] * 300
    elif lens_of == "short":
        lens = torch.randint(0, 36, (260,), generator=g).tolist()
    else:
        lens = (torch.randint(1, 140, (24,), generator=g).tolist() + [1] * 200 + [32, 33, 34, 64, 65])
        order = torch.randperm(len(lens), generator=g).tolist()
        lens = [lens[i] for i in order]
    check(kda, Batch(lens, dtype, 2, 64, "raw", seed=41, null=(5, 7)))


@pytest.mark.parametrize("value", [0.0, -40.0, -200.0, float("-inf")])
@pytest.mark.parametrize("form", ["log", "loghead"])
def test_decays_at_the_ends(kda, value, form):
    b = Batch([200, 130], gate=form, seed=6, init=True)
    pick = torch.rand(b.gate.shape, generator=torch.Generator().manual_seed(1)) < 0.3
    b.gate[pick.cuda()] = value
    check(kda, b)
    b = Batch([200, 130], gate=form, seed=7, init=True)
    b.gate[20:140] = value
    check(kda, b)


@pytest.mark.parametrize("k_scale,v_scale", [(1e-3, 1e3), (1.2, 1e-4), (1.0, 1e4)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_magnitudes(kda, k_scale, v_scale, dtype):
    check(kda, Batch([180, 140], dtype, k_scale=k_scale, v_scale=v_scale if dtype == "bf16" else
                     min(v_scale, 100.0), seed=10, init=True))


def test_no_decay_keeps_every_token(kda):
    """Decays of 1 and orthogonal keys: nothing is forgotten over 1500 tokens, so errors add up."""
    b = Batch([1500], "bf16", 1, 64, "log", gate_mul=0.0, seed=12, init=True)
    b.beta.mul_(0.1)
    check(kda, b)


def test_rows_of_zeros_and_repeated_keys(kda):
    b = Batch([250], heads=2, gate="log", gate_mul=0.0, seed=12, init=True)
    b.k[20:160] = b.k[20]
    b.k[170:175] = 0
    b.q[100:110] = 0
    b.v[180:190] = 0
    b.beta[20:160] = 1.0
    b.beta[190:200] = 0.0
    check(kda, b)


def test_garbage_where_nothing_is_read(kda):
    b = Batch([140, 270, 1, 120], seed=13, null=(3,), init=False)
    want = b.want()
    nan = float("nan")
    owned = torch.zeros(b.tokens, dtype=torch.bool)
    for s, n in zip(b.starts, b.lens):
        owned[s:s + n] = True
    for t in (b.q, b.k, b.v, b.gate, b.beta):
        t[~owned.cuda()] = nan
    b.states.fill_(nan)
    n = kda.delta_rule_workspace(b.tokens, len(b.lens), b.heads, b.dim)
    out = b.run(kda, workspace=torch.full((n + 100,), 255, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    used = [int(x) for x in b.lines if x >= 0]
    rest = [i for i in range(b.states.shape[0]) if i not in used]
    assert torch.isnan(b.states[rest]).all()
    b.states[rest] = want[1][rest].float().cuda()
    compare(b, out, b.states, want)


def test_columns_of_a_projection_and_cache_gaps(kda):
    b = Batch([150, 1, 230], heads=3, packed=True, seed=14)
    want = b.want()
    cache = torch.full((7, 4, 130, 128), 5.0, device="cuda")
    cache[:, :3, :128] = b.states
    b.states = cache[:, :3, :128]
    out = b.run(kda)
    torch.cuda.synchronize()
    compare(b, out, b.states, want)
    assert (cache[:, 3] == 5.0).all() and (cache[:, :, 128:] == 5.0).all()


def test_workspace_bounds(kda):
    """A workspace that is too small or misaligned is refused; one of the stated size
    with guards after it is not written past its end."""
    b = Batch([300, 140], seed=15)
    want = b.want()
    n = kda.delta_rule_workspace(b.tokens, 2, b.heads, b.dim)
    assert n > 0
    big = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
    assert big.data_ptr() % 256 == 0
    keep = b.states.clone()
    with pytest.raises(kda.KdaError) as e:
        b.run(kda, workspace=big[:n - 1])
    assert e.value.status == kda.KDA_ERR_INVALID_ARG
    with pytest.raises(kda.KdaError) as e:
        b.run(kda, workspace=big[16:])
    assert e.value.status == kda.KDA_ERR_MISALIGNED
    with pytest.raises(ValueError):
        b.run(kda, workspace=big.half())
    torch.cuda.synchronize()
    assert torch.equal(b.states, keep)
    out = b.run(kda, workspace=big[:n])
    torch.cuda.synchronize()
    compare(b, out, b.states, want)
    assert (big[n:] == 77).all()
    assert big[:4].view(torch.int32).item() == 0, "a wait inside the kernels ran out"


def test_same_bits_every_time(kda):
    first = None
    for _ in range(4):
        b = Batch([1300, 200, 64, 17, 1], heads=3, dim=64, seed=17)
        out = b.run(kda)
        torch.cuda.synchronize()
        both = (out.clone(), b.states.clone())
        if first is not None:
            assert torch.equal(first[0], both[0]) and torch.equal(first[1], both[1])
        first = both


def test_graph_replays_with_new_lengths(kda):
    a = Batch([300, 3, 840], heads=1, dim=64, seed=18, lead=0, tail=7)
    b = Batch([1, 1080, 69], heads=1, dim=64, seed=19, lead=0, tail=0)
    out = torch.full((1150, 1, 64), 7.0, dtype=a.dtype, device="cuda")
    ws = torch.empty(kda.delta_rule_workspace(1150, 3, 1, 64), dtype=torch.uint8, device="cuda")
    a.run(kda, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(kda, out=out, workspace=ws)
    want = b.want()
    for name in ("q", "k", "v", "gate", "beta", "states", "qsl", "ci", "his", "a_log", "dt_bias"):
        getattr(a, name).copy_(getattr(b, name))
    for _ in range(2):
        a.states.copy_(b.states)
        out.fill_(7.0)
        g.replay()
    torch.cuda.synchronize()
    compare(b, out, a.states, want)


def test_two_streams_with_their_own_workspaces(kda):
    pairs = [Batch([400, 150], seed=50 + i) for i in range(2)]
    wants = [b.want() for b in pairs]
    streams = [torch.cuda.Stream() for _ in pairs]
    outs = [torch.full((b.tokens, 2, 128), 7.0, dtype=b.dtype, device="cuda") for b in pairs]
    torch.cuda.synchronize()
    keep = [b.states.clone() for b in pairs]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s, o, k in zip(pairs, streams, outs, keep):
            with torch.cuda.stream(s):
                b.states.copy_(k)
            b.run(kda, stream=s, out=o)
    torch.cuda.synchronize()
    for b, o, w in zip(pairs, outs, wants):
        compare(b, o, b.states, w)


def test_raw_stream_handle(kda):
    b = Batch([150], seed=60)
    want = b.want()
    s = torch.cuda.Stream()
    out = torch.full((b.tokens, 2, 128), 7.0, dtype=b.dtype, device="cuda")
    torch.cuda.synchronize()
    b.run(kda, stream=s.cuda_stream, out=out)
    s.synchronize()
    compare(b, out, b.states, want)
    assert isinstance(s.cuda_stream, int) and ctypes.sizeof(ctypes.c_void_p) == 8
