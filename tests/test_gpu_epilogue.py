"""The W8A8 linear with bias, activation and residual in its epilogue, on every path (GEMV, one-CTA and CTA-pair
tensor-core GEMMs).  Without an activation, and with ReLU, the fp32 steps are the definition's, so outputs are
compared bit for bit; with the others against 64 bits."""
import math

import numpy as np
import pytest
import torch

from moe_gemm_absmax_b200 import inputs, w8a8
from tests._util import to_dev_bf16

pytestmark = pytest.mark.gpu

ACTS = {"none": w8a8.ACT_NONE, "relu": w8a8.ACT_RELU, "silu": w8a8.ACT_SILU, "gelu": w8a8.ACT_GELU,
        "gelu_tanh": w8a8.ACT_GELU_TANH}


def _case(M, K, N, seed):
    xb, w = inputs.dense_linear(seed, M, K, N)
    g = torch.Generator().manual_seed(seed)
    qw, sw = w8a8.quant_rows_f32(torch.from_numpy(w).cuda())
    bias = (0.5 * torch.randn(N, generator=g)).cuda()
    res = torch.randn((M, N), generator=g).to(torch.bfloat16).cuda()
    return to_dev_bf16(xb), qw, sw, bias, res


def _pre(x, qw, sw):
    """fp32 values of the plain linear: the exact integer sum, times sx, times sw, one rounding each."""
    qx, sx = w8a8.quant_act(x)
    acc = (qx.double() @ qw.double().t()).float()      # below 2^31: float() rounds the integer once, as the kernel
    return acc * sx[:, None] * sw


def _act64(name, v):
    v = v.double()
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def _check(y, x, qw, sw, bias, res, name):
    v = _pre(x, qw, sw)
    if name in ("none", "relu"):
        r = v if bias is None else v + bias
        r = torch.clamp(r, min=0) if name == "relu" else r
        r = r if res is None else r + res.float()
        assert torch.equal(y, r.to(torch.bfloat16))
        return
    b = torch.zeros_like(sw) if bias is None else bias
    t = torch.zeros_like(v) if res is None else res
    a = _act64(name, v.double() + b.double())
    r = a + t.double()
    # bf16's rounding; the sums' (2^-24 each, through a slope below 1.2), the activation's 2^-20; where e^-v
    # overflows the result is 0 for a value below 1e-36
    tol = 2.0 ** -8 * r.abs() + 2.0 ** -20 * (v.abs() + b.abs() + a.abs() + t.abs()) + 1e-36
    bad = (y.double() - r).abs() > tol
    assert not bad.any(), (int(bad.sum()), float((y.double() - r).abs().max()))


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("M,K,N", [(1, 256, 64), (3, 272, 72), (8, 4096, 1024), (9, 256, 136), (37, 1040, 264),
                                   (130, 512, 392), (256, 512, 512), (300, 1024, 264), (513, 528, 1288)])
def test_epilogue_small(M, K, N, name):
    x, qw, sw, bias, res = _case(M, K, N, M + K + N)
    for b in (None, bias):
        for r in (None, res):
            _check(w8a8.linear_epilogue(x, qw, sw, bias=b, act=ACTS[name], residual=r), x, qw, sw, b, r, name)
    assert w8a8.get_device_error() == (w8a8.OK, 0)


@pytest.mark.parametrize("M,K,N", [(1, 16, 8), (8, 16, 8), (9, 16, 8), (33, 144, 8), (129, 16, 136), (700, 32, 24),
                                   # clusters of 2, 4 and 8 along K, uneven shares of its blocks
                                   (5, 2064, 200), (16, 9232, 1024), (40, 4112, 512), (200, 1296, 5120), (7, 17408, 264),
                                   # more tiles than SMs
                                   (128, 256, 40000), (260, 400, 20000)])
def test_epilogue_shapes(M, K, N):
    x, qw, sw, bias, res = _case(M, K, N, 11)
    _check(w8a8.linear_epilogue(x, qw, sw, bias=bias, residual=res), x, qw, sw, bias, res, "none")
    _check(w8a8.linear_epilogue(x, qw, sw, bias=bias, act=w8a8.ACT_GELU), x, qw, sw, bias, None, "gelu")
    assert w8a8.get_device_error() == (w8a8.OK, 0)


@pytest.mark.parametrize("M", [1, 8, 16, 32, 100, 512])
def test_epilogue_none_is_the_linear(M):
    x, qw, sw, _, _ = _case(M, 1024, 512, M)
    assert torch.equal(w8a8.linear_epilogue(x, qw, sw), w8a8.linear(x, qw, sw))


@pytest.mark.parametrize("M,K,N", [(4, 17408, 5120), (40, 5120, 17408), (1000, 5120, 4104)])
def test_epilogue_large(M, K, N):
    x, qw, sw, bias, res = _case(M, K, N, 7)
    _check(w8a8.linear_epilogue(x, qw, sw, bias=bias, act=w8a8.ACT_SILU, residual=res), x, qw, sw, bias, res, "silu")


@pytest.mark.parametrize("M", [1, 5, 20, 70, 300])
def test_epilogue_strided_and_in_place(M):
    K, N = 512, 264
    x, qw, sw, bias, res = _case(M, K, N, M)
    want = w8a8.linear_epilogue(x, qw, sw, bias=bias, act=w8a8.ACT_GELU, residual=res)
    # columns of wider tensors; what lies beside them stays as it was
    wide_x = torch.full((M, K + 48), 3.0, dtype=torch.bfloat16, device="cuda")
    wide_r = torch.full((M, N + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    wide_x[:, 16:16 + K] = x
    wide_r[:, 8:8 + N] = res
    y = w8a8.linear_epilogue(wide_x[:, 16:16 + K], qw, sw, bias=bias, act=w8a8.ACT_GELU, residual=wide_r[:, 8:8 + N],
                             y=wide_r[:, 8:8 + N])
    assert torch.equal(y, want) and torch.equal(wide_r[:, 8:8 + N], want)
    assert bool((wide_r[:, :8] == 5).all()) and bool((wide_r[:, 8 + N:] == 5).all())


@pytest.mark.parametrize("M", [3, 8, 30, 130, 600])
def test_epilogue_leaves_the_rows_behind(M):
    """A padded batch: rows past M of input, residual and output are neither used nor written."""
    K, N = 256, 136
    x, qw, sw, bias, res = _case(M + 9, K, N, M)
    x[M:], res[M:] = float("nan"), float("nan")
    y = torch.full((M + 9, N), 7.0, dtype=torch.bfloat16, device="cuda")
    w8a8.linear_epilogue(x[:M], qw, sw, bias, w8a8.ACT_NONE, res[:M], y=y[:M])
    _check(y[:M], x[:M], qw, sw, bias, res[:M], "none")
    assert bool((y[M:] == 7).all())


# Outputs of more tiles than CTAs can share go to the pair tiles, in each of their widths and epilogues: 256 columns
# with 16 epilogue warps, 160, 144, and 256 with 8 warps (many tiles of 32 k blocks or more).
PAIRS = [(300, 64, 12808), (150, 144, 21536), (300, 64, 10408), (1030, 4096, 15368)]


@pytest.mark.parametrize("M,K,N", PAIRS)
def test_epilogue_pair_tiles(M, K, N):
    x, qw, sw, bias, res = _case(M, K, N, 5)
    for name in ACTS:
        for b, r in ((bias, res), (bias, None), (None, res)):
            _check(w8a8.linear_epilogue(x, qw, sw, bias=b, act=ACTS[name], residual=r), x, qw, sw, b, r, name)
    assert torch.equal(w8a8.linear_epilogue(x, qw, sw), w8a8.linear(x, qw, sw))
    # strided, in place, in a padded batch: nothing beside or behind the output is touched
    want = w8a8.linear_epilogue(x, qw, sw, bias=bias, act=w8a8.ACT_SILU, residual=res)
    wide = torch.full((M + 40, N + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:M, 8:8 + N] = res
    wide_x = torch.full((M, K + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    wide_x[:, 8:8 + K] = x
    y = wide[:M, 8:8 + N]
    for _ in range(2):
        y.copy_(res)
        w8a8.linear_epilogue(wide_x[:, 8:8 + K], qw, sw, bias=bias, act=w8a8.ACT_SILU, residual=y, y=y)
        assert torch.equal(y, want)
    assert bool((wide[:, :8] == 5).all()) and bool((wide[:, 8 + N:] == 5).all()) and bool((wide[M:] == 5).all())
    # non-finite values stay where they belong
    bias[3], res[1, 5], res[M - 1, N - 1] = float("nan"), float("inf"), float("nan")
    y = w8a8.linear_epilogue(x, qw, sw, bias, w8a8.ACT_RELU, res)
    nan = torch.zeros_like(y, dtype=torch.bool)
    nan[:, 3], nan[M - 1, N - 1] = True, True
    assert torch.equal(torch.isnan(y), nan) and y[1, 5] == float("inf")
    assert w8a8.get_device_error() == (w8a8.OK, 0)


def test_epilogue_pair_tiles_captured_and_at_once():
    cases = [_case(M, K, N, 6 + i) for i, (M, K, N) in enumerate(PAIRS[:3])]
    calls = [lambda c=c, **kw: w8a8.linear_epilogue(*c[:3], c[3], w8a8.ACT_GELU_TANH, c[4], **kw) for c in cases]
    want = [f() for f in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[f(stream=s) for f, s in zip(calls, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for row in got for a, b in zip(row, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = [f() for f in calls]
    for c in cases:
        c[0].copy_(torch.roll(c[0], 1, 0))
        c[4].copy_(torch.roll(c[4], 1, 1))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, f()) for a, f in zip(ys, calls))


def test_epilogue_non_finite_residual_and_bias():
    for M in (4, 20, 300):
        x, qw, sw, bias, res = _case(M, 256, 64, M)
        bias[3], res[1, 5], res[2, 6] = float("nan"), float("inf"), float("nan")
        for name in ("none", "relu", "silu", "gelu", "gelu_tanh"):
            y = w8a8.linear_epilogue(x, qw, sw, bias, ACTS[name], res)
            nan = torch.zeros_like(y, dtype=torch.bool)
            nan[:, 3], nan[2, 6] = True, True
            assert torch.equal(torch.isnan(y), nan) and y[1, 5] == float("inf")


def test_epilogue_extreme_values():
    """Zero rows, and pre-activations far out on both sides."""
    M, K, N = 6, 256, 64
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[1:] = 1.0
    qw = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    qw[1::2] = -127
    sw = torch.full((N,), 0.01, device="cuda")     # v = +-325
    bias = torch.linspace(-200, 200, N, device="cuda")
    for name, act in ACTS.items():
        for m in (M, 2):
            _check(w8a8.linear_epilogue(x[:m], qw, sw, bias=bias, act=act), x[:m], qw, sw, bias, None, name)


def test_epilogue_two_streams_and_graph():
    """Two calls at once with workspaces of their own, and a captured call replayed on new data."""
    x, qw, sw, bias, res = _case(8, 17408, 1024, 3)
    x2, qw2, sw2, bias2, res2 = _case(300, 1024, 512, 4)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    want = w8a8.linear_epilogue(x, qw, sw, bias, w8a8.ACT_SILU, res)
    want2 = w8a8.linear_epilogue(x2, qw2, sw2, bias2, w8a8.ACT_RELU, res2)
    torch.cuda.synchronize()
    ys = []
    for _ in range(4):
        ys.append((w8a8.linear_epilogue(x, qw, sw, bias, w8a8.ACT_SILU, res, stream=a),
                   w8a8.linear_epilogue(x2, qw2, sw2, bias2, w8a8.ACT_RELU, res2, stream=b)))
    torch.cuda.synchronize()
    assert all(torch.equal(p, want) and torch.equal(q, want2) for p, q in ys)
    graph, y = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        w8a8.linear_epilogue(x, qw, sw, bias, w8a8.ACT_SILU, res, y=y)
    x.copy_(torch.roll(x, 1, 0))
    graph.replay()
    torch.cuda.synchronize()
    got = y.clone()
    assert torch.equal(got, w8a8.linear_epilogue(x, qw, sw, bias, w8a8.ACT_SILU, res))
