"""The epilogue's activations closer than the output's bf16 shows them: a residual that is the activation's own value in
bf16, negated, takes its leading digits away (the sum is exact), and the output holds the next ones."""
import math

import pytest
import torch

from moe_gemm_absmax_b200 import w8a8

pytestmark = pytest.mark.gpu

#: What the library states for |v| < 8.
BOUND = {"silu": 2.0 ** -18, "gelu": 2.0 ** -18, "gelu_tanh": 2.0 ** -16}


def _exact(name, v):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))


@pytest.mark.parametrize("name", list(BOUND))
@pytest.mark.parametrize("M", [1, 7, 20, 300])
def test_activation_accuracy(M, name):
    act = {"silu": w8a8.ACT_SILU, "gelu": w8a8.ACT_GELU, "gelu_tanh": w8a8.ACT_GELU_TANH}[name]
    N, K = 16384 if M < 100 else 40000, 64
    # one code of 127 a row: the sum is 127 * 127, and sw alone sets v
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    qw = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    qw[:, 0] = 127
    at = torch.linspace(-7.999, 7.999, N, device="cuda")
    sw = at / 127
    qx, sx = w8a8.quant_act(x[:1])
    v = (torch.tensor(127.0 * 127.0, device="cuda") * sx) * sw              # fp32, one rounding each, as the library
    want = _exact(name, v.double())
    res = (-want).to(torch.bfloat16)
    y = w8a8.linear_epilogue(x, qw, sw, act=act, residual=res.expand(M, N).contiguous())
    got = y.double() - res.double()
    # the difference, small where the value is next to a bf16 number, rounds to 2^-8 of itself
    tol = (BOUND[name] * want.abs() + 2.0 ** -8 * (want + res.double()).abs()) * (1 + 2.0 ** -8)
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / want.abs()).max()))
    assert w8a8.get_device_error() == (w8a8.OK, 0)
