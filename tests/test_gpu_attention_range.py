"""The attention of one new token over the paged cache where scales, queries and scores are far apart, against 64 bits."""
import math

import pytest
import torch

from moe_gemm_absmax_b200 import w8a8

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _table(B, pages):
    return torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)


def _int8(B, n, Hkv, D, page=16, seed=0):
    """An int8 cache of B contexts of n tokens, every page full: codes and scales [B, Hkv, tokens, ...] as views."""
    pages = -(-n // page)
    g = _gen(seed)
    c = [torch.randint(-127, 128, (B * pages, Hkv, page, D), generator=g, device="cuda").to(torch.int8) for _ in range(2)]
    s = [0.5 + torch.rand((B * pages, Hkv, page), generator=g, device="cuda") for _ in range(2)]
    return c, s, _table(B, pages), torch.full((B,), n, dtype=torch.int32, device="cuda")


def _held(cache, scale, b, n, table):
    """float64 [Hkv, n, D]"""
    x = cache[table[b].long()].double()
    if scale is not None:
        x = x * scale[table[b].long()].double()[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _at(t, page):
    return t // page, t % page


@pytest.mark.parametrize("D,G", [(64, 1), (128, 3), (128, 9), (256, 2)])
def test_attention_maximum_that_rises_slowly(D, G):
    """Scores that rise a little from tile to tile over a long context whose values are all zero but the first token's:
    the running maximum is raised some hundred times and the first token's part must come through.  (Many sequences over
    the same pages, so that a CTA has a whole context to itself.)"""
    n, page, B = 32768, 256, 640
    c, s, table, _ = _int8(1, n, 1, D, page, seed=D)
    c[0].zero_()
    c[0][..., 0] = 127
    c[1][:] = 0
    c[1][0, 0, 0] = torch.arange(D, device="cuda").to(torch.int8) % 127 + 1
    s[0][:, 0] = torch.arange(n, device="cuda").view(-1, page) / n
    s[1].zero_()                                             # what the append writes for rows of zeros
    s[1][0, 0, 0] = 1.0
    q = torch.zeros((B, G, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = 8 * math.log(2) / 127
    y = w8a8.paged_attention(q, c[0], c[1], table.expand(B, -1).contiguous(), torch.full((B,), n, dtype=torch.int32, device="cuda"),
                             scale=scale, k_scale=s[0], v_scale=s[1])
    p = torch.softmax(8 * math.log(2) * s[0][:, 0].double().flatten(), dim=0)
    want = p[0] * c[1][0, 0, 0].double()
    # bf16's rounding; scores of up to 8 log 2 to three roundings and the exponential's 2^-22, the sum's n terms to 2^-23
    # each (pairwise by lanes, warps and parts), the first token's part raised 256 times, 2^-24 each
    tol = (2.0 ** -8 + 2.0 ** -16 + n / 4 / 32 * 2.0 ** -22) * want
    bad = (y.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), y[bad][:4], want[:4])
    assert w8a8.get_device_error() == (w8a8.OK, 0)
