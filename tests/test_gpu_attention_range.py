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


def _floor(cache, scale, b, n, table, p):
    """What the sum of two fp16 may lose, [Hkv, 1, D]: u = p s is scaled so that the largest of a head lies in
    [2^14, 2^15); fp16's smallest step is 2^-24, so the lower part is off by up to 2^-25, which is 2^-39 of that largest
    u, for each token that has a code at d."""
    codes = _held(cache, None, b, n, table).abs()
    u = _held(torch.ones_like(cache[..., :1]), scale, b, n, table) * p            # [Hkv, n, 1]
    return (2.0 ** -39 * u.amax(dim=1, keepdim=True) * codes.sum(dim=1, keepdim=True))


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


@pytest.mark.parametrize("D,G", [(64, 3), (128, 4), (128, 12), (256, 6), (256, 16)])
@pytest.mark.parametrize("n", [40, 700, 20000])
def test_attention_value_scales_far_apart(n, D, G):
    """One token's values are 2^8 to 2^24 times as loud as the others', but its codes are zero from d = 16 on: there the
    others decide, each of them far below the loudest."""
    page, loud = 16, (8, 14, 17, 20, 24)
    c, s, table, lengths = _int8(len(loud), n, 2, D, page, seed=D + G)
    for b, e in enumerate(loud):
        for t in (3, n - 1, n // 2)[:1 + b % 3]:
            pg, at = _at(t, page)
            pg = int(table[b, pg])
            c[1][pg, :, at, 16:] = 0
            s[1][pg, :, at] = 2.0 ** e
    q = torch.zeros((len(loud), 2 * G, D), dtype=torch.bfloat16, device="cuda")      # every token weighs the same
    y = w8a8.paged_attention(q, c[0], c[1], table, lengths, k_scale=s[0], v_scale=s[1])
    for b in range(len(loud)):
        v = _held(c[1], s[1], b, n, table)
        want, size = v.mean(dim=1)[:, None], v.abs().mean(dim=1)[:, None]
        # bf16's rounding; probability times scale to 2^-20, sums of n terms in fp32 (2^-23 each, pairwise by lanes
        # and warps: no more than n of them)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -20 + n * 2.0 ** -23) * size + _floor(c[1], s[1], b, n, table, 1.0 / n)
        bad = (y[b].double().view(2, G, D) - want).abs() > tol
        assert not bad.any(), (b, int(bad.sum()), float(((y[b].double().view(2, G, D) - want).abs() / tol).max()))
    assert w8a8.get_device_error() == (w8a8.OK, 0)


@pytest.mark.parametrize("D,G", [(64, 3), (128, 4), (128, 12), (256, 6)])
@pytest.mark.parametrize("n", [40, 700, 20000])
def test_attention_quiet_tokens_count_together(n, D, G):
    """A first token that takes nearly all of the probability and whose values are zero from d = 16 on: there the many
    others, of probability 2^-20 to 2^-30 each, are all that the output holds."""
    page = 16
    c, s, table, lengths = _int8(3, n, 2, D, page, seed=n)
    c[0].zero_()
    s[0].fill_(1.0)
    first = table[:, 0].long()
    c[0][first, :, 0, 0] = 64
    c[1][first, :, 0, 16:] = 0
    q = torch.zeros((3, 2 * G, D), dtype=torch.bfloat16, device="cuda")
    for b, e in enumerate((20, 25, 30)):
        q[b, :, 0] = e                                       # the first token's score: 64 e scale = e log 2
    scale = math.log(2) / 64
    y = w8a8.paged_attention(q, c[0], c[1], table, lengths, scale=scale, k_scale=s[0], v_scale=s[1])
    for b, e in enumerate((20, 25, 30)):
        v = _held(c[1], s[1], b, n, table)
        p = torch.full((n,), 2.0 ** -e, dtype=torch.float64, device="cuda")
        p[0] = 1.0
        p /= p.sum()
        want = (p[None, :, None] * v).sum(dim=1)[:, None]
        size = (p[None, :, None] * v.abs()).sum(dim=1)[:, None]
        # a score of e log2 units is off by its three roundings and scale's (2^-22 e together), through the exponential
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -20 + 2.0 ** -22 * e + n * 2.0 ** -23) * size \
            + _floor(c[1], s[1], b, n, table, p[:, None])
        bad = (y[b].double().view(2, G, D) - want).abs() > tol
        assert not bad.any(), (b, int(bad.sum()), float(((y[b].double().view(2, G, D) - want).abs() / tol).max()))
    assert w8a8.get_device_error() == (w8a8.OK, 0)


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("n", [1, 300, 20000])
def test_attention_scores_of_minus_infinity(n, int8):
    """Keys that are infinite: where each of a head's scores is -inf the outputs are NaN, as the formula's; where one
    score is finite they are its value; absent tokens remain absent."""
    D, page, Hkv, G = 64, 16, 2, 3
    c, s, table, lengths = _int8(4, n, Hkv, D, page, seed=5)
    c[0][..., 0] = 100
    s[1].fill_(1.0)
    q = torch.randn((4, Hkv * G, D), generator=_gen(6), device="cuda").to(torch.bfloat16)
    if int8:
        q[..., 1:] = 0
        q[..., 0] = -q[..., 0].abs() - 1                     # every score of an infinite scale is -inf
        s[0][:, 0] = math.inf                                # of the first key-value head
    else:
        c = [x.to(torch.bfloat16) for x in c]
        s = [None, None]
        q[..., 0] = -q[..., 0].abs() - 1
        c[0][:, 0, :, 0] = math.inf
    pg, at = _at(n - 1, page)
    pg = int(table[1, pg])
    if int8:
        s[0][pg, 0, at] = 1.0
    else:
        c[0][pg, 0, at, 0] = 1.0
    lengths[2] = 0
    table[3] = -1
    y = w8a8.paged_attention(q, c[0], c[1], table, lengths, k_scale=s[0], v_scale=s[1])
    assert w8a8.get_device_error()[0] == w8a8.ERR_INVALID_ARG          # the absent pages
    assert bool(torch.isnan(y[0, :G]).all()) and bool(torch.isfinite(y[0, G:]).all())
    assert torch.equal(y[1, :G], c[1][pg, 0, at].to(torch.bfloat16).expand(G, D)) and bool(torch.isfinite(y[1]).all())
    assert not y[2:].any()


@pytest.mark.parametrize("D,G", [(64, 3), (128, 4), (128, 12), (256, 6), (256, 16)])
@pytest.mark.parametrize("n", [40, 700, 20000])
def test_attention_query_elements_far_apart(n, D, G):
    """One query element 2^10 to 2^18 times as large as the others, which meets zero codes: the others decide the scores,
    and each of them counts with all of its digits."""
    page, large = 16, (10, 12, 14, 16, 18)
    c, s, table, lengths = _int8(len(large), n, 2, D, page, seed=n + D)
    c[0][..., 5] = 0
    s[0] *= 1.0 / 64
    q = torch.randn((len(large), 2 * G, D), generator=_gen(G), device="cuda")
    for b, e in enumerate(large):
        q[b, :, 5] = 2.0 ** e * 1.5
    q = q.to(torch.bfloat16)
    y = w8a8.paged_attention(q, c[0], c[1], table, lengths, k_scale=s[0], v_scale=s[1])
    for b in range(len(large)):
        k, v = _held(c[0], s[0], b, n, table), _held(c[1], s[1], b, n, table)
        qb = q[b].double().view(2, G, D)
        l = torch.einsum("hgd,htd->hgt", qb, k) * D ** -0.5
        p = torch.softmax(l, dim=2)
        want, size = torch.einsum("hgt,htd->hgd", p, v), torch.einsum("hgt,htd->hgd", p, v.abs())
        # a score's error: elements rounded to 2^-30 of the largest (2^-22 beyond 8 heads), the sum's three joins, the products with scale and
        # key scale and the subtraction of the maximum, 2^-24 each of what has been summed up
        part = torch.einsum("hgd,htd->hgt", qb.abs(), k.abs()).amax(dim=2, keepdim=True) * D ** -0.5
        small = 2.0 ** (-30 if G <= 8 else -22) * qb.abs().amax(dim=2, keepdim=True) * k.abs().sum(dim=2).amax(dim=1)[:, None, None] * D ** -0.5
        dl = small + 8 * 2.0 ** -24 * part + 2.0 ** -21
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -20 + n * 2.0 ** -23 + 2 * dl) * size \
            + (2.0 ** -39 * p.amax(dim=2, keepdim=True) * 1.5 * _held(c[1], None, b, n, table).abs().sum(dim=1)[:, None])
        bad = (y[b].double().view(2, G, D) - want).abs() > tol
        assert not bad.any(), (b, int(bad.sum()), float(((y[b].double().view(2, G, D) - want).abs() / tol).max()))
    assert w8a8.get_device_error() == (w8a8.OK, 0)
