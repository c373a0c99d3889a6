"""Token log probabilities, entropy and top alternatives against 64 bits."""
import math

import pytest
import torch

from moe_gemm_absmax_b200 import w8a8

pytestmark = pytest.mark.gpu


def _want(x, tokens, k):
    lp = torch.log_softmax(x.double(), dim=1)
    lp = torch.where((x == -math.inf).all(dim=1, keepdim=True), -math.inf, lp)
    h = -torch.where(lp > -math.inf, lp.exp() * lp, 0.0).sum(dim=1)
    ids = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]
    return lp.gather(1, tokens.long()), h, ids.to(torch.int32), lp.gather(1, ids)


def _tol(x):
    """Absolute error of a row's log probabilities, and of its entropy.  s: a thread adds at most V / 512 + 8 terms one
    after the other (2^-24 each), 20 joins, and the exponentials are good to 2^-21 with the rounding of their
    arguments; log s and the difference x - m round to 2^-24 of themselves."""
    V = x.shape[1]
    fin = torch.where(x > -math.inf, x.double(), 0.0)
    far = 2 * fin.abs().amax(dim=1) + math.log(V)
    s = (V / 512 + 28) * 2.0 ** -24 + 2.0 ** -21
    return s + 2.0 ** -22 * far, (2 * s + 2.0 ** -22) * (far + math.log(V) + 1)


def _check(x, tokens, k, **kw):
    t2 = tokens if tokens.dim() == 2 else tokens[:, None]
    logprob, h, ids, top = w8a8.token_logprobs(x, tokens, topk=k, **kw)
    torch.cuda.synchronize()
    lp0, h0, ids0, top0 = _want(x, t2, k)
    tl, th = _tol(x)
    assert logprob.shape == tokens.shape
    for got, want, tol in ((logprob.view(t2.shape), lp0, tl[:, None]), (h, h0, th), *(((top, top0, tl[:, None]),) if k else ())):
        same = (got == want) | ((got.double() - want).abs() <= tol)
        assert same.all(), (got[~same][:5], want[~same][:5])
    if k:
        assert torch.equal(ids, ids0)


def _logits(M, V, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (2.5 * torch.randn((M, V), generator=g, device="cuda")).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V,k", [(1, 1, 1), (2, 7, 7), (3, 31, 32 - 1), (1, 100, 5), (5, 1000, 20), (4, 4097, 32),
                                   (1, 131072, 20), (3, 100003, 20), (40, 32000, 1), (700, 5001, 20), (9, 65536, 0)])
def test_logprobs(M, V, k, dtype):
    x = _logits(M, V, dtype, V)
    tokens = torch.randint(0, V, (M,), device="cuda", dtype=torch.int32)
    _check(x, tokens, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_rows_at_any_element(dtype):
    """Views whose rows start at every element offset from a 16-byte boundary, odd strides."""
    base = _logits(6, 5003, dtype)
    tokens = torch.arange(6, device="cuda", dtype=torch.int32) * 700
    for at in range(9):
        _check(base[:, at:at + 4900 + at], tokens, 20)
    _check(base[1:2, 3:10], tokens[:1], 3)


def test_logprobs_ties_and_order():
    """Equal logits go to the lower index; the large ones together in one thread's elements, or ascending."""
    M, V = 8, 40000
    x = torch.zeros((M, V), dtype=torch.bfloat16, device="cuda")
    x[1] = -0.0
    x[1, 5::7] = 0.0
    x[2] = torch.linspace(-8, 8, V, device="cuda")           # bf16: long runs of equal values, ascending
    x[3] = torch.linspace(8, -8, V, device="cuda")
    x[4, 4096 * 0 + 8:4096 * 0 + 16] = 3.0
    for i in range(9):                                      # one thread's windows, 512 windows of 8 apart
        x[5, i * 4096 + 16:i * 4096 + 24] = 4.0
    x[6, V - 3:] = 1.0
    x[7, :40] = torch.arange(40, device="cuda").to(torch.bfloat16)
    tokens = torch.zeros(M, device="cuda", dtype=torch.int32)
    for k in (1, 20, 32):
        _check(x, tokens, k)
        _check(x.float(), tokens, k)
        _check(x[5:6], tokens[:1], k)


@pytest.mark.parametrize("dtype,per", [(torch.bfloat16, 8), (torch.float32, 4)])
def test_logprobs_tie_with_the_rows_ragged_end(dtype, per):
    """The largest value three times: in the second 16-byte window, in a later one, and behind the last whole one, which
    the second window's thread takes as well."""
    V = 400 * per + 3
    x = torch.zeros((3, V), dtype=dtype, device="cuda")
    for at in (per, 300 * per + 1, V - 1):
        x[0, at] = 4.0
    x[1, V - 1] = x[1, 299 * per] = 4.0
    x[2, per + 2], x[2, V - 2] = 4.0, 5.0
    tokens = torch.zeros(3, device="cuda", dtype=torch.int32)
    for k in (1, 2, 3, 4):
        _check(x, tokens[:1].expand(3).contiguous(), k)
        for i in range(3):
            _check(x[i:i + 1], tokens[:1], k)


def test_logprobs_masked_rows():
    x = _logits(6, 3001, torch.float32)
    x[0, 10:] = -math.inf                                   # fewer left than alternatives asked for
    x[1] = -math.inf                                        # nothing left
    x[2] = torch.finfo(torch.float32).min                   # the type's lowest value everywhere: uniform
    x[3, 1:] = torch.finfo(torch.float32).min
    x[4, ::2] = -math.inf
    tokens = torch.tensor([3, 3, 3, 3, 4, 0], device="cuda", dtype=torch.int32)
    _check(x, tokens, 20)
    h = w8a8.token_logprobs(x)[1]
    assert h[1] == 0 and abs(float(h[2]) - math.log(3001)) < 1e-5 and h[3] == 0
    b = x.to(torch.bfloat16)
    b[2] = torch.finfo(torch.bfloat16).min
    _check(b, tokens, 20)


def test_logprobs_nan_and_inf():
    x = _logits(4, 2000, torch.float32)
    x[1, 77] = math.nan
    x[2, 55] = math.inf
    x[3, 1] = -math.inf
    tokens = torch.tensor([0, 0, 0, 1], device="cuda", dtype=torch.int32)
    lp, h, ids, top = w8a8.token_logprobs(x, tokens, topk=5)
    assert torch.isfinite(lp[0]) and torch.isnan(lp[1]) and torch.isnan(lp[2]) and lp[3] == -math.inf
    assert torch.isnan(h[1]) and torch.isnan(h[2]) and torch.isfinite(h[3])
    assert ids[2, 0] == 55 and 77 not in ids[1].tolist()
    clean = x.clone()
    clean[1, 77] = -math.inf
    assert torch.equal(ids, torch.sort(clean, dim=1, descending=True, stable=True).indices[:, :5].to(torch.int32))
    x = torch.full((1, 20), math.nan, device="cuda")
    ids = w8a8.token_logprobs(x, topk=4)[2]
    assert ids.tolist() == [[0, 1, 2, 3]]


def test_logprobs_many_tokens_and_outside():
    x = _logits(3, 5000, torch.bfloat16)
    tokens = torch.randint(0, 5000, (3, 700), device="cuda", dtype=torch.int32)
    _check(x, tokens, 2)
    tokens[0, 0], tokens[1, 699], tokens[2, 5] = -1, 5000, 2 ** 31 - 1
    lp = w8a8.token_logprobs(x, tokens)[0]
    assert torch.isnan(lp).sum() == 3 and torch.isnan(lp[0, 0]) and torch.isnan(lp[1, 699]) and torch.isnan(lp[2, 5])


def test_logprobs_repeats_and_graph():
    x = _logits(20, 30000, torch.bfloat16)
    tokens = torch.randint(0, 30000, (20,), device="cuda", dtype=torch.int32)
    first = w8a8.token_logprobs(x, tokens, topk=20)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, w8a8.token_logprobs(x, tokens, topk=20)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w8a8.token_logprobs(x, tokens, topk=20)
    x.copy_(_logits(20, 30000, torch.bfloat16, 9))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, w8a8.token_logprobs(x, tokens, topk=20)))
